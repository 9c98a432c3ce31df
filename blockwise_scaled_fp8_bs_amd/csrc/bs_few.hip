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
// bf16 on the way to the matrix cores: e4m3 and e2m1 fit, and MX scales are
// powers of two that the conversion applies, so that this is exact for weights
// from 2^-126 up to bf16's largest (below, MXFP8's smallest codes are rounded to
// multiples of 2^-133; above, they are infinite).  What lies outside the
// operands is read as zeros by the buffers' bounds.
//
// Tokens stay in bf16: quantizing them would save nothing where the weights
// are the traffic.  Sums are in fp32; h alone is rounded on the way, to bf16,
// which is what the matrix instructions take.  Up to 8 tokens it is kept in two
// bf16 parts, h and what its rounding left out, side by side in the instructions'
// 16 columns: the result's error against float64 is then that of its own
// rounding, 0.0016 to 0.0017 of the norm, up to 0.0024 with one part (1 to 4
// tokens take the same time, 5 to 8 0 to 7 % more: a gated FFN of 5120 and 8192
// in MXFP8 44 us, 41 with one).  Beside more tokens the parts would take columns
// of their own, and twice the way through LDS that bounds there: one part (16
// tokens through an FFN of 2048 and 4096 in e4m3 17 us, 20 with two; 24 over 16
// experts of 1024 37 and 44; 64 over 64 e2m1 experts of 2048 181 and 219).
//
// Measured on MI355X: a call of few bytes takes 3.6 us (product) and 5 + 5.5
// (experts), and the weights come on top at up to 6.1 TB/s (24 tokens over 64
// e4m3 experts of 2048, width 4096: 254 us for 1.55 GB).
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

// A unit: HB bytes along each of 16 rows of codes, 128, or 64 beside many
// tokens, whose values would fill the ring.
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

// Stages of a ring: at most 6, and at most 63 loads under way (the counter that
// a wave waits by has six bits).
template <class S>
constexpr int ring_stages(int ring) {
    const int fit = ring / S::kBytes, count = 63 / S::kLoads, most = fit < count ? fit : count;
    return most < 6 ? most : 6;
}

template <int V>
using Int = std::integral_constant<int, V>;

// Bytes of a unit: whole cache lines (64 tokens over 64 experts in 4 bits take
// 119 us in the first kernel, 148 with half ones), but where the tokens would
// leave the ring without a second stage.
template <int KIND, int NT, int RX, int RING>
using UnitBytes = Int<ring_stages<Stage<KIND, 128, NT, RX>>(RING) >= 2 ? 128 : 64>;

// 16 rows of weights.
struct Tile16 {
    i32x4 q, s;  // their codes and scales
};

// The units of a wave: weights' row pieces and tokens' pieces of its lanes.
template <int KIND, int HB, int NT, int RX>
struct Loader {
    using U = Unit<KIND, HB>;
    using S = Stage<KIND, HB, NT, RX>;
    int lane, piece;               // 16-byte piece of the row that the lane fetches, in bytes
    int row[S::kTileLoads];        // offset of its row and piece
    int token[S::kCopies];         // offset of its token and piece (kOut: none)
    int K, row_bytes, ld_s;        // (ld_s in bytes: the scales of a matrix are below 2^31)

    __device__ __forceinline__ void rows(int lane_, int64_t ld_q, int64_t ld_s_, int K_) {
        lane = lane_;
        K = K_;
        row_bytes = KIND == kFewMx4 ? K / 2 : K;
        ld_s = (int)(KIND == kFewE4m3 ? 4 * ld_s_ : ld_s_);
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

    // S::kLoads loads, whatever is there of the unit: what lies past the contraction is fetched from kOut, also the scales
    // (a byte 255 behind the last row of them would make NaN of the zeros in their place)
    __device__ __forceinline__ void load(const Tile16 (&tile)[NT], const i32x4 x, int u, uint32_t lds) const {
        const int at = u * HB;
        const bool in = at + piece < row_bytes;
        int off[S::kCopies > S::kTileLoads ? S::kCopies : S::kTileLoads];
#pragma unroll
        for (int i = 0; i < S::kTileLoads; ++i) off[i] = in ? row[i] : kOut;
#pragma unroll
        for (int n = 0; n < NT; ++n) dma16_run<S::kTileLoads>(tile[n].q, lds + n * S::kTile, off, at);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            if (KIND == kFewE4m3) {
                if (lane == 0)
                    dma4(tile[n].s, lds + S::kScaleAt + n * S::kScales, at < K ? 0 : kOut,
                         (int)((uint32_t)(at / 128) * (uint32_t)ld_s));
            } else {
                if (lane < U::kBlocks)
                    dma16(tile[n].s, lds + S::kScaleAt + n * S::kScales, 32 * (u * U::kBlocks + lane) < K ? lane * ld_s : kOut,
                          (int)((uint32_t)u * U::kBlocks * (uint32_t)ld_s));
            }
        }
        const int xat = u * U::kTokenRow;
#pragma unroll
        for (int i = 0; i < S::kCopies; ++i) off[i] = xat + token_piece(i, lane) < 2 * K ? token[i] : kOut;
        if (RX * S::kSlots >= 64 || lane < RX * S::kSlots) dma16_run<S::kCopies>(x, lds + S::kTokenAt, off, xat);
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
    static constexpr int TT = RX > 16 ? RX / 16 : 1;  // tiles of tokens
    u32x4 a[NT][U::kHalves], x[TT][U::kSteps];
    uint32_t s[NT][U::kHalves];
    float sc[NT];

    __device__ __forceinline__ void read(const uint8_t* stage, int r, int g) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int h = 0; h < U::kHalves; ++h)
                a[n][h] = *reinterpret_cast<const u32x4*>(stage + n * S::kTile + r * HB + 16 * ((4 * h + g) ^ U::key(r)));
#pragma unroll
        for (int t = 0; t < TT; ++t) {
            const int row = 16 * t + (RX < 16 ? r & (RX - 1) : r);  // the columns past the tokens are not used
#pragma unroll
            for (int f = 0; f < U::kSteps; ++f) {
                constexpr int per = U::kSteps / U::kHalves;  // steps, and 16-byte pieces of tokens, of a piece of codes
                const int p = (4 * (f / per) + g) * per + f % per;
                x[t][f] = *reinterpret_cast<const u32x4*>(stage + S::kTokenAt + row * U::kTokenRow + 16 * (p ^ (row & 7)));
            }
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

    __device__ __forceinline__ void multiply(f32x4 (&acc)[NT][TT]) const {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            f32x4 p[TT];
#pragma unroll
            for (int t = 0; t < TT; ++t) p[t] = KIND == kFewE4m3 ? f32x4{0.f, 0.f, 0.f, 0.f} : acc[n][t];
#pragma unroll
            for (int f = 0; f < U::kSteps; ++f) {
                const bf16x8 w = weights<KIND>(a[n], s[n], f);
#pragma unroll
                for (int t = 0; t < TT; ++t)
                    p[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, __builtin_bit_cast(bf16x8, x[t][f]), p[t], 0, 0, 0);
            }
#pragma unroll
            for (int t = 0; t < TT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[n][t][i] = KIND == kFewE4m3 ? __builtin_fmaf(p[t][i], sc[n], acc[n][t][i]) : p[t][i];
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
template <int KIND, int HB, int NT, int RX, int RING, int TT, class Load, class Before>
__device__ __forceinline__ void stream_units(const uint8_t* ring, int units, int r, int g, f32x4 (&acc)[NT][TT], Load load,
                                             Before before) {
    using S = Stage<KIND, HB, NT, RX>;
    constexpr int DEPTH = ring_stages<S>(RING);
    static_assert(DEPTH >= 2, "a ring of two stages at least");
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

// Rows row0 .. of the N of expert e; `there` false: nothing, all of it reads zeros.
template <int KIND>
__device__ __forceinline__ Tile16 tile_rows(const FewWeight& w, int64_t e, int64_t row0, int64_t N, int K, bool there = true) {
    const int row_bytes = KIND == kFewMx4 ? K / 2 : K;
    const int64_t rows = N - row0 < 16 ? N - row0 : 16;
    there &= rows > 0;
    Tile16 t;
    t.q = make_rsrc(w.q + e * w.stride_q + row0 * w.ld_q, there ? (rows - 1) * w.ld_q + row_bytes : 0);
    if (KIND == kFewE4m3)
        t.s = make_rsrc(static_cast<const float*>(w.s) + e * w.stride_s + row0 / 128, there ? ((K / 128 - 1) * w.ld_s + 1) * 4 : 0);
    else
        t.s = make_rsrc(static_cast<const uint8_t*>(w.s) + e * w.stride_s + row0, there ? (K / 32 - 1) * w.ld_s + 16 : 0);
    return t;
}

template <int NT, int TT>
__device__ __forceinline__ void zero(f32x4 (&acc)[NT][TT]) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int t = 0; t < TT; ++t) acc[n][t] = f32x4{0.f, 0.f, 0.f, 0.f};
}

// Each wave's sums into LDS: red[wave][n][t][lane].
template <int NT, int TT>
__device__ __forceinline__ void put_sums(f32x4* red, int wave, int lane, const f32x4 (&acc)[NT][TT]) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int t = 0; t < TT; ++t) red[((wave * NT + n) * TT + t) * 64 + lane] = acc[n][t];
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

// Workgroup: 16 NT columns of up to RX rows; its waves take turns along the
// contraction, so that 4096 columns are enough for every CU.  One row: 4096 x
// 4096 e4m3 6.1 us, 8192 x 5120 e2m1 7.3; 16 rows: 8192 x 5120 e4m3 10.6 (4.0
// TB/s).  Beside many rows the rows bound it, 64 of them 655 kB a workgroup
// through its CU's 64 bytes a clock: 8192 x 5120 e2m1 14.2 us, 5.5 of them that.
template <int KIND, int HB, int NT, int RX, int W, int RING>
__global__ __launch_bounds__(64 * W) void few_mm_kernel(FewMmArgs a) {
    constexpr int TT = RX > 16 ? RX / 16 : 1;
    static_assert(RING >= NT * TT * 1024, "the sums take the ring's place");
    __shared__ __attribute__((aligned(16))) uint8_t s_ring[W * RING];
    const int tile = xcd_tile(blockIdx.x, gridDim.x);
    if (tile >= a.tiles) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int64_t t0 = (int64_t)blockIdx.y * RX, row0 = (int64_t)tile * (16 * NT);
    const int T = (int)(a.T - t0 < RX ? a.T - t0 : RX), K = (int)a.K;
    const i32x4 x = make_rsrc(a.x + t0 * a.ld_x, ((T - 1) * a.ld_x + K) * 2);
    Tile16 rows[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) rows[n] = tile_rows<KIND>(a.w, 0, row0 + 16 * n, a.N, K);
    Loader<KIND, HB, NT, RX> loader;
    loader.rows(lane, a.w.ld_q, a.w.ld_s, K);
    loader.tokens([&](int c) { return c < T ? c * (int)a.ld_x * 2 : kOut; });
    const int units = (K + Unit<KIND, HB>::kCodes - 1) / Unit<KIND, HB>::kCodes;
    f32x4 acc[NT][TT];
    zero(acc);
    stream_units<KIND, HB, NT, RX, RING>(
        s_ring + wave * RING, (units - wave + W - 1) / W, r, g, acc,
        [&](int i, uint32_t lds) { loader.load(rows, x, wave + i * W, lds); }, [](int) {});
    __syncthreads();
    f32x4* const red = reinterpret_cast<f32x4*>(s_ring);
    put_sums(red, wave, lane, acc);
    __syncthreads();
    for (int i = wave; i < NT * TT; i += W) {
        const int64_t n = row0 + 16 * (i / TT) + 4 * g;
        const int t = 16 * (i % TT) + r;
        if (t >= T || n >= a.N) continue;
        const int64_t at = (t0 + t) * a.ld_out + n;
        store4(sum_waves<W, NT * TT>(red, i, lane), a.residual ? a.residual + (t0 + t) * a.ld_res + n : nullptr,
               a.f32 ? (void*)(static_cast<float*>(a.out) + at) : (void*)(static_cast<uint16_t*>(a.out) + at), a.f32, a.vec,
               (int)(a.N - n < 4 ? a.N - n : 4));
    }
}

// ---------------------------------------------------------------------------
// gated experts: h of the routed slots, then their weighted sum
// ---------------------------------------------------------------------------
//
// h has a row (or one for each part) for every token of every expert that it
// chose (one that it names twice counts once), in the order of the experts and, within one, of the
// tokens.  A work item is 16 of an expert's tokens at most, 32 where most
// experts have more than that.

// What a workgroup knows of its chunk of tokens.
struct Routing {
    const uint32_t* item;   // [items + 1]: expert << 16 | first row of h
    const uint8_t* token;   // [row of h]
    const float* weight;    // [row of h]
    int items, most;        // places (a power of two) that the largest item's tokens take
};

// LDS of the table for `slots` choices and `items` items, and what making it
// takes besides: the ring's place.
struct RoutingLayout {
    int weight, item, token, bytes;        // the table
    int chose, w, e, start, scratch;       // the experts' tokens as bits, and the choices
    __host__ __device__ RoutingLayout(int E, int slots, int items) {
        weight = 0;
        item = 4 * slots;
        token = item + 4 * (items + 4);    // and what was found: items, the places of the largest one, an expert named twice
        bytes = (token + slots + 15) / 16 * 16;
        chose = 0;
        w = 8 * E;
        e = w + 4 * slots;
        start = e + 2 * slots;
        scratch = start + 2 * E;
    }
};

__device__ __forceinline__ u64 below(int lane) { return (1ull << lane) - 1; }

// Sum over the lanes up to this one: within rows of 16 by shifts, then the
// rows' last lanes passed on.
__device__ __forceinline__ int prefix_sum(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);  // row_shr 1
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);  // row_shr 2
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);  // row_shr 4
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);  // row_shr 8
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast 15 into rows 1 and 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // row_bcast 31 into rows 2 and 3
    return v;
}

template <int PER, int THREADS>
__device__ __forceinline__ Routing route_chunk(const MoeFewArgs& a, int64_t t0, int slots, uint8_t* lds, uint8_t* scratch) {
    const RoutingLayout at(a.E, slots, a.items);
    float* const weight = reinterpret_cast<float*>(lds + at.weight);
    uint32_t* const item = reinterpret_cast<uint32_t*>(lds + at.item);
    uint32_t* const found = item + a.items + 1;
    uint8_t* const token = lds + at.token;
    u64* const chose = reinterpret_cast<u64*>(scratch + at.chose);
    float* const w = reinterpret_cast<float*>(scratch + at.w);
    int16_t* const expert = reinterpret_cast<int16_t*>(scratch + at.e);
    uint16_t* const start = reinterpret_cast<uint16_t*>(scratch + at.start);
    const int tid = threadIdx.x, lane = tid & 63;
    // (the first choices are on their way while the table is cleared)
    int32_t e0 = -1;
    float w0 = 1.f;
    if (tid < slots) {
        e0 = a.idx ? a.idx[t0 * a.k + tid] : 0;
        if (a.w) w0 = a.w[t0 * a.k + tid];
    }
    for (int i = tid; i < a.E; i += THREADS) chose[i] = 0;
    if (tid == 0) found[2] = 0;
    __syncthreads();
    for (int i = tid; i < slots; i += THREADS) {
        const int32_t e = i == tid ? e0 : a.idx ? a.idx[t0 * a.k + i] : 0;
        const bool routed = (uint32_t)e < (uint32_t)a.E;
        expert[i] = (int16_t)(routed ? e : -1);
        w[i] = i == tid ? w0 : a.w ? a.w[t0 * a.k + i] : 1.f;
        const u64 bit = 1ull << (i / a.k);
        if (routed && (atomicOr(&chose[e], bit) & bit)) found[2] = 1;  // named twice
    }
    __syncthreads();
    if (tid < 64) {
        int items = 0, rows = 0, most = 0;
        for (int e = lane; e - lane < a.E; e += 64) {
            const int n = e < a.E ? __popcll(chose[e]) : 0, its = (n + PER - 1) / PER;
            const int upto = prefix_sum(n | its << 16);  // both sums in one: at most 2048 rows of a chunk
            const int r0 = rows + (upto & 0xffff) - n, i0 = items + (upto >> 16) - its;
            if (e < a.E) start[e] = (uint16_t)r0;
            for (int j = 0; j < its; ++j) item[i0 + j] = (uint32_t)e << 16 | (uint32_t)(r0 + PER * j);
            most = max(most, min(n, PER));
            const int all = __builtin_amdgcn_readlane(upto, 63);
            rows += all & 0xffff;
            items += all >> 16;
        }
        // (PER is a power of two: the largest count's power is the bit that counts)
        int places = 1;
        for (; places < PER && __ballot(most > places); places *= 2) {
        }
        if (lane == 0) {
            item[items] = (uint32_t)rows;
            found[0] = (uint32_t)items;
            found[1] = (uint32_t)places;
        }
    }
    __syncthreads();
    const bool twice = found[2] != 0;
    for (int i = tid; i < slots; i += THREADS) {
        const int e = expert[i], t = i / a.k;
        if (e < 0) continue;
        bool first = true;
        float sum = w[i];
        if (twice) {
            sum = 0.f;
            for (int j = t * a.k; j < (t + 1) * a.k; ++j)
                if (expert[j] == e) {
                    first &= j >= i;
                    sum += w[j];
                }
        }
        if (!first) continue;
        const int row = start[e] + __popcll(chose[e] & below(t));
        token[row] = (uint8_t)t;
        weight[row] = sum;
    }
    __syncthreads();
    return {item, token, weight, __builtin_amdgcn_readfirstlane((int)found[0]),
            __builtin_amdgcn_readfirstlane((int)found[1])};
}

// The same of a single token, a table for each wave, without a barrier.
struct OneToken {
    uint32_t item[34];
    float weight[32];
    uint8_t token[32];
};

__device__ __forceinline__ Routing route_one(const MoeFewArgs& a, OneToken& t) {
    const int lane = threadIdx.x & 63;
    int e = lane < a.k ? (a.idx ? a.idx[lane] : 0) : -1;
    const float w = lane < a.k ? (a.w ? a.w[lane] : 1.f) : 0.f;
    if ((uint32_t)e >= (uint32_t)a.E) e = -1;
    float sum = 0.f;
    bool first = e >= 0;
    int before = 0;  // experts in ascending order, as with more tokens
    for (int j = 0; j < a.k; ++j) {
        const int ej = __builtin_amdgcn_readlane(e, j);
        const float wj = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(w), j));
        if (ej == e) sum += wj, first &= j >= lane;
        before += (uint32_t)ej < (uint32_t)e;
    }
    // an earlier expert that is named twice stands before once
    for (int j = 0; j < a.k; ++j) {
        const int ej = __builtin_amdgcn_readlane(e, j);
        const bool again = !__builtin_amdgcn_readlane((int)first, j);
        if (again && (uint32_t)ej < (uint32_t)e) --before;
    }
    const int items = __popcll(__ballot(first));
    if (first) {
        t.item[before] = (uint32_t)e << 16 | (uint32_t)before;
        t.weight[before] = sum;
        t.token[before] = 0;
    }
    if (lane == 0) t.item[items] = (uint32_t)items;
    wait_lds();
    return {t.item, t.token, t.weight, items, 1};
}

// The it-th item: its expert, first row of h and number of tokens.
template <int PER>
__device__ __forceinline__ int item_rows(const Routing& rt, int it, int& first, int& n) {
    const uint32_t v = __builtin_amdgcn_readfirstlane(rt.item[it]), w = __builtin_amdgcn_readfirstlane(rt.item[it + 1]);
    first = (int)(v & 0xffff);
    n = min(PER, (int)(w & 0xffff) - first);
    return (int)(v >> 16);
}

// Tokens of an item, at most, in kernels for RXMAX tokens.
constexpr int item_tokens(int rxmax) { return rxmax > 16 ? rxmax : 16; }

// Calls run with the tokens' places and the unit's bytes for items of `most`
// places, RXMAX at most.
template <int KIND, int RXMAX, int NT, int RING, class Run>
__device__ __forceinline__ void with_places(int most, Run run) {
    if (RXMAX == 1 || most <= 1) return run(Int<1>{}, UnitBytes<KIND, NT, 1, RING>{});
    if constexpr (RXMAX == 2) return run(Int<2>{}, UnitBytes<KIND, NT, 2, RING>{});
    if constexpr (RXMAX > 2) {
        if (RXMAX == 4 || most <= 4) return run(Int<4>{}, UnitBytes<KIND, NT, 4, RING>{});
    }
    if constexpr (RXMAX > 4) {
        if (RXMAX == 8 || most <= 8) return run(Int<8>{}, UnitBytes<KIND, NT, 8, RING>{});
    }
    if constexpr (RXMAX > 8) {
        if (RXMAX == 16 || most <= 16) return run(Int<16>{}, UnitBytes<KIND, NT, 16, RING>{});
    }
    if constexpr (RXMAX > 16) run(Int<32>{}, UnitBytes<KIND, NT, 32, RING>{});
}

// h of one lane's four columns, weight silu(a) b: rounded to bf16, and with two
// parts what that left out (nothing of an infinity or a NaN) in a row of its own.
__device__ __forceinline__ void store_h(const MoeFewArgs& a, int64_t row, int64_t col, float weight, f32x4 ga, f32x4 up) {
    uint32_t o[4], rest[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float v = weight * (ga[j] / (1.f + __expf(-ga[j])) * up[j]);
        o[j] = bf16_bits(v);
        rest[j] = (o[j] & 0x7f80u) == 0x7f80u ? 0u : bf16_bits(v - bf16_lo(o[j]));
    }
    uint16_t* const h = a.h + row * a.parts * a.H + col;
    *reinterpret_cast<uint2*>(h) = make_uint2(o[0] | o[1] << 16, o[2] | o[3] << 16);
    if (a.parts > 1) *reinterpret_cast<uint2*>(h + a.H) = make_uint2(rest[0] | rest[1] << 16, rest[2] | rest[3] << 16);
}

// Workgroup: 16 columns of h of a work item; its waves take turns along the
// contraction.  One token: 4 experts of 64 tiles, 2048 e4m3 rows 8.3 us (17 MB);
// 2 of 256 tiles, 5120 e2m1 rows 12.6 (45 MB): five microseconds and the bytes.
template <int KIND, int RXMAX, int W, int RING>
__global__ __launch_bounds__(64 * W) void moe_few_up_kernel(MoeFewArgs a) {
    constexpr int PER = item_tokens(RXMAX);
    extern __shared__ __attribute__((aligned(16))) uint8_t s_dyn[];
    __shared__ __attribute__((aligned(16))) uint8_t s_ring[W * RING];
    __shared__ OneToken s_one[RXMAX == 1 ? W : 1];
    const int padded = (int)((a.tiles + 7) & ~7);
    const int it = blockIdx.x / padded, tile = xcd_tile(blockIdx.x % padded, padded);
    if (tile >= a.tiles) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t0 = (int64_t)blockIdx.y * kFewChunk;
    const int T = (int)(a.T - t0 < kFewChunk ? a.T - t0 : kFewChunk);
    const Routing rt = RXMAX == 1 ? route_one(a, s_one[wave]) : route_chunk<PER, 64 * W>(a, t0, T * a.k, s_dyn, s_ring);
    if (it >= rt.items) return;
    int first, n;
    const int e = item_rows<PER>(rt, it, first, n);

    const int r = lane & 15, g = lane >> 4, D = (int)a.D;
    const int64_t h0 = 16 * (int64_t)tile;
    const Tile16 rows[2] = {tile_rows<KIND>(a.w12, e, h0, a.H, D), tile_rows<KIND>(a.w12, e, a.H + h0, 2 * a.H, D)};
    const i32x4 x = make_rsrc(a.x + t0 * a.ld_x, ((T - 1) * a.ld_x + D) * 2);
    with_places<KIND, RXMAX, 2, RING>(n, [&](auto rx, auto hb) {
        constexpr int RX = decltype(rx)::value, HB = decltype(hb)::value, TT = RX > 16 ? RX / 16 : 1;
        static_assert(RING >= 2 * TT * 1024, "the sums take the ring's place");
        Loader<KIND, HB, 2, RX> loader;
        loader.rows(lane, a.w12.ld_q, a.w12.ld_s, D);
        loader.tokens([&](int c) { return c < n ? rt.token[first + c] * (int)a.ld_x * 2 : kOut; });
        const int units = (D + Unit<KIND, HB>::kCodes - 1) / Unit<KIND, HB>::kCodes;
        f32x4 acc[2][TT];
        zero(acc);
        stream_units<KIND, HB, 2, RX, RING>(
            s_ring + wave * RING, (units - wave + W - 1) / W, r, g, acc,
            [&](int i, uint32_t lds) { loader.load(rows, x, wave + i * W, lds); }, [](int) {});
        __syncthreads();
        f32x4* const red = reinterpret_cast<f32x4*>(s_ring);
        put_sums(red, wave, lane, acc);
        __syncthreads();
        const int c = 16 * wave + r;
        if (wave < TT && c < n)
            store_h(a, t0 * a.k + first + c, h0 + 4 * g, rt.weight[first + c], sum_waves<W, 2 * TT>(red, wave, lane),
                    sum_waves<W, 2 * TT>(red, TT + wave, lane));
    });
}

// The same where there are many tiles: every wave streams whole tiles (16 NH
// columns), one after the other, without a barrier; an XCD's waves walk
// neighbouring tiles.  24 tokens over 64 experts of 128 tiles, 4096 e4m3 rows:
// 175 us, 5.9 TB/s; 64 tokens, e2m1: 120 us, 4.8 TB/s (2 tiles a wave; 153 with
// one, which fetches the tokens twice as often).
template <int KIND, int RXMAX, int NH, int W, int RING>
__global__ __launch_bounds__(64 * W) void moe_few_up_tiles_kernel(MoeFewArgs a) {
    constexpr int PER = item_tokens(RXMAX), NT = 2 * NH;
    extern __shared__ __attribute__((aligned(16))) uint8_t s_dyn[];
    __shared__ __attribute__((aligned(16))) uint8_t s_ring[W * RING];
    __shared__ OneToken s_one[RXMAX == 1 ? W : 1];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t0 = (int64_t)blockIdx.y * kFewChunk;
    const int T = (int)(a.T - t0 < kFewChunk ? a.T - t0 : kFewChunk);
    const Routing rt = RXMAX == 1 ? route_one(a, s_one[wave]) : route_chunk<PER, 64 * W>(a, t0, T * a.k, s_dyn, s_ring);

    const int r = lane & 15, g = lane >> 4, D = (int)a.D;
    const i32x4 x = make_rsrc(a.x + t0 * a.ld_x, ((T - 1) * a.ld_x + D) * 2);
    const int share = (int)((a.tiles + 7) >> 3), tile0 = (blockIdx.x & 7) * share;  // of this XCD
    const int width = max(0, min(share, (int)a.tiles - tile0));
    const int q0 = (blockIdx.x >> 3) * W + wave, step = (gridDim.x >> 3) * W, all = rt.items * width;
    if (q0 >= all) return;
    const int mine = (all - q0 + step - 1) / step;
    with_places<KIND, RXMAX, NT, RING>(rt.most, [&](auto rx, auto hb) {
        constexpr int RX = decltype(rx)::value, HB = decltype(hb)::value, TT = RX > 16 ? RX / 16 : 1;
        const int units = (D + Unit<KIND, HB>::kCodes - 1) / Unit<KIND, HB>::kCodes;
        Loader<KIND, HB, NT, RX> loader;
        loader.rows(lane, a.w12.ld_q, a.w12.ld_s, D);
        Tile16 rows[NT];
        int l_q = q0, l_u = 0;  // of the next unit to load
        auto select = [&] {
            const bool there = l_q < all;
            const int q = there ? l_q : q0;
            int first, n;
            const int e = item_rows<PER>(rt, q / width, first, n);
            const int64_t h0 = 16 * NH * (int64_t)(tile0 + q % width);
#pragma unroll
            for (int i = 0; i < NH; ++i) {
                rows[2 * i] = tile_rows<KIND>(a.w12, e, h0 + 16 * i, a.H, D, there);
                rows[2 * i + 1] = tile_rows<KIND>(a.w12, e, a.H + h0 + 16 * i, 2 * a.H, D, there);
            }
            loader.tokens([&](int c) { return c < n && there ? rt.token[first + c] * (int)a.ld_x * 2 : kOut; });
        };
        select();
        f32x4 acc[NT][TT];
        zero(acc);
        int m_q = q0, m_u = 0;  // of the next one to multiply
        auto put = [&] {
            int first, n;
            item_rows<PER>(rt, m_q / width, first, n);
            const int64_t h0 = 16 * NH * (int64_t)(tile0 + m_q % width) + 4 * g;
#pragma unroll
            for (int t = 0; t < TT; ++t)
#pragma unroll
                for (int i = 0; i < NH; ++i)
                    if (16 * t + r < n && (NH == 1 || h0 + 16 * i < a.H))
                        store_h(a, t0 * a.k + first + 16 * t + r, h0 + 16 * i, rt.weight[first + 16 * t + r], acc[2 * i][t],
                                acc[2 * i + 1][t]);
            zero(acc);
        };
        stream_units<KIND, HB, NT, RX, RING>(
            s_ring + wave * RING, mine * units, r, g, acc,
            [&](int, uint32_t lds) {
                loader.load(rows, x, l_u, lds);
                if (++l_u == units) l_u = 0, l_q += step, select();
            },
            [&](int) {
                if (m_u == units) put(), m_u = 0, m_q += step;
                ++m_u;
            });
        put();
    });
}

// Workgroup: 16 NT columns of the output of every token of the chunk, or with
// a.splits > 1 its share of them.  The items' units follow one another; each
// wave streams an equal share of them and adds what an item gave to sums of its
// own for every token (the weights are in h already), added up at the end in
// the order of the waves.  Where few columns leave CUs idle, several
// workgroups share the units, and each leaves its sums in the workspace (the
// last one adding them up behind a fence took 10 to 30 us more than a kernel).
// 24 tokens over 64 experts of 2048, 4096 e4m3 columns: 79 us, 6.5 TB/s; 64
// tokens, e2m1, 2 tiles a wave and 2 shares: 62 + 4.7 us, 4.3 TB/s (95 with one
// tile and none).
template <int KIND, int RXMAX, int NT, int W, int RING>
__global__ __launch_bounds__(64 * W) void moe_few_down_kernel(MoeFewArgs a) {
    constexpr int PER = item_tokens(RXMAX), Q = 4 * NT;     // f32x4 of a token
    constexpr int PLACES = RXMAX <= 8 ? 2 * RXMAX : RXMAX;  // both parts of h, where there are two
    extern __shared__ __attribute__((aligned(16))) uint8_t s_dyn[];
    __shared__ __attribute__((aligned(16))) uint8_t s_ring[W * RING];
    __shared__ OneToken s_one[RXMAX == 1 ? W : 1];
    const int split = (int)(blockIdx.x % a.splits), tile = xcd_tile(blockIdx.x / a.splits, gridDim.x / a.splits);
    if (tile >= a.tiles) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t0 = (int64_t)blockIdx.y * kFewChunk;
    const int T = (int)(a.T - t0 < kFewChunk ? a.T - t0 : kFewChunk);
    f32x4* const sums = reinterpret_cast<f32x4*>(s_dyn);  // [wave][token][Q]
    f32x4* const own = sums + wave * T * Q;
    for (int i = lane; i < T * Q; i += 64) own[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    const Routing rt = RXMAX == 1 ? route_one(a, s_one[wave])
                                  : route_chunk<PER, 64 * W>(a, t0, T * a.k, s_dyn + W * T * 16 * Q, s_ring);

    const int r = lane & 15, g = lane >> 4, H = (int)a.H;
    const int64_t d0 = 16 * NT * (int64_t)tile;
    const bool two = RXMAX <= 8 && a.parts > 1;
    with_places<KIND, PLACES, NT, RING>(rt.most << two, [&](auto rx, auto hb) {
        constexpr int RX = decltype(rx)::value, HB = decltype(hb)::value, TT = RX > 16 ? RX / 16 : 1;
        const int units = (H + Unit<KIND, HB>::kCodes - 1) / Unit<KIND, HB>::kCodes;
        const int all = rt.items * units, shares = W * a.splits, share = (all + shares - 1) / shares;
        const int u0 = min(all, (split * W + wave) * share), mine = min(share, all - u0);
        if (mine <= 0) return;
        Loader<KIND, HB, NT, RX> loader;
        loader.rows(lane, a.wo.ld_q, a.wo.ld_s, H);
        loader.tokens([&](int c) { return c * H * 2; });  // (those past the item's are outside the buffer)
        int l_item = u0 / units, l_u = u0 % units, l_left = mine;  // of the next unit to load
        int m_item = l_item, m_u = l_u;                            // of the next one to multiply
        Tile16 rows[NT];
        i32x4 h;
        auto select = [&] {
            const bool there = l_left > 0;
            int first, n;
            const int e = item_rows<PER>(rt, there ? l_item : 0, first, n);
#pragma unroll
            for (int i = 0; i < NT; ++i) rows[i] = tile_rows<KIND>(a.wo, e, d0 + 16 * i, a.D, H, there);
            h = make_rsrc(a.h + ((t0 * a.k + first) << two) * a.H, there ? ((int64_t)n << two) * H * 2 : 0);
        };
        select();
        f32x4 acc[NT][TT];
        zero(acc);
        auto put = [&] {
            int first, n;
            item_rows<PER>(rt, m_item, first, n);
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                if (two) {  // a token's parts are neighbours
#pragma unroll
                    for (int i = 0; i < NT; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            acc[i][t][j] += __uint_as_float(
                                __builtin_amdgcn_mov_dpp((int)__float_as_uint(acc[i][t][j]), 0xB1, 0xF, 0xF, false));  // quad_perm 1,0,3,2
                }
                const int c = (16 * t + r) >> two;
                if (c < n && !(two && (r & 1))) {
                    f32x4* const s = own + rt.token[first + c] * Q + g;
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        const f32x4 v = s[4 * i], p = acc[i][t];
                        s[4 * i] = f32x4{v[0] + p[0], v[1] + p[1], v[2] + p[2], v[3] + p[3]};
                    }
                }
            }
            zero(acc);
        };
        stream_units<KIND, HB, NT, RX, RING>(
            s_ring + wave * RING, mine, r, g, acc,
            [&](int, uint32_t lds) {
                loader.load(rows, h, l_u, lds);
                --l_left;
                if (++l_u == units || l_left == 0) l_u = 0, ++l_item, select();
            },
            [&](int) {
                if (m_u == units) put(), m_u = 0, ++m_item;
                ++m_u;
            });
        put();
    });
    __syncthreads();
    for (int i = threadIdx.x; i < T * Q; i += 64 * W) {
        f32x4 v = sums[i];
#pragma unroll
        for (int w = 1; w < W; ++w) {
            const f32x4 o = sums[w * T * Q + i];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] += o[j];
        }
        const int64_t t = t0 + i / Q, d = d0 + 4 * (i % Q);
        if (d >= a.D) continue;
        if (a.splits > 1)
            a.part[(split * a.T + t) * (a.D / 4) + d / 4] = v;
        else
            store4(v, a.residual ? a.residual + t * a.ld_res + d : nullptr, a.out + t * a.ld_out + d, false, a.vec, 4);
    }
}

// The sums of the workgroups that shared columns, in their order.
__global__ __launch_bounds__(256) void moe_few_join_kernel(MoeFewArgs a) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, n = a.T * (a.D / 4);
    if (i >= n) return;
    f32x4 v = a.part[i];
    for (int p = 1; p < a.splits; ++p) {
        const f32x4 o = a.part[p * n + i];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] += o[j];
    }
    const int64_t t = i / (a.D / 4), d = 4 * (i % (a.D / 4));
    store4(v, a.residual ? a.residual + t * a.ld_res + d : nullptr, a.out + t * a.ld_out + d, false, a.vec, 4);
}

// The launchers below only say in `plan` what they would run where there is one.
template <int KIND, int NT, int RX, int W, int RING>
hipError_t mm(FewMmArgs a, hipStream_t stream, FewMmPlan* plan) {
    a.tiles = (a.N + 16 * NT - 1) / (16 * NT);
    if (plan) {
        *plan = {RX, NT, (a.tiles + 7) & ~(int64_t)7, 64 * W};
        return hipSuccess;
    }
    const dim3 grid((unsigned)((a.tiles + 7) & ~7), (unsigned)((a.T + RX - 1) / RX));
    hipLaunchKernelGGL((few_mm_kernel<KIND, UnitBytes<KIND, NT, RX, RING>::value, NT, RX, W, RING>), grid, dim3(64 * W), 0, stream,
                       a);
    return hipGetLastError();
}

template <int KIND>
hipError_t mm_kind(const FewMmArgs& a, hipStream_t stream, FewMmPlan* plan) {
    // Up to 16 rows, workgroups of 80 KiB, two on a CU.
    if (a.T <= 1) return mm<KIND, 1, 1, 8, 9728>(a, stream, plan);
    if (a.T <= 4) return mm<KIND, 1, 4, 8, 9728>(a, stream, plan);
    if (a.T <= 8) return mm<KIND, 1, 8, 8, 9728>(a, stream, plan);
    if (a.T <= 16) return mm<KIND, 1, 16, 4, 19200>(a, stream, plan);
    // Beside more, a workgroup fills its CU, and two tiles of columns at a time halve what is fetched of x: taken where one
    // would need a second round of the CUs.  64 rows of 5120 by e4m3 weights, one tile and two: 4096 columns 15.7 and 19.3
    // us, 4352 27.3 and 19.5, 6144 28.1 and 20.3, 8192 29.0 and 21.0, 16384 55 and 40; 128 rows of 2048: 2048 columns 7.4 and
    // 9.0, 2304 12.6 and 9.0.  (17 to 256 rows of 1024 to 5120, the other formats: the same side is the faster one.)
    const int64_t rows = a.T <= 32 ? 32 : 64, groups = (a.N + 15) / 16 * ((a.T + rows - 1) / rows);
    const bool wide = groups > kCus;
    if (a.T <= 32) return wide ? mm<KIND, 2, 32, 4, 40960>(a, stream, plan) : mm<KIND, 1, 32, 4, 40960>(a, stream, plan);
    return wide ? mm<KIND, 2, 64, 4, 40960>(a, stream, plan) : mm<KIND, 1, 64, 4, 40960>(a, stream, plan);
}

constexpr int kLds = 160 * 1024;  // of a CU

// Workgroups that share the units of 16 nt columns of the output: enough to
// give every CU one where a wave without sharing has 20 units and more (half a
// microsecond each; joining the shares costs four).
int down_splits(int64_t T, int64_t D, int64_t H, int64_t E, int64_t k, int nt, int waves) {
    const int64_t chunks = (T + kFewChunk - 1) / kFewChunk, tokens = T < kFewChunk ? T : kFewChunk;
    const int64_t groups = (D + 16 * nt - 1) / (16 * nt) * chunks, slots = tokens * k;
    const int64_t units = (slots < E ? slots : E) * ((H + 127) / 128);  // of a workgroup, about
    const int64_t wanted = kCus / groups, room = units / (10 * waves);
    const int64_t n = wanted < room ? wanted : room;
    return n < 1 ? 1 : n > kMaxSplits ? kMaxSplits : (int)n;
}

// NH, NT: tiles of h and of the output a wave takes at a time; W, RING of the
// three kernels.
template <int KIND, int RXMAX, int RING_U, int NH, int RING_T, int NT, int WD, int RING_D>
hipError_t moe(MoeFewArgs a, hipStream_t stream, MoeFewPlan* plan) {
    constexpr int PER = item_tokens(RXMAX), W = 4;
    const int64_t chunks = (a.T + kFewChunk - 1) / kFewChunk, tokens = a.T < kFewChunk ? a.T : kFewChunk;
    const int slots = (int)(tokens * a.k);
    a.items = (slots < a.E ? slots : a.E) + (tokens > PER ? slots / PER : 0);
    const int table = RXMAX == 1 ? 0 : RoutingLayout(a.E, slots, a.items).bytes;
    a.splits = down_splits(a.T, a.D, a.H, a.E, a.k, NT, WD);
    a.part = reinterpret_cast<f32x4*>(a.h + a.parts * a.T * a.k * a.H);
    // The waves of a workgroup share a tile (four microseconds of its own a workgroup, half a microsecond a unit and
    // wave), or each streams whole tiles: one token over 2 experts of 256 tiles and 5120 rows in 4 bits takes 12 us
    // shared, 64 tokens of a single e4m3 expert of 512 tiles and 5120 rows 52 shared and 37 by tiles, 32 tokens over 16
    // experts of 64 tiles and 2048 rows 19 and 28.
    constexpr int64_t kShared = kCus * (2 * W * RING_U <= kLds ? 2 : 1), kTiles = kCus * (2 * W * RING_T <= kLds ? 2 : 1);
    constexpr int kCodes = Unit<KIND, 128>::kCodes;
    const int64_t narrow = (a.H + 15) / 16, wide = (a.H + 16 * NH - 1) / (16 * NH), units = (a.D + kCodes - 1) / kCodes;
    const int64_t shared = (a.items * narrow + kShared - 1) / kShared * (8 + (units + W - 1) / W);
    const int64_t by_tiles = 8 + (a.items * wide + kTiles * W - 1) / (kTiles * W) * units * NH;
    if (plan) {
        *plan = {PER, a.items, by_tiles < shared ? NH : 0, kTiles * W, NT, a.splits};
        return hipSuccess;
    }
    if (by_tiles < shared) {
        a.tiles = wide;
        hipLaunchKernelGGL((moe_few_up_tiles_kernel<KIND, RXMAX, NH, W, RING_T>), dim3((unsigned)kTiles, (unsigned)chunks), dim3(64 * W),
                           table, stream, a);
    } else {
        a.tiles = narrow;
        const int64_t padded = (a.tiles + 7) & ~7;
        hipLaunchKernelGGL((moe_few_up_kernel<KIND, RXMAX, W, RING_U>), dim3((unsigned)(a.items * padded), (unsigned)chunks),
                           dim3(64 * W), table, stream, a);
    }
    hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    a.tiles = (a.D + 16 * NT - 1) / (16 * NT);
    hipLaunchKernelGGL((moe_few_down_kernel<KIND, RXMAX, NT, WD, RING_D>),
                       dim3((unsigned)(((a.tiles + 7) & ~7) * a.splits), (unsigned)chunks), dim3(64 * WD),
                       table + WD * tokens * 64 * NT, stream, a);
    err = hipGetLastError();
    if (a.splits == 1 || err != hipSuccess) return err;
    hipLaunchKernelGGL(moe_few_join_kernel, dim3((unsigned)((a.T * (a.D / 4) + 255) / 256)), dim3(256), 0, stream, a);
    return hipGetLastError();
}

template <int KIND>
hipError_t moe_kind(const MoeFewArgs& a, hipStream_t stream, MoeFewPlan* plan) {
    // Up to 8 tokens, workgroups of 80 KiB, two on a CU (from 5 on with longer rings for fewer waves in the second kernel:
    // 5 tokens through an FFN of 5120 and 8192 in e4m3 39 us, 43 with eight waves).
    if (a.T <= 1) return moe<KIND, 1, 19200, 1, 19200, 1, 8, 9728>(a, stream, plan);
    if (a.T <= 4) return moe<KIND, 4, 19200, 1, 19200, 1, 8, 9728>(a, stream, plan);
    if (a.T <= 8) return moe<KIND, 8, 19200, 1, 19200, 1, 4, 19200>(a, stream, plan);
    // Beside more tokens of an expert a wave takes two tiles at a time, which halves what it fetches of tokens, in rings
    // of a whole CU (64 tokens over 64 e2m1 experts of 2048, width 4096: 119 + 63 us, 153 + 95 with one).  In the second
    // kernel where one tile would need a second round of the CUs, or where workgroups that share the tiles fill them:
    // both kernels in us with one and two, a gated FFN of 8192 in e4m3 of 64 tokens, width 4096 54.9 and 58.8, 5120 85 and
    // 69, of 128 tokens, width 2048 54 and 58, 2560 78 and 66, 4096 95 and 81; 64 tokens over 16 experts of 1024, width 2560
    // 48 and 45 (three shares), 4096 64 and 63 (two).  Chunks count by their tokens (65 of them, width 2560, 16 experts: 59
    // and 65).  Where experts have more than 12 tokens, many have more than 16: items of 32 read their weights once (64
    // tokens of one e4m3 expert of 8192, width 5120: 37 + 30 us, 62 + 49 by items of 16).
    const int64_t tokens = a.T < kFewChunk ? a.T : kFewChunk;
    const int64_t work = a.D * (a.T > kFewChunk ? a.T : kFewChunk), round = kCus * 16 * kFewChunk;
    const bool wide = work > round || (2 * work > round && down_splits(a.T, a.D, a.H, a.E, a.k, 2, 4) > 1);
    const int slots = (int)(tokens * a.k), items = (slots < a.E ? slots : a.E) + slots / 16;
    const int table = RoutingLayout(a.E, slots, items).bytes + 512;
    if (tokens * a.k > 12 * a.E && tokens > 16) {
        if (wide) return moe<KIND, 32, 31104, 1, 33792, 2, 4, 25600>(a, stream, plan);
        return moe<KIND, 32, 31104, 1, 33792, 1, 4, 20992>(a, stream, plan);
    }
    if (tokens * a.k >= 5 * a.E) {
        if (wide && table + 4 * 38400 <= kLds) return moe<KIND, 16, 19200, 2, 38400, 2, 4, 25600>(a, stream, plan);
        return moe<KIND, 16, 19200, 2, 36864, 1, 8, 12800>(a, stream, plan);
    }
    if (table + 8 * (tokens * 64 + 15552) <= kLds) return moe<KIND, 16, 19200, 1, 19200, 1, 8, 15552>(a, stream, plan);
    return moe<KIND, 16, 19200, 1, 19200, 1, 8, 12800>(a, stream, plan);
}

}  // namespace

hipError_t launch_few_mm(const FewMmArgs& a, FewKind kind, hipStream_t stream, FewMmPlan* plan) {
    return kind == kFewE4m3 ? mm_kind<kFewE4m3>(a, stream, plan)
           : kind == kFewMx8 ? mm_kind<kFewMx8>(a, stream, plan) : mm_kind<kFewMx4>(a, stream, plan);
}

int64_t moe_few_shares_bytes(int64_t T, int64_t D, int64_t H, int64_t E, int64_t k) {
    int most = 1;
    for (int nt = 1; nt <= 2; ++nt) {
        const int n = down_splits(T, D, H, E, k, nt, nt == 1 ? 8 : 4);
        most = n > most ? n : most;
    }
    return most > 1 ? most * T * D * 4 : 0;
}

hipError_t launch_moe_few(const MoeFewArgs& a, FewKind kind, hipStream_t stream, MoeFewPlan* plan) {
    return kind == kFewE4m3 ? moe_kind<kFewE4m3>(a, stream, plan)
           : kind == kFewMx8 ? moe_kind<kFewMx8>(a, stream, plan) : moe_kind<kFewMx4>(a, stream, plan);
}

}  // namespace bs
