// Dispatch and combine of an MoE layer for gfx950: the stable sort of the
// routed slots by expert, the gather of their rows fused with the 1x128
// quantizer, and the weighted sum back into token order with its gradients.
#include "bs_moe.h"
#include "bs_tile.h"

namespace bs {

namespace {

// ---- plan: a stable counting sort of the slots (token, choice) by expert ----
// One block sorts 512 * chunks consecutive slots; its 8 waves own consecutive
// stretches, so that (block, wave, chunk, lane) is slot order.  Within a
// chunk of 64 slots the lanes with the same expert are found with one ballot
// per bit of the expert index; a slot's rank is its expert's running count
// plus the matching lanes below it.  No order depends on an atomic: the
// atomics only count.  Bound by latency: 192 slots of 64 experts 4.2 us (one
// launch), 128000 slots of 8 experts 5.6 us for the counts and 7.3 us for the
// places.
constexpr int kPlanThreads = 512;
constexpr int kPlanWaves = kPlanThreads / 64;

// Rows of a group; unsigned, since the sum may pass 2^31 where its result does not.
__device__ __forceinline__ int32_t padded(int32_t slots, int32_t align) {
    return (int32_t)(((uint32_t)slots + (uint32_t)align - 1u) / (uint32_t)align * (uint32_t)align);
}

__global__ __launch_bounds__(kPlanThreads) void plan_hist_kernel(PlanArgs a) {
    __shared__ int32_t cnt[kMaxExperts];
    for (int e = threadIdx.x; e < a.E; e += kPlanThreads) cnt[e] = 0;
    __syncthreads();
    const int64_t s0 = (int64_t)blockIdx.x * kPlanThreads * a.chunks;
    for (int c = 0; c < a.chunks; ++c) {
        const int64_t s = s0 + (int64_t)c * kPlanThreads + threadIdx.x;
        if (s < a.n) {
            const int32_t e = a.idx[s];
            if (e >= 0 && e < a.E) atomicAdd(&cnt[e], 1);
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += kPlanThreads) a.hist[(int64_t)blockIdx.x * a.E + e] = cnt[e];
}

__global__ __launch_bounds__(kPlanThreads) void plan_place_kernel(PlanArgs a) {
    extern __shared__ int32_t s_plan[];
    const int E = a.E;
    int32_t* const tot = s_plan;       // [E] slots of each expert
    int32_t* const pre = s_plan + E;   // [E] those of the blocks before this one
    int32_t* const start = pre + E;    // [E] first row of each group
    int32_t* const cnt = start + E;    // [waves][E]
    __shared__ int32_t s_total;

    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int64_t n = a.n;
    const int64_t w0 = (int64_t)blockIdx.x * kPlanThreads * a.chunks + (int64_t)wave * 64 * a.chunks;

    for (int i = t; i < (3 + kPlanWaves) * E; i += kPlanThreads) s_plan[i] = 0;
    __syncthreads();
    // slots of each expert per wave of this block
    for (int c = 0; c < a.chunks; ++c) {
        const int64_t s = w0 + c * 64 + lane;
        const int32_t e = s < n ? a.idx[s] : -1;
        if (e >= 0 && e < E) atomicAdd(&cnt[wave * E + e], 1);
    }
    // totals over all blocks and over those before this one
    if (a.blocks > 1) {
        int ep = 1;
        while (ep < E && ep < kPlanThreads) ep <<= 1;
        const int parts = kPlanThreads / ep, part = t / ep;
        for (int e = t % ep; e < E; e += ep) {
            int32_t all = 0, before = 0;
            for (int b = part; b < a.blocks; b += parts) {
                const int32_t h = a.hist[(int64_t)b * E + e];
                all += h;
                before += b < (int)blockIdx.x ? h : 0;
            }
            if (all) atomicAdd(&tot[e], all);
            if (before) atomicAdd(&pre[e], before);
        }
    }
    __syncthreads();
    if (a.blocks == 1) {
        for (int e = t; e < E; e += kPlanThreads) {
            int32_t all = 0;
            for (int w = 0; w < kPlanWaves; ++w) all += cnt[w * E + e];
            tot[e] = all;
        }
        __syncthreads();
    }
    // first rows of the padded groups: a scan by one wave, consecutive experts per lane
    if (wave == 0) {
        const int per = (E + 63) / 64;
        int32_t own = 0;
        for (int i = 0; i < per; ++i) {
            const int e = lane * per + i;
            if (e < E) own += padded(tot[e], a.align);
        }
        int32_t upto = own;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int32_t x = __shfl_up(upto, d);
            if (lane >= d) upto += x;
        }
        int32_t at = upto - own;
        for (int i = 0; i < per; ++i) {
            const int e = lane * per + i;
            if (e < E) {
                start[e] = at;
                at += padded(tot[e], a.align);
                if (blockIdx.x == 0) {
                    a.group_end[e] = at;
                    a.counts[e] = tot[e];
                }
            }
        }
        if (lane == 63) s_total = upto;
    }
    __syncthreads();
    // each wave's next row of each expert
    for (int e = t; e < E; e += kPlanThreads) {
        int32_t at = start[e] + pre[e];
        for (int w = 0; w < kPlanWaves; ++w) {
            const int32_t c = cnt[w * E + e];
            cnt[w * E + e] = at;
            at += c;
        }
    }
    __syncthreads();
    int bits = 0;
    while ((1 << bits) < E) ++bits;
    for (int c = 0; c < a.chunks; ++c) {
        const int64_t s = w0 + c * 64 + lane;
        const int32_t e = s < n ? a.idx[s] : -1;
        const bool routed = e >= 0 && e < E;
        uint64_t same = __ballot(routed);
        for (int b = 0; b < bits; ++b) {
            const bool bit = (e >> b) & 1;
            const uint64_t v = __ballot(bit);
            same &= bit ? v : ~v;
        }
        int32_t row = -1;
        const int leader = same ? __builtin_ctzll(same) : lane;
        int32_t first = 0;
        if (routed && lane == leader) first = atomicAdd(&cnt[wave * E + e], (int32_t)__popcll(same));
        first = __shfl(first, leader);
        if (routed) row = first + (int32_t)__popcll(same & ((1ull << lane) - 1));
        if (s < n) {
            a.slot_row[s] = row;
            if (row >= 0 && row < a.M) a.row_slot[row] = (int32_t)s;
        }
    }
    // rows that no slot takes: the padding of this block's share of the groups, and of the end
    for (int e = blockIdx.x + wave * a.blocks; e < E; e += a.blocks * kPlanWaves) {
        const int32_t from = start[e] + tot[e];
        const int32_t to = start[e] + padded(tot[e], a.align);
        for (int32_t r = from + lane; r < to; r += 64)
            if (r < a.M) a.row_slot[r] = -1;
    }
    for (int64_t r = s_total + (int64_t)blockIdx.x * kPlanThreads + t; r < a.M; r += (int64_t)a.blocks * kPlanThreads)
        a.row_slot[r] = -1;
}

constexpr int kGatherSpan = 4;

// ---- gather fused with the 1x128 quantizer ----
// Row r of the result is row row_slot[r] / k of x (times w[row_slot[r]]), zero
// where the slot is negative.  As the quantizer's one-workgroup-per-tile form,
// with the tile's rows taken from wherever their tokens lie.  Bound by HBM: at
// 128000 slots of 64000 tokens of 5120 in rows and columns 437 us (1.28 GB read,
// half of it out of the last-level cache, 1.36 GB written: 6.0 TB/s), 450
// weighted, 297 in rows alone, 425 to bf16 (455, 472, 306 and 430 on another
// card); with the blocks of rows outermost, so that every slot's row
// comes from HBM, 522, 525 and 367.  With one slot a token nothing is read
// twice: 526 that way, 542 the other.
// NEAR: x within 2 GiB, its rows addressed by 32-bit offsets into one buffer
// (absent rows past its end, where loads give zeros): registers for four waves
// on a SIMD instead of three.
template <bool ROW, bool COL, bool W, bool NEAR>
__global__ __launch_bounds__(kThreads) void moe_gather_quant_kernel(GatherArgs a, int32_t span) {
    __shared__ float s_colmax[4][kTile];
    __shared__ __attribute__((aligned(16))) uint8_t s_tr[COL ? kTile * kTile : 16];

    const int t = threadIdx.x;
    const int tr = t >> 4, tc = t & 15;
    const int wave = t >> 6;
    const int col_tiles = (int)(a.D / kTile);
    // with several slots a token all row blocks of one strip of columns before
    // the next strip: its rows are read again, by other experts' blocks, while
    // the strip is still in the last-level cache
    const unsigned blocks = (unsigned)((a.M + kTile - 1) / kTile), strips = (unsigned)((col_tiles + span - 1) / span);
    const unsigned rb = a.k > 1 ? blockIdx.x % blocks : blockIdx.x / strips;
    const unsigned strip = a.k > 1 ? blockIdx.x / blocks : blockIdx.x % strips;
    const int64_t r0 = (int64_t)rb * kTile;
    const int first = (int)strip * span;
    const int last = first + span < col_tiles ? first + span : col_tiles;
    const int64_t rows = (a.M - r0) < kTile ? (a.M - r0) : kTile;
    const int64_t n = a.T * a.k;

    const __amdgpu_buffer_rsrc_t rx = rsrc(a.x, NEAR ? a.T * a.ld_x * 2 : 0);
    uint32_t off[8];
    const uint16_t* src[8];
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t r = r0 + 8 * tr + i;
        const int32_t slot = r < a.M ? a.row_slot[r] : -1;
        if (NEAR) off[i] = 0x80000000u;
        else src[i] = nullptr;
        if (W) w[i] = 0.f;
        if (slot >= 0 && slot < n) {
            const uint32_t tok = a.k_mul ? __umulhi((uint32_t)slot, a.k_mul) >> a.k_shift : (uint32_t)slot;
            if (NEAR) off[i] = tok * (uint32_t)(a.ld_x * 2) + 16 * tc;
            else src[i] = a.x + (int64_t)tok * a.ld_x + 8 * tc;
            if (W) w[i] = a.w[slot];
        }
    }
    for (int ct = first; ct < last; ++ct) {
        const int64_t c0 = (int64_t)ct * kTile;
        Raw raw;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (NEAR) {
                const u32x4 v =
                    __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rx, (int)off[i], (int)(c0 * 2), 0));
                raw.v[i] = make_uint4(v[0], v[1], v[2], v[3]);
            } else {
                raw.v[i] = src[i] != nullptr ? *reinterpret_cast<const uint4*>(src[i] + c0) : make_uint4(0, 0, 0, 0);
            }
        }
        TileRegs tl;
        unpack_tile(raw, tl);
        if (W) {
            // the product stays in fp32: what is quantized is not rounded to bf16 first
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) tl.f[i][j] *= w[i];
        }
        if (a.y != nullptr) {
            if (W) pack_tile(tl, raw);
            store_raw(raw, a.y + r0 * a.ld_y + c0, a.ld_y, rows, tr, tc);
        }
        if (ROW)
            quant_tile_rows(tl, rows, a.q_row + r0 * a.ld_qr + c0, a.ld_qr, a.s_row + (c0 / kTile) * a.ld_sr + r0,
                            tr, tc);
        // its two barriers also part one tile's LDS reads from the next one's writes
        if (COL)
            quant_tile_cols(tl, a.q_col + c0 * a.ld_qc + r0, a.ld_qc, a.s_col + (r0 / kTile) * a.ld_sc + c0,
                            s_colmax, s_tr, tr, tc, wave);
    }
}

// ---- combine ----
// One thread per token and 16 bytes of its row: the k rows of y are read at
// once, the sum is kept in fp32 in the order of the slots and rounded once.
// Bound by HBM: 64000 tokens of 2 slots, 5120 columns and a residual 442 us
// (2.62 GB, 5.9 TB/s).
__global__ __launch_bounds__(kThreads) void moe_combine_kernel(CombineArgs a, uint32_t nchunk) {
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t tok = i / nchunk;
    if (tok >= a.T) return;
    const int64_t c = (i - tok * nchunk) * 8;
    float acc[8];
    if (a.residual != nullptr) {
        unpack8(*reinterpret_cast<const uint4*>(a.residual + tok * a.ld_res + c), acc);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] = 0.f;
    }
    for (int j0 = 0; j0 < a.k; j0 += 4) {
        uint4 v[4];
        float w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = make_uint4(0, 0, 0, 0);
            w[j] = 0.f;
            if (j0 + j < a.k) {
                const int32_t row = a.slot_row[tok * a.k + j0 + j];
                if (row >= 0 && row < a.M) {
                    v[j] = *reinterpret_cast<const uint4*>(a.y + row * a.ld_y + c);
                    w[j] = a.w != nullptr ? a.w[tok * a.k + j0 + j] : 1.f;
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float f[8];
            unpack8(v[j], f);
#pragma unroll
            for (int q = 0; q < 8; ++q) acc[q] = __builtin_fmaf(w[j], f[q], acc[q]);
        }
    }
    *reinterpret_cast<uint4*>(a.out + tok * a.ld_out + c) =
        make_uint4(pack_bf16(acc[0], acc[1]), pack_bf16(acc[2], acc[3]), pack_bf16(acc[4], acc[5]),
                   pack_bf16(acc[6], acc[7]));
}

// dw[t, j] = <dout[t], y[slot_row[t, j]]>: one wave per token, dout read once
// for four slots at a time.  Bound by HBM: at those sizes 333 us (1.97 GB,
// 5.9 TB/s).
__global__ __launch_bounds__(kThreads) void moe_combine_dw_kernel(CombineDwArgs a) {
    const int lane = threadIdx.x & 63;
    const int64_t tok = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
    if (tok >= a.T) return;
    for (int j0 = 0; j0 < a.k; j0 += 4) {
        const uint16_t* p[4];
        float acc[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            acc[j] = 0.f;
            p[j] = nullptr;
            if (j0 + j < a.k) {
                const int32_t row = a.slot_row[tok * a.k + j0 + j];
                if (row >= 0 && row < a.M) p[j] = a.y + row * a.ld_y;
            }
        }
        for (int64_t c = lane * 8; c < a.D; c += 512) {
            float d[8];
            unpack8(*reinterpret_cast<const uint4*>(a.dout + tok * a.ld_dout + c), d);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (p[j] != nullptr) {
                    float f[8];
                    unpack8(*reinterpret_cast<const uint4*>(p[j] + c), f);
#pragma unroll
                    for (int q = 0; q < 8; ++q) acc[j] = __builtin_fmaf(d[q], f[q], acc[j]);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
            for (int s = 1; s < 64; s <<= 1) acc[j] += __shfl_xor(acc[j], s);
            if (lane == 0 && j0 + j < a.k) a.dw[tok * a.k + j0 + j] = acc[j];
        }
    }
}

}  // namespace

void plan_blocks(int64_t n, int32_t* blocks, int32_t* chunks) {
    // up to 8192 slots one block sorts alone (one launch); beyond, at most
    // about 128 blocks, whose histograms every block adds up by itself
    int64_t c = 1;
    if (n <= 16 * kPlanThreads) {
        c = (n + kPlanThreads - 1) / kPlanThreads;
    } else {
        while ((n + c * kPlanThreads - 1) / (c * kPlanThreads) > 128) c *= 2;
    }
    if (c < 1) c = 1;
    *chunks = (int32_t)c;
    const int64_t b = (n + c * kPlanThreads - 1) / (c * kPlanThreads);
    *blocks = (int32_t)(b < 1 ? 1 : b);
}

hipError_t launch_plan(const PlanArgs& a, hipStream_t stream) {
    if (a.blocks > 1)
        hipLaunchKernelGGL(plan_hist_kernel, dim3(a.blocks), dim3(kPlanThreads), 0, stream, a);
    const size_t lds = (size_t)(3 + kPlanWaves) * a.E * sizeof(int32_t);
    hipLaunchKernelGGL(plan_place_kernel, dim3(a.blocks), dim3(kPlanThreads), lds, stream, a);
    return hipGetLastError();
}

hipError_t launch_gather(const GatherArgs& a, hipStream_t stream) {
    const int64_t blocks = (a.M + kTile - 1) / kTile, tiles = a.D / kTile;
    // several column tiles per workgroup share one reading of the row list (at
    // 1007 x 40 tiles: 455 us with 4, 500 with 1, 457 with 2, 476 with 8) where
    // that still leaves a few workgroups for every place on the GPU
    const int span = blocks * tiles >= 4 * kGatherSpan * 1024 ? kGatherSpan : 1;
    const dim3 grid((unsigned)(blocks * ((tiles + span - 1) / span))), block(kThreads);
    const bool row = a.q_row != nullptr, col = a.q_col != nullptr;
    const bool near = a.T * a.ld_x * 2 < (int64_t)0x7fffffff;
#define BS_GATHER_W(R, C, W)                                                                                        \
    if (near) hipLaunchKernelGGL((moe_gather_quant_kernel<R, C, W, true>), grid, block, 0, stream, a, span);        \
    else hipLaunchKernelGGL((moe_gather_quant_kernel<R, C, W, false>), grid, block, 0, stream, a, span);
#define BS_GATHER(R, C)                             \
    if (a.w != nullptr) { BS_GATHER_W(R, C, true) } \
    else { BS_GATHER_W(R, C, false) }
    if (row && col) { BS_GATHER(true, true) }
    else if (row) { BS_GATHER(true, false) }
    else if (col) { BS_GATHER(false, true) }
    else { BS_GATHER(false, false) }
#undef BS_GATHER
#undef BS_GATHER_W
    return hipGetLastError();
}

hipError_t launch_combine(const CombineArgs& a, hipStream_t stream) {
    const uint32_t nchunk = (uint32_t)(a.D / 8);
    const int64_t blocks = (a.T * nchunk + kThreads - 1) / kThreads;
    hipLaunchKernelGGL(moe_combine_kernel, dim3((unsigned)blocks), dim3(kThreads), 0, stream, a, nchunk);
    return hipGetLastError();
}

hipError_t launch_combine_dw(const CombineDwArgs& a, hipStream_t stream) {
    const int64_t blocks = (a.T + kThreads / 64 - 1) / (kThreads / 64);
    hipLaunchKernelGGL(moe_combine_dw_kernel, dim3((unsigned)blocks), dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace bs
