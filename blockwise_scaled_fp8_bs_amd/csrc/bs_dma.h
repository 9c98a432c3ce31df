// Copies from global memory into LDS that bypass the registers (buffer loads
// with the lds bit), shared by the kernels that stream their operands
// (bs_gemm.hip, bs_few.hip).  gfx950 only.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace bs {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// Raw buffer resource (gfx9 layout): offsets at or beyond `bytes` read as zero.
__device__ __forceinline__ i32x4 make_rsrc(const void* base, int64_t bytes) {
    const uint64_t a = reinterpret_cast<uint64_t>(base);
    const int32_t n = bytes > 0x7fffffff ? 0x7fffffff : (bytes < 0 ? 0 : (int32_t)bytes);
    return i32x4{(int32_t)(uint32_t)a, (int32_t)((a >> 32) & 0xffffu), n, 0x00020000};
}

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
    return (uint32_t)(size_t)(__attribute__((address_space(3))) const char*)p;
}

// Global -> LDS copies (buffer_load ... lds): lane i's bytes land at
// lds_base + i * size.  Issued through inline asm so that the compiler does
// not wait for them before every LDS read of the other stage (it cannot tell
// the two stages apart); the kernel waits for them explicitly (vmcnt(0))
// before the barrier that publishes the stage.
// Byte address = buffer base + voffset (per lane) + soffset (uniform).
//
// The compiler keeps the wait states that gfx9 asks of software for its own
// instructions, not for those in inline asm: one between a write of m0 and a
// load into LDS, five between a vector instruction's write of a scalar register
// (v_readfirstlane, and v_readlane where scalar registers were spilled) and a
// vector memory instruction that reads it.  The operands are there before the
// asm begins, so s_mov_b32 and the four states of s_nop 3 are both.
__device__ __forceinline__ void dma16(i32x4 rs, uint32_t lds_base, int voffset, int soffset) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :: "s"(__builtin_amdgcn_readfirstlane(lds_base)), "v"(voffset), "s"(rs),
                    "s"(__builtin_amdgcn_readfirstlane(soffset)) : "memory");
}

__device__ __forceinline__ void dma4(i32x4 rs, uint32_t lds_base, int voffset, int soffset) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dword %1, %2, %3 offen lds"
                 :: "s"(__builtin_amdgcn_readfirstlane(lds_base)), "v"(voffset), "s"(rs),
                    "s"(__builtin_amdgcn_readfirstlane(soffset)) : "memory");
}

// Two of them, of two buffers, at soffset + step each, that share the five
// states; two of them add up the offsets (the MoE wgrad 1 % faster than with
// both added up before, in a loop that issues little else beside its MFMAs).
__device__ __forceinline__ void dma16_pair(i32x4 rs0, uint32_t lds0, int voffset0, int step0, i32x4 rs1, uint32_t lds1,
                                           int voffset1, int step1, int soffset) {
    int so0, so1;
    asm volatile("s_add_u32 %0, %8, %6\n\ts_add_u32 %1, %8, %7\n\ts_mov_b32 m0, %2\n\ts_nop 1\n\t"
                 "buffer_load_dwordx4 %4, %9, %0 offen lds\n\t"
                 "s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %5, %10, %1 offen lds"
                 : "=&s"(so0), "=&s"(so1)
                 : "s"(__builtin_amdgcn_readfirstlane(lds0)), "s"(__builtin_amdgcn_readfirstlane(lds1)), "v"(voffset0),
                   "v"(voffset1), "s"(__builtin_amdgcn_readfirstlane(step0)), "s"(__builtin_amdgcn_readfirstlane(step1)),
                   "s"(__builtin_amdgcn_readfirstlane(soffset)), "s"(rs0), "s"(rs1)
                 : "memory", "scc");
}

// N of them from one buffer and uniform offset, 1 KiB after the other in LDS:
// the five states once, then one after each step of m0.
template <int N>
__device__ __forceinline__ void dma16_run(i32x4 rs, uint32_t lds_base, const int* voffset, int soffset) {
    static_assert(N == 1 || N == 2 || N % 4 == 0, "in fours");
#define BS_DMA_NEXT "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\tbuffer_load_dwordx4 "
    const uint32_t m0 = __builtin_amdgcn_readfirstlane(lds_base);
    const int so = __builtin_amdgcn_readfirstlane(soffset);
    if constexpr (N == 1) {
        dma16(rs, lds_base, voffset[0], soffset);
    } else if constexpr (N == 2) {
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %3, %4 offen lds\n\t"
                     BS_DMA_NEXT "%2, %3, %4 offen lds"
                     :: "s"(m0), "v"(voffset[0]), "v"(voffset[1]), "s"(rs), "s"(so) : "memory", "scc");
    } else {
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %5, %6 offen lds\n\t"
                     BS_DMA_NEXT "%2, %5, %6 offen lds\n\t"
                     BS_DMA_NEXT "%3, %5, %6 offen lds\n\t"
                     BS_DMA_NEXT "%4, %5, %6 offen lds"
                     :: "s"(m0), "v"(voffset[0]), "v"(voffset[1]), "v"(voffset[2]), "v"(voffset[3]), "s"(rs), "s"(so)
                     : "memory", "scc");
        if constexpr (N > 4) dma16_run<N - 4>(rs, lds_base + 4096, voffset + 4, soffset);
    }
#undef BS_DMA_NEXT
}

__device__ __forceinline__ void wait_dma() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

}  // namespace bs
