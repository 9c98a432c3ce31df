// C ABI of serving few tokens from quantized weights: host-side validation,
// then the launches on the caller's stream.  Contracts: include/bs.h.
#include "bs_check.h"
#include "bs_few.h"
#include "bs_moe.h"

using bs::aligned16;
using bs::hip_status;
using bs::kMaxLd;
using bs::ok;

namespace {

typedef long long ll;

constexpr int64_t kMaxI32 = 0x7fffffff;
constexpr int64_t kMaxTokens = (int64_t)1 << 21;   // 32768 chunks: the launch grid's second axis
constexpr int64_t kMaxThreads = 0xffffffffll;      // of a launch along one axis
constexpr int64_t kMaxScales = (int64_t)1 << 30;   // bytes of a matrix's scales: 32-bit offsets, past its end too

bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

#define CHECK(call)                   \
    do {                              \
        const bs_status st_ = (call); \
        if (st_ != BS_OK) return st_; \
    } while (0)

// Tokens [T, cols] bf16 whose rows are read 16 bytes at a time.
bs_status check_tokens(const char* fn, const void* x, int64_t cols, int64_t ld) {
    REQUIRE(x, BS_ERR_NULL, "x is NULL");
    REQUIRE(ld >= cols && ld < kMaxLd, BS_ERR_LAYOUT, "ld_x=%lld must be >= %lld columns and < 2^22", (ll)ld, (ll)cols);
    REQUIRE(aligned16(x) && ld % 8 == 0, BS_ERR_ALIGN, "x must be 16-byte aligned with ld_x %% 8 == 0");
    return BS_OK;
}

// Codes and scales of weights [N, K] (E of them, `name` and its scales).
bs_status check_weight(const char* fn, const char* name, bs_weight_kind kind, int64_t E, int64_t N, int64_t K,
                       const bs::FewWeight& w) {
    REQUIRE(w.q && w.s, BS_ERR_NULL, "%s and its scales must be non-NULL", name);
    if (kind == BS_WEIGHT_E4M3_128X128) {
        REQUIRE(N % 128 == 0 && K % 128 == 0, BS_ERR_SHAPE, "%s is %lld x %lld: both must be multiples of 128 (128x128 scales)",
                name, (ll)N, (ll)K);
    } else {
        REQUIRE(K % 32 == 0, BS_ERR_SHAPE, "%s has %lld columns: they must be a multiple of 32 (1x32 scales)", name, (ll)K);
    }
    const int64_t row = kind == BS_WEIGHT_MXFP4 ? K / 2 : K;
    REQUIRE(w.ld_q >= row && w.ld_q < kMaxLd, BS_ERR_LAYOUT, "ld of %s = %lld must be >= %lld bytes and < 2^22", name,
            (ll)w.ld_q, (ll)row);
    REQUIRE(aligned16(w.q) && w.ld_q % 16 == 0 && w.stride_q % 16 == 0, BS_ERR_ALIGN,
            "%s must be 16-byte aligned, its ld and stride multiples of 16", name);
    const int64_t cols = kind == BS_WEIGHT_E4M3_128X128 ? N / 128 : N;
    REQUIRE(w.ld_s >= cols, BS_ERR_LAYOUT, "ld of the scales of %s = %lld must be >= %lld (K-major)", name, (ll)w.ld_s,
            (ll)cols);
    const int64_t blocks = kind == BS_WEIGHT_E4M3_128X128 ? K / 128 : K / 32;
    REQUIRE(w.ld_s <= kMaxScales / (blocks > 8 ? blocks : 8) / (kind == BS_WEIGHT_E4M3_128X128 ? 4 : 1), BS_ERR_LAYOUT,
            "the scales of %s, %lld rows of %lld, must be below 2^30 bytes", name, (ll)blocks, (ll)w.ld_s);
    if (kind == BS_WEIGHT_E4M3_128X128)
        REQUIRE(aligned_to(w.s, 4), BS_ERR_ALIGN, "the scales of %s must be aligned to their type", name);
    else
        REQUIRE(aligned16(w.s) && w.ld_s % 16 == 0 && w.stride_s % 16 == 0, BS_ERR_ALIGN,
                "the scales of %s must be 16-byte aligned, their ld and stride multiples of 16", name);
    if (E > 1) REQUIRE(w.stride_q >= 0 && w.stride_s >= 0, BS_ERR_LAYOUT, "the strides of %s must not be negative", name);
    return BS_OK;
}

bs_status check_kind(const char* fn, bs_weight_kind kind) {
    REQUIRE(kind == BS_WEIGHT_E4M3_128X128 || kind == BS_WEIGHT_MXFP8 || kind == BS_WEIGHT_MXFP4, BS_ERR_MODE,
            "kind=%d must be BS_WEIGHT_E4M3_128X128, BS_WEIGHT_MXFP8 or BS_WEIGHT_MXFP4", (int)kind);
    return BS_OK;
}

bs::FewKind few_kind(bs_weight_kind kind) {
    return kind == BS_WEIGHT_E4M3_128X128 ? bs::kFewE4m3 : kind == BS_WEIGHT_MXFP8 ? bs::kFewMx8 : bs::kFewMx4;
}

}  // namespace

extern "C" {

bs_status bs_mx4_quant_1x32(const uint16_t* x, int64_t R, int64_t C, int64_t ld_x, uint8_t* q, int64_t ld_q, uint8_t* s,
                            int64_t ld_s, uint16_t* y, int64_t ld_y, hipStream_t stream) {
    static const char* fn = "bs_mx4_quant_1x32";
    REQUIRE(R >= 0 && R <= kMaxI32 && C >= 0, BS_ERR_SHAPE, "R=%lld must be in [0, 2^31) and C=%lld >= 0", (ll)R, (ll)C);
    REQUIRE(C % 32 == 0, BS_ERR_SHAPE, "C=%lld must be a multiple of 32 (1x32 blocks)", (ll)C);
    if (R == 0 || C == 0) return ok();
    REQUIRE(x && q && s, BS_ERR_NULL, "x, q and s must be non-NULL");
    REQUIRE(ld_x >= C && ld_x < kMaxLd, BS_ERR_LAYOUT, "ld_x=%lld must be >= C=%lld and < 2^22", (ll)ld_x, (ll)C);
    REQUIRE(aligned16(x) && ld_x % 8 == 0, BS_ERR_ALIGN, "x must be 16-byte aligned with ld_x %% 8 == 0");
    REQUIRE(ld_q >= C / 2 && ld_q < kMaxLd, BS_ERR_LAYOUT, "ld_q=%lld must be >= C / 2 = %lld bytes and < 2^22", (ll)ld_q,
            (ll)(C / 2));
    REQUIRE(aligned16(q) && ld_q % 16 == 0, BS_ERR_ALIGN, "q must be 16-byte aligned with ld_q %% 16 == 0");
    REQUIRE(ld_s >= R && ld_s % 16 == 0, BS_ERR_LAYOUT,
            "ld_s=%lld must be >= R=%lld and a multiple of 16 (s is K-major [C/32][ld_s] bytes)", (ll)ld_s, (ll)R);
    REQUIRE(aligned16(s), BS_ERR_ALIGN, "s must be 16-byte aligned");
    if (y) {
        REQUIRE(ld_y >= C && ld_y < kMaxLd, BS_ERR_LAYOUT, "ld_y=%lld must be >= C=%lld and < 2^22", (ll)ld_y, (ll)C);
        REQUIRE(aligned16(y) && ld_y % 8 == 0, BS_ERR_ALIGN, "y must be 16-byte aligned with ld_y %% 8 == 0");
    }
    const int64_t tiles = (R + 31) / 32 * ((C + 255) / 256);  // of 256 threads; launched in eights
    REQUIRE((tiles + 7) / 8 * 8 * 256 <= kMaxThreads, BS_ERR_SHAPE, "%lld x %lld is more than one launch takes", (ll)R, (ll)C);
    return hip_status(bs::launch_mx4_quant({x, R, C, ld_x, q, ld_q, s, ld_s, y, ld_y, 0}, stream), fn);
}

bs_status bs_few_mm(bs_weight_kind kind, int64_t T, int64_t N, int64_t K, const uint16_t* x, int64_t ld_x, const uint8_t* w,
                    int64_t ld_w, const void* s, int64_t ld_s, const uint16_t* residual, int64_t ld_res, void* out,
                    int64_t ld_out, bs_dtype out_dtype, hipStream_t stream) {
    static const char* fn = "bs_few_mm";
    CHECK(check_kind(fn, kind));
    REQUIRE(out_dtype == BS_OUT_BF16 || out_dtype == BS_OUT_F32, BS_ERR_MODE, "out_dtype=%d must be BF16 or F32",
            (int)out_dtype);
    REQUIRE(T >= 0 && T <= kMaxTokens, BS_ERR_SHAPE, "T=%lld must be in [0, 2^21]", (ll)T);
    REQUIRE(N >= 0 && N <= kMaxI32 && K >= 1, BS_ERR_SHAPE, "N=%lld must be in [0, 2^31) and K=%lld >= 1", (ll)N, (ll)K);
    if (T == 0 || N == 0) return ok();
    CHECK(check_tokens(fn, x, K, ld_x));
    bs::FewMmArgs a{};
    a.w = {w, 0, ld_w, s, 0, ld_s};
    CHECK(check_weight(fn, "w", kind, 1, N, K, a.w));
    const bool f32 = out_dtype == BS_OUT_F32;
    REQUIRE(out, BS_ERR_NULL, "out is NULL");
    REQUIRE(ld_out >= N, BS_ERR_LAYOUT, "ld_out=%lld < N=%lld: out is row-major [T, N]", (ll)ld_out, (ll)N);
    REQUIRE(aligned_to(out, f32 ? 4 : 2), BS_ERR_ALIGN, "out must be aligned to its type");
    if (residual) {
        REQUIRE(ld_res >= N, BS_ERR_LAYOUT, "ld_res=%lld < N=%lld: the residual is row-major [T, N]", (ll)ld_res, (ll)N);
        REQUIRE(aligned_to(residual, 2), BS_ERR_ALIGN, "residual must be aligned to its type");
    }
    a.T = T; a.N = N; a.K = K; a.x = x; a.ld_x = ld_x;
    a.residual = residual; a.ld_res = ld_res; a.out = out; a.ld_out = ld_out; a.f32 = f32;
    a.vec = N % 4 == 0 && ld_out % 4 == 0 && aligned_to(out, f32 ? 16 : 8) &&
            (!residual || (ld_res % 4 == 0 && aligned_to(residual, 8)));
    bs::FewMmPlan plan;
    CHECK(hip_status(bs::launch_few_mm(a, few_kind(kind), stream, &plan), fn));
    REQUIRE(plan.workgroups * plan.threads <= kMaxThreads, BS_ERR_SHAPE, "N=%lld with T=%lld is more than one launch takes", (ll)N,
            (ll)T);
    return hip_status(bs::launch_few_mm(a, few_kind(kind), stream), fn);
}

int64_t bs_moe_few_workspace_bytes(int64_t T, int64_t D, int64_t H, int64_t E, int64_t k) {
    if (T < 0 || T > kMaxTokens || D < 0 || D > bs::kMaxFewDim || H < 0 || H > bs::kMaxFewDim || E < 1 || E > bs::kMaxExperts ||
        k < 1 || k > bs::kMaxTopK)
        return 0;
    return T == 0 || D == 0 ? 0 : T * k * H * 2 + bs::moe_few_shares_bytes(T, D, H, E, k);
}

int64_t bs_moe_few_full_workspace_bytes(int64_t T, int64_t D, int64_t H, int64_t E, int64_t k) {
    const int64_t n = bs_moe_few_workspace_bytes(T, D, H, E, k);
    return n > 0 && T <= bs::kTwoParts ? n + T * k * H * 2 : n;
}

bs_status bs_moe_few(bs_weight_kind kind, int64_t T, int64_t D, int64_t H, int64_t E, int64_t k, const uint16_t* x,
                     int64_t ld_x, const int32_t* idx, const float* w, const uint8_t* w12, int64_t stride_w12,
                     int64_t ld_w12, const void* s12, int64_t stride_s12, int64_t ld_s12, const uint8_t* out_proj,
                     int64_t stride_wo, int64_t ld_wo, const void* s_out, int64_t stride_so, int64_t ld_so,
                     const uint16_t* residual, int64_t ld_res, uint16_t* out, int64_t ld_out, void* workspace,
                     int64_t workspace_bytes, hipStream_t stream) {
    static const char* fn = "bs_moe_few";
    CHECK(check_kind(fn, kind));
    REQUIRE(T >= 0 && T <= kMaxTokens, BS_ERR_SHAPE, "T=%lld must be in [0, 2^21]", (ll)T);
    REQUIRE(E >= 1 && E <= bs::kMaxExperts, BS_ERR_SHAPE, "E=%lld must be in [1, 1024]", (ll)E);
    REQUIRE(k >= 1 && k <= E && k <= bs::kMaxTopK, BS_ERR_SHAPE, "k=%lld must be in [1, min(E, 32)]", (ll)k);
    const int64_t step = kind == BS_WEIGHT_E4M3_128X128 ? 128 : 32;
    REQUIRE(D >= 1 && D <= bs::kMaxFewDim && D % step == 0 && H >= 1 && H <= bs::kMaxFewDim && H % step == 0, BS_ERR_SHAPE,
            "D=%lld and H=%lld must be multiples of %lld, at least that and at most 262144", (ll)D, (ll)H, (ll)step);
    REQUIRE(idx || (E == 1 && k == 1), BS_ERR_NULL, "idx may be NULL only with E = 1 and k = 1");
    if (T == 0) return ok();
    CHECK(check_tokens(fn, x, D, ld_x));
    bs::MoeFewArgs a{};
    a.w12 = {w12, stride_w12, ld_w12, s12, stride_s12, ld_s12};
    a.wo = {out_proj, stride_wo, ld_wo, s_out, stride_so, ld_so};
    CHECK(check_weight(fn, "w12", kind, E, 2 * H, D, a.w12));
    CHECK(check_weight(fn, "out_proj", kind, E, D, H, a.wo));
    REQUIRE(aligned_to(idx, 4) && aligned_to(w, 4), BS_ERR_ALIGN, "idx and w must be aligned to their types");
    REQUIRE(out, BS_ERR_NULL, "out is NULL");
    REQUIRE(ld_out >= D, BS_ERR_LAYOUT, "ld_out=%lld < D=%lld: out is row-major [T, D]", (ll)ld_out, (ll)D);
    REQUIRE(aligned_to(out, 2), BS_ERR_ALIGN, "out must be aligned to its type");
    if (residual) {
        REQUIRE(ld_res >= D, BS_ERR_LAYOUT, "ld_res=%lld < D=%lld: the residual is row-major [T, D]", (ll)ld_res, (ll)D);
        REQUIRE(aligned_to(residual, 2), BS_ERR_ALIGN, "residual must be aligned to its type");
    }
    REQUIRE(workspace && workspace_bytes >= bs_moe_few_workspace_bytes(T, D, H, E, k), BS_ERR_SHAPE,
            "the workspace has %lld bytes: this needs %lld", (ll)(workspace ? workspace_bytes : 0),
            (ll)bs_moe_few_workspace_bytes(T, D, H, E, k));
    REQUIRE(aligned16(workspace), BS_ERR_ALIGN, "workspace must be 16-byte aligned");
    a.T = T; a.D = D; a.H = H; a.E = (int32_t)E; a.k = (int32_t)k;
    a.x = x; a.ld_x = ld_x; a.idx = idx; a.w = w;
    a.residual = residual; a.ld_res = ld_res; a.out = out; a.ld_out = ld_out;
    a.vec = ld_out % 4 == 0 && aligned_to(out, 8) && (!residual || (ld_res % 4 == 0 && aligned_to(residual, 8)));
    a.h = static_cast<uint16_t*>(workspace);
    a.parts = T <= bs::kTwoParts && workspace_bytes >= bs_moe_few_full_workspace_bytes(T, D, H, E, k) ? 2 : 1;
    return hip_status(bs::launch_moe_few(a, few_kind(kind), stream), fn);
}

bs_status bs_diag_few_mm_plan(bs_weight_kind kind, int64_t T, int64_t N, int64_t K, int64_t* plan) {
    static const char* fn = "bs_diag_few_mm_plan";
    CHECK(check_kind(fn, kind));
    REQUIRE(plan, BS_ERR_NULL, "plan is NULL");
    REQUIRE(T >= 1 && T <= kMaxTokens && N >= 1 && N <= kMaxI32 && K >= 1, BS_ERR_SHAPE,
            "T=%lld must be in [1, 2^21], N=%lld in [1, 2^31), K=%lld >= 1", (ll)T, (ll)N, (ll)K);
    bs::FewMmArgs a{};
    a.T = T; a.N = N; a.K = K;
    bs::FewMmPlan p;
    const bs_status st = hip_status(bs::launch_few_mm(a, few_kind(kind), nullptr, &p), fn);
    if (st == BS_OK) plan[0] = p.rows, plan[1] = p.tiles, plan[2] = p.workgroups, plan[3] = p.threads;
    return st;
}

bs_status bs_diag_moe_few_plan(bs_weight_kind kind, int64_t T, int64_t D, int64_t H, int64_t E, int64_t k, int64_t* plan) {
    static const char* fn = "bs_diag_moe_few_plan";
    CHECK(check_kind(fn, kind));
    REQUIRE(plan, BS_ERR_NULL, "plan is NULL");
    REQUIRE(T >= 1 && D >= 1 && H >= 1 && bs_moe_few_workspace_bytes(T, D, H, E, k) > 0 && k <= E, BS_ERR_SHAPE,
            "T=%lld, D=%lld, H=%lld, E=%lld or k=%lld is out of range", (ll)T, (ll)D, (ll)H, (ll)E, (ll)k);
    bs::MoeFewArgs a{};
    a.T = T; a.D = D; a.H = H; a.E = (int32_t)E; a.k = (int32_t)k;
    bs::MoeFewPlan p;
    const bs_status st = hip_status(bs::launch_moe_few(a, few_kind(kind), nullptr, &p), fn);
    if (st == BS_OK)
        plan[0] = p.tokens, plan[1] = p.items, plan[2] = p.up_tiles, plan[3] = p.up_waves, plan[4] = p.out_tiles, plan[5] = p.splits;
    return st;
}

}  // extern "C"
