// C ABI around the experts' products of an MoE block: host-side validation,
// then the launches on the caller's stream.  Contracts: include/bs.h.
#include <cmath>

#include "bs_check.h"
#include "bs_moe.h"
#include "bs_norm.h"

using bs::aligned16;
using bs::hip_status;
using bs::kMaxLd;
using bs::ok;

namespace {

typedef long long ll;

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

constexpr int64_t kMaxI32 = 0x7fffffff;

// A bf16 matrix [rows, cols] with 16-byte rows.
bs_status check_bf16(const char* fn, const char* name, const void* p, int64_t cols, int64_t ld) {
    REQUIRE(ld >= cols && ld < kMaxLd, BS_ERR_LAYOUT, "ld of %s = %lld must be >= %lld columns and < 2^22", name,
            (ll)ld, (ll)cols);
    REQUIRE(aligned16(p) && ld % 8 == 0, BS_ERR_ALIGN, "%s must be 16-byte aligned with ld %% 8 == 0", name);
    return BS_OK;
}

// Row and column outputs of a 1x128 quantization of an [R, C] matrix.
bs_status check_codes(const char* fn, int64_t R, int64_t C, const uint8_t* q_row, int64_t ld_qr, const float* s_row,
                      int64_t ld_sr, const uint8_t* q_col, int64_t ld_qc, const float* s_col, int64_t ld_sc) {
    const bool row = q_row || s_row, col = q_col || s_col;
    const bool empty = R == 0 || C == 0;  // codes without elements may be NULL beside scales that are not
    REQUIRE(!row || (q_row && s_row) || empty, BS_ERR_NULL, "q_row and s_row must both be set or both NULL");
    REQUIRE(!col || (q_col && s_col) || empty, BS_ERR_NULL, "q_col and s_col must both be set or both NULL");
    if (row || col)
        REQUIRE(C % 128 == 0, BS_ERR_SHAPE, "%lld columns must be a multiple of 128 (1x128 blocks along rows)", (ll)C);
    if (row) {
        REQUIRE(ld_qr >= C && ld_qr < kMaxLd, BS_ERR_LAYOUT, "ld_qr=%lld must be >= %lld and < 2^22", (ll)ld_qr,
                (ll)C);
        REQUIRE(ld_sr >= R && ld_sr % 4 == 0, BS_ERR_LAYOUT,
                "ld_sr=%lld must be >= %lld rows and a multiple of 4 (s_row is K-major)", (ll)ld_sr, (ll)R);
        REQUIRE(aligned16(q_row) && ld_qr % 16 == 0 && aligned16(s_row), BS_ERR_ALIGN,
                "q_row and s_row must be 16-byte aligned with ld_qr %% 16 == 0");
    }
    if (col) {
        REQUIRE(R % 128 == 0, BS_ERR_SHAPE, "%lld rows must be a multiple of 128 for the column output", (ll)R);
        REQUIRE(ld_qc >= R && ld_qc < kMaxLd, BS_ERR_LAYOUT,
                "ld_qc=%lld must be >= %lld (q_col is the transpose) and < 2^22", (ll)ld_qc, (ll)R);
        REQUIRE(ld_sc >= C && ld_sc % 4 == 0, BS_ERR_LAYOUT,
                "ld_sc=%lld must be >= %lld columns and a multiple of 4 (s_col is K-major)", (ll)ld_sc, (ll)C);
        REQUIRE(aligned16(q_col) && ld_qc % 16 == 0 && aligned16(s_col), BS_ERR_ALIGN,
                "q_col and s_col must be 16-byte aligned with ld_qc %% 16 == 0");
    }
    return BS_OK;
}

#define CHECK(call)                              \
    do {                                         \
        const bs_status st_ = (call);            \
        if (st_ != BS_OK) return st_;            \
    } while (0)

bs_status check_route(const char* fn, const void* logits, bs_dtype dtype, int64_t T, int64_t E, int64_t ld_l,
                      bs_score_kind score, int64_t k, float scale, const void* idx, const void* w) {
    REQUIRE(dtype == BS_OUT_BF16 || dtype == BS_OUT_F32, BS_ERR_MODE, "dtype=%d must be BF16 or F32", (int)dtype);
    REQUIRE(score == BS_SCORE_SOFTMAX || score == BS_SCORE_SIGMOID, BS_ERR_MODE,
            "score=%d must be BS_SCORE_SOFTMAX or BS_SCORE_SIGMOID", (int)score);
    REQUIRE(T >= 0 && T <= kMaxI32, BS_ERR_SHAPE, "T=%lld must be in [0, 2^31)", (ll)T);
    REQUIRE(E >= 1 && E <= bs::kMaxExperts, BS_ERR_SHAPE, "E=%lld must be in [1, 1024]", (ll)E);
    REQUIRE(k >= 1 && k <= E && k <= bs::kMaxTopK, BS_ERR_SHAPE, "k=%lld must be in [1, min(E, 32)]", (ll)k);
    REQUIRE(std::isfinite(scale) && scale != 0.f, BS_ERR_MODE, "scale must be finite and not 0");
    REQUIRE((logits && idx && w) || T == 0, BS_ERR_NULL, "logits, idx and w must be non-NULL");
    REQUIRE(ld_l >= E, BS_ERR_LAYOUT, "ld_l=%lld < E=%lld: logits are row-major [T, E]", (ll)ld_l, (ll)E);
    REQUIRE((reinterpret_cast<uintptr_t>(logits) & (dtype == BS_OUT_F32 ? 3u : 1u)) == 0 && aligned4(idx) &&
                aligned4(w),
            BS_ERR_ALIGN, "logits, idx and w must be aligned to their types");
    return BS_OK;
}

bool vec_rows(const void* p, int64_t ld, bs_dtype dtype) {
    return aligned16(p) && ld % (dtype == BS_OUT_F32 ? 4 : 8) == 0;
}

}  // namespace

extern "C" {

bs_status bs_moe_route(const void* logits, bs_dtype dtype, int64_t T, int64_t E, int64_t ld_l, const float* bias,
                       bs_score_kind score, int64_t k, int64_t n_group, int64_t topk_group, int64_t group_best,
                       int renormalize, float scale, int32_t* idx, float* w, hipStream_t stream) {
    static const char* fn = "bs_moe_route";
    CHECK(check_route(fn, logits, dtype, T, E, ld_l, score, k, scale, idx, w));
    REQUIRE(n_group >= 1 && E % n_group == 0, BS_ERR_SHAPE, "n_group=%lld must divide E=%lld", (ll)n_group, (ll)E);
    REQUIRE(topk_group >= 1 && topk_group <= n_group, BS_ERR_SHAPE, "topk_group=%lld must be in [1, n_group=%lld]",
            (ll)topk_group, (ll)n_group);
    REQUIRE(group_best == 1 || group_best == 2, BS_ERR_MODE, "group_best=%lld must be 1 or 2", (ll)group_best);
    REQUIRE(aligned4(bias), BS_ERR_ALIGN, "bias must be aligned to its type");
    if (T == 0) return ok();
    bs::RouteArgs a{};
    a.logits = logits; a.bf16 = dtype == BS_OUT_BF16;
    a.T = T; a.E = E; a.ld = ld_l;
    a.bias = bias; a.sigmoid = score == BS_SCORE_SIGMOID;
    a.k = (int32_t)k; a.n_group = (int32_t)n_group; a.topk_group = (int32_t)topk_group;
    a.group_best = (int32_t)group_best;
    a.renorm = renormalize != 0; a.scale = scale; a.idx = idx; a.w = w;
    a.vec = vec_rows(logits, ld_l, dtype);
    a.vec_bias = aligned16(bias);
    // groups that are all kept decide nothing
    if (topk_group == n_group) a.n_group = a.topk_group = 1;
    return hip_status(bs::launch_route(a, stream), fn);
}

bs_status bs_moe_route_bwd(const void* logits, bs_dtype dtype, int64_t T, int64_t E, int64_t ld_l,
                           bs_score_kind score, int64_t k, int renormalize, float scale, const int32_t* idx,
                           const float* w, const float* dw, void* dlogits, int64_t ld_d, hipStream_t stream) {
    static const char* fn = "bs_moe_route_bwd";
    CHECK(check_route(fn, logits, dtype, T, E, ld_l, score, k, scale, idx, w));
    REQUIRE((dw && dlogits) || T == 0, BS_ERR_NULL, "dw and dlogits must be non-NULL");
    REQUIRE(ld_d >= E, BS_ERR_LAYOUT, "ld_d=%lld < E=%lld: dlogits are row-major [T, E]", (ll)ld_d, (ll)E);
    REQUIRE((reinterpret_cast<uintptr_t>(dlogits) & (dtype == BS_OUT_F32 ? 3u : 1u)) == 0 && aligned4(dw),
            BS_ERR_ALIGN, "dlogits and dw must be aligned to their types");
    if (T == 0) return ok();
    bs::RouteBwdArgs a{};
    a.logits = logits; a.bf16 = dtype == BS_OUT_BF16;
    a.T = T; a.E = E; a.ld = ld_l;
    a.sigmoid = score == BS_SCORE_SIGMOID; a.k = (int32_t)k; a.renorm = renormalize != 0; a.scale = scale;
    a.idx = idx; a.w = w; a.dw = dw; a.dlogits = dlogits; a.ld_d = ld_d;
    a.vec = vec_rows(logits, ld_l, dtype);
    a.vec_d = vec_rows(dlogits, ld_d, dtype);
    return hip_status(bs::launch_route_bwd(a, stream), fn);
}

int64_t bs_moe_plan_rows(int64_t T, int64_t k, int64_t E, int64_t align) {
    if (T < 0 || k < 1 || k > bs::kMaxTopK || E < 1 || E > bs::kMaxExperts || align < 1 || T > kMaxI32 / k ||
        align > bs::kMaxAlign)
        return 0;
    const int64_t n = T * k, groups = n < E ? n : E;
    return (n + groups * (align - 1)) / align * align;
}

int64_t bs_moe_plan_workspace_bytes(int64_t T, int64_t k, int64_t E) {
    if (bs_moe_plan_rows(T, k, E, 1) == 0) return 0;
    int32_t blocks, chunks;
    bs::plan_blocks(T * k, &blocks, &chunks);
    return blocks > 1 ? (int64_t)blocks * E * 4 : 0;
}

bs_status bs_moe_plan(const int32_t* idx, int64_t T, int64_t k, int64_t E, int64_t align, int64_t M,
                      int32_t* group_end, int32_t* counts, int32_t* slot_row, int32_t* row_slot, void* workspace,
                      int64_t workspace_bytes, hipStream_t stream) {
    static const char* fn = "bs_moe_plan";
    REQUIRE(E >= 1 && E <= bs::kMaxExperts, BS_ERR_SHAPE, "E=%lld must be in [1, 1024]", (ll)E);
    REQUIRE(k >= 1 && k <= bs::kMaxTopK, BS_ERR_SHAPE, "k=%lld must be in [1, 32]", (ll)k);
    REQUIRE(T >= 0 && T <= kMaxI32 / k, BS_ERR_SHAPE, "T=%lld must be >= 0 with T * k < 2^31", (ll)T);
    REQUIRE(align >= 1 && align <= bs::kMaxAlign, BS_ERR_SHAPE, "align=%lld must be in [1, 65536]", (ll)align);
    const int64_t need = bs_moe_plan_rows(T, k, E, align);
    REQUIRE(M >= need && M <= kMaxI32, BS_ERR_SHAPE,
            "M=%lld must be >= %lld (every group padded to %lld, whatever the routing) and < 2^31", (ll)M, (ll)need,
            (ll)align);
    REQUIRE(group_end && counts, BS_ERR_NULL, "group_end and counts must be non-NULL");
    REQUIRE((idx && slot_row) || T == 0, BS_ERR_NULL, "idx and slot_row must be non-NULL");
    REQUIRE(row_slot || M == 0, BS_ERR_NULL, "row_slot must be non-NULL");
    REQUIRE(aligned4(idx) && aligned4(group_end) && aligned4(counts) && aligned4(slot_row) && aligned4(row_slot),
            BS_ERR_ALIGN, "index arrays must be aligned to their type");
    const int64_t ws = bs_moe_plan_workspace_bytes(T, k, E);
    REQUIRE(workspace_bytes >= ws, BS_ERR_SHAPE, "workspace of %lld bytes < %lld (bs_moe_plan_workspace_bytes)",
            (ll)workspace_bytes, (ll)ws);
    REQUIRE(workspace || ws == 0, BS_ERR_NULL, "workspace is NULL");
    REQUIRE(aligned16(workspace), BS_ERR_ALIGN, "workspace must be 16-byte aligned");
    bs::PlanArgs a{};
    a.idx = idx; a.n = T * k; a.E = (int32_t)E; a.align = (int32_t)align; a.M = M;
    a.group_end = group_end; a.counts = counts; a.slot_row = slot_row; a.row_slot = row_slot;
    a.hist = static_cast<int32_t*>(workspace);
    bs::plan_blocks(a.n, &a.blocks, &a.chunks);
    return hip_status(bs::launch_plan(a, stream), fn);
}

bs_status bs_moe_gather_quant_1x128(const uint16_t* x, int64_t T, int64_t D, int64_t ld_x, int64_t k,
                                    const int32_t* row_slot, int64_t M, const float* w, uint16_t* y, int64_t ld_y,
                                    uint8_t* q_row, int64_t ld_qr, float* s_row, int64_t ld_sr, uint8_t* q_col,
                                    int64_t ld_qc, float* s_col, int64_t ld_sc, hipStream_t stream) {
    static const char* fn = "bs_moe_gather_quant_1x128";
    REQUIRE(k >= 1 && k <= bs::kMaxTopK, BS_ERR_SHAPE, "k=%lld must be in [1, 32]", (ll)k);
    REQUIRE(T >= 0 && T <= kMaxI32 / k && M >= 0 && M <= kMaxI32 && D >= 0, BS_ERR_SHAPE,
            "T=%lld, M=%lld, D=%lld must be >= 0 with T * k and M < 2^31", (ll)T, (ll)M, (ll)D);
    REQUIRE(D % 128 == 0, BS_ERR_SHAPE, "D=%lld must be a multiple of 128", (ll)D);
    const bool empty = M == 0 || D == 0;
    REQUIRE(x || T == 0 || empty, BS_ERR_NULL, "x is NULL");
    REQUIRE(row_slot || empty, BS_ERR_NULL, "row_slot is NULL");
    REQUIRE(y || q_row || s_row || q_col || s_col || empty, BS_ERR_NULL,
            "no output requested (y, q_row/s_row and q_col/s_col are all NULL)");
    CHECK(check_bf16(fn, "x", x, D, ld_x));
    if (y) CHECK(check_bf16(fn, "y", y, D, ld_y));
    CHECK(check_codes(fn, M, D, q_row, ld_qr, s_row, ld_sr, q_col, ld_qc, s_col, ld_sc));
    REQUIRE(aligned4(row_slot) && aligned4(w), BS_ERR_ALIGN, "row_slot and w must be aligned to their types");
    REQUIRE((M + 127) / 128 * (D / 128) <= kMaxI32, BS_ERR_SHAPE, "M=%lld x D=%lld has too many tiles", (ll)M, (ll)D);
    if (empty) return ok();
    bs::GatherArgs a{};
    a.x = x; a.T = T; a.D = D; a.ld_x = ld_x; a.k = (int32_t)k;
    // slot / k for slots < 2^31: a 32-bit multiply whose error e < k gives slot * e < 2^(32 + floor(log2 k))
    uint32_t fl = 0;
    while ((2u << fl) <= (uint32_t)k) ++fl;
    if ((k & (k - 1)) == 0) {
        a.k_mul = k == 1 ? 0u : 0x80000000u;
        a.k_shift = k == 1 ? 0u : fl - 1;
    } else {
        a.k_mul = (uint32_t)((((uint64_t)1 << (32 + fl)) + (uint64_t)k - 1) / (uint64_t)k);
        a.k_shift = fl;
    }
    a.row_slot = row_slot; a.M = M; a.w = w; a.y = y; a.ld_y = ld_y;
    a.q_row = q_row; a.ld_qr = ld_qr; a.s_row = s_row; a.ld_sr = ld_sr;
    a.q_col = q_col; a.ld_qc = ld_qc; a.s_col = s_col; a.ld_sc = ld_sc;
    return hip_status(bs::launch_gather(a, stream), fn);
}

bs_status bs_moe_combine(const uint16_t* y, int64_t M, int64_t D, int64_t ld_y, const int32_t* slot_row,
                         const float* w, int64_t T, int64_t k, const uint16_t* residual, int64_t ld_res,
                         uint16_t* out, int64_t ld_out, hipStream_t stream) {
    static const char* fn = "bs_moe_combine";
    REQUIRE(k >= 1 && k <= bs::kMaxTopK, BS_ERR_SHAPE, "k=%lld must be in [1, 32]", (ll)k);
    REQUIRE(T >= 0 && T <= kMaxI32 / k && M >= 0 && M <= kMaxI32 && D >= 0, BS_ERR_SHAPE,
            "T=%lld, M=%lld, D=%lld must be >= 0 with T * k and M < 2^31", (ll)T, (ll)M, (ll)D);
    REQUIRE(D % 8 == 0, BS_ERR_SHAPE, "D=%lld must be a multiple of 8 (16-byte rows)", (ll)D);
    const bool empty = T == 0 || D == 0;
    REQUIRE(y || M == 0 || empty, BS_ERR_NULL, "y is NULL");
    REQUIRE((slot_row && out) || empty, BS_ERR_NULL, "slot_row and out must be non-NULL");
    CHECK(check_bf16(fn, "y", y, D, ld_y));
    CHECK(check_bf16(fn, "out", out, D, ld_out));
    if (residual) CHECK(check_bf16(fn, "residual", residual, D, ld_res));
    REQUIRE(aligned4(slot_row) && aligned4(w), BS_ERR_ALIGN, "slot_row and w must be aligned to their types");
    REQUIRE(T * (D / 8) / 256 < kMaxI32, BS_ERR_SHAPE, "T=%lld x D=%lld is too large", (ll)T, (ll)D);
    if (empty) return ok();
    bs::CombineArgs a{y, M, D, ld_y, slot_row, w, T, (int32_t)k, residual, ld_res, out, ld_out};
    return hip_status(bs::launch_combine(a, stream), fn);
}

bs_status bs_moe_combine_dw(const uint16_t* dout, int64_t T, int64_t D, int64_t ld_dout, const uint16_t* y,
                            int64_t M, int64_t ld_y, const int32_t* slot_row, int64_t k, float* dw,
                            hipStream_t stream) {
    static const char* fn = "bs_moe_combine_dw";
    REQUIRE(k >= 1 && k <= bs::kMaxTopK, BS_ERR_SHAPE, "k=%lld must be in [1, 32]", (ll)k);
    REQUIRE(T >= 0 && T <= kMaxI32 / k && M >= 0 && M <= kMaxI32 && D >= 0, BS_ERR_SHAPE,
            "T=%lld, M=%lld, D=%lld must be >= 0 with T * k and M < 2^31", (ll)T, (ll)M, (ll)D);
    REQUIRE(D % 8 == 0, BS_ERR_SHAPE, "D=%lld must be a multiple of 8 (16-byte rows)", (ll)D);
    REQUIRE((slot_row && dw) || T == 0, BS_ERR_NULL, "slot_row and dw must be non-NULL");
    REQUIRE(dout || T == 0 || D == 0, BS_ERR_NULL, "dout is NULL");
    REQUIRE(y || M == 0 || D == 0, BS_ERR_NULL, "y is NULL");
    CHECK(check_bf16(fn, "dout", dout, D, ld_dout));
    CHECK(check_bf16(fn, "y", y, D, ld_y));
    REQUIRE(aligned4(slot_row) && aligned4(dw), BS_ERR_ALIGN, "slot_row and dw must be aligned to their types");
    if (T == 0) return ok();
    bs::CombineDwArgs a{dout, ld_dout, y, M, D, ld_y, slot_row, T, (int32_t)k, dw};
    return hip_status(bs::launch_combine_dw(a, stream), fn);
}

bs_status bs_resid_norm(const uint16_t* x, const uint16_t* u, int64_t R, int64_t D, int64_t ld_x, int64_t ld_u,
                        const void* w_post, const void* gate, int64_t ld_gate, int64_t rows_per_gate,
                        const void* w_pre, bs_dtype w_dtype, float alpha, float eps, uint16_t* r, int64_t ld_r,
                        float* rstd_u, float* rstd_r, uint16_t* h, int64_t ld_h, uint8_t* q_row, int64_t ld_qr,
                        float* s_row, int64_t ld_sr, uint8_t* q_col, int64_t ld_qc, float* s_col, int64_t ld_sc,
                        hipStream_t stream) {
    static const char* fn = "bs_resid_norm";
    REQUIRE(w_dtype == BS_OUT_BF16 || w_dtype == BS_OUT_F32, BS_ERR_MODE, "w_dtype=%d must be BF16 or F32",
            (int)w_dtype);
    REQUIRE(R >= 0 && R <= kMaxI32 && D >= 0, BS_ERR_SHAPE, "R=%lld, D=%lld must be >= 0", (ll)R, (ll)D);
    REQUIRE(D % 8 == 0 && D <= bs::kMaxNormDim, BS_ERR_SHAPE,
            "D=%lld must be a multiple of 8 (16-byte rows), at most 16384", (ll)D);
    REQUIRE(std::isfinite(alpha) && std::isfinite(eps) && eps >= 0.f, BS_ERR_MODE,
            "alpha must be finite and eps finite and >= 0");
    const bool empty = R == 0 || D == 0;
    const bool codes = q_row || s_row || q_col || s_col;
    REQUIRE(x || empty, BS_ERR_NULL, "x is NULL");
    REQUIRE(!u || r || empty, BS_ERR_NULL, "r must be set with u");
    REQUIRE(u || empty || (!r && !w_post && !gate && !rstd_u), BS_ERR_NULL,
            "r, w_post, gate and rstd_u need u (without it r is x)");
    REQUIRE(!rstd_u || w_post, BS_ERR_NULL, "rstd_u needs w_post");
    REQUIRE(w_pre || (!h && !codes && !rstd_r), BS_ERR_NULL, "h, its codes and rstd_r need w_pre");
    REQUIRE(r || h || codes || rstd_r || empty, BS_ERR_NULL, "no output requested");
    REQUIRE(!(q_col || s_col) || rstd_r || empty, BS_ERR_NULL, "the column output needs rstd_r");
    CHECK(check_bf16(fn, "x", x, D, ld_x));
    if (u) {
        CHECK(check_bf16(fn, "u", u, D, ld_u));
        CHECK(check_bf16(fn, "r", r, D, ld_r));
    }
    if (h) CHECK(check_bf16(fn, "h", h, D, ld_h));
    CHECK(check_codes(fn, R, D, q_row, ld_qr, s_row, ld_sr, q_col, ld_qc, s_col, ld_sc));
    if (gate) {
        REQUIRE(rows_per_gate >= 1 && R % rows_per_gate == 0, BS_ERR_SHAPE,
                "rows_per_gate=%lld must divide R=%lld", (ll)rows_per_gate, (ll)R);
        REQUIRE(ld_gate >= D && ld_gate < kMaxLd, BS_ERR_LAYOUT, "ld_gate=%lld must be >= D=%lld and < 2^22",
                (ll)ld_gate, (ll)D);
        REQUIRE(ld_gate % (w_dtype == BS_OUT_F32 ? 4 : 8) == 0, BS_ERR_ALIGN, "gate rows must be 16-byte aligned");
    }
    REQUIRE(aligned16(w_post) && aligned16(gate) && aligned16(w_pre), BS_ERR_ALIGN,
            "w_post, gate and w_pre must be 16-byte aligned");
    REQUIRE(aligned4(rstd_u) && aligned4(rstd_r) && (!q_col || aligned16(rstd_r)), BS_ERR_ALIGN,
            "rstd_u and rstd_r must be aligned (rstd_r to 16 bytes with the column output)");
    if (empty) return ok();
    bs::ResidNormArgs a{};
    a.x = x; a.u = u; a.R = R; a.D = D; a.ld_x = ld_x; a.ld_u = ld_u;
    a.w_post = w_post; a.gate = gate; a.w_pre = w_pre; a.w_bf16 = w_dtype == BS_OUT_BF16;
    a.ld_gate = ld_gate; a.rows_per_gate = gate ? rows_per_gate : R; a.alpha = alpha; a.eps = eps;
    a.r = r; a.ld_r = ld_r; a.rstd_u = rstd_u; a.rstd_r = rstd_r; a.h = h; a.ld_h = ld_h;
    a.q_row = q_row; a.ld_qr = ld_qr; a.s_row = s_row; a.ld_sr = ld_sr;
    a.q_col = q_col; a.ld_qc = ld_qc; a.s_col = s_col; a.ld_sc = ld_sc;
    return hip_status(bs::launch_resid_norm(a, stream), fn);
}

int64_t bs_resid_norm_bwd_workspace_bytes(int64_t R, int64_t D, int64_t rows_per_gate) {
    if (R < 1 || R > kMaxI32 || D < 1 || D > bs::kMaxNormDim || rows_per_gate < 1 || R % rows_per_gate != 0) return 0;
    const bs::NormBwdSplit sp = bs::norm_bwd_split(R, D, rows_per_gate);
    return (2 * sp.blocks + (sp.chunks > 1 ? sp.segs * sp.chunks : 0)) * D * 4;
}

bs_status bs_resid_norm_bwd(const uint16_t* r, const uint16_t* u, const uint16_t* dh, const uint16_t* dr, int64_t R,
                            int64_t D, int64_t ld_r, int64_t ld_u, int64_t ld_dh, int64_t ld_dr, const void* w_post,
                            const void* gate, int64_t ld_gate, int64_t rows_per_gate, const void* w_pre,
                            bs_dtype w_dtype, float alpha, const float* rstd_u, const float* rstd_r, uint16_t* dx,
                            int64_t ld_dx, uint16_t* du, int64_t ld_du, float* dw_pre, float* dw_post, float* dgate,
                            void* workspace, int64_t workspace_bytes, hipStream_t stream) {
    static const char* fn = "bs_resid_norm_bwd";
    REQUIRE(w_dtype == BS_OUT_BF16 || w_dtype == BS_OUT_F32, BS_ERR_MODE, "w_dtype=%d must be BF16 or F32",
            (int)w_dtype);
    REQUIRE(R >= 0 && R <= kMaxI32 && D >= 0, BS_ERR_SHAPE, "R=%lld, D=%lld must be >= 0", (ll)R, (ll)D);
    REQUIRE(D % 8 == 0 && D <= bs::kMaxNormDim, BS_ERR_SHAPE,
            "D=%lld must be a multiple of 8 (16-byte rows), at most 16384", (ll)D);
    REQUIRE(std::isfinite(alpha), BS_ERR_MODE, "alpha must be finite");
    REQUIRE(R > 0 || (!dw_pre && !dw_post && !dgate), BS_ERR_SHAPE, "R=0 has no sums over rows");
    const bool empty = R == 0 || D == 0;
    REQUIRE(dx || empty, BS_ERR_NULL, "dx is NULL");
    REQUIRE(!w_pre || (r && dh && rstd_r) || empty, BS_ERR_NULL, "r, dh and rstd_r must be set with w_pre");
    REQUIRE(w_pre || (dr && !dh && !dw_pre) || empty, BS_ERR_NULL, "without w_pre dr must be set, dh and dw_pre NULL");
    REQUIRE(u || (!w_post && !gate && !du && !dw_post && !dgate) || empty, BS_ERR_NULL,
            "w_post, gate, du, dw_post and dgate need u");
    REQUIRE(!u || du || empty, BS_ERR_NULL, "du must be set with u");
    REQUIRE(!w_post || rstd_u || empty, BS_ERR_NULL, "rstd_u must be set with w_post");
    REQUIRE((!dw_post || w_post) && (!dgate || gate), BS_ERR_NULL, "dw_post needs w_post, dgate needs gate");
    if (r) CHECK(check_bf16(fn, "r", r, D, ld_r));
    if (u) CHECK(check_bf16(fn, "u", u, D, ld_u));
    if (dh) CHECK(check_bf16(fn, "dh", dh, D, ld_dh));
    if (dr) CHECK(check_bf16(fn, "dr", dr, D, ld_dr));
    CHECK(check_bf16(fn, "dx", dx, D, ld_dx));
    if (du) CHECK(check_bf16(fn, "du", du, D, ld_du));
    const int64_t S = gate ? rows_per_gate : (R > 0 ? R : 1);
    if (gate) {
        REQUIRE(S >= 1 && R % S == 0, BS_ERR_SHAPE, "rows_per_gate=%lld must divide R=%lld", (ll)S, (ll)R);
        REQUIRE(ld_gate >= D && ld_gate < kMaxLd, BS_ERR_LAYOUT, "ld_gate=%lld must be >= D=%lld and < 2^22",
                (ll)ld_gate, (ll)D);
        REQUIRE(ld_gate % (w_dtype == BS_OUT_F32 ? 4 : 8) == 0, BS_ERR_ALIGN, "gate rows must be 16-byte aligned");
    }
    REQUIRE(aligned16(w_post) && aligned16(gate) && aligned16(w_pre) && aligned16(dw_pre) && aligned16(dw_post) &&
                aligned16(dgate) && aligned16(workspace),
            BS_ERR_ALIGN, "parameters, their gradients and the workspace must be 16-byte aligned");
    REQUIRE(aligned4(rstd_u) && aligned4(rstd_r), BS_ERR_ALIGN, "rstd_u and rstd_r must be aligned to their type");
    if (empty) return ok();
    const int64_t need = bs_resid_norm_bwd_workspace_bytes(R, D, S);
    REQUIRE(workspace && workspace_bytes >= need, BS_ERR_SHAPE,
            "workspace of %lld bytes < %lld (bs_resid_norm_bwd_workspace_bytes)", (ll)workspace_bytes, (ll)need);
    bs::ResidNormBwdArgs a{};
    a.r = r; a.u = u; a.dh = dh; a.dr = dr; a.R = R; a.D = D;
    a.ld_r = ld_r; a.ld_u = ld_u; a.ld_dh = ld_dh; a.ld_dr = ld_dr;
    a.w_post = w_post; a.gate = gate; a.w_pre = w_pre; a.w_bf16 = w_dtype == BS_OUT_BF16;
    a.ld_gate = ld_gate; a.rows_per_gate = S; a.alpha = alpha; a.rstd_u = rstd_u; a.rstd_r = rstd_r;
    a.dx = dx; a.du = du; a.ld_dx = ld_dx; a.ld_du = ld_du;
    a.dw_pre = dw_pre; a.dw_post = dw_post; a.dgate = dgate; a.ws = static_cast<float*>(workspace);
    return hip_status(bs::launch_resid_norm_bwd(a, stream), fn);
}

bs_status bs_swiglu_quant_1x128_ckpt(const uint16_t* a, const uint16_t* b, int64_t R, int64_t C, int64_t ld_a,
                                     int64_t ld_b, uint8_t* ck, int64_t ld_ck, float* s_ck, int64_t ld_sck,
                                     uint8_t* q_row, int64_t ld_qr, float* s_row, int64_t ld_sr, uint8_t* q_col,
                                     int64_t ld_qc, float* s_col, int64_t ld_sc, hipStream_t stream) {
    static const char* fn = "bs_swiglu_quant_1x128_ckpt";
    REQUIRE(R >= 0 && C >= 0, BS_ERR_SHAPE, "R=%lld C=%lld must be >= 0", (ll)R, (ll)C);
    REQUIRE(C % 128 == 0, BS_ERR_SHAPE, "C=%lld must be a multiple of 128", (ll)C);
    const bool empty = R == 0 || C == 0;
    REQUIRE((a && b && ck && s_ck) || empty, BS_ERR_NULL, "a, b, ck and s_ck must be non-NULL");
    REQUIRE(q_row || s_row || q_col || s_col || empty, BS_ERR_NULL,
            "no output requested (q_row/s_row and q_col/s_col are all NULL)");
    CHECK(check_bf16(fn, "a", a, C, ld_a));
    CHECK(check_bf16(fn, "b", b, C, ld_b));
    if (!empty) {
        CHECK(check_codes(fn, R, C, q_row, ld_qr, s_row, ld_sr, q_col, ld_qc, s_col, ld_sc));
        REQUIRE(ld_ck >= 2 * C && ld_ck < kMaxLd, BS_ERR_LAYOUT, "ld_ck=%lld must be >= 2C=%lld and < 2^22",
                (ll)ld_ck, (ll)(2 * C));
        REQUIRE(ld_sck >= R && ld_sck % 4 == 0, BS_ERR_LAYOUT,
                "ld_sck=%lld must be >= R=%lld and a multiple of 4 (s_ck is K-major)", (ll)ld_sck, (ll)R);
        REQUIRE(aligned16(ck) && ld_ck % 16 == 0 && aligned16(s_ck), BS_ERR_ALIGN,
                "ck and s_ck must be 16-byte aligned with ld_ck %% 16 == 0");
        REQUIRE((R + 127) / 128 * (C / 128) <= kMaxI32, BS_ERR_SHAPE, "too many tiles");
    }
    if (empty) return ok();
    bs::SwigluCkptArgs g{a, b, R, C, ld_a, ld_b, ck, ld_ck, s_ck, ld_sck, q_row, ld_qr, s_row, ld_sr, q_col, ld_qc,
                         s_col, ld_sc};
    return hip_status(bs::launch_swiglu_ckpt(g, stream), fn);
}

bs_status bs_swiglu_bwd_quant_1x128_ckpt(const uint8_t* ck, int64_t R, int64_t C, int64_t ld_ck, const float* s_ck,
                                         int64_t ld_sck, const uint16_t* dh, int64_t ld_dh, uint8_t* q_row,
                                         int64_t ld_qr, float* s_row, int64_t ld_sr, uint8_t* q_col, int64_t ld_qc,
                                         float* s_col, int64_t ld_sc, hipStream_t stream) {
    static const char* fn = "bs_swiglu_bwd_quant_1x128_ckpt";
    REQUIRE(R >= 0 && C >= 0, BS_ERR_SHAPE, "R=%lld C=%lld must be >= 0", (ll)R, (ll)C);
    REQUIRE(C % 128 == 0, BS_ERR_SHAPE, "C=%lld must be a multiple of 128", (ll)C);
    const bool empty = R == 0 || C == 0;
    REQUIRE((ck && s_ck && dh) || empty, BS_ERR_NULL, "ck, s_ck and dh must be non-NULL");
    REQUIRE(q_row || s_row || q_col || s_col || empty, BS_ERR_NULL,
            "no output requested (q_row/s_row and q_col/s_col are all NULL)");
    CHECK(check_bf16(fn, "dh", dh, C, ld_dh));
    if (!empty) {
        CHECK(check_codes(fn, R, 2 * C, q_row, ld_qr, s_row, ld_sr, q_col, ld_qc, s_col, ld_sc));
        REQUIRE(ld_ck >= 2 * C && ld_ck < kMaxLd, BS_ERR_LAYOUT, "ld_ck=%lld must be >= 2C=%lld and < 2^22",
                (ll)ld_ck, (ll)(2 * C));
        REQUIRE(ld_sck >= R && ld_sck % 4 == 0, BS_ERR_LAYOUT,
                "ld_sck=%lld must be >= R=%lld and a multiple of 4 (s_ck is K-major)", (ll)ld_sck, (ll)R);
        REQUIRE(aligned16(ck) && ld_ck % 16 == 0 && aligned16(s_ck), BS_ERR_ALIGN,
                "ck and s_ck must be 16-byte aligned with ld_ck %% 16 == 0");
        REQUIRE((R + 127) / 128 * (C / 128) <= kMaxI32, BS_ERR_SHAPE, "too many tiles");
    }
    if (empty) return ok();
    bs::SwigluBwdCkptArgs g{ck, R, C, ld_ck, s_ck, ld_sck, dh, ld_dh, q_row, ld_qr, s_row, ld_sr, q_col, ld_qc,
                            s_col, ld_sc};
    return hip_status(bs::launch_swiglu_bwd_ckpt(g, stream), fn);
}

}  // extern "C"
