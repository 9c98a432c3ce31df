// Router of an MoE layer for gfx950: scores, balance bias, expert groups,
// top-k and weights, and the gradient of the logits.
//
// A token is owned by L lanes of a wave (L a power of two, by the expert
// count), each holding V consecutive experts in registers, so that a wave
// routes 64 / L tokens at once and a reduction over a token's experts is
// log2(L) lane exchanges.  The choice is between values that may lie next to
// one another and has to be exact: by the logits themselves where neither bias
// nor groups are in play (scores rise with their logits), else by scores in
// fp32 with a bound on their error, and in float64 for the tokens (some in a
// thousand) whose choice that leaves in doubt.  Equal keys go to the lowest
// expert: a lane's experts are consecutive, so that is the lowest lane of the
// ballot and its first maximum.
//
// Bound by a wave's vector instructions and chain of reductions, not by bytes:
// 256 experts in 8 groups with a bias, top 8: one token 5.6 us (an empty launch
// is 3.8), 16384 tokens 18 us (17 MB would take 3.5; 1200 vector instructions a
// wave of 4 tokens, 9 us) and 9 us back, of them about 2 for the last wave with
// a token in doubt; without groups or bias the
// choice is by the logits: 128000 tokens of 8 experts 3.8 us and 3.6 back.
// Weights are computed in fp32, also where the choice went by float64.
#include "bs_moe.h"
#include "bs_device.h"

namespace bs {

namespace {

constexpr int kThreads = 256;
constexpr float kTinySum = 1e-20f;  // added to the sum of the chosen sigmoid scores
constexpr float kUp = 18446744073709551616.0f;  // 2^64: scores may be far below 1e-20, and fp32 ends at 1e-38

// ---- reductions over the L lanes of a token; every lane gets the result ----
// Steps 1 and 2 are quad permutes; 4 and 8 mirror halves of a 16-lane row
// whose quads (halves) already agree; 16 and 32 go through the LDS crossbar.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp32(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, false);
}

template <int STEP, typename T>
__device__ __forceinline__ T lane_swap(T v) {
    if constexpr (STEP >= 16) {
        return __shfl_xor(v, STEP);
    } else {
        constexpr int C = STEP == 1 ? 0xB1 : STEP == 2 ? 0x4E : STEP == 4 ? 0x141 : 0x140;
        if constexpr (sizeof(T) == 8) {
            const uint64_t b = __builtin_bit_cast(uint64_t, v);
            const uint64_t r = (uint64_t)dpp32<C>((uint32_t)b) | ((uint64_t)dpp32<C>((uint32_t)(b >> 32)) << 32);
            return __builtin_bit_cast(T, r);
        } else {
            return __builtin_bit_cast(T, dpp32<C>(__builtin_bit_cast(uint32_t, v)));
        }
    }
}

template <int L, typename T, typename F>
__device__ __forceinline__ T seg_reduce(T v, F f) {
    if constexpr (L > 1) v = f(v, lane_swap<1>(v));
    if constexpr (L > 2) v = f(v, lane_swap<2>(v));
    if constexpr (L > 4) v = f(v, lane_swap<4>(v));
    if constexpr (L > 8) v = f(v, lane_swap<8>(v));
    if constexpr (L > 16) v = f(v, lane_swap<16>(v));
    if constexpr (L > 32) v = f(v, lane_swap<32>(v));
    return v;
}
template <int L>
__device__ __forceinline__ float seg_max(float v) {
    return seg_reduce<L>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int L>
__device__ __forceinline__ double seg_max(double v) {
    return seg_reduce<L>(v, [](double a, double b) { return fmax(a, b); });
}
template <int L, typename T>
__device__ __forceinline__ T seg_sum(T v) {
    return seg_reduce<L>(v, [](T a, T b) { return a + b; });
}

__device__ __forceinline__ float load_logit(const void* p, bool bf16, int64_t i) {
    return bf16 ? __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(p)[i] << 16)
                : reinterpret_cast<const float*>(p)[i];
}

constexpr float kNegInf = -__builtin_inff();

// V logits from expert e0 on; experts past E read as -inf.
template <bool BF16, int V>
__device__ __forceinline__ void load_logits(const void* base, int64_t row, int e0, int E, bool vec, float* f) {
    constexpr bool kWhole = V % (BF16 ? 8 : 4) == 0;  // whole 16-byte loads
    if (kWhole && vec && e0 + V <= E) {
        if constexpr (BF16) {
            const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(base) + row + e0);
#pragma unroll
            for (int i = 0; i < V / 8; ++i) unpack8(p[i], f + 8 * i);
        } else {
            const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(base) + row + e0);
#pragma unroll
            for (int i = 0; i < V / 4; ++i) {
                const float4 v = p[i];
                f[4 * i] = v.x; f[4 * i + 1] = v.y; f[4 * i + 2] = v.z; f[4 * i + 3] = v.w;
            }
        }
    } else {
        // the last expert stands in for those past it, so that no load is conditional
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float x = load_logit(base, BF16, row + (e0 + v < E ? e0 + v : E - 1));
            f[v] = e0 + v < E ? x : kNegInf;
        }
    }
}

// LDS writes of this wave before it are seen by the wave's reads after it
// (they run in order; this keeps the compiler from moving them).
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ __forceinline__ double sigmoid64(double l) { return 1.0 / (1.0 + exp(-l)); }

// 2^64 sigmoid(d), and 1 - sigmoid(d) without its cancellation, in fp32: of
// h = exp(-|d| / 2), whose square would vanish where the scaled one does not.
__device__ __forceinline__ float sigmoid_up(float d, float& other) {
    const float h = expf(-0.5f * fabsf(d)), hu = h * 4294967296.0f;
    const float r = 1.0f / __builtin_fmaf(h, h, 1.0f);
    other = d < 0.f ? r : h * h * r;
    return d < 0.f ? hu * hu * r : kUp * r;
}

// exp(x) for the choice: the product's rounding makes it err by |x| units of
// 2^-24 and the hardware exponential by 2 more, where what counts is the error
// of a score, exp(x) of the largest: at most 3 units.  Infinities and NaN come
// out as they should.
__device__ __forceinline__ float exp_fast(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896f); }

// Largest of V values with its place, the first of equals: halves compared
// pairwise, since a chain of V dependent steps would take V latencies.  (By
// recursion on values: a loop over arrays is turned into indexing them by the
// result of a comparison.)
template <typename Key>
struct Placed {
    Key value;
    int place;
};
template <int V, int FROM = 0, typename Key>
__device__ __forceinline__ Placed<Key> first_max(const Key* key) {
    if constexpr (V == 1) {
        return {key[FROM], FROM};
    } else {
        const Placed<Key> x = first_max<V / 2, FROM>(key), y = first_max<V / 2, FROM + V / 2>(key);
        const bool up = y.value > x.value;
        return {up ? y.value : x.value, up ? y.place : x.place};
    }
}
template <int V, int FROM = 0>
__device__ __forceinline__ uint32_t tree_max(const uint32_t* key) {
    if constexpr (V == 1) {
        return key[FROM];
    } else {
        const uint32_t x = tree_max<V / 2, FROM>(key), y = tree_max<V / 2, FROM + V / 2>(key);
        return x > y ? x : y;
    }
}

// The lowest expert among the lanes of a token that offer one (kMaxExperts: none).
template <int L>
__device__ __forceinline__ int lowest(bool offer, int e) {
    return seg_reduce<L>(offer ? e : (int)kMaxExperts, [](int x, int y) { return x < y ? x : y; });
}

// k rounds over a token's keys: the best one left, ties to the lowest expert;
// slot j's expert goes to lane j % L.
template <int L, int V, int KR, typename Key>
__device__ __forceinline__ void select_k(Key* key, int k, int l, int32_t* mine_idx) {
    constexpr Key kNone = -(Key)__builtin_inff();
#pragma unroll
    for (int r = 0; r < KR; ++r) {
        mine_idx[r] = -1;
        for (int q = 0; q < L; ++q) {
            if (r * L + q >= k) break;
            const Placed<Key> best = first_max<V>(key);
            const Key mx = seg_max<L>(best.value);
            const int e = lowest<L>(best.value == mx, l * V + best.place);
#pragma unroll
            for (int v = 0; v < V; ++v) key[v] = l * V + v == e ? kNone : key[v];
            if (q == l && mx > kNone) mine_idx[r] = e;
        }
    }
}

// The choice in float64, from the logits on: what the definition says.  By all
// 64 lanes, slot j's expert to lane j.
template <bool BF16, int L, int V, int KR>
__device__ __forceinline__ void route_exact(const RouteArgs& a, int64_t row, int l, double* mine, int32_t* mine_idx) {
    constexpr double kNone = -__builtin_inf();
    const int E = (int)a.E, e0 = l * V;
    float lg[V];
    load_logits<BF16, V>(a.logits, row, e0, E, a.vec, lg);
    double key[V];
    float m = kNegInf;
    if (!a.sigmoid) {
#pragma unroll
        for (int v = 0; v < V; ++v) m = fmaxf(m, lg[v]);
        m = seg_max<L>(m);
    }
    double sum = 0.0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const double d = lg[v];
        key[v] = a.sigmoid ? sigmoid64(d) : (lg[v] == kNegInf ? 0.0 : exp(d - (double)m));
        sum += key[v];
    }
    if (!a.sigmoid) {
        sum = seg_sum<L>(sum);
        const double r = 1.0 / sum;
        // a NaN or +inf logit makes every score NaN: it counts as the largest, and the others as 0
#pragma unroll
        for (int v = 0; v < V; ++v)
            key[v] = sum == sum ? key[v] * r : lg[v] < __builtin_inff() ? 0.0 : __builtin_inf();
    }
    if (a.bias != nullptr) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float b = e0 + v < E ? a.bias[e0 + v] : 0.f;
            key[v] = b == kNegInf ? kNone : key[v] + (double)b;  // (masked, also where the score is not finite)
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (key[v] != key[v]) key[v] = __builtin_inf();  // NaN ranks first
        if (lg[v] == kNegInf) key[v] = kNone;            // and a masked expert never
    }
    if (a.n_group > 1) {
        // Group scores: the keys go to LDS, one element more than Eg per
        // group (lanes that read different groups then use different
        // banks, and that element takes the group's score, then whether it
        // is kept); lane l takes the groups l, l + L, ... of its token.  A
        // token's lanes are in one wave: its LDS operations run in order.
        const int G = a.n_group, Eg = E / G;
        const int g_first = e0 / Eg;
        int at = e0 + g_first, left = Eg - (e0 - g_first * Eg);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (e0 + v < E) mine[at] = key[v];
            left -= 1;
            at += left == 0 ? 2 : 1;
            left = left == 0 ? Eg : left;
        }
        wave_sync();
        for (int g = l; g < G; g += L) {
            double b1 = kNone, b2 = kNone;
#pragma unroll 4
            for (int i = 0; i < Eg; ++i) {
                const double x = mine[g * (Eg + 1) + i];
                b2 = fmax(b2, fmin(b1, x));
                b1 = fmax(b1, x);
            }
            if (a.group_best > 1 && b2 > kNone) b1 += b2;
            mine[g * (Eg + 1) + Eg] = b1;
        }
        wave_sync();
        // a group is kept if fewer than topk_group are better
        uint32_t kept = 0;  // bit i: group l + i L (at most V of them)
        for (int g = l, i = 0; g < G; g += L, ++i) {
            const double own = mine[g * (Eg + 1) + Eg];
            int better = 0;
#pragma unroll 4
            for (int h = 0; h < G; ++h) {
                const double o = mine[h * (Eg + 1) + Eg];
                better += (o > own) | ((o == own) & (h < g));
            }
            kept |= (better < a.topk_group ? 1u : 0u) << i;
        }
        wave_sync();
        for (int g = l, i = 0; g < G; g += L, ++i) mine[g * (Eg + 1) + Eg] = (double)((kept >> i) & 1u);
        wave_sync();
        at = g_first * (Eg + 1) + Eg;
        left = Eg - (e0 - g_first * Eg);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (e0 + v < E && mine[at] == 0.0) key[v] = kNone;
            left -= 1;
            at += left == 0 ? Eg + 1 : 0;
            left = left == 0 ? Eg : left;
        }
        if (a.bias == nullptr) {  // without a bias experts are ranked by their logits
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (key[v] != kNone) key[v] = lg[v] != lg[v] ? __builtin_inf() : (double)lg[v];
        }
    }
    select_k<L, V, KR>(key, a.k, l, mine_idx);
}

// Order-preserving image of a float in unsigned integers, and back.
__device__ __forceinline__ uint32_t to_ordered(float f) {
    const uint32_t b = __float_as_uint(f);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// The choice in fp32 where that is certain.  Scores err by at most 8 (sigmoid,
// of values up to 1) or 32 (softmax, of the largest: exponent, sum and
// quotient) units of 2^-24, a sum with the bias by one more of itself, and a
// key gives up its lowest log2(V) bits to the expert's place in its lane, so
// that a maximum finds both: two choices nearer than twice that are
// uncertain, unless logit and bias are the same and so the tie is real.
// Returns whether the token's choice is uncertain (then route_exact decides).
// whole: every group is a power of two of whole lanes (see route_lv).
template <int L, int V, int KR>
__device__ __forceinline__ bool route_fast(const RouteArgs& a, const float* lg, const float* bias,
                                           const float* row_lds, int l, float* group_lds, bool whole,
                                           int32_t* mine_idx) {
    const int E = (int)a.E, e0 = l * V;
    constexpr float u = 5.9604645e-08f;  // 2^-24
    float c[V];
    float err = 16.f * u;
    if (a.sigmoid) {
#pragma unroll
        for (int v = 0; v < V; ++v) c[v] = __builtin_amdgcn_rcpf(1.0f + exp_fast(-lg[v]));
    } else {
        float m = kNegInf, sum = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) m = fmaxf(m, lg[v]);
        m = seg_max<L>(m);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            c[v] = lg[v] == kNegInf ? 0.f : exp_fast(lg[v] - m);
            sum += c[v];
        }
        const float r = 1.0f / seg_sum<L>(sum);
#pragma unroll
        for (int v = 0; v < V; ++v) c[v] *= r;
        err = 64.f * u * r;  // r: the largest score
    }
    if (a.bias != nullptr) {
#pragma unroll
        for (int v = 0; v < V; ++v) c[v] += bias[v];
    }
    // masked experts at -inf (where a bias of -inf puts them by itself)
#pragma unroll
    for (int v = 0; v < V; ++v) c[v] = lg[v] == kNegInf ? kNegInf : c[v];
    bool unsure = false, out = false;  // out: this lane's group does not stay
    // Groups better than g, surely and maybe, from their scores `stride` apart:
    // true if g stays.
    const auto stays = [&](const float* score, int stride, int g, float own) {
        int surely = 0, maybe = 0;
        const float w0 = 2.f * err + 4.f * u * fabsf(own);
#pragma unroll 4
        for (int h = 0; h < a.n_group; ++h) {
            const float o = score[h * stride], w = w0 + 4.f * u * fabsf(o);
            surely += o - own > w;
            maybe += (h != g) & (o != kNegInf) & !(own - o > w);
        }
        const bool keep = surely < a.topk_group;
        unsure |= own != kNegInf && keep != (maybe < a.topk_group);
        return keep;
    };
    if (a.n_group > 1 && whole) {
        // the two best of a lane, then of the group's lanes
        const int G = a.n_group, lanes = E / G / V, g = l / lanes;
        float b1 = kNegInf, b2 = kNegInf;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            unsure |= c[v] != c[v];
            b2 = __builtin_amdgcn_fmed3f(b1, b2, c[v]);
            b1 = fmaxf(b1, c[v]);
        }
#define BS_MERGE(STEP)                                                            \
        if constexpr (L > STEP) {                                                 \
            if (lanes > STEP) {                                                   \
                const float o1 = lane_swap<STEP>(b1), o2 = lane_swap<STEP>(b2);   \
                b2 = fmaxf(fminf(b1, o1), fmaxf(b2, o2));                         \
                b1 = fmaxf(b1, o1);                                               \
            }                                                                     \
        }
        BS_MERGE(1) BS_MERGE(2) BS_MERGE(4) BS_MERGE(8) BS_MERGE(16) BS_MERGE(32)
#undef BS_MERGE
        const float own = a.group_best > 1 && b2 > kNegInf ? b1 + b2 : b1;
        if (g < G) group_lds[g] = own;
        wave_sync();
        out = !stays(group_lds, 1, g, own);
        wave_sync();  // the next use of group_lds
    } else if (a.n_group > 1) {
        // groups of any size: through LDS, laid out as in route_exact (16
        // experts in 4 groups, 8192 tokens: 7 us; by route_exact alone 41)
        const int G = a.n_group, Eg = E / G, g_first = e0 / Eg;
        int at = e0 + g_first, left = Eg - (e0 - g_first * Eg);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            unsure |= c[v] != c[v];
            if (e0 + v < E) group_lds[at] = c[v];
            left -= 1;
            at += left == 0 ? 2 : 1;
            left = left == 0 ? Eg : left;
        }
        wave_sync();
        for (int g = l; g < G; g += L) {
            float b1 = kNegInf, b2 = kNegInf;
#pragma unroll 4
            for (int i = 0; i < Eg; ++i) {
                const float x = group_lds[g * (Eg + 1) + i];
                b2 = fmaxf(b2, fminf(b1, x));
                b1 = fmaxf(b1, x);
            }
            group_lds[g * (Eg + 1) + Eg] = a.group_best > 1 && b2 > kNegInf ? b1 + b2 : b1;
        }
        wave_sync();
        uint32_t kept = 0;  // bit i: group l + i L (at most V of them)
        for (int g = l, i = 0; g < G; g += L, ++i)
            kept |= (uint32_t)stays(group_lds + Eg, Eg + 1, g, group_lds[g * (Eg + 1) + Eg]) << i;
        wave_sync();
        for (int g = l, i = 0; g < G; g += L, ++i) group_lds[g * (Eg + 1) + Eg] = (float)((kept >> i) & 1u);
        wave_sync();
        at = g_first * (Eg + 1) + Eg;
        left = Eg - (e0 - g_first * Eg);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (e0 + v < E && group_lds[at] == 0.f) c[v] = kNegInf;
            left -= 1;
            at += left == 0 ? Eg + 1 : 0;
            left = left == 0 ? Eg : left;
        }
        wave_sync();  // the next use of group_lds
    }
    if (a.bias == nullptr) {  // ranked by their logits, exactly
        float key[V];
#pragma unroll
        for (int v = 0; v < V; ++v)
            key[v] = out || c[v] == kNegInf ? kNegInf : lg[v] != lg[v] ? __builtin_inff() : lg[v];
        select_k<L, V, KR>(key, a.k, l, mine_idx);
        return unsure;
    }
    constexpr uint32_t kPlace = V - 1, kNone = 0x007FFFFFu;  // kNone: to_ordered(-inf); its keys are not over it
    uint32_t key[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        unsure |= c[v] != c[v];
        key[v] = (to_ordered(c[v]) & ~kPlace) | (uint32_t)(kPlace - v);
    }
    // A lane's keys differ, and they are taken in descending order: those left
    // are the ones below the last that was taken (limit; 0: none yet), and
    // since key - limit wraps for just those, the largest of the differences
    // finds the best of them.
    uint32_t limit = 0;
    const auto best_left = [&] {
        uint32_t d[V];
#pragma unroll
        for (int v = 0; v < V; ++v) d[v] = key[v] - limit;
        const uint32_t t = tree_max<V>(d);
        return out || t < 0u - limit ? 0u : t + limit;
    };
    float prev = 0.f;
    int prev_e = -1;
    const auto near = [&](float cur) {  // to the value before it in the order
        return !(prev - cur > err + (float)(2 * V + 2) * 2.f * u * fmaxf(fabsf(prev), fabsf(cur)));
    };
#pragma unroll
    for (int r = 0; r < KR; ++r) {
        mine_idx[r] = -1;
        for (int q = 0; q < L; ++q) {
            const int j = r * L + q;
            if (j >= a.k) break;
            const uint32_t best = best_left(), top = best & ~kPlace;
            const uint32_t mx = seg_reduce<L>(top, [](uint32_t x, uint32_t y) { return x > y ? x : y; });
            if (mx <= kNone) break;
            const int own_e = e0 + (int)(kPlace - (best & kPlace));
            const int e = lowest<L>(top == mx, own_e);
            limit = e == own_e ? best : limit;
            const float cur = from_ordered(mx);
            if (prev_e >= 0 && near(cur))
                unsure |= row_lds[prev_e] != row_lds[e] || a.bias[prev_e] != a.bias[e];
            prev = cur;
            prev_e = e;
            if (q == l) mine_idx[r] = e;
        }
    }
    // those left out against the last that was chosen, every one that is near
    // it: one that ties with it may have another next to it
    const uint32_t left = best_left();
    if (left > kNone && near(from_ordered(left & ~kPlace))) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (key[v] <= left && key[v] > kNone && near(from_ordered(key[v] & ~kPlace)))
                unsure |= row_lds[prev_e] != row_lds[e0 + v] || a.bias[prev_e] != a.bias[e0 + v];
        }
    }
    return unsure;
}

// A lane's logits to its token's row in LDS.
template <int V>
__device__ __forceinline__ void keep_row(float* lds, const float* lg) {
    wave_sync();
#pragma unroll
    for (int v = 0; v < V; v += 4)
        *reinterpret_cast<float4*>(lds + v) = make_float4(lg[v], lg[v + 1], lg[v + 2], lg[v + 3]);
    wave_sync();
}

// SCORES: the choice goes by scores (a bias or groups are in play); without,
// by the logits, and exactly so in fp32.
template <bool BF16, int L, int V, bool SCORES>
__global__ __launch_bounds__(kThreads) void route_kernel(RouteArgs a, bool whole) {
    extern __shared__ double s_dyn[];
    constexpr int TPB = kThreads / L;  // tokens of a block
    constexpr int KR = (int)kMaxTopK < V * L ? ((int)kMaxTopK + L - 1) / L : V;  // slots a lane may hold

    const int l = threadIdx.x % L, tb = threadIdx.x / L;
    const int seg = (threadIdx.x & 63) / L * L;  // first lane of the token
    const int64_t tok = (int64_t)blockIdx.x * TPB + tb;
    const bool real = tok < a.T;
    const int64_t row = (real ? tok : a.T - 1) * a.ld;
    const int E = (int)a.E, e0 = l * V;

    // the one trip to memory: the logits (also to LDS, where the chosen ones
    // are looked up at the end) and the bias
    float* const row_lds = reinterpret_cast<float*>(s_dyn) + tb * a.lds_token;
    float lg[V], bias[V];
    load_logits<BF16, V>(a.logits, row, e0, E, a.vec, lg);
    if (SCORES && a.bias != nullptr) load_logits<false, V>(a.bias, 0, e0, E, a.vec_bias, bias);
    keep_row<V>(row_lds + e0, lg);
    float m = kNegInf, z = 0.f;  // softmax over all experts: the largest logit, the sum of exp(l - m)
    if (!a.sigmoid && !a.renorm) {
#pragma unroll
        for (int v = 0; v < V; ++v) m = fmaxf(m, lg[v]);
        m = seg_max<L>(m);
#pragma unroll
        for (int v = 0; v < V; ++v) z += lg[v] == kNegInf ? 0.f : expf(lg[v] - m);
        z = seg_sum<L>(z);
    }

    int32_t mine_idx[KR];
    if constexpr (SCORES) {
        const bool unsure = route_fast<L, V, KR>(a, lg, bias, row_lds, l, row_lds + L * V, whole, mine_idx);
        // rare: the tokens in doubt one after another, each by the whole wave
        // (a wave that redid its tokens as they lie would take 12 us more at
        // 256 experts, and some wave always has one)
        uint64_t some = __ballot(unsure && real);
        while (some != 0) {
            const int lane = threadIdx.x & 63, at = __builtin_ctzll(some) / L * L;
            constexpr uint64_t kToken = L < 64 ? (1ull << L) - 1 : ~0ull;
            some &= ~(kToken << at);
            const int tw = (threadIdx.x & ~63) / L + at / L;  // the token's place in the block
            const int64_t t = (int64_t)blockIdx.x * TPB + tw;
            float* const lds = reinterpret_cast<float*>(s_dyn) + tw * a.lds_token;
            constexpr int VW = V * L > 64 ? V * L / 64 : 1;
            int32_t exact[1];
            route_exact<BF16, 64, VW, 1>(a, t * a.ld, lane, reinterpret_cast<double*>(lds), exact);
#pragma unroll
            for (int r = 0; r < KR; ++r) {
                const int32_t e = __shfl(exact[0], (r * L + l) & 63);
                if (seg == at) mine_idx[r] = r * L + l < a.k ? e : -1;
            }
            if (seg == at) keep_row<V>(row_lds + e0, lg);  // (the exact keys took its place)
        }
    } else {
        float key[V];
#pragma unroll
        for (int v = 0; v < V; ++v) key[v] = lg[v] != lg[v] ? __builtin_inff() : lg[v];
        select_k<L, V, KR>(key, a.k, l, mine_idx);
    }

    // weights of the chosen experts, in fp32
    float s[KR];
    float top = kNegInf;
    if (!a.sigmoid && a.renorm) {
#pragma unroll
        for (int r = 0; r < KR; ++r) {
            if (r * L >= a.k) break;
            if (mine_idx[r] >= 0) top = fmaxf(top, row_lds[mine_idx[r]]);
        }
        top = seg_max<L>(top);
    }
    float sum = 0.f;
#pragma unroll
    for (int r = 0; r < KR; ++r) {
        s[r] = 0.f;
        if (r * L >= a.k) continue;
        if (mine_idx[r] >= 0) {
            const float d = row_lds[mine_idx[r]];
            float other;
            s[r] = a.sigmoid ? sigmoid_up(d, other) : a.renorm ? expf(d - top) : expf(d - m) / z;
        }
        sum += s[r];
    }
    float f = a.sigmoid ? a.scale * (1.f / kUp) : a.scale;
    if (a.renorm) {
        sum = seg_sum<L>(sum);
        if (a.sigmoid) sum += kTinySum * kUp;
        f = a.scale / sum;
    }
    if (!real) return;
#pragma unroll
    for (int r = 0; r < KR; ++r) {
        const int j = r * L + l;
        if (j < a.k) {
            a.idx[tok * a.k + j] = mine_idx[r];
            a.w[tok * a.k + j] = mine_idx[r] >= 0 ? s[r] * f : 0.f;
        }
    }
}

// Gradient of the logits.  The k contributions of a token are placed in an
// LDS row, which the lanes then add to what they hold and write out whole.
// With p_j the chosen experts' shares of their sum (renormalized weights over
// scale) it takes g_j - sum p_i g_i, which vanishes for k = 1 and nearly so
// for an expert with nearly all of the sum.  With g_0 that of the largest
// share and rest = 1 - sum p_i (of the sigmoid's 1e-20; 0 for the softmax) it
// is (g_j - g_0) - sum p_i (g_i - g_0) + rest g_0, where nothing cancels.
// Not renormalized, the softmax's shares are of all experts, g of those that
// were not chosen 0: for the largest share that was chosen it is (1 - p_0) g_0
// less the others' p_i g_i, with 1 - p_0 from the exponentials of all others;
// the rest have p_j <= 1/2, and g_j - sum p_i g_i loses no more than a bit.
template <bool BF16, int L, int V>
__global__ __launch_bounds__(kThreads) void route_bwd_kernel(RouteBwdArgs a) {
    constexpr int TPB = kThreads / L;
    constexpr int KR = (int)kMaxTopK < V * L ? ((int)kMaxTopK + L - 1) / L : V;
    __shared__ __attribute__((aligned(16))) float s_row[TPB][L * V];
    const int l = threadIdx.x % L, tb = threadIdx.x / L;
    const int64_t tok = (int64_t)blockIdx.x * TPB + tb;
    const bool real = tok < a.T;
    const int64_t t = real ? tok : a.T - 1;
    const int E = (int)a.E, e0 = l * V;
    const bool all = !a.sigmoid && !a.renorm;  // every logit of the row has a gradient
    // an expert that was not chosen: no result of arithmetic has these bits (a signalling NaN)
    constexpr uint32_t kNotChosen = 0x7FBADBADu;
#pragma unroll
    for (int v = 0; v < V; ++v) s_row[tb][e0 + v] = all ? __uint_as_float(kNotChosen) : 0.f;
    __syncthreads();

    float m = kNegInf, z = 1.f;
    float lg[V];
    if (all) {
        load_logits<BF16, V>(a.logits, t * a.ld, e0, E, a.vec, lg);
#pragma unroll
        for (int v = 0; v < V; ++v) m = fmaxf(m, lg[v]);
        m = seg_max<L>(m);
        float sum = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            lg[v] = lg[v] == kNegInf ? 0.f : expf(lg[v] - m);
            sum += lg[v];
        }
        z = seg_sum<L>(sum);
    }
    int32_t e[KR];
    float w[KR], g[KR], s[KR], ns[KR];
    float dot = 0.f, ssum = 0.f;
    const float inv_scale = 1.f / a.scale;
#pragma unroll
    for (int r = 0; r < KR; ++r) {
        const int j = r * L + l;
        e[r] = -1;
        w[r] = g[r] = s[r] = ns[r] = 0.f;
        if (r * L >= a.k) continue;
        if (j < a.k) {
            const int32_t x = a.idx[t * a.k + j];
            if (x >= 0 && x < E) {
                e[r] = x;
                w[r] = a.w[t * a.k + j] * inv_scale;
                g[r] = a.dw[t * a.k + j];
                if (a.sigmoid) {
                    const float d = load_logit(a.logits, BF16, t * a.ld + x);
                    s[r] = sigmoid_up(d, ns[r]);
                }
            }
        }
        ssum += s[r];
    }
    float f = a.scale * (1.f / kUp), rest = 0.f;
    if (a.sigmoid && a.renorm) {
        const float sum = seg_sum<L>(ssum), total = sum + kTinySum * kUp;
        f = a.scale / total;
        rest = (total - sum) / total;  // 0 where the sum does not feel the 1e-20: over 2^-42
    }
    float g0 = 0.f;
    if (a.renorm) {
        uint64_t top = 0;  // the largest share with its g
#pragma unroll
        for (int r = 0; r < KR; ++r) {
            const uint64_t x = ((uint64_t)__float_as_uint(fabsf(w[r])) << 32) | __float_as_uint(g[r]);
            if (e[r] >= 0 && x > top) top = x;
        }
        top = seg_reduce<L>(top, [](uint64_t x, uint64_t y) { return x > y ? x : y; });
        g0 = __uint_as_float((uint32_t)top);
    }
    int e_top = -1;  // the largest share that was chosen, of all experts
    float p0 = 0.f, others = 0.f;  // it, and 1 - p_0
    if (all) {
        uint64_t top = 0;
#pragma unroll
        for (int r = 0; r < KR; ++r) {
            const uint64_t x = ((uint64_t)__float_as_uint(fabsf(w[r])) << 32) | (uint32_t)(e[r] + 1);
            if (x > top) top = x;
        }
        top = seg_reduce<L>(top, [](uint64_t x, uint64_t y) { return x > y ? x : y; });
        p0 = __uint_as_float((uint32_t)(top >> 32));
        e_top = (int)(uint32_t)top - 1;
#pragma unroll
        for (int v = 0; v < V; ++v) others += e0 + v == e_top ? 0.f : lg[v];
        others = seg_sum<L>(others) / z;
    }
    float g_top = 0.f;
#pragma unroll
    for (int r = 0; r < KR; ++r) {
        g[r] = e[r] >= 0 ? g[r] - g0 : 0.f;
        if (all && e[r] == e_top) g_top = g[r];
        else dot += w[r] * g[r];
    }
    dot = seg_sum<L>(dot);  // all: without the largest share's
    const float mean = all ? dot + p0 * seg_sum<L>(g_top) : dot;
#pragma unroll
    for (int r = 0; r < KR; ++r) {
        if (e[r] >= 0) {
            float d = g[r];
            if (a.renorm) d = (g[r] - dot) + rest * g0;
            else if (all) d = e[r] == e_top ? others * g[r] - dot : g[r] - mean;
            s_row[tb][e[r]] = a.sigmoid ? f * d * s[r] * ns[r] : a.scale * w[r] * d;
        }
    }
    __syncthreads();
    if (!real) return;
    float o[V];
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] = s_row[tb][e0 + v];
    if (all) {
        const float c = z != 0.f ? a.scale * mean / z : 0.f;  // 0: every expert is masked
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = __float_as_uint(o[v]) == kNotChosen ? 0.f - c * lg[v] : o[v];
    }
    const int64_t at = tok * a.ld_d + e0;
    if constexpr (BF16) {
        uint16_t* p = reinterpret_cast<uint16_t*>(a.dlogits) + at;
        uint16_t h[V];
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = __builtin_bit_cast(uint16_t, (__bf16)o[v]);
        if (a.vec_d && e0 + V <= E) {
#pragma unroll
            for (int i = 0; i < V / 8; ++i) {
                uint4 q;
                q.x = h[8 * i] | ((uint32_t)h[8 * i + 1] << 16);
                q.y = h[8 * i + 2] | ((uint32_t)h[8 * i + 3] << 16);
                q.z = h[8 * i + 4] | ((uint32_t)h[8 * i + 5] << 16);
                q.w = h[8 * i + 6] | ((uint32_t)h[8 * i + 7] << 16);
                reinterpret_cast<uint4*>(p)[i] = q;
            }
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (e0 + v < E) p[v] = h[v];
        }
    } else {
        float* p = reinterpret_cast<float*>(a.dlogits) + at;
        if (a.vec_d && e0 + V <= E) {
#pragma unroll
            for (int i = 0; i < V / 4; ++i)
                reinterpret_cast<float4*>(p)[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (e0 + v < E) p[v] = o[v];
        }
    }
}

template <int L, int V>
hipError_t route_lv(RouteArgs a, hipStream_t stream) {
    constexpr int TPB = kThreads / L;
    const dim3 grid((unsigned)((a.T + TPB - 1) / TPB)), block(kThreads);
    const bool scores = a.bias != nullptr || a.n_group > 1;
    // Every group a power of two of whole lanes: its best are found between
    // lanes.  LDS of a token: its logits, then the groups' scores, or with
    // other groups E keys and those; the exact path puts E + n_group float64
    // keys in the place of all that.
    const int64_t lanes = a.E / a.n_group / V;
    const bool whole = lanes * V * a.n_group == a.E && (lanes & (lanes - 1)) == 0;
    int64_t words = L * V;
    if (a.n_group > 1) {
        words += a.n_group + (whole ? 0 : a.E);
        if (2 * (a.E + a.n_group) > words) words = 2 * (a.E + a.n_group);
    }
    a.lds_token = (int32_t)((words + 3) / 4 * 4);
    const size_t lds = (size_t)TPB * a.lds_token * sizeof(float);
    if (a.bf16 && scores) hipLaunchKernelGGL((route_kernel<true, L, V, true>), grid, block, lds, stream, a, whole);
    else if (a.bf16) hipLaunchKernelGGL((route_kernel<true, L, V, false>), grid, block, lds, stream, a, whole);
    else if (scores) hipLaunchKernelGGL((route_kernel<false, L, V, true>), grid, block, lds, stream, a, whole);
    else hipLaunchKernelGGL((route_kernel<false, L, V, false>), grid, block, lds, stream, a, whole);
    return hipGetLastError();
}

template <int L, int V>
hipError_t route_bwd_lv(const RouteBwdArgs& a, hipStream_t stream) {
    constexpr int TPB = kThreads / L;
    const dim3 grid((unsigned)((a.T + TPB - 1) / TPB)), block(kThreads);
    if (a.bf16) hipLaunchKernelGGL((route_bwd_kernel<true, L, V>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((route_bwd_kernel<false, L, V>), grid, block, 0, stream, a);
    return hipGetLastError();
}

}  // namespace

// Lanes per token by the expert count: the fewest whose registers hold the
// row at 8 or 16 experts a lane.
#define BS_ROUTE_BY_E(FN)                       \
    if (a.E <= 8) return FN<1, 8>(a, stream);   \
    if (a.E <= 32) return FN<4, 8>(a, stream);  \
    if (a.E <= 64) return FN<8, 8>(a, stream);  \
    if (a.E <= 128) return FN<16, 8>(a, stream);  \
    if (a.E <= 256) return FN<16, 16>(a, stream); \
    if (a.E <= 512) return FN<32, 16>(a, stream); \
    return FN<64, 16>(a, stream);

hipError_t launch_route(const RouteArgs& a, hipStream_t stream) { BS_ROUTE_BY_E(route_lv) }
hipError_t launch_route_bwd(const RouteBwdArgs& a, hipStream_t stream) { BS_ROUTE_BY_E(route_bwd_lv) }

}  // namespace bs
