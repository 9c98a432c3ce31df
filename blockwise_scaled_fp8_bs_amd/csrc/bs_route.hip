// Router of an MoE layer for gfx950: scores, balance bias, expert groups,
// top-k and weights, and the gradient of the logits.
//
// A token is owned by L lanes of a wave (L a power of two, by the expert
// count), each holding V consecutive experts in registers, so that a wave
// routes 64 / L tokens at once and a reduction over a token's experts is
// log2(L) lane exchanges.  The choice is between values that may lie next to
// one another, so it is made on exact keys: the logits themselves where no
// bias is added (scores rise with their logits), float64 scores otherwise
// (gfx950 runs float64 vector arithmetic at the unpacked fp32 rate).  Equal
// keys go to the lowest expert: a lane's experts are consecutive, so that is
// the lowest lane of the ballot and its first maximum.
#include "bs_moe.h"
#include "bs_device.h"

namespace bs {

namespace {

constexpr int kThreads = 256;
constexpr double kTinySum = 1e-20;  // added to the sum of the chosen sigmoid scores

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
    if (vec && e0 + V <= E) {
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
#pragma unroll
        for (int v = 0; v < V; ++v) f[v] = e0 + v < E ? load_logit(base, BF16, row + e0 + v) : kNegInf;
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

// F64: the keys are float64 scores (a bias or groups are in play).
template <bool BF16, int L, int V, bool F64>
__global__ __launch_bounds__(kThreads) void route_kernel(RouteArgs a) {
    extern __shared__ double s_dyn[];
    using Key = typename std::conditional<F64, double, float>::type;
    constexpr Key kNone = -(Key)__builtin_inff();
    constexpr int TPB = kThreads / L;  // tokens of a block
    constexpr int KR = (int)kMaxTopK < V * L ? ((int)kMaxTopK + L - 1) / L : V;  // slots a lane may hold

    const int l = threadIdx.x % L, tb = threadIdx.x / L;
    const int seg = (threadIdx.x & 63) / L * L;  // first lane of the token
    const int64_t tok = (int64_t)blockIdx.x * TPB + tb;
    const bool real = tok < a.T;
    const int64_t row = (real ? tok : a.T - 1) * a.ld;
    const int E = (int)a.E, e0 = l * V;

    float lg[V];
    load_logits<BF16, V>(a.logits, row, e0, E, a.vec, lg);

    float m = 0.f;
    double z = 1.0;  // softmax: the largest logit and the sum of exp(l - m)
    const bool need_z = !a.sigmoid && (F64 || !a.renorm);
    if (need_z) {
        m = kNegInf;
#pragma unroll
        for (int v = 0; v < V; ++v) m = fmaxf(m, lg[v]);
        m = seg_max<L>(m);
    }
    Key key[V];
    if constexpr (F64) {
        double sum = 0.0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const double d = lg[v];
            key[v] = a.sigmoid ? sigmoid64(d) : (lg[v] == kNegInf ? 0.0 : exp(d - (double)m));
            sum += key[v];
        }
        if (!a.sigmoid) {
            z = seg_sum<L>(sum);
            const double r = 1.0 / z;
#pragma unroll
            for (int v = 0; v < V; ++v) key[v] *= r;
        }
        if (a.bias != nullptr) {
#pragma unroll
            for (int v = 0; v < V; ++v) key[v] += e0 + v < E ? (double)a.bias[e0 + v] : 0.0;
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
            double* const mine = s_dyn + tb * (E + G);
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
    } else {
        if (need_z) {
            float sum = 0.f;
#pragma unroll
            for (int v = 0; v < V; ++v) sum += lg[v] == kNegInf ? 0.f : expf(lg[v] - m);
            z = (double)seg_sum<L>(sum);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) key[v] = lg[v] != lg[v] ? __builtin_inff() : lg[v];
    }

    // k rounds: the best key left, its expert to the lane that holds slot j
    int32_t mine_idx[KR];
#pragma unroll
    for (int r = 0; r < KR; ++r) {
        mine_idx[r] = -1;
        for (int q = 0; q < L; ++q) {
            if (r * L + q >= a.k) break;
            Key bm = key[0];
            int bi = 0;
#pragma unroll
            for (int v = 1; v < V; ++v) {
                if (key[v] > bm) {
                    bm = key[v];
                    bi = v;
                }
            }
            int e = e0 + bi;
            Key mx = bm;
            bool win = true;
            if constexpr (L > 1) {
                mx = seg_max<L>(bm);
                uint64_t vote = __ballot(bm == mx) >> seg;
                if constexpr (L < 64) vote &= (1ull << L) - 1;
                const int first = __builtin_ctzll(vote);
                win = first == l;
                e = __shfl(e, seg + first);
            }
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (win && v == bi) key[v] = kNone;
            if (q == l && mx > kNone) mine_idx[r] = e;
        }
    }

    // weights of the chosen experts, in float64 (a few values per token)
    double s[KR];
    float top = kNegInf;
    if (!a.sigmoid && a.renorm) {
#pragma unroll
        for (int r = 0; r < KR; ++r) {
            if (r * L >= a.k) break;
            if (mine_idx[r] >= 0) top = fmaxf(top, load_logit(a.logits, BF16, row + mine_idx[r]));
        }
        top = seg_max<L>(top);
    }
    double sum = 0.0;
#pragma unroll
    for (int r = 0; r < KR; ++r) {
        s[r] = 0.0;
        if (r * L >= a.k) continue;
        if (mine_idx[r] >= 0) {
            const double d = load_logit(a.logits, BF16, row + mine_idx[r]);
            s[r] = a.sigmoid ? sigmoid64(d) : a.renorm ? exp(d - (double)top) : exp(d - (double)m) / z;
        }
        sum += s[r];
    }
    double f = a.scale;
    if (a.renorm) {
        sum = seg_sum<L>(sum);
        if (a.sigmoid) sum += kTinySum;
        f /= sum;
    }
    if (!real) return;
#pragma unroll
    for (int r = 0; r < KR; ++r) {
        const int j = r * L + l;
        if (j < a.k) {
            a.idx[tok * a.k + j] = mine_idx[r];
            a.w[tok * a.k + j] = mine_idx[r] >= 0 ? (float)(s[r] * f) : 0.f;
        }
    }
}

// Gradient of the logits.  The k contributions of a token are placed in an
// LDS row, which the lanes then add to what they hold and write out whole.
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
#pragma unroll
    for (int v = 0; v < V; ++v) s_row[tb][e0 + v] = 0.f;
    __syncthreads();

    float m = kNegInf, z = 1.f;
    float lg[V];
    const bool all = !a.sigmoid && !a.renorm;  // every logit of the row has a gradient
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
                    s[r] = 1.f / (1.f + expf(-d));
                    ns[r] = 1.f / (1.f + expf(d));  // 1 - s, without the cancellation
                }
            }
        }
        dot += w[r] * g[r];
        ssum += s[r];
    }
    dot = seg_sum<L>(dot);
    float f = a.scale;
    if (a.sigmoid && a.renorm) f = a.scale / (seg_sum<L>(ssum) + (float)kTinySum);
#pragma unroll
    for (int r = 0; r < KR; ++r) {
        if (e[r] >= 0) {
            const float d = a.renorm ? g[r] - dot : g[r];
            s_row[tb][e[r]] = a.sigmoid ? f * d * s[r] * ns[r] : a.scale * w[r] * d;
        }
    }
    __syncthreads();
    if (!real) return;
    float o[V];
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] = s_row[tb][e0 + v];
    if (all) {
        const float c = z != 0.f ? a.scale * dot / z : 0.f;  // 0: every expert is masked
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] -= c * lg[v];
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
hipError_t route_lv(const RouteArgs& a, hipStream_t stream) {
    constexpr int TPB = kThreads / L;
    const dim3 grid((unsigned)((a.T + TPB - 1) / TPB)), block(kThreads);
    const bool f64 = a.bias != nullptr || a.n_group > 1;
    const size_t lds = a.n_group > 1 ? (size_t)TPB * (a.E + a.n_group) * sizeof(double) : 0;
    if (a.bf16 && f64) hipLaunchKernelGGL((route_kernel<true, L, V, true>), grid, block, lds, stream, a);
    else if (a.bf16) hipLaunchKernelGGL((route_kernel<true, L, V, false>), grid, block, 0, stream, a);
    else if (f64) hipLaunchKernelGGL((route_kernel<false, L, V, true>), grid, block, lds, stream, a);
    else hipLaunchKernelGGL((route_kernel<false, L, V, false>), grid, block, 0, stream, a);
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
