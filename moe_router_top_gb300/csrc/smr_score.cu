// smr_score.cu -- scores, groups and top-k of token rows whose logits are in
// memory: softmax or sigmoid scores, a balance bias that acts on the choice
// alone, groups of experts of which only the best stay, weights renormalised
// or not and scaled ("[AMD] One-launch small-M MoE router for Qwen3.5 on
// gfx950", Modifications, names the fused gate with groups and a bias as what
// its unit test compares with).
//
// For a row of logits x (NaN and -inf count as the lowest finite number, +inf
// as the largest), scores s = sigmoid(x) or softmax(x) and choices c = s + b:
//   group value = sum of the `best` (1 or 2) largest c of the group;
//   the `kept` groups of the largest values stay (ties: the lower index);
//   slots = the k largest c of those, ordered by (c desc, id asc);
//   weight = s (over the sum of the selected s) * routed_scale.
// The choice is taken as in 64 bits. Without a bias c is ordered like x, so x
// itself is compared. With one, c is evaluated in 32 bits with a bound on its
// error; a row where two choices that the bound does not tell apart would
// decide (about one in 500) is decided again in 64 bits.
//
// One warp per row. A group's experts lie next to each other on L lanes
// (groups as many as the next power of two, L = 32 / groups), nk of them on a
// lane, so that ids ascend with (lane, place) and a group is a range of lanes.
#include <float.h>

#include "smr_device.cuh"
#include "smr_launch.h"

namespace smr {

constexpr int kScoreWarps = 8;

// Where a lane's experts are.
struct ScoreLane {
    int first, count;  // its first expert; how many it holds
    int nk;            // places a lane has
    int L;             // lanes of a group
};
__device__ __forceinline__ ScoreLane score_lane(const ScoreLaunch &p, int lane) {
    ScoreLane s;
    s.L = 32 >> p.log_groups;
    const int gs = p.group_size, g = lane / s.L, sub = lane % s.L;
    s.nk = p.nk;
    s.first = g * gs + sub * s.nk;
    s.count = g < p.groups ? max(0, min(s.nk, gs - sub * s.nk)) : 0;
    return s;
}

// The finite value that a logit or a bias counts as.
__device__ __forceinline__ float to_finite(float x) { return fminf(fmaxf(x, -FLT_MAX), FLT_MAX) + 0.0f; }

template <bool F32>
__device__ __forceinline__ float load_logit(const ScoreLaunch &p, int64_t row, int e) {
    if constexpr (F32) return to_finite(__ldcg(static_cast<const float *>(p.logits) + row * p.ld + e));
    else return to_finite(__uint_as_float((uint32_t)__ldcg(static_cast<const uint16_t *>(p.logits) + row * p.ld + e) << 16));
}
__device__ __forceinline__ float load_bias(const ScoreLaunch &p, int e) { return to_finite(__ldcg(p.bias + e)); }

// A float's bits as an unsigned number of the same order (0 below them all).
__device__ __forceinline__ uint32_t ordered(float v) {
    const uint32_t b = __float_as_uint(v);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t u) {
    return __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
}

__device__ __forceinline__ float exp2_fast(float t) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(t));
    return r;
}
constexpr float kLog2e = 1.44269504f;
// sigmoid(x) within 4e-7: with t = -x log2(e) (relative error 2^-23) and e =
// 2^t, e's relative error is below |x| 2^-23 + 2^-22 and moves s by s (1 - s)
// times that, at most 0.23 * 2^-23 + 2^-24; the sum and its reciprocal add
// 2^-24 + 2^-23 of s.
__device__ __forceinline__ float sigmoid_fast(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + exp2_fast(x * -kLog2e)));
    return r;
}

// The choice of a row in 64 bits: what the 32-bit one cannot tell apart. Lane
// j gets slot j's expert. Rare, so it reads the row again and takes its time.
template <int NK, bool F32>
__device__ __noinline__ int select_in_64_bits(const ScoreLaunch &p, int64_t row) {
    const int lane = threadIdx.x & 31;
    const ScoreLane at = score_lane(p, lane);
    double c[NK];
    double top = -DBL_MAX;
#pragma unroll 1
    for (int i = 0; i < at.count; ++i) {
        c[i] = (double)load_logit<F32>(p, row, at.first + i);
        top = fmax(top, c[i]);
    }
    double sum = 0.0;
    if (!p.sigmoid) {
#pragma unroll 1
        for (int o = 16; o >= 1; o >>= 1) top = fmax(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll 1
        for (int i = 0; i < at.count; ++i) sum += c[i] = exp(c[i] - top);
#pragma unroll 1
        for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    double m1 = -INFINITY, m2 = -INFINITY;  // the lane's two largest
#pragma unroll 1
    for (int i = 0; i < at.count; ++i) {
        double s = p.sigmoid ? 1.0 / (1.0 + exp(-c[i])) : c[i] / sum;
        if (p.bias != nullptr) s += (double)load_bias(p, at.first + i);
        c[i] = s;
        m2 = fmax(m2, fmin(m1, s));
        m1 = fmax(m1, s);
    }
    __syncwarp();
    bool stays = at.count > 0;
    if (p.groups > 1) {
#pragma unroll 1
        for (int o = at.L >> 1; o >= 1; o >>= 1) {
            const double o1 = __shfl_xor_sync(0xffffffffu, m1, o), o2 = __shfl_xor_sync(0xffffffffu, m2, o);
            m2 = fmax(fmin(m1, o1), fmax(m2, o2));
            m1 = fmax(m1, o1);
        }
        const double value = p.best == 2 ? m1 + m2 : m1;
        const int g = lane / at.L;
        int above = 0;
#pragma unroll 1
        for (int h = 0; h < p.groups; ++h) {
            const double v = __shfl_sync(0xffffffffu, value, h * at.L);
            above += v > value || (v == value && h < g);
        }
        stays = stays && above < p.kept;
    }
    if (p.bias == nullptr)  // as above: in the logits' order
#pragma unroll 1
        for (int i = 0; i < at.count; ++i) c[i] = (double)load_logit<F32>(p, row, at.first + i);
    __syncwarp();
    uint32_t taken = 0u;
    int mine = 0;
#pragma unroll 1
    for (int j = 0; j < p.k; ++j) {
        double best = -INFINITY;
        int id = 0x7FFFFFFF;
        if (stays)
#pragma unroll 1
            for (int i = 0; i < at.count; ++i)
                if (!(taken >> i & 1u) && (c[i] > best || id == 0x7FFFFFFF)) {
                    best = c[i];
                    id = at.first + i;
                }
        __syncwarp();
#pragma unroll 1
        for (int o = 16; o >= 1; o >>= 1) {
            const double ob = __shfl_xor_sync(0xffffffffu, best, o);
            const int oi = __shfl_xor_sync(0xffffffffu, id, o);
            if (ob > best || (ob == best && oi < id)) {
                best = ob;
                id = oi;
            }
        }
        if (id >= at.first && id < at.first + at.count) taken |= 1u << (id - at.first);
        if (lane == j) mine = id;
    }
    return mine;
}

// Bound by its instructions for large batches and by latency for small ones;
// what it reads is the logits, once.
template <int NK, bool F32>
__global__ void __launch_bounds__(32 * kScoreWarps) select_experts_kernel(const ScoreLaunch p) {
    griddep_launch_dependents();  // the next kernel may launch; it waits for this grid
    griddep_wait();               // the logits come from the previous kernel
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * kScoreWarps + (threadIdx.x >> 5);
    if (row >= p.M) return;  // warp-uniform
    const ScoreLane at = score_lane(p, lane);
    float x[NK];
#pragma unroll
    for (int i = 0; i < NK; ++i) x[i] = i < at.count ? load_logit<F32>(p, row, at.first + i) : -INFINITY;
    if (p.logits_out != nullptr) {
#pragma unroll
        for (int i = 0; i < NK; ++i)
            if (i < at.count)
                p.logits_out[row * p.E + at.first + i] = __ldcg(static_cast<const uint16_t *>(p.logits) + row * p.ld + at.first + i);
    }

    // softmax: the row's largest logit and the sum of the exponentials
    float top = 0.0f, den = 1.0f;
    const bool soft = !p.sigmoid;
    if (soft && (p.bias != nullptr || !p.renorm || p.best == 2)) {
        float m = x[0];
#pragma unroll
        for (int i = 1; i < NK; ++i) m = fmaxf(m, x[i]);
        top = unordered(__reduce_max_sync(0xffffffffu, ordered(m)));
        float e[NK];
#pragma unroll
        for (int i = 0; i < NK; ++i) e[i] = exp2_fast((x[i] - top) * kLog2e);  // (0 where there is no expert)
#pragma unroll
        for (int h = NK / 2; h >= 1; h >>= 1)
#pragma unroll
            for (int i = 0; i < h; ++i) e[i] += e[i + h];
        den = e[0];
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    }
    const float inv = __frcp_rn(den);

    // choices; without a bias the logits themselves, which have their order
    float c[NK];
    // how far a choice in 32 bits may be off, twice: 4e-7 of a sigmoid, 2e-6
    // of a softmax (its sum of up to ten roundings), half a unit of c itself
    const float slack = p.bias == nullptr ? 0.0f : (soft ? 4e-6f : 8e-7f);
    if (p.bias != nullptr) {
#pragma unroll
        for (int i = 0; i < NK; ++i) {
            const float s = soft ? exp2_fast((x[i] - top) * kLog2e) * inv : sigmoid_fast(x[i]);
            c[i] = i < at.count ? s + load_bias(p, at.first + i) : -INFINITY;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NK; ++i) c[i] = x[i];
    }

    bool unsure = false;
    if (p.groups > 1) {
        float m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll
        for (int i = 0; i < NK; ++i) {
            m2 = fmaxf(m2, fminf(m1, c[i]));
            m1 = fmaxf(m1, c[i]);
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) {
            if (o >= at.L) continue;
            const float o1 = __shfl_xor_sync(0xffffffffu, m1, o), o2 = __shfl_xor_sync(0xffffffffu, m2, o);
            m2 = fmaxf(fminf(m1, o1), fmaxf(m2, o2));
            m1 = fmaxf(m1, o1);
        }
        float value = m1, mag = fabsf(m1);  // (mag: what its rounding goes by)
        if (p.best == 2) {
            if (p.bias == nullptr) {  // of logits: their scores
                m1 = soft ? exp2_fast((m1 - top) * kLog2e) : sigmoid_fast(m1);
                m2 = soft ? exp2_fast((m2 - top) * kLog2e) : sigmoid_fast(m2);
            }
            value = fmaxf(m1 + m2, -FLT_MAX);
            mag = fabsf(m1) + fabsf(m2);
        }
        const int g = lane / at.L;
        if (g >= p.groups) {
            value = -INFINITY;
            mag = 0.0f;
        }
        int above = 0;
#pragma unroll 1
        for (int h = 0; h < p.groups; ++h) {
            const float v = __shfl_sync(0xffffffffu, value, h * at.L);
            above += v > value || (v == value && h < g);
        }
        const bool stays = above < p.kept;
        if (p.bias != nullptr || p.best == 2) {
            // the least of the groups that stay and the best of the others
            const float lo = unordered(__reduce_min_sync(0xffffffffu, ordered(stays ? value : INFINITY)));
            const float hi = unordered(__reduce_max_sync(0xffffffffu, ordered(stays ? -INFINITY : value)));
            const float most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mag)));
            unsure = hi > -INFINITY && !(lo - hi > 2.0f * (soft ? 4e-6f : 8e-7f) + 5e-7f * most);
        }
        if (!stays) {
#pragma unroll
            for (int i = 0; i < NK; ++i) c[i] = -INFINITY;
        }
        __syncwarp();
    }

    // the k largest, and the one after them; lane j keeps slot j
    float cj = 0.0f, xj = 0.0f, ca = -INFINITY, xa = 0.0f;  // (a: the one after)
    int ej = 0, ea = -1;
    float best = -INFINITY;
    int bi = 0;
#pragma unroll
    for (int i = 0; i < NK; ++i)
        if (c[i] > best) {
            best = c[i];
            bi = i;
        }
    const int rounds = p.bias != nullptr ? p.k + 1 : p.k;
#pragma unroll 1
    for (int j = 0; j < rounds; ++j) {
        const uint32_t u = ordered(best), m = __reduce_max_sync(0xffffffffu, u);
        const int w = __ffs(__ballot_sync(0xffffffffu, u == m)) - 1;
        float bx = 0.0f;
        if (lane == w) {
            float b2 = -INFINITY;
            int i2 = 0;
#pragma unroll
            for (int i = 0; i < NK; ++i) {
                if (i == bi) {
                    bx = x[i];
                    c[i] = -INFINITY;
                }
                if (c[i] > b2) {
                    b2 = c[i];
                    i2 = i;
                }
            }
            ea = at.first + bi;  // (passed on below)
            best = b2;
            bi = i2;
        }
        __syncwarp();
        const float cw = unordered(m), xw = __shfl_sync(0xffffffffu, bx, w);
        const int ew = __shfl_sync(0xffffffffu, ea, w);
        if (lane == j && j < p.k) {
            cj = cw;
            xj = xw;
            ej = ew;
        }
        if (j == p.k) {
            ca = cw;
            xa = xw;
            ea = ew;
        }
    }
    if (p.bias != nullptr) {
        // every slot against the next: told apart, or equal in logit and bias
        // (then equal, and the lower id comes first)
        float cn = __shfl_down_sync(0xffffffffu, cj, 1), xn = __shfl_down_sync(0xffffffffu, xj, 1);
        int en = __shfl_down_sync(0xffffffffu, ej, 1);
        if (lane == p.k - 1) {
            cn = ca;
            xn = xa;
            en = ea;
        }
        bool close = lane < p.k && cn > -INFINITY && !(cj - cn > slack + 2.5e-7f * fmaxf(fabsf(cj), fabsf(cn)));
        if (close && xj == xn) close = load_bias(p, ej) != load_bias(p, en);
        unsure = unsure || __any_sync(0xffffffffu, close);
    }
    if (__any_sync(0xffffffffu, unsure)) {
        ej = select_in_64_bits<NK, F32>(p, row);
        if (lane < p.k) xj = load_logit<F32>(p, row, ej);
        __syncwarp();
    }

    // weights
    const bool slot = lane < p.k;
    float n;
    if (soft) {
        if (p.renorm) top = unordered(__reduce_max_sync(0xffffffffu, ordered(slot ? xj : -FLT_MAX)));
        n = expf(xj - top);
    } else {
        // s = e^x / (1 + e^x) below 0, 1 / (1 + e^-x) above; renormalised
        // scores of logits that are all negative are taken relative to the
        // largest e^x, so that they keep their ratios however small they are
        float shift = 0.0f;
        if (p.renorm) shift = fminf(0.0f, unordered(__reduce_max_sync(0xffffffffu, ordered(slot ? xj : -FLT_MAX))));
        n = xj < 0.0f ? expf(xj - shift) / (1.0f + expf(xj)) : 1.0f / (1.0f + expf(-xj));
    }
    float sum = slot ? n : 0.0f;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float w = (p.renorm ? n / sum : (soft ? n / den : n)) * p.routed_scale;
    const int width = p.k + p.S;
    if (slot) {
        p.ids[row * width + lane] = ej;
        p.wts[row * width + lane] = w;
    } else if (p.S != 0 && lane == p.k && !p.shared_done) {
        float v = p.shared_scale;
        if (p.shared != nullptr) {
            const float s = __ldcg(p.shared + row);
            v *= sigmoid_stable(p.shared_bf16 ? round_bf16(s) : s);
        }
        p.ids[row * width + p.k] = p.E;
        p.wts[row * width + p.k] = v;
    }
}

int score_places(int E, int groups, int *log_groups) {
    int lg = 0;
    while ((1 << lg) < groups) ++lg;
    if (log_groups) *log_groups = lg;
    const int L = 32 >> lg;
    return L < 1 ? 1 << 30 : (E / groups + L - 1) / L;
}

template <int NK>
static cudaError_t launch_nk(const ScoreLaunch &a, const cudaLaunchConfig_t &cfg) {
    return a.f32 ? cudaLaunchKernelEx(&cfg, select_experts_kernel<NK, true>, a)
                 : cudaLaunchKernelEx(&cfg, select_experts_kernel<NK, false>, a);
}

cudaError_t launch_select_experts(const ScoreLaunch &in, cudaStream_t stream) {
    ScoreLaunch a = in;
    a.nk = score_places(a.E, a.groups, &a.log_groups);
    a.group_size = a.E / a.groups;
    a.best = a.groups == 1 ? 1 : (a.best < a.group_size ? a.best : a.group_size);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.M + kScoreWarps - 1) / kScoreWarps), 1, 1);
    cfg.blockDim = dim3(32 * kScoreWarps, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (a.nk <= 4) return launch_nk<4>(a, cfg);
    if (a.nk <= 8) return launch_nk<8>(a, cfg);
    if (a.nk <= 16) return launch_nk<16>(a, cfg);
    return a.nk <= kScoreMaxPlaces ? launch_nk<32>(a, cfg) : cudaErrorNotSupported;
}

}  // namespace smr
