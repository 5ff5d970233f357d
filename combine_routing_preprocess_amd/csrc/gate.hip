// The gate: the top-k experts of each token and their weights from the
// router's logits, written in the handle's routing format, and its gradient.
//
//   score   s_e = softmax(l)_e  or  sigmoid(l_e)
//   choice  the K largest keys, key_e = l_e, or s_e + bias_e with a bias; ties
//           go to the lowest expert; an expert whose logit or key is NaN or
//           -inf is never chosen and has no share of the softmax
//   weight  p_j = scale * s_j, or scale * s_j / (sum of the chosen s)
//   gradient, with G_j the weight's and q_j = s_j / (sum of the chosen s):
//     softmax               gl_e = scale * s_e * (G_e [chosen] - sum_j G_j s_j)
//     softmax, normalised   gl_j = scale * q_j * (G_j - sum_i G_i q_i)
//     sigmoid               gl_j = scale * G_j * s_j * (1 - s_j)
//     sigmoid, normalised   gl_j = scale * q_j * (1 - s_j) * (G_j - sum_i G_i q_i)
//
// One wavefront per token; lane l holds experts l, l + 64, ... (EPL of them).
// Neither direction moves many bytes (a row of logits, K weights): the time
// goes into the K selection rounds and the 64-bit scores, so that is what the
// layout is for.
//  * With a bias the keys are 64-bit floats: score + bias decides between
//    experts that 32 bits cannot tell apart, and the choice is an integer that
//    must not hang on a rounding.  Without one the logits themselves rank the
//    experts, exactly.  Either way a key becomes an unsigned integer of the
//    same order; a round takes the maximum of the upper 32 bits over the lanes
//    (lane permutes, no LDS), a ballot finds who holds it, and the lower 32 bits
//    are looked at only where several do.  The winner is scalar, so lane j
//    keeps slot j's expert and logit without any exchange.
//  * exp and the reciprocal below are for arguments that occur here (x <= 0
//    and 1 <= d <= 2) and take some 20 and 6 instructions instead of the
//    library's general forms.
//  * Measured on MI355X, 256 experts top-8 with bias, in long runs of calls:
//    8192 tokens in 9.6 us, 11.1 in a run of a dozen (the logits alone would
//    take 1.7 us; with shuffles through LDS and the library's exp 26 us), 16
//    tokens in 4.4 us; gradient of 8192 tokens 7.9 us, of a Boolean map 10 us
//    (softmax over the row 13).  More than 64 slots: 8192 tokens, 160 experts
//    top-96 in 49 us, their gradient in 48.
#include "wave_ops.h"

namespace moe {
namespace {

using namespace ops;

constexpr double kOut = -INFINITY;   // logit or key of an expert that is no candidate
constexpr double kTiny = 1e-260;     // sums of sigmoids below this are formed from logarithms, so that the largest
                                     // scale over a sum (3.4e38 / 1e-260) stays a 64-bit number

// exp(x) for x <= 0 (0 for NaN): x = n ln 2 + r with |r| <= ln 2 / 2 (ln 2 in
// two parts), the Taylor polynomial of degree 13 at r (next term 4e-18),
// scaled by 2^n.
__device__ __forceinline__ double exp_neg(double x) {
    x = fmax(x, -1100.0);
    const double n = rint(x * 1.4426950408889634);
    double r = fma(n, -0x1.62e42fefa3800p-1, x);      // the upper 42 bits of ln 2: n times it is exact
    r = fma(n, -0x1.ef35793c76730p-45, r);
    double p = 1.0 / 6227020800.0;
    p = fma(p, r, 1.0 / 479001600.0);
    p = fma(p, r, 1.0 / 39916800.0);
    p = fma(p, r, 1.0 / 3628800.0);
    p = fma(p, r, 1.0 / 362880.0);
    p = fma(p, r, 1.0 / 40320.0);
    p = fma(p, r, 1.0 / 5040.0);
    p = fma(p, r, 1.0 / 720.0);
    p = fma(p, r, 1.0 / 120.0);
    p = fma(p, r, 1.0 / 24.0);
    p = fma(p, r, 1.0 / 6.0);
    p = fma(p, r, 0.5);
    p = fma(p, r, 1.0);
    p = fma(p, r, 1.0);
    return __builtin_amdgcn_ldexp(p, (int)n);
}

// sigmoid(l) and sigmoid(-l): with e = exp(-|l|), 1 / (1 + e) and e / (1 + e);
// the reciprocal from the hardware's estimate by two Newton steps.
__device__ __forceinline__ void sigmoids(double l, double* s, double* other) {
    const double e = exp_neg(-fabs(l)), d = 1.0 + e;
    double y = __builtin_amdgcn_rcp(d);
    y = fma(y, fma(-d, y, 1.0), y);
    y = fma(y, fma(-d, y, 1.0), y);
    const double z = e * y;
    *s = l < 0.0 ? z : y;
    *other = l < 0.0 ? y : z;
}
__device__ __forceinline__ double sigmoid_of(double l) {
    double s, o;
    sigmoids(l, &s, &o);
    return s;
}
__device__ __forceinline__ double log_sigmoid(double l) { return fmin(l, 0.0) - log1p(exp(-fabs(l))); }

// A logit as a float (exact); NaN reads as no candidate, -0 as 0.
template <typename LT>
__device__ __forceinline__ float load_logit(const LT* p) {
    float v;
    if constexpr (sizeof(LT) == 2) v = __uint_as_float((uint32_t)*p << 16);
    else v = *p;
    return v == v ? v + 0.f : -INFINITY;
}

// Unsigned integers in the order of the floats (all above 0 but -inf and NaN,
// which the callers leave out).
__device__ __forceinline__ uint32_t ordered(float v) {
    const uint32_t u = __float_as_uint(v);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint64_t ordered(double v) {
    const uint64_t u = (uint64_t)__double_as_longlong(v);
    return u ^ ((uint64_t)((int64_t)u >> 63) | 0x8000000000000000ull);
}

// Maximum of the row's logits and the sum of exp(l - max) (softmax).
template <int EPL>
__device__ __forceinline__ void softmax_terms(const float (&l)[EPL], double* m, double* sum) {
    float top = l[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) top = fmaxf(top, l[i]);
    *m = wave_max_dpp((double)top);
    double a = 0.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) a += l[i] == -INFINITY ? 0.0 : exp_neg((double)l[i] - *m);
    *sum = wave_sum_dpp(a);
}

// The K choices, one per round.  On return lane j < n holds slot j's expert
// (the first 64), and with TAKEN taken[i] says in which slot the lane's expert
// i is.  Who holds the round's largest key is looked up by ballots, so that
// this work is scalar: ordering each lane's experts first, for rounds that
// look at the lanes' heads only, took 14.4 us against 11.2 at 8192 x 256.
template <int EPL, bool BIAS, bool SIGMOID, bool TAKEN>
__device__ __forceinline__ int choose(const float (&l)[EPL], const float* bias, int E, int K, double m, double sum,
                                      int lane, int* my_e, int (&taken)[EPL]) {
    uint32_t hi[EPL], lo[EPL];
    const double inv = BIAS && !SIGMOID ? 1.0 / sum : 0.0;
    float be[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        if (BIAS) be[i] = bias[min(lane + 64 * i, E - 1)];
        if (TAKEN) taken[i] = -1;
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        lo[i] = 0u;
        if constexpr (BIAS) {
            const double s = SIGMOID ? sigmoid_of((double)l[i]) : exp_neg((double)l[i] - m) * inv;
            const double key = s + (double)be[i] + 0.0;
            const uint64_t u = l[i] != -INFINITY && key > kOut ? ordered(key) : 0u;
            hi[i] = (uint32_t)(u >> 32);
            lo[i] = (uint32_t)u;
        } else {
            hi[i] = l[i] != -INFINITY ? ordered(l[i]) : 0u;
        }
    }
    int n = 0;
    for (; n < K; ++n) {
        uint32_t top = hi[0];
#pragma unroll
        for (int i = 1; i < EPL; ++i) top = max(top, hi[i]);
        top = wave_max_dpp(top);
        if (top == 0u) break;   // no candidate is left
        uint64_t has[EPL];
#pragma unroll
        for (int i = 0; i < EPL; ++i) has[i] = __ballot(hi[i] == top);
        if (BIAS) {   // several holders: the lower halves decide
            int holders = 0;
#pragma unroll
            for (int i = 0; i < EPL; ++i) holders += __popcll(has[i]);
            if (holders > 1) {
                uint32_t low = 0u;
#pragma unroll
                for (int i = 0; i < EPL; ++i) low = max(low, hi[i] == top ? lo[i] : 0u);
                low = wave_max_dpp(low);
#pragma unroll
                for (int i = 0; i < EPL; ++i) has[i] = __ballot(hi[i] == top && lo[i] == low);
            }
        }
        bool found = false;   // the lowest expert: lowest i, then lowest lane
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (!found && has[i]) {
                found = true;
                const int at = __ffsll((unsigned long long)has[i]) - 1;
                if (lane == n) *my_e = at + 64 * i;
                if (lane == at) {
                    if (TAKEN) taken[i] = n;
                    hi[i] = 0u;
                }
            }
    }
    return n;
}

// K <= 64: a slot per lane.
template <typename LT, int FMT, int EPL, bool BIAS, bool SIGMOID>
__global__ __launch_bounds__(256) void k_gate(const LT* __restrict__ logits, int T, int E, int K,
                                              const float* __restrict__ bias, int normalize, float scale,
                                              void* __restrict__ routing, float* __restrict__ probs) {
    const int lane = threadIdx.x & 63;
    const long long t = (long long)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= T) return;
    const LT* row = logits + t * E;
    float l[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) l[i] = lane + 64 * i < E ? load_logit(row + lane + 64 * i) : -INFINITY;
    double m = 0.0, sum = 1.0;
    if (!SIGMOID && (BIAS || !normalize)) softmax_terms<EPL>(l, &m, &sum);
    int my_e = -1, taken[EPL];
    const int n = choose<EPL, BIAS, SIGMOID, FMT == MOE_ROUTE_SPARSE_BOOL>(l, bias, E, K, m, sum, lane, &my_e, taken);
    // weight of the lane's slot; its logit comes once more from the cache
    const bool on = lane < n;
    const double le = on ? (double)load_logit(row + my_e) : kOut;
    double w;
    if (SIGMOID) {
        w = on ? sigmoid_of(le) : 0.0;
        if (normalize) {
            sum = wave_sum_dpp(w);
            if (sum < kTiny) {   // the same for every lane
                const double ls = on ? log_sigmoid(le) : kOut;
                const double top = wave_max_dpp(ls);
                w = on ? exp(ls - top) : 0.0;
                sum = wave_sum_dpp(w);
            }
        }
    } else {
        if (normalize) m = wave_max_dpp(le);
        w = on ? exp_neg(le - m) : 0.0;
        if (normalize) sum = wave_sum_dpp(w);
    }
    const float p = on ? (float)(w * ((double)scale / sum)) : 0.f;
    if constexpr (FMT == MOE_ROUTE_SPARSE_BOOL) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = lane + 64 * i;
            const float pe = __shfl(p, taken[i] & 63, 64);
            if (e < E) {
                ((uint8_t*)routing)[t * E + e] = taken[i] >= 0;
                probs[t * E + e] = taken[i] >= 0 ? pe : 0.f;
            }
        }
    } else if (lane < K) {
        using IT = std::conditional_t<FMT == MOE_ROUTE_DENSE_I16, int16_t, int32_t>;
        ((IT*)routing)[t * K + lane] = (IT)my_e;
        probs[t * K + lane] = p;
    }
}

// Any K: slots stay with the experts' lanes.
template <typename LT, int FMT, int EPL>
__global__ __launch_bounds__(256) void k_gate_many(const LT* __restrict__ logits, int T, int E, int K,
                                                   const float* __restrict__ bias, int sigmoid, int normalize,
                                                   float scale, void* __restrict__ routing,
                                                   float* __restrict__ probs) {
    const int lane = threadIdx.x & 63;
    const long long t = (long long)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= T) return;
    float l[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) l[i] = lane + 64 * i < E ? load_logit(logits + t * E + lane + 64 * i) : -INFINITY;
    double m = 0.0, sum = 1.0;
    if (!sigmoid && (bias || !normalize)) softmax_terms<EPL>(l, &m, &sum);
    int my_e = -1, taken[EPL];
    const int n = !bias     ? choose<EPL, false, true, true>(l, bias, E, K, m, sum, lane, &my_e, taken)
                  : sigmoid ? choose<EPL, true, true, true>(l, bias, E, K, m, sum, lane, &my_e, taken)
                            : choose<EPL, true, false, true>(l, bias, E, K, m, sum, lane, &my_e, taken);
    double w[EPL], part = 0.0;
    if (normalize && !sigmoid) {
        m = kOut;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (taken[i] >= 0) m = fmax(m, (double)l[i]);
        m = wave_max_dpp(m);
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        w[i] = 0.0;
        if (taken[i] >= 0) w[i] = sigmoid ? sigmoid_of((double)l[i]) : exp_neg((double)l[i] - m);
        part += w[i];
    }
    if (normalize) {
        sum = wave_sum_dpp(part);
        if (sigmoid && sum < kTiny) {
            double top = kOut;
            part = 0.0;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                w[i] = taken[i] >= 0 ? log_sigmoid((double)l[i]) : kOut;
                top = fmax(top, w[i]);
            }
            top = wave_max_dpp(top);
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                w[i] = taken[i] >= 0 ? exp(w[i] - top) : 0.0;
                part += w[i];
            }
            sum = wave_sum_dpp(part);
        }
    }
    const double f = (double)scale / sum;
    if constexpr (FMT == MOE_ROUTE_SPARSE_BOOL) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = lane + 64 * i;
            if (e < E) {
                ((uint8_t*)routing)[t * E + e] = taken[i] >= 0;
                probs[t * E + e] = taken[i] >= 0 ? (float)(w[i] * f) : 0.f;
            }
        }
    } else {
        using IT = std::conditional_t<FMT == MOE_ROUTE_DENSE_I16, int16_t, int32_t>;
        IT* idx = (IT*)routing + t * K;
        float* p = probs + t * K;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (taken[i] >= 0) {
                idx[taken[i]] = (IT)(lane + 64 * i);
                p[taken[i]] = (float)(w[i] * f);
            }
        for (int j = n + lane; j < K; j += 64) {
            idx[j] = (IT)-1;
            p[j] = 0.f;
        }
    }
}

template <typename LT>
__device__ __forceinline__ void store_grad(LT* p, double v) {
    if constexpr (sizeof(LT) == 2) *p = (LT)f32_to_bf16((float)v);
    else *p = (float)v;
}

// Both backward kernels read all they need of a row before they write it: the
// gradient may take the logits' place.
//
// Dense routing, K <= 64: lane j has slot j.  Only the chosen experts' logits
// are read, but for the softmax over the whole row.
template <typename LT, typename IT, int EPL>
__global__ __launch_bounds__(256) void k_gate_backward(const float* __restrict__ grad_probs,
                                                       const LT* logits, const IT* __restrict__ routing, int T, int E,
                                                       int K, int sigmoid, int normalize, float scale,
                                                       LT* grad_logits) {
    const int lane = threadIdx.x & 63;
    const long long t = (long long)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= T) return;
    const LT* row = logits + t * E;
    const int e = lane < K ? (int)routing[t * K + lane] : -1;
    float le = -INFINITY;
    if (e >= 0 && e < E) le = load_logit(row + e);
    const bool on = le != -INFINITY;
    const double g = on ? (double)grad_probs[t * K + lane] : 0.0;
    double m = 0.0, sum = 1.0, o[EPL];
    const bool whole = !sigmoid && !normalize;
    float l[EPL];
    if (whole) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) l[i] = lane + 64 * i < E ? load_logit(row + lane + 64 * i) : -INFINITY;
        softmax_terms<EPL>(l, &m, &sum);
    } else if (!sigmoid) {
        m = wave_max_dpp((double)le);
    }
    double p = 0.0, rest = 1.0;   // the slot's score or share, and 1 - score of a sigmoid
    if (sigmoid) sigmoids((double)le, &p, &rest);
    else p = exp_neg((double)le - m);
    if (!on) p = 0.0;
    if (normalize) {
        sum = wave_sum_dpp(p);
        if (sigmoid && sum < kTiny) {
            const double ls = on ? log_sigmoid((double)le) : kOut, top = wave_max_dpp(ls);
            p = on ? exp(ls - top) : 0.0;
            sum = wave_sum_dpp(p);
        }
    }
    // a quotient and not a product with 1 / sum: a share that is all of the sum is exactly 1, its gradient exactly 0
    p = on ? p / sum : 0.0;
    double dot = 0.0;
    if (!sigmoid || normalize) dot = wave_sum_dpp(g * p);
    const double v = on ? p * rest * (whole ? g : g - dot) * (double)scale : 0.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        o[i] = whole && l[i] != -INFINITY ? -dot * (exp_neg((double)l[i] - m) / sum) * (double)scale : 0.0;
    // the slots' gradients to their experts, one after the other (a repeated expert adds)
    for (int j = 0; j < K; ++j) {
        const int ej = (int)readlane((uint32_t)e, j);
        if (ej < 0 || ej >= E) continue;
        const double vj = readlane(v, j);
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (ej >> 6 == i) o[i] += lane == (ej & 63) ? vj : 0.0;
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        if (lane + 64 * i < E) store_grad(grad_logits + t * E + lane + 64 * i, o[i]);
}

// Boolean map, or any K: slots counted at the experts' lanes.
template <typename LT, int FMT, int EPL>
__global__ __launch_bounds__(256) void k_gate_backward_many(const float* __restrict__ grad_probs,
                                                            const LT* logits, const void* __restrict__ routing, int T,
                                                            int E, int K, int sigmoid, int normalize, float scale,
                                                            LT* grad_logits) {
    const int lane = threadIdx.x & 63;
    const long long t = (long long)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= T) return;
    float l[EPL];
    double g[EPL];
    int cnt[EPL];   // slots that hold this expert (a repeated index adds its slots)
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = lane + 64 * i;
        l[i] = e < E ? load_logit(logits + t * E + e) : -INFINITY;
        g[i] = 0.0;
        cnt[i] = 0;
    }
    if constexpr (FMT == MOE_ROUTE_SPARSE_BOOL) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = lane + 64 * i;
            if (e < E && l[i] != -INFINITY && ((const uint8_t*)routing)[t * E + e]) {
                cnt[i] = 1;
                g[i] = (double)grad_probs[t * E + e];
            }
        }
    } else {
        using IT = std::conditional_t<FMT == MOE_ROUTE_DENSE_I16, int16_t, int32_t>;
        for (int j0 = 0; j0 < K; j0 += 64) {
            int my = -1;
            float mg = 0.f;
            if (j0 + lane < K) {
                my = (int)((const IT*)routing)[t * K + j0 + lane];
                mg = grad_probs[t * K + j0 + lane];
            }
            const int nj = min(64, K - j0);
            for (int j = 0; j < nj; ++j) {
                const int e = (int)readlane((uint32_t)my, j);
                const float ge = readlane(mg, j);
#pragma unroll
                for (int i = 0; i < EPL; ++i)
                    if (e == lane + 64 * i && l[i] != -INFINITY) {
                        ++cnt[i];
                        g[i] += (double)ge;
                    }
            }
        }
    }
    // p = scores (or the chosen scores' shares), dot = sum over the slots of G p
    const bool whole = !sigmoid && !normalize;
    auto has_share = [&](int i) { return whole ? l[i] != -INFINITY : cnt[i] > 0; };
    double m = 0.0, sum = 1.0, p[EPL], rest[EPL], part = 0.0;
    if (whole) {
        softmax_terms<EPL>(l, &m, &sum);
    } else if (!sigmoid) {
        m = kOut;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (cnt[i]) m = fmax(m, (double)l[i]);
        m = wave_max_dpp(m);
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        p[i] = 0.0;
        rest[i] = 1.0;
        if (has_share(i)) {
            if (sigmoid) sigmoids((double)l[i], &p[i], &rest[i]);
            else p[i] = exp_neg((double)l[i] - m);
        }
        part += cnt[i] * p[i];
    }
    if (normalize) {
        sum = wave_sum_dpp(part);
        if (sigmoid && sum < kTiny) {
            double top = kOut;
            part = 0.0;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                p[i] = cnt[i] ? log_sigmoid((double)l[i]) : kOut;
                top = fmax(top, p[i]);
            }
            top = wave_max_dpp(top);
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                p[i] = cnt[i] ? exp(p[i] - top) : 0.0;
                part += cnt[i] * p[i];
            }
            sum = wave_sum_dpp(part);
        }
    }
    double dot = 0.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        p[i] = has_share(i) ? p[i] / sum : 0.0;   // exactly 1 where it is all of the sum; NaN in the row of a +inf
        dot += g[i] * p[i];
    }
    dot = !sigmoid || normalize ? wave_sum_dpp(dot) : 0.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = lane + 64 * i;
        if (e >= E) continue;
        // a slot's own gradient less, through the sum that divides it, the dot:
        // with the chosen scores' sum each slot of the expert carries it once
        const double o = p[i] * rest[i] * (g[i] - (normalize ? cnt[i] : 1) * dot) * (double)scale;
        store_grad(grad_logits + t * E + e, has_share(i) ? o : 0.0);
    }
}

template <typename F>
void by_epl(int E, F go) {
    const int epl = (E + 63) / 64;
    if (epl <= 1) go(std::integral_constant<int, 1>{});
    else if (epl <= 2) go(std::integral_constant<int, 2>{});
    else if (epl <= 4) go(std::integral_constant<int, 4>{});
    else if (epl <= 8) go(std::integral_constant<int, 8>{});
    else go(std::integral_constant<int, 16>{});
}

template <typename F>
void by_type(int logit_dtype, int fmt, F go) {
    auto f = [&](auto lt) {
        if (fmt == MOE_ROUTE_DENSE_I16) go(lt, std::integral_constant<int, MOE_ROUTE_DENSE_I16>{});
        else if (fmt == MOE_ROUTE_DENSE_I32) go(lt, std::integral_constant<int, MOE_ROUTE_DENSE_I32>{});
        else go(lt, std::integral_constant<int, MOE_ROUTE_SPARSE_BOOL>{});
    };
    if (logit_dtype == MOE_BF16) f(uint16_t{});
    else f(float{});
}

}  // namespace

hipError_t launch_gate(const moe_handle* h, const void* logits, int logit_dtype, const float* bias, int sigmoid,
                       int normalize, float scale, void* routing, float* probs, hipStream_t s) {
    const moe_desc& d = h->desc;
    if (d.T == 0) return hipSuccess;
    const dim3 grid((unsigned)((d.T + 3ll) / 4));
    by_type(logit_dtype, d.route_fmt, [&](auto lt, auto fmt) {
        by_epl(d.E, [&](auto epl) {
            using LT = decltype(lt);
            constexpr int FMT = decltype(fmt)::value, EPL = decltype(epl)::value;
            auto go = [&](auto kernel) {
                hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, (const LT*)logits, d.T, d.E, d.K, bias, normalize,
                                   scale, routing, probs);
            };
            if (d.K > 64)
                hipLaunchKernelGGL((k_gate_many<LT, FMT, EPL>), grid, dim3(256), 0, s, (const LT*)logits, d.T, d.E,
                                   d.K, bias, sigmoid, normalize, scale, routing, probs);
            else if (bias && sigmoid) go(k_gate<LT, FMT, EPL, true, true>);
            else if (bias) go(k_gate<LT, FMT, EPL, true, false>);
            else if (sigmoid) go(k_gate<LT, FMT, EPL, false, true>);
            else go(k_gate<LT, FMT, EPL, false, false>);
        });
    });
    return hipGetLastError();
}

hipError_t launch_gate_backward(const moe_handle* h, const float* grad_probs, const void* logits, int logit_dtype,
                                const void* routing, int sigmoid, int normalize, float scale, void* grad_logits,
                                hipStream_t s) {
    const moe_desc& d = h->desc;
    if (d.T == 0) return hipSuccess;
    const dim3 grid((unsigned)((d.T + 3ll) / 4));
    by_type(logit_dtype, d.route_fmt, [&](auto lt, auto fmt) {
        by_epl(d.E, [&](auto epl) {
            using LT = decltype(lt);
            constexpr int FMT = decltype(fmt)::value, EPL = decltype(epl)::value;
            if constexpr (FMT != MOE_ROUTE_SPARSE_BOOL) {
                using IT = std::conditional_t<FMT == MOE_ROUTE_DENSE_I16, int16_t, int32_t>;
                if (d.K <= 64) {
                    hipLaunchKernelGGL((k_gate_backward<LT, IT, EPL>), grid, dim3(256), 0, s, grad_probs,
                                       (const LT*)logits, (const IT*)routing, d.T, d.E, d.K, sigmoid, normalize,
                                       scale, (LT*)grad_logits);
                    return;
                }
            }
            hipLaunchKernelGGL((k_gate_backward_many<LT, FMT, EPL>), grid, dim3(256), 0, s, grad_probs,
                               (const LT*)logits, routing, d.T, d.E, d.K, sigmoid, normalize, scale,
                               (LT*)grad_logits);
        });
    });
    return hipGetLastError();
}

}  // namespace moe
