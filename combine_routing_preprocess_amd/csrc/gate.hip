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
// Keys are 64-bit floats: score + bias decides between experts that 32 bits
// cannot tell apart, and the choice is an integer that must not hang on a
// rounding.  Scores are held as their logarithm (l - m for the softmax,
// log sigmoid otherwise), so that the normalised weights, a softmax over the
// chosen logarithms, stay finite where every chosen score underflows.
#include "moe_internal.h"

namespace moe {
namespace {

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, 64);
    return v;
}
__device__ __forceinline__ double wave_max(double v) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v = fmax(v, __shfl_xor(v, m, 64));
    return v;
}

constexpr double kOut = -INFINITY;   // key of an expert that is not (or no longer) a candidate

template <typename LT>
__device__ __forceinline__ double load_logit(const LT* p) {
    if constexpr (sizeof(LT) == 2) return (double)__uint_as_float((uint32_t)*p << 16);
    else return (double)*p;
}

// Logarithm of the score, up to the row's constant in the softmax case.
__device__ __forceinline__ double log_score(double l, int sigmoid) {
    return sigmoid ? fmin(l, 0.0) - log1p(exp(-fabs(l))) : l;
}

// Logits of a lane's experts (NaN and experts past E read as kOut), and the
// row's maximum and sum of exp(l - max) for the softmax.
template <typename LT, int EPL>
__device__ __forceinline__ void load_row(const LT* row, int E, int lane, int sigmoid, double (&l)[EPL], double* m,
                                         double* sum) {
    *m = kOut;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = lane + 64 * i;
        l[i] = e < E ? load_logit(row + e) : kOut;
        if (!(l[i] == l[i])) l[i] = kOut;
        *m = fmax(*m, l[i]);
    }
    *sum = 1.0;
    if (sigmoid) return;
    *m = wave_max(*m);
    double a = 0.0;
    if (*m != kOut) {
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (l[i] != kOut) a += exp(l[i] - *m);
    }
    *sum = wave_sum(a);
}

template <typename LT, int FMT, int EPL>
__global__ __launch_bounds__(256) void k_gate(const LT* __restrict__ logits, int T, int E, int K,
                                              const float* __restrict__ bias, int sigmoid, int normalize, float scale,
                                              void* __restrict__ routing, float* __restrict__ probs) {
    const int lane = threadIdx.x & 63;
    const long long t = (long long)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= T) return;
    double l[EPL], key[EPL], m, sum;
    int slot[EPL];
    load_row<LT, EPL>(logits + t * E, E, lane, sigmoid, l, &m, &sum);
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = lane + 64 * i;
        key[i] = l[i];
        if (bias && l[i] != kOut) {
            const double s = sigmoid ? 1.0 / (1.0 + exp(-l[i])) : exp(l[i] - m) / sum;
            key[i] = s + (double)bias[e];
            if (!(key[i] == key[i])) key[i] = kOut;
        }
        slot[i] = -1;
    }
    int n = 0;   // chosen so far
    for (; n < K; ++n) {
        double best = kOut;
        int at = 1 << 30;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (key[i] > best) {
                best = key[i];
                at = lane + 64 * i;
            }
#pragma unroll
        for (int x = 32; x >= 1; x >>= 1) {
            const double ob = __shfl_xor(best, x, 64);
            const int oa = __shfl_xor(at, x, 64);
            if (ob > best || (ob == best && oa < at)) {
                best = ob;
                at = oa;
            }
        }
        if (best == kOut) break;   // the same for every lane
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (at == lane + 64 * i) {
                slot[i] = n;
                key[i] = kOut;
            }
    }
    // weights of the chosen
    double top = kOut, part = 0.0, w[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        w[i] = slot[i] >= 0 ? log_score(l[i], sigmoid) : kOut;
        top = fmax(top, w[i]);
    }
    if (normalize) top = wave_max(top);
    else top = sigmoid ? 0.0 : m;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        w[i] = slot[i] >= 0 ? exp(w[i] - top) : 0.0;
        part += w[i];
    }
    const double f = (double)scale / (normalize ? wave_sum(part) : sum);
    if constexpr (FMT == MOE_ROUTE_SPARSE_BOOL) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = lane + 64 * i;
            if (e < E) {
                ((uint8_t*)routing)[t * E + e] = slot[i] >= 0;
                probs[t * E + e] = slot[i] >= 0 ? (float)(w[i] * f) : 0.f;
            }
        }
    } else {
        using IT = std::conditional_t<FMT == MOE_ROUTE_DENSE_I16, int16_t, int32_t>;
        IT* idx = (IT*)routing + t * K;
        float* p = probs + t * K;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (slot[i] >= 0) {
                idx[slot[i]] = (IT)(lane + 64 * i);
                p[slot[i]] = (float)(w[i] * f);
            }
        for (int j = n + lane; j < K; j += 64) {
            idx[j] = (IT)-1;
            p[j] = 0.f;
        }
    }
}

template <typename LT, int FMT, int EPL>
__global__ __launch_bounds__(256) void k_gate_backward(const float* __restrict__ grad_probs,
                                                       const LT* __restrict__ logits,
                                                       const void* __restrict__ routing, int T, int E, int K,
                                                       int sigmoid, int normalize, float scale,
                                                       LT* __restrict__ grad_logits) {
    const int lane = threadIdx.x & 63;
    const long long t = (long long)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= T) return;
    double l[EPL], g[EPL], m, sum;
    int cnt[EPL];   // slots that hold this expert (a repeated index adds its slots)
    load_row<LT, EPL>(logits + t * E, E, lane, sigmoid, l, &m, &sum);
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        g[i] = 0.0;
        cnt[i] = 0;
    }
    if constexpr (FMT == MOE_ROUTE_SPARSE_BOOL) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const int e = lane + 64 * i;
            if (e < E && l[i] != kOut && ((const uint8_t*)routing)[t * E + e]) {
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
                const int e = __shfl(my, j, 64);
                const float ge = __shfl(mg, j, 64);
#pragma unroll
                for (int i = 0; i < EPL; ++i)
                    if (e == lane + 64 * i && l[i] != kOut) {
                        ++cnt[i];
                        g[i] += (double)ge;
                    }
            }
        }
    }
    // p = scores (or the chosen scores' shares), dot = sum over the slots of G p
    double top = kOut, p[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        p[i] = normalize && !cnt[i] ? kOut : log_score(l[i], sigmoid);
        if (l[i] == kOut) p[i] = kOut;
        if (p[i] != kOut) top = fmax(top, p[i]);
    }
    if (normalize) top = wave_max(top);
    else top = sigmoid ? 0.0 : m;
    double part = 0.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        p[i] = p[i] != kOut ? exp(p[i] - top) : 0.0;
        part += cnt[i] * p[i];
    }
    const double inv = 1.0 / (normalize ? wave_sum(part) : sum);
    double dot = 0.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        p[i] = p[i] != 0.0 ? p[i] * inv : 0.0;
        dot += g[i] * p[i];
    }
    if (normalize || !sigmoid) dot = wave_sum(dot);
    else dot = 0.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = lane + 64 * i;
        if (e >= E) continue;
        // a slot's own gradient less, through the sum that divides it, the dot:
        // with the chosen scores' sum each slot of the expert carries it once
        double o = p[i] * (g[i] - (normalize ? cnt[i] : 1) * dot);
        if (sigmoid) o *= 1.0 / (1.0 + exp(l[i]));   // 1 - s
        o = p[i] != 0.0 ? o * (double)scale : 0.0;
        if constexpr (sizeof(LT) == 2) grad_logits[t * E + e] = (LT)f32_to_bf16((float)o);
        else grad_logits[t * E + e] = (float)o;
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
            hipLaunchKernelGGL((k_gate<LT, decltype(fmt)::value, decltype(epl)::value>), grid, dim3(256), 0, s,
                               (const LT*)logits, d.T, d.E, d.K, bias, sigmoid, normalize, scale, routing, probs);
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
            hipLaunchKernelGGL((k_gate_backward<LT, decltype(fmt)::value, decltype(epl)::value>), grid, dim3(256), 0,
                               s, grad_probs, (const LT*)logits, routing, d.T, d.E, d.K, sigmoid, normalize, scale,
                               (LT*)grad_logits);
        });
    });
    return hipGetLastError();
}

}  // namespace moe
