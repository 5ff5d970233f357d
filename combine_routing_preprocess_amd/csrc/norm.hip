// Layer norm of token rows, forward and backward, with the reduction of the
// weight's and bias's gradients: the norm in front of the MoE layer.
//
//   forward   y = (x - mu) * r * w + b,  mu = mean(x),  r = 1 / sqrt(mean((x - mu)^2) + eps)
//   backward  xh = (x - mu) * r,  g = gy * w,
//             gx = r * (g - mean(g) - xh * mean(g * xh)),
//             gw = sum over the rows of gy * xh,  gb = sum over the rows of gy
//
// Both directions are bound by HBM: the forward reads x and writes y once, the
// backward reads x and gy and writes gx once.  A row is held in registers by W
// wavefronts, 8 elements (one chunk) per lane and step, at most NC steps; G
// rows share a workgroup when they are short.  Workgroups walk the rows with a
// stride, so weight and bias are loaded once per workgroup, and the next row's
// loads are issued before the current row's reductions.
//
// Statistics are fp32 and need one barrier per row.  Each wavefront takes the
// mean m of its own part, then the sum e and the square sum q of what is left,
// x - m: e is the rounding that m carries, so the part's mean is m + e / n and
// its centred square sum q - e^2 / n, without the cancellation of E[x^2] -
// mu^2.  The parts join by the exact rule for means and square sums of
// disjoint sets, relative to the first part's m, so that a row whose offset is
// far larger than its spread keeps its precision.
//
// Rows need no alignment beyond their element's: chunks are loaded and stored
// as 16-byte accesses at element alignment, which the memory pipeline takes
// (the whole-line rows of a width that is a multiple of 8 are just the fast
// case), and a last partial chunk goes element by element.
#include "moe_internal.h"

namespace moe {
namespace {

typedef u32x4 u32x4_e __attribute__((aligned(2)));   // 16 bytes at element alignment

// Eight consecutive elements as loaded: one 16-byte word per 8 bf16, two per 8 fp32.
template <typename XT>
struct Chunk {
    u32x4 w[sizeof(XT) / 2];
};

// Elements 0 .. n-1 of a chunk (n <= 8; the rest reads as zero).
template <typename XT>
__device__ __forceinline__ Chunk<XT> load_chunk(const XT* p, int n) {
    Chunk<XT> c;
    if (n >= 8) {
#pragma unroll
        for (int i = 0; i < (int)(sizeof(XT) / 2); ++i) c.w[i] = ((const u32x4_e*)p)[i];
        return c;
    }
    if constexpr (sizeof(XT) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = 2 * i < n ? p[2 * i] : 0u, hi = 2 * i + 1 < n ? p[2 * i + 1] : 0u;
            c.w[0][i] = lo | (hi << 16);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) c.w[i / 4][i % 4] = i < n ? __float_as_uint(p[i]) : 0u;
    }
    return c;
}

template <typename XT>
__device__ __forceinline__ void unpack(const Chunk<XT>& c, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (sizeof(XT) == 2) v[i] = i & 1 ? bf16_hi(c.w[0][i / 2]) : bf16_lo(c.w[0][i / 2]);
        else v[i] = __uint_as_float(c.w[i / 4][i % 4]);
    }
}

template <typename XT>
__device__ __forceinline__ void store_chunk(XT* p, int n, const float (&v)[8]) {
    if (n >= 8) {
        if constexpr (sizeof(XT) == 2) {
            *(u32x4_e*)p = u32x4{bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]), bf16x2_rne(v[4], v[5]),
                                 bf16x2_rne(v[6], v[7])};
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                ((u32x4_e*)p)[i] = u32x4{__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                                         __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3])};
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) {
            if constexpr (sizeof(XT) == 2) p[i] = (uint16_t)f32_to_bf16(v[i]);
            else p[i] = v[i];
        }
}

// Chunk of a weight or bias vector; `fill` where there is none.
__device__ __forceinline__ void load_param(const void* p, int dtype, int c, int n, float fill, float (&v)[8]) {
    if (!p) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = fill;
    } else if (dtype == MOE_BF16) {
        unpack(load_chunk((const uint16_t*)p + 8 * c, n), v);
    } else {
        unpack(load_chunk((const float*)p + 8 * c, n), v);
    }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, 64);
    return v;
}

constexpr int kMaxWaves = 16;   // wavefronts of a workgroup

// Elements that wavefront i of a row's W holds in all its NC steps.
template <int NC>
__device__ __forceinline__ int part_elems(int H, int W, int i) {
    int n = 0;
#pragma unroll
    for (int k = 0; k < NC; ++k) n += min(max(H - 512 * (i + k * W), 0), 512);
    return n;
}

template <typename XT, typename YT, int NC>
__global__ __launch_bounds__(1024) void k_layer_norm(const XT* __restrict__ x, int T, int H, int W, int G,
                                                     const void* __restrict__ weight, const void* __restrict__ bias,
                                                     int wdtype, float eps, YT* __restrict__ y,
                                                     float* __restrict__ mean, float* __restrict__ rstd) {
    __shared__ float s_m[2][kMaxWaves], s_e[2][kMaxWaves], s_q[2][kMaxWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int grp = wave / W, part = wave - grp * W;
    int col[NC], n[NC];
    float w[NC][8], b[NC][8];
#pragma unroll
    for (int k = 0; k < NC; ++k) {
        const int c = (part + k * W) * 64 + lane;
        col[k] = 8 * c;
        n[k] = min(max(H - col[k], 0), 8);
        load_param(weight, wdtype, c, n[k], 1.f, w[k]);
        load_param(bias, wdtype, c, n[k], 0.f, b[k]);
    }
    const float inv_h = 1.f / (float)H;
    const float inv_mine = 1.f / (float)part_elems<NC>(H, W, part);
    const long long stride = (long long)gridDim.x * G;
    long long row = (long long)blockIdx.x * G + grp;
    Chunk<XT> next[NC];
#pragma unroll
    for (int k = 0; k < NC; ++k) next[k] = load_chunk(x + row * H + col[k], row < T ? n[k] : 0);
    int par = 0;
    // the workgroup's rows advance together, so every wavefront meets the barrier
    for (long long row0 = (long long)blockIdx.x * G; row0 < T; row0 += stride, row += stride, par ^= 1) {
        const bool ok = row < T;
        float v[NC][8];
#pragma unroll
        for (int k = 0; k < NC; ++k) unpack(next[k], v[k]);
#pragma unroll
        for (int k = 0; k < NC; ++k)
            next[k] = load_chunk(x + (row + stride) * H + col[k], row + stride < T ? n[k] : 0);
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < NC; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) s += v[k][i];
        // through a scalar register: m is one rounded value everywhere below (contracted into v - m, the
        // product would enter unrounded there and rounded elsewhere, and e would not be its rounding)
        float m = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(wave_sum(s) * inv_mine)));
        float e = 0.f, q = 0.f;
#pragma unroll
        for (int k = 0; k < NC; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float d = i < n[k] ? v[k][i] - m : 0.f;
                e += d;
                q = fmaf(d, d, q);
            }
        e = wave_sum(e);
        q = wave_sum(q);
        float delta, sq;   // mean relative to m, centred square sum of the row
        if (W == 1) {
            delta = e * inv_h;
            sq = q - e * delta;
        } else {
            if (lane == 0) {
                s_m[par][wave] = m;
                s_e[par][wave] = e;
                s_q[par][wave] = q;
            }
            __syncthreads();   // the other parity's readers passed the barrier before this one's writers run again
            const int w0 = grp * W;
            m = s_m[par][w0];
            float sum = 0.f;
            for (int i = 0; i < W; ++i)
                sum += fmaf((float)part_elems<NC>(H, W, i), s_m[par][w0 + i] - m, s_e[par][w0 + i]);
            delta = sum * inv_h;
            sq = 0.f;
            for (int i = 0; i < W; ++i) {
                const float ni = (float)part_elems<NC>(H, W, i), ei = s_e[par][w0 + i];
                const float off = (s_m[par][w0 + i] - m) - delta;      // part's m relative to the row's mean
                sq += s_q[par][w0 + i] + off * fmaf(ni, off, 2.f * ei);
            }
        }
        if (sq < 0.f) sq = 0.f;   // NaN stays
        const float r = 1.f / sqrtf(fmaf(sq, inv_h, eps));
        if (ok) {
#pragma unroll
            for (int k = 0; k < NC; ++k) {
                float o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = fmaf(((v[k][i] - m) - delta) * r, w[k][i], b[k][i]);
                store_chunk(y + row * H + col[k], n[k], o);
            }
            if (part == 0 && lane == 0) {
                if (mean) mean[row] = m + delta;
                if (rstd) rstd[row] = r;
            }
        }
    }
}

// Row gradients of the workgroup's rows, and its sums of gy * xh and gy per
// column into part[2 * blockIdx][H] and part[2 * blockIdx + 1][H] (straight
// into gw and gb when one workgroup has every row).
template <typename XT, typename YT, int NC>
__global__ __launch_bounds__(1024) void k_layer_norm_backward(const YT* __restrict__ gy, const XT* __restrict__ x,
                                                              const float* __restrict__ mean,
                                                              const float* __restrict__ rstd, int T, int H, int W,
                                                              int G, const void* __restrict__ weight, int wdtype,
                                                              XT* __restrict__ gx, float* __restrict__ pw,
                                                              float* __restrict__ pb, long long pstride) {
    extern __shared__ float s_cols[];   // [2][H], G > 1 only
    __shared__ float s_a[2][kMaxWaves], s_b[2][kMaxWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int grp = wave / W, part = wave - grp * W;
    int col[NC], n[NC];
    float w[NC][8], aw[NC][8], ab[NC][8];
#pragma unroll
    for (int k = 0; k < NC; ++k) {
        const int c = (part + k * W) * 64 + lane;
        col[k] = 8 * c;
        n[k] = min(max(H - col[k], 0), 8);
        load_param(weight, wdtype, c, n[k], 1.f, w[k]);
#pragma unroll
        for (int i = 0; i < 8; ++i) aw[k][i] = ab[k][i] = 0.f;
    }
    const float inv_h = 1.f / (float)H;
    const long long stride = (long long)gridDim.x * G;
    long long row = (long long)blockIdx.x * G + grp;
    Chunk<XT> nx[NC];
    Chunk<YT> ng[NC];
    float nm = 0.f, nr = 0.f;
    auto fetch = [&](long long r) {
        const bool ok = r < T;
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            nx[k] = load_chunk(x + r * H + col[k], ok ? n[k] : 0);
            ng[k] = load_chunk(gy + r * H + col[k], ok ? n[k] : 0);
        }
        nm = ok ? mean[r] : 0.f;
        nr = ok ? rstd[r] : 0.f;
    };
    fetch(row);
    int par = 0;
    for (long long row0 = (long long)blockIdx.x * G; row0 < T; row0 += stride, row += stride, par ^= 1) {
        const bool ok = row < T;
        const float m = nm, r = nr;
        float xh[NC][8], g[NC][8];
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int k = 0; k < NC; ++k) {
            unpack(nx[k], xh[k]);
            unpack(ng[k], g[k]);
        }
        fetch(row + stride);
#pragma unroll
        for (int k = 0; k < NC; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // past the row's end gy reads as 0; xh must be 0 there too (0 * inf)
                xh[k][i] = i < n[k] ? (xh[k][i] - m) * r : 0.f;
                aw[k][i] = fmaf(g[k][i], xh[k][i], aw[k][i]);
                ab[k][i] += g[k][i];
                g[k][i] *= w[k][i];
                a += g[k][i];
                b = fmaf(g[k][i], xh[k][i], b);
            }
        a = wave_sum(a);
        b = wave_sum(b);
        if (W > 1) {
            if (lane == 0) {
                s_a[par][wave] = a;
                s_b[par][wave] = b;
            }
            __syncthreads();
            a = b = 0.f;
            for (int i = 0; i < W; ++i) {
                a += s_a[par][grp * W + i];
                b += s_b[par][grp * W + i];
            }
        }
        a *= inv_h;
        b *= inv_h;
        if (ok) {
#pragma unroll
            for (int k = 0; k < NC; ++k) {
                float o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = r * (g[k][i] - a - xh[k][i] * b);
                store_chunk(gx + row * H + col[k], n[k], o);
            }
        }
    }
    if (!pw && !pb) return;
    if (G > 1) {   // the row groups' columns, one group after the other
        for (int turn = 0; turn < G; ++turn) {
            if (grp == turn) {
#pragma unroll
                for (int k = 0; k < NC; ++k)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (i < n[k]) {
                            float* pa = s_cols + col[k] + i;
                            pa[0] = turn ? pa[0] + aw[k][i] : aw[k][i];
                            pa[H] = turn ? pa[H] + ab[k][i] : ab[k][i];
                        }
            }
            __syncthreads();
        }
        for (int h = threadIdx.x; h < H; h += blockDim.x) {
            if (pw) pw[(long long)blockIdx.x * pstride + h] = s_cols[h];
            if (pb) pb[(long long)blockIdx.x * pstride + h] = s_cols[H + h];
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < NC; ++k) {
        if (pw) store_chunk(pw + (long long)blockIdx.x * pstride + col[k], n[k], aw[k]);
        if (pb) store_chunk(pb + (long long)blockIdx.x * pstride + col[k], n[k], ab[k]);
    }
}

// gw / gb = sum over the nb workgroups' partials [nb][2][H], in a fixed order
// (no atomics, so a call repeats bit for bit): 32 columns x 8 slices of the
// partials per workgroup.  nb = 0 (no rows) writes zeros.
__global__ __launch_bounds__(256) void k_norm_param_grads(const float* __restrict__ part, int nb, int H,
                                                          float* __restrict__ gw, float* __restrict__ gb) {
    __shared__ float s[8][33];
    const int cl = threadIdx.x & 31, sl = threadIdx.x >> 5;
    const long long c = (long long)blockIdx.x * 32 + cl;   // column of [2][H]
    float v = 0.f;
    if (c < 2ll * H)
        for (int i = sl; i < nb; i += 8) v += part[(long long)i * 2 * H + c];
    s[sl][cl] = v;
    __syncthreads();
    if (sl == 0 && c < 2ll * H) {
        float o = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) o += s[i][cl];
        if (c < H) {
            if (gw) gw[c] = o;
        } else if (gb) {
            gb[c - H] = o;
        }
    }
}

constexpr int kMaxRowElems = 64 * 8 * kMaxWaves * 4;   // 4 steps of 16 wavefronts
static_assert(kMaxRowElems == MOE_NORM_MAX_H, "norm row limit");
constexpr int kBackwardBlocks = 256;                   // one workgroup per CU walks the rows

// Steps per lane and wavefronts per row.
void row_shape(int H, int* NC, int* W) {
    const int groups = (H + 511) / 512;   // 64-lane groups of chunks
    *NC = groups <= kMaxWaves ? 1 : groups <= 2 * kMaxWaves ? 2 : 4;
    *W = (groups + *NC - 1) / *NC;
}

int backward_blocks(int T, int G) { return min(kBackwardBlocks, (int)(((long long)T + G - 1) / G)); }

}  // namespace

size_t norm_backward_scratch_bytes(int T, int H) {
    int NC, W;
    row_shape(H, &NC, &W);
    return (size_t)backward_blocks(T, kMaxWaves / W) * 2 * H * sizeof(float);
}

hipError_t launch_layer_norm(int T, int H, int x_dtype, int y_dtype, int w_dtype, const void* x, const void* weight,
                             const void* bias, float eps, void* y, float* mean, float* rstd, int num_cu,
                             hipStream_t s) {
    if (T == 0) return hipSuccess;
    int NC, W;
    row_shape(H, &NC, &W);
    const int G = W >= 4 ? 1 : 4 / W;
    const int per_cu = max(1, 32 / (W * G));
    const long long want = ((long long)T + G - 1) / G, most = (long long)num_cu * per_cu;
    const unsigned grid = (unsigned)(want < most ? want : most);
    auto go = [&](auto xt, auto yt, auto nc) {
        using XT = decltype(xt);
        using YT = decltype(yt);
        hipLaunchKernelGGL((k_layer_norm<XT, YT, decltype(nc)::value>), dim3(grid), dim3(64 * W * G), 0, s,
                           (const XT*)x, T, H, W, G, weight, bias, w_dtype, eps, (YT*)y, mean, rstd);
    };
    auto by_nc = [&](auto xt, auto yt) {
        if (NC == 1) go(xt, yt, std::integral_constant<int, 1>{});
        else if (NC == 2) go(xt, yt, std::integral_constant<int, 2>{});
        else go(xt, yt, std::integral_constant<int, 4>{});
    };
    const bool xb = x_dtype == MOE_BF16, yb = y_dtype == MOE_BF16;
    if (xb && yb) by_nc(uint16_t{}, uint16_t{});
    else if (xb) by_nc(uint16_t{}, float{});
    else if (yb) by_nc(float{}, uint16_t{});
    else by_nc(float{}, float{});
    return hipGetLastError();
}

hipError_t launch_layer_norm_backward(int T, int H, int x_dtype, int y_dtype, int w_dtype, const void* gy,
                                      const void* x, const float* mean, const float* rstd, const void* weight,
                                      void* gx, float* gw, float* gb, void* scratch, hipStream_t s) {
    int NC, W;
    row_shape(H, &NC, &W);
    const int G = kMaxWaves / W;
    const int nb = T > 0 ? backward_blocks(T, G) : 0;
    const bool params = gw || gb;
    if (nb > 0) {
        float* part = (float*)scratch;
        float* pw = nb == 1 ? gw : params ? part : nullptr;
        float* pb = nb == 1 ? gb : params ? part + H : nullptr;
        const size_t lds = params && G > 1 ? (size_t)2 * H * sizeof(float) : 0;
        auto go = [&](auto xt, auto yt, auto nc) {
            using XT = decltype(xt);
            using YT = decltype(yt);
            hipLaunchKernelGGL((k_layer_norm_backward<XT, YT, decltype(nc)::value>), dim3(nb), dim3(64 * W * G), lds,
                               s, (const YT*)gy, (const XT*)x, mean, rstd, T, H, W, G, weight, w_dtype, (XT*)gx, pw,
                               pb, 2ll * H);
        };
        auto by_nc = [&](auto xt, auto yt) {
            if (NC == 1) go(xt, yt, std::integral_constant<int, 1>{});
            else if (NC == 2) go(xt, yt, std::integral_constant<int, 2>{});
            else go(xt, yt, std::integral_constant<int, 4>{});
        };
        const bool xb = x_dtype == MOE_BF16, yb = y_dtype == MOE_BF16;
        if (xb && yb) by_nc(uint16_t{}, uint16_t{});
        else if (xb) by_nc(uint16_t{}, float{});
        else if (yb) by_nc(float{}, uint16_t{});
        else by_nc(float{}, float{});
        hipError_t e = hipGetLastError();
        if (e != hipSuccess || nb == 1) return e;
    }
    if (!params) return hipSuccess;
    hipLaunchKernelGGL(k_norm_param_grads, dim3((unsigned)((2ll * H + 31) / 32)), dim3(256), 0, s,
                       (const float*)scratch, nb, H, gw, gb);
    return hipGetLastError();
}

}  // namespace moe
