// The products grouped by expert for many rows per expert: one workgroup of
// eight wavefronts per CU walks tiles of 256 features x 256 rows (half the
// operand bytes per product of two workgroups of 256 x 128).
//
// A wavefront holds 64 features x 128 rows.  Stages of 64 elements of the sum in
// two slots of LDS, so that operands that are not read across arrive in whole
// lines (with 32 and four slots: 1978 us against 1876 for the case below); step s
// is loaded while step s - 1 is multiplied, the last one's products follow the
// next stage's barrier; the next tile's first stage is fetched while the last is
// multiplied, and is waited for before the outputs' stores, so that it does not
// wait for those.  The tile's second stage does: its wait counts stores like
// transfers, and they were issued before it.  They have one stage's time then,
// which long sums do not notice; with the four or five stages of a weight's
// gradient of 256 rows the stores' 2.2 us show.  Up to eight tiles of rows take
// a feature tile one after the other: an expert's weights are then read from HBM
// once (32 experts of 1000 rows: 8, 4 and 2 tiles together 1761, 1787 and 1884
// us).
//
// Measured on MI355X: 32768 rows over 32 experts, 7168 x 4096, 1.72 ms (1120
// TFLOP/s; transposed 1.71), its weight's gradient 1.44 ms, [256,7168,2048] of
// 65536 rows 2.80 ms (7.5 GB written); 11804 rows over 60 uneven experts, 2056 x
// 1416 transposed, 134 to 142 us (505 TFLOP/s; the tiles of 256 x 128 take 141);
// one expert, 8192 x 8192 x 8192, 0.86 ms (1270 TFLOP/s, where a library product
// of that size reaches 1445).  The matrix pipe is busy 46 to 59 % of the cycles
// in the sizes of 32 experts (31 % in the weight's gradient of 256 rows each) at
// the 1.9 to 2.2 GHz that the chip holds: a stage of 2048 matrix cycles takes 3300, of which the waits for its
// transfers are 2 to 4 %.  With transfers that always hit L2 it takes 83 % of
// that, without transfers in the loop 72 %.
#include "grouped.h"

namespace moe {
namespace grouped {
namespace {

constexpr int kTile = 256, kThreads = 512;
constexpr int kBK = 64;                          // sum's elements per stage
constexpr int kOperand = kTile * kBK * 2, kSlot = 2 * kOperand;
constexpr int kStage = 16 * 144;                 // epilogue bytes of a wavefront
constexpr int kGroup = 8;                        // tiles of rows that take a feature tile one after the other
constexpr int kLds = 2 * kSlot + 8 * kStage;
static_assert(kLds + 8 * kMaxE + 64 <= 160 * 1024 && 8 * 272 <= kStage, "LDS budget");

// Where tile t lies: expert, rows, first feature and row.
struct Place {
    int e, rows, a0, b0, nb;
    long long seg;
};

// A stage's transfers, four per operand and wavefront: eight rows of 128 bytes,
// or two rows (across) of 512, each.
template <bool AX, bool BX, bool KEEP>
struct Transfers {
    static constexpr int Q = 4;
    uint32_t a[Q], b[Q];
    int nb_mine;
    uint32_t pitch_a, pitch_b;
    gchar *A, *B;
    int nk;

    // 16-byte chunk of its row that this lane fetches
    static __device__ __forceinline__ int chunk(int wave, int lane) { return (lane & 7) ^ ((4 * wave + (lane >> 4)) & 7); }

    __device__ __forceinline__ void init(const Args& p, const Place& t, int wave, int lane) {
        constexpr bool WEIGHT = BX;
        nk = WEIGHT ? t.rows : p.nk;
        pitch_a = (uint32_t)(AX ? p.na : nk) * 2u;
        pitch_b = (uint32_t)(BX ? p.nb : nk) * 2u;
        A = uniform_ptr(WEIGHT ? p.a + (size_t)t.seg * p.na : p.a + (size_t)t.e * (KEEP ? 2 : 1) * p.na * p.nk);
        B = uniform_ptr(WEIGHT ? p.b + (size_t)t.seg * p.nb : p.b + (size_t)(t.seg + t.b0) * p.nk);
        const uint32_t c = (uint32_t)chunk(wave, lane) * 16u;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int r = 64 * q + 8 * wave + (lane >> 3), k = 16 * q + 2 * wave + (lane >> 5);
            const int cx = (lane & 31) ^ ((k & 3) << 2);
            if (AX) {
                a[q] = (uint32_t)k * pitch_a + (uint32_t)min(t.a0 + 8 * cx, p.na - 8) * 2u;
            } else if (KEEP) {      // of 64 rows: 32 gate features, the same 32 up
                const int f = min(t.a0 + r / 64 * 32 + r % 32, p.na - 1);
                a[q] = (uint32_t)(f + (r % 64) / 32 * p.na) * pitch_a + c;
            } else {
                a[q] = (uint32_t)min(t.a0 + r, p.na - 1) * pitch_a + c;
            }
            if (BX) b[q] = (uint32_t)k * pitch_b + (uint32_t)min(t.b0 + 8 * cx, p.nb - 8) * 2u;
            else b[q] = (uint32_t)min(r, t.nb - t.b0 - 1) * pitch_b + c;
        }
        const int blocks = (t.nb - t.b0 + 31) / 32;
        nb_mine = BX ? Q : (4 * blocks - wave + 7) / 8;
    }

    // Stage kt into LDS from byte address `lds` on; elements past the sum's end read valid memory again.
    __device__ __forceinline__ void issue(int kt, uint32_t lds, int wave, int lane) const {
        gchar* Ak = A + (AX ? (size_t)kt * kBK * pitch_a : (size_t)kt * kBK * 2);
        gchar* Bk = B + (BX ? (size_t)kt * kBK * pitch_b : (size_t)kt * kBK * 2);
        const int rem = nk - kt * kBK;
        uint32_t va[Q], vb[Q];
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            va[q] = a[q];
            vb[q] = b[q];
        }
        if (rem < kBK) {
            const uint32_t c = (uint32_t)chunk(wave, lane);
            const uint32_t back = (int)(8 * c) >= rem ? 16u * c : 0u;
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                const uint32_t past = (uint32_t)max(16 * q + 2 * wave + (lane >> 5) - (rem - 1), 0);
                va[q] -= AX ? past * pitch_a : back;
                vb[q] -= BX ? past * pitch_b : back;
            }
        }
        base_ready(Ak, Bk);
#pragma unroll
        for (int q = 0; q < Q; ++q) to_lds16(Ak, va[q], lds + (uint32_t)(8 * q + wave) * 1024u);
#pragma unroll
        for (int q = 0; q < Q; ++q)
            if (BX || q < nb_mine) to_lds16(Bk, vb[q], lds + kOperand + (uint32_t)(8 * q + wave) * 1024u);
    }
};

template <bool AX, bool BX, Epilogue EPI, int NTB, typename Next>
__device__ __forceinline__ void run_tile(const Args& p, Place t, Transfers<AX, BX, EPI == kSwigluKeep>& tr, lchar* lds,
                                         uint32_t base, int& slot, int wave, int lane, Next next) {
    Fragments<AX, kBK, kTile * 2, 2> fa;
    constexpr int ND = NTB > 0 ? NTB : 1;
    Fragments<BX, kBK, kTile * 2, ND> fb;
    fa.init(2 * (wave & 3), 1, lane);
    fb.init(wave >> 2, 2, lane);
    f32x16 acc[2][ND];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < ND; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[j][i][r] = 0.f;
    const int nk = tr.nk, n = (nk + kBK - 1) / kBK;
    u32x4 a[2][2] = {}, b[2][ND] = {};
    auto mul = [&](int buf) {
#pragma unroll
        for (int i = 0; i < NTB; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) acc[j][i] = multiply(a[buf][j], b[buf][i], acc[j][i]);
    };
    // Step s of a stage is loaded while step s - 1 is multiplied; the last one's products follow the next stage's barrier.
    auto stage = [&]() {
        lchar* s0 = lds + slot * kSlot;
#pragma unroll
        for (int s = 0; s < (NTB > 0 ? kBK / 16 : 0); ++s) {
            const int buf = s & 1;
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 0; j < 2; ++j) a[buf][j] = fa.load(s0, s, j);
#pragma unroll
            for (int i = 0; i < NTB; ++i) b[buf][i] = fb.load(s0 + kOperand, s, i);
            mul(buf ^ 1);
#pragma unroll
            for (int i = 0; i < 2 * NTB; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        slot ^= 1;
    };
    auto store = [&]() {
        if constexpr (NTB > 0)
            store_tile<EPI, 16, 8>(p, t.a0 + (EPI == kSwigluKeep ? 32 : 64) * (wave & 3), t.b0, t.nb - t.b0, wave >> 2, 2,
                               t.seg, t.e, acc, lds + 2 * kSlot + wave * kStage, lane);
    };
    if (BX && n == 0) {        // an expert without rows
        next(slot);
        wait_vm<0>();
        if (EPI != kWeight16Add && !(EPI == kWeight32 && p.accumulate)) store();
        return;
    }
    // this wavefront's part of stage 0 is there
    for (int kt = 0; kt + 1 < n; ++kt) {
        if (kt > 0) wait_vm<0>();
        lds_barrier();         // stage kt is there, and every wavefront has read stage kt - 1
        tr.issue(kt + 1, base + (slot ^ 1) * kSlot, wave, lane);
        stage();
    }
    if (n > 1) wait_vm<0>();
    lds_barrier();
    next(slot ^ 1);            // the next tile's first stage
    // the last one: as many steps as there are, elements past the sum's end zero in both operands
    mul(1);
    for (int s = 0, left = nk - (n - 1) * kBK; NTB > 0 && left > 0; ++s, left -= 16) {
        lchar* s0 = lds + slot * kSlot;
#pragma unroll
        for (int j = 0; j < 2; ++j) a[0][j] = keep_first(fa.load(s0, s, j), left - 8 * (lane >> 5));
#pragma unroll
        for (int i = 0; i < NTB; ++i) b[0][i] = keep_first(fb.load(s0 + kOperand, s, i), left - 8 * (lane >> 5));
        mul(0);
    }
    slot ^= 1;
    wait_vm<0>();              // before the stores, so that the next tile's first stage waits for none of them
    store();
}

template <bool AX, bool BX, Epilogue EPI>
__global__ __launch_bounds__(kThreads, 2) void k_grouped_wide(Args p) {
    constexpr bool WEIGHT = BX;
    constexpr int AW = EPI == kSwigluKeep ? kTile / 2 : kTile;
    __shared__ u32x4 s_ring[kLds / 16];
    __shared__ int s_first[kMaxE + 1];     // first tile of rows of each expert
    __shared__ int s_rows[kMaxE];
    __shared__ int s_wave[8];
    lchar* lds = (lchar*)(__attribute__((address_space(3))) u32x4*)s_ring;
    const uint32_t base = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)lds);
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int ta = (p.na + AW - 1) / AW;
    int run_rows[2], sum = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int e = 2 * tid + i;
        long long seg;
        run_rows[i] = e < p.E ? expert_rows(p, e, &seg) : 0;
        sum += (run_rows[i] + kTile - 1) / kTile;
    }
    int run = sum;
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(run, d);
        if (lane >= d) run += o;
    }
    if (lane == 63) s_wave[wave] = run;
    __syncthreads();
    int before = run - sum, all = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        if (w < wave) before += s_wave[w];
        all += s_wave[w];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int e = 2 * tid + i;
        if (e < p.E) {
            s_first[e] = before;
            s_rows[e] = run_rows[i];
        }
        before += (run_rows[i] + kTile - 1) / kTile;
    }
    if (tid == 0) s_first[p.E] = all;
    __syncthreads();
    const int tb = WEIGHT ? (p.nb + kTile - 1) / kTile : 0;
    const long long total = WEIGHT ? (long long)p.E * ta * tb : (long long)uniform(all) * ta;
    const int xcd = blockIdx.x % kNxcd;
    const long long hi = total * (xcd + 1) / kNxcd, step = gridDim.x / kNxcd;
    auto place = [&](long long t) {
        Place r;
        int at, tiles;
        if (WEIGHT) {
            r.e = (int)(t / ((long long)ta * tb));
            at = (int)(t - (long long)r.e * ta * tb);
            tiles = tb;
            r.nb = p.nb;
        } else {
            const int u = (int)(t / ta);
            int e = 0;         // experts whose tiles all lie before u
            for (int c = 0; c < p.E; c += 64)
                e += __popcll(__ballot(c + lane < p.E && s_first[c + lane + 1] <= u));
            r.e = uniform(e);
            const int first = uniform(s_first[r.e]);
            tiles = uniform(s_first[r.e + 1]) - first;
            at = (int)(t - (long long)first * ta);
        }
        r.rows = uniform(s_rows[r.e]);
        r.seg = p.seg_off[r.e];
        const int g = at / (kGroup * ta), in = at - g * kGroup * ta, wide = min(kGroup, tiles - g * kGroup);
        r.a0 = (in / wide) * AW;
        const int bt = g * kGroup + in % wide;
        if (WEIGHT) {
            r.b0 = bt * kTile;
        } else {
            const int blocks = ((r.rows + 31) / 32 + tiles - 1) / tiles;
            r.b0 = bt * blocks * 32;
            r.nb = min(r.rows, r.b0 + blocks * 32);
        }
        return r;
    };
    long long t = total * xcd / kNxcd + blockIdx.x / kNxcd;
    if (t >= hi) return;
    Place cur = place(t);
    Transfers<AX, BX, EPI == kSwigluKeep> tr;
    tr.init(p, cur, wave, lane);
    int slot = 0;
    if (tr.nk > 0) tr.issue(0, base, wave, lane);
    wait_vm<0>();
    while (t < hi) {
        const long long t2 = t + step;
        const Place then = t2 < hi ? place(t2) : cur;
        auto next = [&](int sl) {
            if (t2 < hi) {
                tr.init(p, then, wave, lane);
                if (tr.nk > 0) tr.issue(0, base + sl * kSlot, wave, lane);
            }
        };
        // row blocks of this wavefront's half of the tile: every other one
        switch (((min(cur.nb - cur.b0, kTile) + 31) / 32 - (wave >> 2) + 1) / 2) {
            case 0: run_tile<AX, BX, EPI, 0>(p, cur, tr, lds, base, slot, wave, lane, next); break;
            case 1: run_tile<AX, BX, EPI, 1>(p, cur, tr, lds, base, slot, wave, lane, next); break;
            case 2: run_tile<AX, BX, EPI, 2>(p, cur, tr, lds, base, slot, wave, lane, next); break;
            case 3: run_tile<AX, BX, EPI, 3>(p, cur, tr, lds, base, slot, wave, lane, next); break;
            default: run_tile<AX, BX, EPI, 4>(p, cur, tr, lds, base, slot, wave, lane, next); break;
        }
        cur = then;
        t = t2;
    }
}

}  // namespace

hipError_t launch_wide(Epilogue epi, bool across, const Args& p, int num_cu, hipStream_t s) {
    int grid = num_cu - num_cu % kNxcd;
    if (grid < kNxcd) grid = kNxcd;
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(grid), dim3(kThreads), 0, s, p); };
    switch (epi) {
        case kRows:
            if (across) go(k_grouped_wide<true, false, kRows>);
            else go(k_grouped_wide<false, false, kRows>);
            break;
        case kSwigluKeep: go(k_grouped_wide<false, false, kSwigluKeep>); break;
        case kSwigluGrad: go(k_grouped_wide<true, false, kSwigluGrad>); break;
        case kWeight16: go(k_grouped_wide<true, true, kWeight16>); break;
        case kWeight16Add: go(k_grouped_wide<true, true, kWeight16Add>); break;
        case kWeight32: go(k_grouped_wide<true, true, kWeight32>); break;
    }
    return hipGetLastError();
}

}  // namespace grouped
}  // namespace moe
