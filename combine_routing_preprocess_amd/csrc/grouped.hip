// Matrix products grouped by expert over the dispatched rows, for sizes that
// are any multiple of 8: the rows' product with the expert's weight and with
// its transpose, the weight's gradient, and the two products of the SwiGLU
// MLP's training passes with the activation in their epilogue.
//
// Every one is C[b][a] = sum over k of A[a][k] * B[b][k] for one expert, fp32
// sums of bf16 products (MFMA), one rounding at the end:
//   product            a = feature of w, b = row, k = column of the rows
//   its transpose      the same with w read across its rows (k = row of w)
//   weight's gradient  a = column of the rows, b = column of the gradient, k = row (both read across)
// An operand is "across" when its k runs over rows of the array; it is staged as
// it lies and turned by the transposing LDS read on its way to the MFMA.
//
// This file: four wavefronts per workgroup, two workgroups per CU, so that one's
// prologue, barriers and epilogue fall into the other's products.  Both operands
// go straight to LDS, in stages of 32 elements of the sum (a ring of three or
// four), the last step of a stage is multiplied behind the next stage's barrier.
// Tiles of 256 features x 128 rows, or of 128 x 128 with four stages where those
// go into fewer rounds (narrow below): such calls are bound by the latency of a
// stage (0.6 us), not by bandwidth.  Measured on MI355X: 16 tokens, 256 experts
// top-8, 7168 x 4096 transposed 1.02 ms (5.8 TB/s of the touched weights); one
// token 85 to 91 us (5.1 to 5.5 TB/s; 138 us with the tiles of 256 features);
// 2048 tokens over the same experts, transposed, 2.82 ms (5.5 TB/s).  The weight's
// gradient of 1501 tokens over 24 experts, 1048 x 904: bf16 31 us, added 56, fp32
// 43, added 79; of 1024 rows over 32 experts, 4096 x 7168, 304 us (6.2 TB/s).
//
// An expert's rows are cut into tiles of nearly one size and each XCD takes one
// contiguous run of the tiles, so that the tiles that share an expert's rows and
// weights meet in one L2.
#include "grouped.h"

namespace moe {

using namespace grouped;

namespace {

constexpr int kTB = 128;                    // rows (weight's gradient: columns of the gradient) of a tile
constexpr int kBK = 32;                     // sum's elements per stage
constexpr int kBBytes = kTB * kBK * 2;
constexpr int kPerThread = kMaxE / 256;     // experts whose tiles one thread counts

// A tile's features: 64 for each of FW wavefronts, which share the rows with
// the other 4 / FW, every other block of 32 each.
template <int FW>
struct Geometry {
    static constexpr int TA = 64 * FW, HALVES = 4 / FW;
    static constexpr int ABytes = TA * kBK * 2, Slot = ABytes + kBBytes;
    static constexpr int Slots = FW == 4 ? 3 : 4;                      // stages in LDS: two workgroups per CU
    static constexpr int R16 = FW == 4 ? 32 : 16, R32 = R16 / 2;       // epilogue rows that fit a quarter of a slot
    static_assert(R16 * 144 <= Slot / 4 && R32 * 272 <= Slot / 4 && Slots * Slot <= 76 * 1024, "LDS budget");
};

// A stage's transfers.  Not across: rows of 64 bytes, four chunks of 16, chunk
// c of row r at place c ^ (r / 4) % 4.  Across: rows of 128 FW (B: 256) bytes,
// one per element of the sum, in units of 64 bytes, unit u of row k at place
// u ^ k % 4.  Either way the reads below touch every bank once.
template <bool AX, bool BX, bool KEEP, int FW>
struct Transfers {
    uint32_t a[FW], b[2];     // per-lane offsets
    int nb_mine;              // B transfers of this wavefront
    uint32_t pitch_a, pitch_b;

    // row of an across operand of which this lane fetches a chunk: 1024 / BYTES rows of BYTES bytes per transfer
    template <int BYTES>
    static __device__ __forceinline__ int across_row(int q, int wave, int lane) {
        return (1024 / BYTES) * (4 * q + wave) + lane / (BYTES / 16);
    }
    template <int BYTES>
    static __device__ __forceinline__ int across_chunk(int k, int lane) {
        return (lane & (BYTES / 16 - 1)) ^ ((k & 3) << 2);
    }

    __device__ __forceinline__ void init(const Args& p, const Tile& t, int wave, int lane) {
        pitch_a = (uint32_t)(AX ? p.na : t.nk) * 2u;
        pitch_b = (uint32_t)(BX ? p.nb : t.nk) * 2u;
        const uint32_t c4 = (uint32_t)((lane & 3) ^ ((lane >> 4) & 3)) * 16u;
#pragma unroll
        for (int q = 0; q < FW; ++q) {
            const int r = 64 * q + 16 * wave + (lane >> 2);
            if (AX) {
                const int k = across_row<128 * FW>(q, wave, lane);
                a[q] = (uint32_t)k * pitch_a + (uint32_t)min(t.a0 + 8 * across_chunk<128 * FW>(k, lane), p.na - 8) * 2u;
            } else if (KEEP) {      // rows 64 q .. of the tile: 32 gate features, the same 32 up
                const int f = min(t.a0 + r / 64 * 32 + r % 32, p.na - 1);
                a[q] = (uint32_t)(f + (r % 64) / 32 * p.na) * pitch_a + c4;
            } else {
                a[q] = (uint32_t)min(t.a0 + r, p.na - 1) * pitch_a + c4;
            }
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            if (BX) {
                const int k = across_row<256>(q, wave, lane);
                b[q] = (uint32_t)k * pitch_b + (uint32_t)min(t.b0 + 8 * across_chunk<256>(k, lane), t.nb - 8) * 2u;
            } else {
                b[q] = (uint32_t)min(64 * q + 16 * wave + (lane >> 2), t.nb - t.b0 - 1) * pitch_b + c4;
            }
        }
        nb_mine = BX ? 2 : (2 * ((t.nb - t.b0 + 31) / 32) - wave + 3) / 4;
    }
    __device__ __forceinline__ int count() const { return FW + nb_mine; }

    // Stage kt into LDS from byte address `lds` on; elements past the sum's end read valid memory again.
    __device__ __forceinline__ void issue(const Tile& t, int kt, uint32_t lds, int wave, int lane) const {
        gchar* Ak = t.A + (AX ? (size_t)kt * kBK * pitch_a : (size_t)kt * kBK * 2);
        gchar* Bk = t.B + (BX ? (size_t)kt * kBK * pitch_b : (size_t)kt * kBK * 2);
        const int rem = t.nk - kt * kBK;
        uint32_t va[FW], vb[2];
#pragma unroll
        for (int q = 0; q < FW; ++q) va[q] = a[q];
#pragma unroll
        for (int q = 0; q < 2; ++q) vb[q] = b[q];
        if (rem < kBK) {
            const uint32_t c = (uint32_t)((lane & 3) ^ ((lane >> 4) & 3));
            const uint32_t back = (int)(8 * c) >= rem ? 16u * c : 0u;
#pragma unroll
            for (int q = 0; q < FW; ++q)
                va[q] -= AX ? (uint32_t)max(across_row<128 * FW>(q, wave, lane) - (rem - 1), 0) * pitch_a : back;
#pragma unroll
            for (int q = 0; q < 2; ++q)
                vb[q] -= BX ? (uint32_t)max(across_row<256>(q, wave, lane) - (rem - 1), 0) * pitch_b : back;
        }
        base_ready(Ak, Bk);
#pragma unroll
        for (int q = 0; q < FW; ++q) to_lds16(Ak, va[q], lds + (uint32_t)(4 * q + wave) * 1024u);
#pragma unroll
        for (int q = 0; q < 2; ++q)
            if (BX || q < nb_mine)
                to_lds16(Bk, vb[q], lds + Geometry<FW>::ABytes + (uint32_t)(4 * q + wave) * 1024u);
    }
};

// At most n of this wavefront's transfers in flight (fewer where n has no case).
__device__ __forceinline__ void wait_transfers(int n) {
    if (n >= 8) wait_vm<8>();
    else if (n >= 6) wait_vm<6>();
    else if (n == 5) wait_vm<5>();
    else if (n == 4) wait_vm<4>();
    else if (n == 3) wait_vm<3>();
    else if (n == 2) wait_vm<2>();
    else wait_vm<0>();
}

// One tile; `seg` (rows) or `e` (weight's gradient) says where its outputs go.
// NTB: blocks of 32 rows of each half.
template <bool AX, bool BX, Epilogue EPI, int FW, int NTB>
__device__ __forceinline__ void run_tile(const Args& p, const Tile& t, long long seg, int e, lchar* lds, int wave,
                                         int lane) {
    using G = Geometry<FW>;
    constexpr int S = G::Slots;
    const int fw = wave % FW, half = wave / FW;
    Transfers<AX, BX, EPI == kSwigluKeep, FW> tr;
    tr.init(p, t, wave, lane);
    Fragments<AX, kBK, G::TA * 2, 2> fa;
    Fragments<BX, kBK, kTB * 2, NTB> fb;
    fa.init(2 * fw, 1, lane);
    fb.init(half, G::HALVES, lane);
    f32x16 acc[2][NTB];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < NTB; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[j][i][r] = 0.f;
    const uint32_t base = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)lds);
    const int n = (t.nk + kBK - 1) / kBK;
    int slot = 0;             // of the stage that is multiplied
#pragma unroll
    for (int i = 0; i < S - 1; ++i)
        if (n > i) tr.issue(t, i, base + i * G::Slot, wave, lane);
    u32x4 a[2][2] = {}, b[2][NTB] = {};
    auto load = [&](lchar* s0, int s, int buf) {
#pragma unroll
        for (int j = 0; j < 2; ++j) a[buf][j] = fa.load(s0, s, j);
#pragma unroll
        for (int i = 0; i < NTB; ++i) b[buf][i] = fb.load(s0 + G::ABytes, s, i);
    };
    auto mul = [&](int buf) {
#pragma unroll
        for (int i = 0; i < NTB; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) acc[j][i] = multiply(a[buf][j], b[buf][i], acc[j][i]);
    };
    // Stage kt has landed when at most the transfers of the S - 2 stages after
    // it are in flight; past the barrier every wavefront's have, and the slot
    // of stage kt - 1, which all have read, takes stage kt + S - 1.  A step is
    // loaded while the one before it is multiplied; a stage's last products
    // follow the next stage's barrier.
    for (int kt = 0; kt + 1 < n; ++kt) {
        wait_transfers(tr.count() * min(S - 2, n - 1 - kt));
        lds_barrier();
        if (kt + S - 1 < n) tr.issue(t, kt + S - 1, base + (slot == 0 ? S - 1 : slot - 1) * G::Slot, wave, lane);
        lchar* s0 = lds + slot * G::Slot;
        load(s0, 0, 0);
        mul(1);
        __builtin_amdgcn_sched_barrier(0);
        load(s0, 1, 1);
        mul(0);
        __builtin_amdgcn_sched_barrier(0);
        slot = slot == S - 1 ? 0 : slot + 1;
    }
    if (n > 0) {
        // the last one: as many steps as there are, elements past the sum's end zero in both operands
        wait_vm<0>();
        lds_barrier();
        mul(1);
        for (int s = 0, left = t.nk - (n - 1) * kBK; left > 0; ++s, left -= 16) {
            load(lds + slot * G::Slot, s, 0);
#pragma unroll
            for (int j = 0; j < 2; ++j) a[0][j] = keep_first(a[0][j], left - 8 * (lane >> 5));
#pragma unroll
            for (int i = 0; i < NTB; ++i) b[0][i] = keep_first(b[0][i], left - 8 * (lane >> 5));
            mul(0);
        }
        slot = slot == S - 1 ? 0 : slot + 1;
    }
    // the slot behind the last stage's was read S - 1 stages ago, before a barrier that all have passed
    store_tile<EPI, G::R16, G::R32>(p, t.a0 + (EPI == kSwigluKeep ? 32 : 64) * fw, t.b0, t.nb - t.b0, half, G::HALVES,
                                    seg, e, acc, lds + slot * G::Slot + wave * (G::Slot / 4), lane);
}

// run_tile for as many blocks of 32 rows as the tile has.
template <bool AX, bool BX, Epilogue EPI, int FW>
__device__ __forceinline__ void run_blocks(const Args& p, const Tile& t, long long seg, int e, lchar* lds, int wave,
                                           int lane) {
    const int blocks = (min(t.nb - t.b0, kTB) + 31) / 32;
    if constexpr (FW == 4) {
        switch (blocks) {
            case 1: run_tile<AX, BX, EPI, FW, 1>(p, t, seg, e, lds, wave, lane); break;
            case 2: run_tile<AX, BX, EPI, FW, 2>(p, t, seg, e, lds, wave, lane); break;
            case 3: run_tile<AX, BX, EPI, FW, 3>(p, t, seg, e, lds, wave, lane); break;
            default: run_tile<AX, BX, EPI, FW, 4>(p, t, seg, e, lds, wave, lane); break;
        }
    } else {
        if (blocks <= 2) run_tile<AX, BX, EPI, FW, 1>(p, t, seg, e, lds, wave, lane);
        else run_tile<AX, BX, EPI, FW, 2>(p, t, seg, e, lds, wave, lane);
    }
}

// Products of rows: one workgroup per tile.
template <bool AX, Epilogue EPI, int FW>
__global__ __launch_bounds__(256, 2) void k_grouped_rows(Args p) {
    using G = Geometry<FW>;
    constexpr int AW = EPI == kSwigluKeep ? G::TA / 2 : G::TA;     // features of a tile
    __shared__ u32x4 s_ring[G::Slots * G::Slot / 16];
    __shared__ int s_wave[4];
    __shared__ int s_expert, s_first, s_tiles, s_rows;
    __shared__ long long s_seg;
    lchar* lds = (lchar*)(__attribute__((address_space(3))) u32x4*)s_ring;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int ta = (p.na + AW - 1) / AW;
    // the tiles of rows of every expert, counted by each workgroup
    int mine[kPerThread], rows[kPerThread], sum = 0;
    const int per = (p.E + 255) / 256;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const int e = tid * per + i;
        long long seg;
        rows[i] = i < per && e < p.E ? expert_rows(p, e, &seg) : 0;
        mine[i] = (rows[i] + kTB - 1) / kTB;
        sum += mine[i];
    }
    int run = sum;            // inclusive over the wavefront's lanes
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(run, d);
        if (lane >= d) run += o;
    }
    if (lane == 63) s_wave[wave] = run;
    __syncthreads();
    int before = run - sum, all = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        if (w < wave) before += s_wave[w];
        all += s_wave[w];
    }
    const long long total = (long long)all * ta;
    // each XCD takes one contiguous run of the tiles, so that tiles that share rows or weights share an L2
    const int xcd = blockIdx.x % kNxcd;
    const long long hi = total * (xcd + 1) / kNxcd;
    for (long long t = total * xcd / kNxcd + blockIdx.x / kNxcd; t < hi; t += gridDim.x / kNxcd) {
        const int u = (int)(t / ta);
#pragma unroll
        for (int i = 0, at = before; i < kPerThread; at += mine[i], ++i)
            if (u >= at && u < at + mine[i]) {
                s_expert = tid * per + i;
                s_first = at;
                s_tiles = mine[i];
                s_rows = rows[i];
                s_seg = p.seg_off[tid * per + i];
            }
        __syncthreads();
        const int e = uniform(s_expert), tiles = uniform(s_tiles), nrows = uniform(s_rows);
        const int at = (int)(t - (long long)uniform(s_first) * ta);
        const long long seg = (long long)(((uint64_t)__builtin_amdgcn_readfirstlane((uint32_t)(s_seg >> 32)) << 32) |
                                          __builtin_amdgcn_readfirstlane((uint32_t)s_seg));
        // an expert's rows in tiles of nearly one size, whole blocks of 32; its tiles of rows are neighbours
        const int blocks = ((nrows + 31) / 32 + tiles - 1) / tiles;
        Tile tile;
        tile.a0 = (at / tiles) * AW;
        tile.b0 = (at % tiles) * blocks * 32;
        tile.nb = min(nrows, tile.b0 + blocks * 32);
        tile.nk = p.nk;
        tile.A = uniform_ptr(p.a + (size_t)e * (EPI == kSwigluKeep ? 2 : 1) * p.na * p.nk);
        tile.B = uniform_ptr(p.b + (size_t)(seg + tile.b0) * p.nk);
        run_blocks<AX, false, EPI, FW>(p, tile, seg, e, lds, wave, lane);
        lds_barrier();        // the slots are free for the next tile
    }
}

// Weight's gradient, one workgroup per tile.
template <Epilogue EPI, int FW>
__global__ __launch_bounds__(256, 2) void k_grouped_weight(Args p) {
    using G = Geometry<FW>;
    __shared__ u32x4 s_ring[G::Slots * G::Slot / 16];
    lchar* lds = (lchar*)(__attribute__((address_space(3))) u32x4*)s_ring;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int ta = (p.na + G::TA - 1) / G::TA, tb = (p.nb + kTB - 1) / kTB, each = ta * tb;
    const long long total = (long long)p.E * each;
    const int xcd = blockIdx.x % kNxcd;
    const long long hi = total * (xcd + 1) / kNxcd;
    for (long long t = total * xcd / kNxcd + blockIdx.x / kNxcd; t < hi; t += gridDim.x / kNxcd) {
        const int e = (int)(t / each), at = (int)(t - (long long)e * each);
        long long seg;
        Tile tile;
        tile.nk = expert_rows(p, e, &seg);
        if (tile.nk == 0 && p.accumulate) continue;
        tile.a0 = (at % ta) * G::TA;
        tile.b0 = (at / ta) * kTB;
        tile.nb = p.nb;
        tile.A = uniform_ptr(p.a + (size_t)seg * p.na);
        tile.B = uniform_ptr(p.b + (size_t)seg * p.nb);
        run_blocks<true, true, EPI, FW>(p, tile, 0, e, lds, wave, lane);
        lds_barrier();        // the slots are free for the next tile
    }
}

// Workgroups; more tiles than that are walked.  us at 2^16 and 2^20, weight
// gradients of 256 experts: fp32 accumulated, 7168 x 2048, 6850 and 6980; bf16
// written, 7168 x 4096, 2303 and 2295.
constexpr long long kMaxGrid = 1 << 16;

unsigned grid_for(long long tiles) {
    const long long g = (tiles + kNxcd - 1) / kNxcd * kNxcd;
    return (unsigned)(g < kMaxGrid ? g : kMaxGrid);
}

Args make_args(const moe_handle* h) {
    Args p = {};
    p.seg_off = h->seg_off;
    p.kept = h->kept;
    p.R = h->desc.out_rows;
    p.E = h->desc.E;
    return p;
}

long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

long long copies(const moe_handle* h) { return (long long)h->desc.T * h->desc.K; }

// Which kernel.  The host knows the copies and the experts, not who has how
// many: rows below are the mean.  Measured in us, this file's kernel (two
// workgroups of 256 x 128 per CU) against the wide one (one of 256 x 256):
//   rows, 32 experts, 2048 x 2048: 64 rows each 53 and 61, 128 rows 82 and 67, 512 rows 189 and 169; 256 experts,
//   7168 x 4096: 64 rows 2970 and 3330, 128 rows 3610 and 3550, 256 rows 5000 and 4730; 16 experts, 1024 x 1024, 256
//   rows (128 wide tiles for 256 CUs) 23 and 27
//   weights, 64 experts, 4096 x 7168: 8 rows 620 and 730, 64 rows 760 and 710, 512 rows 2600 and 2120; 32 experts,
//   1024 x 2048 (1024 wide tiles), 1024 rows 148 and 139; 24 experts, 1048 x 904 (480 wide tiles) 78 and 105
// The mean also stands for uneven rows.  With an offset per expert of standard
// deviation 3 in the router's logits, us in the small and the wide tiles, 7168 -> 4096 transposed: 32
// experts, 512 tokens top-8, 448 and 478 (even: 487 and 436), 4096 tokens 2015 and
// 1869 (1944 and 1750); 256 experts, 2048 tokens, 2320 and 2612 (2819 and 3163).
bool wide_rows(const moe_handle* h, int na, int width, int num_cu) {
    const long long rows = copies(h) / h->desc.E;
    return rows >= 96 && h->desc.E * ceil_div(rows, 256) * ceil_div(na, width) >= num_cu;
}
bool wide_weight(const moe_handle* h, int na, int nb, int num_cu) {
    return copies(h) / h->desc.E >= 64 && h->desc.E * ceil_div(na, 256) * ceil_div(nb, 256) >= 4ll * num_cu;
}
// Whether tiles of 128 features take `tiles` of 256 features more evenly: two
// workgroups per CU work through them in rounds, and a round of the smaller
// ones takes half the time.  Worth it up to two rounds.  us of the smaller and
// the larger tiles: 16 experts, 1024 x 1024, 64 tokens 13 and 17, 512 tokens 15
// and 23; 64 experts, 4096 x 4096, 16 rows 89 and 94; one token, 8 experts of
// 7168 x 4096, 85 and 138; but 32 experts, 2048 x 2048, 64 rows each (one round of
// 384 larger tiles, two of the smaller) 61 and 53.
bool narrow(long long tiles, int features, int width, int num_cu) {
    const long long wide = tiles * ceil_div(features, width), small = tiles * ceil_div(features, width / 2);
    return wide < 4ll * num_cu && ceil_div(small, 2 * num_cu) < 2 * ceil_div(wide, 2 * num_cu);
}
// Weights that are not read across, streamed for few rows: the expert MLP's FC2
// kernel, which takes a unit's rows all at once and keeps two stages of weights
// in registers on their way.  us of it and of the better of the two above:
//   256 experts, 7168 -> 4096: 16 tokens 1010 and 1100, 64 rows each 2740 and 2990, 256 rows 4110 and 4850, 512 rows
//   8780 and 7610
//   7168 -> 4096, 1, 16, 64 and 256 rows each: 64 experts (3.8 GB) 406 606 656 1045 and 447 666 713 1179; 32 experts
//   (512 units) 259 298 325 562 and 270 335 377 604; 16 experts (256 units, left to the others) 131 155 165 323 and
//   143 174 186 372; 8 experts (128 units) 125 126 117 157 and 85 87 96 167
//   2048 -> 7168, the same rows: 64 experts (1.9 GB) 220 371 403 562 and 219 340 362 612; 32 experts 141 206 225 307
//   and 134 195 207 344; 16 experts (448 units, left to the others) 94 105 116 177 and 78 101 110 178
//   1024 -> 7168: 64 experts (0.9 GB) 114 179 194 309 and 108 171 202 330; 32 experts (0.5 GB) 71 99 110 171 and 63 91
//   106 185; 16 experts (0.2 GB, left to the others) 50 53 60 101 and 39 47 57 98
//   32 experts, 2048 x 2048 (0.3 GB), 1 to 64 rows 47 to 76 and 38 to 72
// Nearer to the border either side is up to 13 % ahead.  Uneven rows cost it more
// than the others: beyond 320 rows of an expert the weights are streamed again.
// 7168 -> 4096 with the offsets above: 32 experts, 512 tokens, 622 and 546 (even:
// 366 and 406); 256 experts, 2048 tokens, 3496 and 2626 (2555 and 2808).
bool stream_weights(const moe_handle* h, int N, int M, int num_cu) {
    const long long touched = copies(h) < h->desc.E ? copies(h) : h->desc.E;
    return N % 256 == 0 && M % 128 == 0 && copies(h) <= 320ll * h->desc.E && touched * N * M * 2 > (384ll << 20) &&
           touched * (N / 256) >= 2ll * num_cu;
}

template <bool AX, Epilogue EPI>
hipError_t launch_rows(const moe_handle* h, const Args& p, int num_cu, hipStream_t s) {
    constexpr int AW = EPI == kSwigluKeep ? 128 : 256;
    if (p.R == 0 || copies(h) == 0) return hipSuccess;
    if (wide_rows(h, p.na, AW, num_cu)) return launch_wide(EPI, AX, p, num_cu, s);
    // most tiles that the rows can make: each expert's last one may be partial
    const long long tiles = copies(h) / kTB + (copies(h) < h->desc.E ? copies(h) : h->desc.E);
    if (narrow(tiles, p.na, AW, num_cu))
        hipLaunchKernelGGL((k_grouped_rows<AX, EPI, 2>), dim3(grid_for(tiles * ceil_div(p.na, AW / 2))), dim3(256), 0, s, p);
    else
        hipLaunchKernelGGL((k_grouped_rows<AX, EPI, 4>), dim3(grid_for(tiles * ceil_div(p.na, AW))), dim3(256), 0, s, p);
    return hipGetLastError();
}

template <Epilogue EPI>
hipError_t launch_weight(const moe_handle* h, const Args& p, int num_cu, hipStream_t s) {
    if (wide_weight(h, p.na, p.nb, num_cu)) return launch_wide(EPI, true, p, num_cu, s);
    const long long tiles = p.E * ceil_div(p.nb, kTB);
    if (narrow(tiles, p.na, 256, num_cu))
        hipLaunchKernelGGL((k_grouped_weight<EPI, 2>), dim3(grid_for(tiles * ceil_div(p.na, 128))), dim3(256), 0, s, p);
    else
        hipLaunchKernelGGL((k_grouped_weight<EPI, 4>), dim3(grid_for(tiles * ceil_div(p.na, 256))), dim3(256), 0, s, p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_grouped_product(const moe_handle* h, int N, int M, int transpose, const void* rows, const void* w,
                                  void* out, int num_cu, hipStream_t s) {
    if (!transpose && stream_weights(h, N, M, num_cu)) {
        moe_handle g = *h;     // the same segments, rows of N
        g.desc.H = N;
        return launch_gemm_bf16(&g, 1, M, rows, w, out, nullptr, num_cu, s);
    }
    Args p = make_args(h);
    p.a = (const uint16_t*)w;
    p.b = (const uint16_t*)rows;
    p.out = out;
    p.na = transpose ? M : N;
    p.nk = transpose ? N : M;
    return transpose ? launch_rows<true, kRows>(h, p, num_cu, s) : launch_rows<false, kRows>(h, p, num_cu, s);
}

hipError_t launch_grouped_swiglu_keep(const moe_handle* h, int F, const void* rows, const void* w1, void* hout,
                                      void* act, int num_cu, hipStream_t s) {
    Args p = make_args(h);
    p.a = (const uint16_t*)w1;
    p.b = (const uint16_t*)rows;
    p.out = hout;
    p.out2 = (uint16_t*)act;
    p.na = F;
    p.nk = h->desc.H;
    return launch_rows<false, kSwigluKeep>(h, p, num_cu, s);
}

hipError_t launch_grouped_swiglu_grad(const moe_handle* h, int F, const void* grad_out, const void* w2, const void* hin,
                                      void* grad_h, void* act, int num_cu, hipStream_t s) {
    Args p = make_args(h);
    p.a = (const uint16_t*)w2;
    p.b = (const uint16_t*)grad_out;
    p.h = (const uint16_t*)hin;
    p.out = grad_h;
    p.out2 = (uint16_t*)act;
    p.na = F;
    p.nk = h->desc.H;
    return launch_rows<true, kSwigluGrad>(h, p, num_cu, s);
}

hipError_t launch_grouped_weight_grad(const moe_handle* h, int N, int M, int out_dtype, int accumulate,
                                      const void* grad, const void* rows, void* out, int num_cu, hipStream_t s) {
    Args p = make_args(h);
    p.a = (const uint16_t*)rows;
    p.b = (const uint16_t*)grad;
    p.out = out;
    p.na = M;
    p.nb = N;
    p.accumulate = accumulate;
    if (out_dtype != MOE_BF16) return launch_weight<kWeight32>(h, p, num_cu, s);
    if (accumulate) return launch_weight<kWeight16Add>(h, p, num_cu, s);
    return launch_weight<kWeight16>(h, p, num_cu, s);
}

}  // namespace moe
