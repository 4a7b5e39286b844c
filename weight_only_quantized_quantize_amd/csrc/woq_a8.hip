// Products of INT8 weights with INT8 activation rows on the int8 matrix cores.
//
//   y[r, n] = fp16(sw(n) sx(r) sum_k code[n, k] q[r, k])
//
// The integer sums are exact (int32), so neither the tiling nor the order of
// the sum changes a bit of the result.  The weights are the INT8 device
// layout, bytes code + 128; flipping the top bit of a byte gives the code in
// two's complement (one v_xor_b32 per four codes).
//
// Few rows are bound by the weights' bytes (one row of 8192 x 3584 8.4 us from
// HBM, 3.5 TB/s, 7.1-7.3 where three such weights in turn stay in the last-level
// cache, 1.55 of either the launch; 61 rows of 28672 x 3584 23-24 us, 4.4-4.6
// TB/s, 224 of the 256 compute units at work), many by the matrix cores (4095
// rows of 28672 x 3584 411-430 us, 1.96-2.05 POP/s, level with the library's
// product of that shape); between them tiles small enough to fill the device are
// bound by what LDS moves (509 rows of 3584 x 14336 48 us, 1.1 POP/s).  Both operands pass through LDS: a
// lane per row, the matrix instruction's order, would cost the address unit a
// lookup per lane and, of the weights, a load per row of tiles.
#include <hip/hip_runtime.h>

#include "woq_gemv.h"
#include "woq_internal.h"

namespace {

using namespace woqk;

typedef int i32x4 __attribute__((ext_vector_type(4)));

struct A8Args {
    const uint8_t* codes;     // [N4][Kd]
    const int8_t* q;          // [b][ldq]
    const float* qs;          // [b]
    uint16_t* y;              // [b][ldy]
    int64_t ldq, ldy, b;
    int N, K, Kd, nseg;
    int tiles_m, tiles_n, GM; // tiles of activation and weight rows; token tiles side by side
    int vec;                  // y may be written in 8-byte pieces
    int seg_end[WOQ_MAX_SEGMENTS];
    float seg_scale[WOQ_MAX_SEGMENTS];
};

__device__ __forceinline__ float row_scale(const A8Args& a, int n) {
    float s = a.seg_scale[0];
#pragma unroll
    for (int i = 1; i < WOQ_MAX_SEGMENTS; ++i)
        if (i < a.nseg && n >= a.seg_end[i - 1]) s = a.seg_scale[i];
    return s;
}

// One workgroup: BM activation rows x BN weight rows, WM x WN x WK waves.
template <int BM, int BN, int WM, int WN, int WK, int KS, int PF, bool EARLY>
__global__ __launch_bounds__(64 * WM * WN * WK) void qgemm_int8_a8_lds(A8Args a) {
    constexpr int T = 64 * WM * WN * WK;
    constexpr int CPS = KS / 16;                       // 16-byte chunks of a row per stage
    constexpr int MT = BM / WM / 16, NT = BN / WN / 16;
    constexpr int STEPS = KS / 64 / WK;                // 64-channel steps of a wave per stage
    constexpr int LW = (BN * CPS + T - 1) / T, LX = (BM * CPS + T - 1) / T;
    static_assert(BM % (16 * WM) == 0 && BN % (16 * WN) == 0 && KS % (64 * WK) == 0 && KS % 128 == 0, "tile");
    constexpr int STAGE = (BM + BN) * KS;
    constexpr int RED = (WK - 1) * BM * BN * 4;
    __shared__ __align__(16) uint8_t lds[2 * STAGE > RED ? 2 * STAGE : RED];

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wk = wave / (WM * WN), wm = wave / WN % WM, wn = wave % WN;
    const int m = lane & 15, c = lane >> 4;
    // tiles: a contiguous range per XCD (workgroups go round the XCDs), and in
    // it groups of GM token tiles side by side over all weight tiles
    int tm, tn;
    {
        const int total = (int)gridDim.x, xcd = blockIdx.x & 7, q = total >> 3, rem = total & 7;
        const int pid = xcd * q + min(xcd, rem) + ((int)blockIdx.x >> 3);
        const int g = pid / (a.GM * a.tiles_n), first = g * a.GM, size = min(a.GM, a.tiles_m - first);
        const int in = pid - g * a.GM * a.tiles_n;
        tm = first + in % size;
        tn = in / size;
    }
    const int n0 = tn * BN;
    const int64_t r0 = (int64_t)tm * BM;
    const int n4 = (a.N + 3) & ~3, chunks_w = a.Kd >> 4, chunks_x = (a.K + 15) >> 4;
    const int rows_x = (int)min((int64_t)BM, a.b - r0);
    const uint8_t* wbase = a.codes + (int64_t)n0 * a.Kd;
    const int8_t* xbase = a.q + r0 * a.ldq;

    // chunk p of a stage: row p / CPS, chunk p % CPS; it lies in LDS at chunk
    // position (p % CPS) ^ swizzle(row), so that the eight lanes of a fragment
    // read that go together fall on different banks
    auto swz_w = [](int row) { return row / NT & 7; };
    auto swz_x = [](int row) { return row & 7; };
    uint4 sw[PF][LW], sx[PF][LX];
    auto load = [&](uint4 (&lw)[LW], uint4 (&lx)[LX], int s) {
#pragma unroll
        for (int i = 0; i < LW; ++i) {
            const int p = tid + i * T, row = p / CPS, ch = s * CPS + p % CPS;
            const bool ok = (BN * CPS % T == 0 || p < BN * CPS) && n0 + row < n4 && ch < chunks_w;
            lw[i] = gload_u4(reinterpret_cast<const uint4*>(ok ? wbase + (int64_t)row * a.Kd + 16 * ch : a.codes));
        }
#pragma unroll
        for (int i = 0; i < LX; ++i) {
            const int p = tid + i * T, row = p / CPS, ch = s * CPS + p % CPS;
            const bool ok = (BM * CPS % T == 0 || p < BM * CPS) && row < rows_x && ch < chunks_x;
            lx[i] = gload_u4(reinterpret_cast<const uint4*>(ok ? xbase + row * a.ldq + 16 * ch : a.q));
        }
    };
    auto store = [&](const uint4 (&lw)[LW], const uint4 (&lx)[LX], int s, uint8_t* buf) {
#pragma unroll
        for (int i = 0; i < LW; ++i) {
            const int p = tid + i * T, row = p / CPS, ch = p % CPS;
            if (BN * CPS % T == 0 || p < BN * CPS)
                *(__attribute__((address_space(3))) u32x4*)(buf + row * KS + 16 * (ch ^ swz_w(row))) =
                    u32x4{lw[i].x ^ 0x80808080u, lw[i].y ^ 0x80808080u, lw[i].z ^ 0x80808080u, lw[i].w ^ 0x80808080u};
        }
#pragma unroll
        for (int i = 0; i < LX; ++i) {
            const int p = tid + i * T, row = p / CPS, ch = p % CPS;
            if (BM * CPS % T == 0 || p < BM * CPS) {
                // chunks past the row meet whatever the weight chunk was read
                // from: they have to be zero here
                const bool ok = s * CPS + ch < chunks_x;
                *(__attribute__((address_space(3))) u32x4*)(buf + (BN + row) * KS + 16 * (ch ^ swz_x(row))) =
                    u32x4{ok ? lx[i].x : 0, ok ? lx[i].y : 0, ok ? lx[i].z : 0, ok ? lx[i].w : 0};
            }
        }
    };

    i32x4 acc[NT][MT];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < MT; ++i) acc[j][i] = i32x4{0, 0, 0, 0};
    // the activations are the first operand and the weights the second, with
    // column m of tile j the weight row NT m + j: a lane then has NT adjacent
    // outputs of four rows, and the 16 lanes of a row 16 NT adjacent ones
    const int wrow = wn * 16 * NT + NT * m, xrow = wm * 16 * MT + m;
    i32x4 wf[NT], xf[MT];
    auto fragments = [&](const uint8_t* buf, int t) {
        const int ch = (wk * STEPS + t) * 4 + c;
#pragma unroll
        for (int j = 0; j < NT; ++j)
            wf[j] = *(const __attribute__((address_space(3))) i32x4*)(buf + (wrow + j) * KS + 16 * (ch ^ swz_w(wrow + j)));
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int row = xrow + 16 * i;
            xf[i] = *(const __attribute__((address_space(3))) i32x4*)(buf + (BN + row) * KS + 16 * (ch ^ swz_x(row)));
        }
    };
    auto multiply = [&]() {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < MT; ++i) acc[j][i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(xf[i], wf[j], acc[j][i], 0, 0, 0);
    };

    // Register set u holds the stages that are u modulo PF, read PF turns ahead
    // (stages past the end read the first chunk over and over: loads that always
    // happen let every wait count exactly).  In turn s, stage s is multiplied
    // out of its buffer and stage s + 1 goes into the other one, which was last
    // read before the previous barrier:
    //   EARLY: between the first operand reads and the products, which then hide
    //   the writes (where the products of a turn take longer than the loads);
    //   else after the products, so that the loads have that much longer.
    const int S = (a.Kd + KS - 1) / KS;
    auto buf = [&](int s) { return lds + (s & 1) * STAGE; };
    static_assert(PF == 1 || PF % 2 == 0, "the buffers alternate within one round of the register sets");
#pragma unroll
    for (int u = 0; u < PF; ++u) load(sw[u], sx[u], u);
    store(sw[0], sx[0], 0, buf(0));
    if constexpr (EARLY) load(sw[0], sx[0], PF);
    __syncthreads();
    // set: of stage s + 1; own: of stage s
    auto turn = [&](int s, int set, int own, const uint8_t* from, uint8_t* to) {
        if constexpr (!EARLY) load(sw[own], sx[own], s + PF);
        // only the products of turns past the end are left out, not their loads
        if (PF == 1 || s < S) fragments(from, 0);
        if constexpr (EARLY) {
            store(sw[set], sx[set], s + 1, to);
            load(sw[set], sx[set], s + 1 + PF);
        }
        if (PF == 1 || s < S) {
            multiply();
#pragma unroll
            for (int t = 1; t < STEPS; ++t) {
                fragments(from, t);
                multiply();
            }
        }
        if constexpr (!EARLY) store(sw[set], sx[set], s + 1, to);
        __syncthreads();
    };
    if constexpr (PF == 1) {
        for (int s = 0; s < S; ++s) turn(s, 0, 0, buf(s), buf(s + 1));
    } else {
        for (int s = 0; s < S; s += PF) {
#pragma unroll
            for (int u = 0; u < PF; ++u)
                turn(s + u, (u + 1) % PF, u, buf(u), buf(u + 1));
        }
    }

    if constexpr (WK > 1) {
        // the K groups' sums meet in the first group
        i32x4* red = reinterpret_cast<i32x4*>(lds);
        if (wk > 0) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < MT; ++i)
                    *(__attribute__((address_space(3))) i32x4*)&red[(((wk - 1) * WM * WN + wave % (WM * WN)) * NT * MT + j * MT + i) * 64 + lane] = acc[j][i];
        }
        __syncthreads();
        if (wk > 0) return;
#pragma unroll
        for (int g = 0; g < WK - 1; ++g)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < MT; ++i)
                    acc[j][i] += *(const __attribute__((address_space(3))) i32x4*)&red[((g * WM * WN + wave) * NT * MT + j * MT + i) * 64 + lane];
    }

    const int nl = n0 + wn * 16 * NT + NT * m;         // this lane's NT outputs
    if (nl >= a.N) return;
    float scale[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) scale[j] = row_scale(a, nl + j);
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int row = wm * 16 * MT + 16 * i + 4 * c + e;
            if (row >= rows_x) continue;
            const float sx1 = *gptr(a.qs + r0 + row);
            uint16_t* yr = a.y + (r0 + row) * a.ldy + nl;
            uint16_t h[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) h[j] = f_to_h((float)acc[j][i][e] * (sx1 * scale[j]));
            if (NT == 4 && a.vec && nl + 4 <= a.N) {
                *(__attribute__((address_space(1))) u32x2*)yr = u32x2{h[0] | (uint32_t)h[1 % NT] << 16, h[2 % NT] | (uint32_t)h[3 % NT] << 16};
            } else if (NT == 2 && a.vec && nl + 2 <= a.N) {
                *gptr(reinterpret_cast<uint32_t*>(yr)) = h[0] | (uint32_t)h[1 % NT] << 16;
            } else {
#pragma unroll
                for (int j = 0; j < NT; ++j)
                    if (nl + j < a.N) *gptr(yr + j) = h[j];
            }
        }
}

template <int BM, int BN, int WM, int WN, int WK, int KS, int PF, bool EARLY>
hipError_t launch_lds(A8Args a, hipStream_t s) {
    a.tiles_m = (int)woq::ceil_div(a.b, BM);
    a.tiles_n = (int)woq::ceil_div(a.N, BN);
    a.GM = 8;
    void* argv[] = {&a};
    return hipLaunchKernel(reinterpret_cast<const void*>(&qgemm_int8_a8_lds<BM, BN, WM, WN, WK, KS, PF, EARLY>),
                           dim3((unsigned)((int64_t)a.tiles_m * a.tiles_n)), dim3(64 * WM * WN * WK), argv, 0, s);
}

// Tiles from small to large, each with the fastest division into waves, stage
// length and prefetch depth of a sweep on MI355X (rows 1 to 2048, weights
// 8192 x 3584, 28672 x 3584, 3584 x 14336, 3584 x 4096 and 1024 x 1024).
// The 64 x 128 tile has two: with one row of tiles the weights stream from HBM
// and the loop with the fewest operand reads is ahead (61 rows of 28672 x 3584:
// 23.5 us against 24.2), with several they come from L2 and two K halves side by
// side are (256 rows of 8192 x 3584: 16.5 against 17.1).
struct A8Plan {
    int bm, bn;
    bool rounds;              // of the tiles as tall, the one for several rounds of workgroups
    hipError_t (*launch)(A8Args, hipStream_t);
};
const A8Plan PLANS[] = {
    {16, 16, false, &launch_lds<16, 16, 1, 1, 8, 512, 2, true>},
    {16, 32, false, &launch_lds<16, 32, 1, 2, 4, 512, 2, false>},
    {16, 64, true, &launch_lds<16, 64, 1, 4, 2, 256, 2, true>},
    {32, 32, false, &launch_lds<32, 32, 1, 2, 4, 512, 2, false>},
    {16, 128, false, &launch_lds<16, 128, 1, 4, 2, 256, 2, false>},
    {32, 64, true, &launch_lds<32, 64, 1, 2, 4, 256, 2, false>},
    {64, 64, false, &launch_lds<64, 64, 2, 2, 4, 256, 2, true>},
    {64, 128, true, [](A8Args a, hipStream_t s) {
         return a.b <= 64 ? launch_lds<64, 128, 2, 4, 1, 128, 4, false>(a, s)
                          : launch_lds<64, 128, 1, 4, 2, 128, 4, false>(a, s);
     }},
    {128, 128, true, &launch_lds<128, 128, 2, 4, 1, 128, 2, false>},
    {128, 256, false, &launch_lds<128, 256, 2, 4, 1, 128, 2, true>},
    {256, 256, true, &launch_lds<256, 256, 2, 4, 1, 128, 1, true>},
};

// The smallest tile that still gives at most one workgroup to a compute unit: a
// second round of workgroups cost more than the reuse that a larger tile adds
// (256 rows of 8192 x 3584: 64 x 128 tiles 16.5 us, 64 x 64 17.3; 1021 rows:
// 128 x 256 36.8, 128 x 128 38.9; 509 rows of 28672 x 3584: 256 x 256 60.9,
// 128 x 256 75.5), and idle compute units cost more than that reuse gains (256
// rows of 3584 x 14336: 64 x 64 33.4 us, 64 x 128, half the workgroups, 46).  Of
// two tiles of one size, the one with more workgroups.
//
// Rows of a tile past the batch reuse nothing, and tall tiles read ahead the
// least: up to 64 rows take no tile of more than 64, and where no tile fits one
// round, a batch takes several rounds of the lowest one that holds it.  us, that
// one | the 128 x 256 tile where it fits one round, else 256 x 256:
//   32784 x 3584:   1 row 25 | 33, 17 rows 29 | 34, 61 rows 38 | 37
//   57344 x 3584:   1 row 37 | 38, 17 rows 40 | 40, 61 rows 44 | 43
//   57344 x 8192:   1 row 85 | 103, 17 rows 88 | 105, 61 rows 99 | 111
//   152064 x 3584:  1 row 91 | 146, 17 rows 101 | 148, 61 rows 111 | 158, 128 rows 130 | 173
//   256000 x 1024:  1 row 44 | 70, 17 rows 60 | 74, 61 rows 66 | 85, 128 rows 80 | 104
const A8Plan& choose_plan(int64_t N, int64_t b) {
    const A8Plan *const largest = PLANS + sizeof(PLANS) / sizeof(PLANS[0]) - 1, *best = nullptr;
    const int64_t cus = woq::compute_units();
    auto tiles = [&](const A8Plan& p) { return woq::ceil_div(b, p.bm) * woq::ceil_div(N, p.bn); };
    for (const A8Plan& p : PLANS) {
        if (b <= 64 && p.bm > 64) continue;
        if (best && p.bm * p.bn > best->bm * best->bn) break;
        if (tiles(p) <= cus && (!best || tiles(p) > tiles(*best))) best = &p;
    }
    if (best) return *best;
    for (const A8Plan& p : PLANS)      // a launch has fewer than 2^32 threads, 512 to a workgroup
        if (p.rounds && b <= p.bm && tiles(p) < 1 << 23) return p;
    return *largest;
}

}  // namespace

extern "C" int woq_qgemm_int8_a8_tile(int64_t N, int64_t b, int32_t* rows, int32_t* cols) {
    if (N < 1 || b < 1 || !rows || !cols) return WOQ_EINVAL;
    if (N > (int64_t)INT32_MAX - 512 || b > (int64_t)INT32_MAX - 512) return WOQ_EUNSUPPORTED;
    const A8Plan& p = choose_plan(N, b);
    *rows = p.bm;
    *cols = p.bn;
    return WOQ_OK;
}

extern "C" int woq_qgemm_int8_a8(const woq_int8_w* w, const int8_t* xq, int64_t ldq, const float* xs, int64_t b,
                                 uint16_t* y, int64_t ldy, void* stream) {
    if (!w || w->N < 0 || w->K < 1 || b < 0 || ldq < w->K || ldy < w->N) return WOQ_EINVAL;
    if (w->nseg < 1 || w->nseg > WOQ_MAX_SEGMENTS || w->seg_end[w->nseg - 1] != w->N) return WOQ_EINVAL;
    for (int i = 0; i < w->nseg; ++i) {
        const int64_t lo = i ? w->seg_end[i - 1] : 0;
        if (w->seg_end[i] < lo) return WOQ_EINVAL;
    }
    if (b == 0 || w->N == 0) return WOQ_OK;
    if (!w->codes || !xq || !xs || !y) return WOQ_EINVAL;
    if (!woq::aligned16(w->codes) || !woq::aligned16(xq) || (ldq & 15) || ((uintptr_t)xs & 3u) || ((uintptr_t)y & 1u))
        return WOQ_EALIGN;
    if (w->K > WOQ_A8_MAX_K || w->N > (int64_t)INT32_MAX - 512 || b > (int64_t)INT32_MAX - 512 ||
        woq::ceil_div(b, 256) * woq::ceil_div(w->N, 256) > (int64_t)UINT32_MAX / 1024)
        return WOQ_EUNSUPPORTED;     // a launch has fewer than 2^32 threads
    A8Args a;
    a.codes = static_cast<const uint8_t*>(w->codes);
    a.q = xq;
    a.qs = xs;
    a.y = y;
    a.ldq = ldq;
    a.ldy = ldy;
    a.b = b;
    a.N = (int)w->N;
    a.K = (int)w->K;
    a.Kd = (int)woq::round_up(w->K, 64);
    a.nseg = w->nseg;
    for (int i = 0; i < WOQ_MAX_SEGMENTS; ++i) {
        a.seg_end[i] = i < w->nseg ? (int)w->seg_end[i] : (int)w->N;
        a.seg_scale[i] = i < w->nseg ? w->seg_scale[i] : 0.0f;
    }
    a.vec = ((uintptr_t)y & 7u) == 0 && (ldy & 3) == 0;
    const hipError_t e = choose_plan(a.N, a.b).launch(a, (hipStream_t)stream);
    if (e != hipSuccess) {
        woq::set_hip_error((int)e);
        return WOQ_EHIP;
    }
    return WOQ_OK;
}
