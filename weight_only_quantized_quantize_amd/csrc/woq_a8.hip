// Products of INT8 weights with INT8 activation rows on the int8 matrix cores.
//
//   y[r, n] = fp16(sw(n) sx(r) sum_k code[n, k] q[r, k])
//
// The integer sums are exact (int32), so neither the tiling nor the order of
// the sum changes a bit of the result.  The weights are the INT8 device
// layout, bytes code + 128; flipping the top bit of a byte gives the code in
// two's complement (one v_xor_b32 per four codes).
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
    int vec;                  // y may be written in 16-byte pieces
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
template <int BM, int BN, int WM, int WN, int WK, int KS, int PF>
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
    auto swz_w = [](int row) { return (row & 3) | ((row >> 2) / NT & 1) << 2; };
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
    // weight row of fragment j, lane row m: the 4 NT rows of a lane's results
    // are adjacent, so its part of an output row is one piece
    const int wrow = wn * 16 * NT + (m >> 2) * 4 * NT + (m & 3), xrow = wm * 16 * MT + m;
    auto compute = [&](const uint8_t* buf) {
#pragma unroll
        for (int t = 0; t < STEPS; ++t) {
            const int ch = (wk * STEPS + t) * 4 + c;
            i32x4 wf[NT], xf[MT];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int row = wrow + 4 * j;
                wf[j] = *(const __attribute__((address_space(3))) i32x4*)(buf + row * KS + 16 * (ch ^ swz_w(row)));
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const int row = xrow + 16 * i;
                xf[i] = *(const __attribute__((address_space(3))) i32x4*)(buf + (BN + row) * KS + 16 * (ch ^ swz_x(row)));
            }
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < MT; ++i)
                    acc[j][i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[j], xf[i], acc[j][i], 0, 0, 0);
        }
    };

    const int S = (a.Kd + KS - 1) / KS;
    uint8_t *b0 = lds, *b1 = lds + STAGE;
    static_assert(PF == 1 || PF % 2 == 0, "the buffers alternate within one turn of the register sets");
#pragma unroll
    for (int u = 0; u < PF; ++u) load(sw[u], sx[u], u);
    store(sw[0], sx[0], 0, b0);
    __syncthreads();
    if constexpr (PF == 1) {
        for (int s = 0; s < S; ++s) {
            if (s + 1 < S) load(sw[0], sx[0], s + 1);
            compute(s & 1 ? b1 : b0);
            if (s + 1 < S) store(sw[0], sx[0], s + 1, s & 1 ? b0 : b1);
            __syncthreads();
        }
    } else {
        for (int s = 0; s < S; s += PF) {
#pragma unroll
            for (int u = 0; u < PF; ++u) {
                load(sw[u], sx[u], s + u + PF);
                if (s + u < S) compute(u & 1 ? b1 : b0);
                store(sw[(u + 1) % PF], sx[(u + 1) % PF], s + u + 1, u & 1 ? b0 : b1);
                __syncthreads();
            }
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

    const int nl = n0 + wn * 16 * NT + c * 4 * NT;     // this lane's 4 NT outputs
    if (nl >= a.N) return;
    float scale[4 * NT];
#pragma unroll
    for (int j = 0; j < 4 * NT; ++j) scale[j] = row_scale(a, nl + j);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int row = xrow + 16 * i;
        if (row >= rows_x) continue;
        const float sx1 = *gptr(a.qs + r0 + row);
        uint16_t* yr = a.y + (r0 + row) * a.ldy + nl;
        uint32_t h[2 * NT];
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                h[2 * j + e] = (uint32_t)f_to_h((float)acc[j][i][2 * e] * (sx1 * scale[4 * j + 2 * e])) |
                               (uint32_t)f_to_h((float)acc[j][i][2 * e + 1] * (sx1 * scale[4 * j + 2 * e + 1])) << 16;
        if (a.vec && nl + 4 * NT <= a.N) {
            if constexpr (NT % 2 == 0) {
#pragma unroll
                for (int j = 0; j < NT; j += 2)
                    gstore_u4(reinterpret_cast<uint4*>(yr + 4 * j), make_uint4(h[2 * j], h[2 * j + 1], h[2 * j + 2], h[2 * j + 3]));
            } else {
#pragma unroll
                for (int j = 0; j < NT; ++j) *(__attribute__((address_space(1))) u32x2*)(yr + 4 * j) = u32x2{h[2 * j], h[2 * j + 1]};
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4 * NT; ++j)
                if (nl + j < a.N) *gptr(yr + j) = (uint16_t)(h[j >> 1] >> (16 * (j & 1)));
        }
    }
}

template <int BM, int BN, int WM, int WN, int WK, int KS, int PF>
hipError_t launch_lds(A8Args a, hipStream_t s) {
    a.tiles_m = (int)woq::ceil_div(a.b, BM);
    a.tiles_n = (int)woq::ceil_div(a.N, BN);
    a.GM = 8;
    void* argv[] = {&a};
    return hipLaunchKernel(reinterpret_cast<const void*>(&qgemm_int8_a8_lds<BM, BN, WM, WN, WK, KS, PF>),
                           dim3((unsigned)((int64_t)a.tiles_m * a.tiles_n)), dim3(64 * WM * WN * WK), argv, 0, s);
}

hipError_t launch_a8(const A8Args& a, hipStream_t s) {
    if (a.b <= 16) {
        if (a.N > 16384) return launch_lds<16, 64, 1, 2, 4, 512, 1>(a, s);
        return launch_lds<16, 16, 1, 1, 8, 512, 2>(a, s);
    }
    if (a.b <= 64) {
        if (a.N > 16384) return launch_lds<64, 128, 2, 4, 1, 128, 4>(a, s);
        return launch_lds<64, 16, 1, 1, 8, 512, 2>(a, s);
    }
    if (a.b <= 256) return launch_lds<64, 64, 2, 2, 2, 128, 4>(a, s);
    if (a.b <= 512) return launch_lds<64, 128, 1, 4, 2, 128, 2>(a, s);
    if (a.b <= 1024) return launch_lds<128, 256, 2, 4, 1, 128, 2>(a, s);
    return launch_lds<256, 256, 4, 4, 1, 128, 1>(a, s);
}

}  // namespace

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
    if (w->K > WOQ_A8_MAX_K || w->N > (int64_t)INT32_MAX - 64 || b > 16 * 65535) return WOQ_EUNSUPPORTED;
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
    a.vec = woq::aligned16(y) && (ldy & 7) == 0;
    const hipError_t e = launch_a8(a, (hipStream_t)stream);
    if (e != hipSuccess) {
        woq::set_hip_error((int)e);
        return WOQ_EHIP;
    }
    return WOQ_OK;
}
