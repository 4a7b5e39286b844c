// Low-rank adapters of many requests beside a shared projection:
//
//   y[r, n] = fp16(base[r, n] + scale[a] sum_j B[a][n, j] h[r, seg(n) R + j]),
//   h[r, i] = sum_k A[a][i, k] x[r, k],   a = ids[r],
//
// with y = base on rows without an adapter.  Two launches: the inner products
// h into the workspace (fp32, one partial sum per K range), and the outer
// ones added to the base.
//
// Both run on the fp16 matrix cores with 16 ranks (or 16 outputs) of ONE
// adapter against 16 rows: rows that share an adapter share its bytes, and a
// result column belongs to one row, so rows never mix.  h is not rounded to
// fp16 on the way: a row of h is scaled by a power of two to below 2^14 and
// split into two fp16 halves, hi + lo, at least 22 bits; one 16x16x32 step
// multiplies 16 ranks of B with both.
//
// A decode batch is bound by the bytes of the adapters that its rows name (or,
// at a few rows, by the two launches); a prompt by the base and the output.
#include <hip/hip_runtime.h>

#include "woq_gemv.h"
#include "woq_internal.h"

namespace {

using namespace woqk;

typedef unsigned long long u64;

struct LoraArgs {
    const uint16_t* A;        // [count][nseg R][lda]
    const uint16_t* B;        // [count][N][R]
    const float* scale;       // [count]
    const int32_t* rank;      // [count], or null
    const uint16_t* x;
    const int32_t* ids;
    const uint16_t* base;     // null: zeros
    uint16_t* y;
    float* h;                 // [splits][b][nseg R]
    int64_t ldx, ldbase, ldy, lda;
    int b, N, K, R, count, nseg, splits;
    int vec;                  // rows of base and y may be read and written in 16-byte pieces
    int seg_end[WOQ_MAX_SEGMENTS];
    int tile0[WOQ_MAX_SEGMENTS + 1];   // output tiles before each segment
};

__device__ __forceinline__ int rank_of(const LoraArgs& a, int id) {
    return a.rank ? min(max(*gptr(a.rank + id), 0), a.R) : a.R;
}

__device__ __forceinline__ h8 as_h8(uint4 v) { return __builtin_bit_cast(h8, v); }

// Values k .. k + 7 of a row, zero from `end` on (which nothing past is read).
__device__ __forceinline__ uint4 load8_until(const uint16_t* row, int k, int end) {
    if (k + 8 <= end) return gload_u4(reinterpret_cast<const uint4*>(row + k));
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (k + j < end) w[j >> 1] |= (uint32_t)*gptr(row + k + j) << (16 * (j & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The inner products.  blockIdx.y names RT rank tiles of 16 in one segment,
// blockIdx.z one of the K ranges; the W waves split the range and add their
// sums in LDS in a fixed order.
//   LEADER (few rows): one workgroup per row; it works if its row is the first
//     of its adapter, for all rows of that adapter (so distinct adapters run
//     side by side, and a shared one is read once).
//   otherwise: one workgroup per window of 32 rows, one adapter of the window
//     after another (a packed prompt has one or two in a window).
template <int W, int RT, bool LEADER>
__global__ __launch_bounds__(64 * W) void lora_down_kernel(LoraArgs a) {
    constexpr int WIN = LEADER ? 256 : 32;
    constexpr int UNR = 4;
    static_assert(!LEADER || 64 * W >= WIN, "a thread per row of the window");
    __shared__ int sid[WIN], list[WIN], cnt[W];
    __shared__ __align__(16) f4 red[W][RT * 2][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int m = lane & 15, c = lane >> 4;
    const int groups = (a.R + 16 * RT - 1) / (16 * RT);
    const int seg = blockIdx.y / groups, j0 = (blockIdx.y % groups) * 16 * RT;
    const int w0 = LEADER ? 0 : blockIdx.x * WIN;
    const int nwin = min(a.b - w0, WIN);
    if (tid < nwin) sid[tid] = *gptr(a.ids + w0 + tid);
    __syncthreads();

    // this wave's 32-channel steps
    const int steps = (a.K + 31) / 32, full = a.K / 32;
    const int units = a.splits * W, unit = blockIdx.z * W + wave;
    const int lo = (int)((int64_t)steps * unit / units), hi = (int)((int64_t)steps * (unit + 1) / units);
    const int hi_full = min(hi, full);

    for (int p = LEADER ? (int)blockIdx.x : 0; p < (LEADER ? (int)blockIdx.x + 1 : nwin); ++p) {
        const int id = __builtin_amdgcn_readfirstlane(sid[p]);
        if ((unsigned)id >= (unsigned)a.count || j0 >= rank_of(a, id)) continue;
        const bool match = tid < nwin && sid[tid] == id;
        const u64 mask = __ballot(match);
        if (lane == 0) cnt[wave] = __popcll(mask);
        if (__syncthreads_or(match && tid < p)) continue;   // not the first of its adapter
        int before = 0, total = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            if (w < wave) before += cnt[w];
            total += cnt[w];
        }
        if (match) list[before + __popcll(mask & ((1ull << lane) - 1))] = tid;
        __syncthreads();

        const uint16_t* ap[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t)
            ap[t] = a.A + (((int64_t)id * a.nseg + seg) * a.R + min(j0 + 16 * t + m, a.R - 1)) * a.lda;
        for (int c0 = 0; c0 < total; c0 += 32) {
            // columns past the list repeat its first row; their results are dropped
            const bool two = total - c0 > 16;
            const uint16_t* xp[2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                xp[i] = a.x + (int64_t)(w0 + list[c0 + 16 * i + m < total ? c0 + 16 * i + m : c0]) * a.ldx;
            f4 acc[RT][2];
#pragma unroll
            for (int t = 0; t < RT; ++t) acc[t][0] = acc[t][1] = f4{0.f, 0.f, 0.f, 0.f};
            int s = lo;
            for (; s + UNR <= hi_full; s += UNR) {
                uint4 av[UNR][RT], xv[UNR][2];
#pragma unroll
                for (int u = 0; u < UNR; ++u) {
#pragma unroll
                    for (int t = 0; t < RT; ++t) av[u][t] = gload_u4(reinterpret_cast<const uint4*>(ap[t] + (s + u) * 32 + 8 * c));
                    xv[u][0] = gload_u4(reinterpret_cast<const uint4*>(xp[0] + (s + u) * 32 + 8 * c));
                    if (two) xv[u][1] = gload_u4(reinterpret_cast<const uint4*>(xp[1] + (s + u) * 32 + 8 * c));
                }
#pragma unroll
                for (int u = 0; u < UNR; ++u) {
#pragma unroll
                    for (int t = 0; t < RT; ++t)
                        acc[t][0] = __builtin_amdgcn_mfma_f32_16x16x32_f16(as_h8(av[u][t]), as_h8(xv[u][0]), acc[t][0], 0, 0, 0);
                    if (two) {
#pragma unroll
                        for (int t = 0; t < RT; ++t)
                            acc[t][1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(as_h8(av[u][t]), as_h8(xv[u][1]), acc[t][1], 0, 0, 0);
                    }
                }
            }
            for (; s < hi; ++s) {                      // what is left, the row's last piece among it
                const int k = s * 32 + 8 * c;
                const h8 x0 = as_h8(load8_until(xp[0], k, a.K)), x1 = as_h8(load8_until(xp[1], k, a.K));
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    const h8 av = as_h8(load8_until(ap[t], k, a.K));
                    acc[t][0] = __builtin_amdgcn_mfma_f32_16x16x32_f16(av, x0, acc[t][0], 0, 0, 0);
                    acc[t][1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(av, x1, acc[t][1], 0, 0, 0);
                }
            }
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                red[wave][2 * t][lane] = acc[t][0];
                red[wave][2 * t + 1][lane] = acc[t][1];
            }
            __syncthreads();
            for (int i = tid; i < RT * 2 * 64; i += 64 * W) {
                const int l = i & 63, t = i >> 7, col = c0 + 16 * (i >> 6 & 1) + (l & 15), j = j0 + 16 * t + 4 * (l >> 4);
                if (col < total && j < a.R) {
                    f4 v = red[0][i >> 6][l];
#pragma unroll
                    for (int w = 1; w < W; ++w) v += red[w][i >> 6][l];
                    *(__attribute__((address_space(1))) f4*)(a.h + (((int64_t)blockIdx.z * a.b + w0 + list[col]) * a.nseg + seg) * a.R + j) = v;
                }
            }
            __syncthreads();
        }
    }
}

// The outer products: 16 MU rows x 64 J outputs of one segment per workgroup
// of four waves, J output tiles a wave; ID adapters at a time, so that a decode
// batch of many adapters has the loads of several in flight.
template <int MU, int J, int ID>
__global__ __launch_bounds__(256) void lora_up_kernel(LoraArgs a) {
    constexpr int TM = 16 * MU, TPR = 256 / TM;        // rows, threads per row
    extern __shared__ __align__(16) uint32_t hp[];     // [TM][Rp + 4]: hi | lo << 16
    __shared__ int sid[TM], sexp[TM];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int m = lane & 15, c = lane >> 4;
    const int Rp = (a.R + 15) & ~15, ldh = Rp + 4;
    int seg = 0;
#pragma unroll
    for (int i = 1; i < WOQ_MAX_SEGMENTS; ++i)
        if (i < a.nseg && (int)blockIdx.x >= a.tile0[i]) seg = i;
    const int seg_lo = seg ? a.seg_end[seg - 1] : 0, seg_hi = a.seg_end[seg];
    const int n0 = seg_lo + ((int)blockIdx.x - a.tile0[seg]) * 64 * J;
    const int r0 = blockIdx.y * TM, rows = min(a.b - r0, TM);
    // a lane's 4 J outputs of a row are adjacent
    const int nw = n0 + wave * 16 * J, nl = nw + c * 4 * J;
    const bool whole = a.vec && (n0 & 7) == 0 && nl + 4 * J <= seg_hi;

    // the base, on its way while h is made ready
    uint32_t base[MU][2 * J];
#pragma unroll
    for (int i = 0; i < MU; ++i) {
        const int r = 16 * i + m;
#pragma unroll
        for (int e = 0; e < 2 * J; ++e) base[i][e] = 0;
        if (!a.base || r >= rows || nl >= seg_hi) continue;
        const uint16_t* br = a.base + (int64_t)(r0 + r) * a.ldbase + nl;
        if (whole) {
            if constexpr (J % 2 == 0) {
#pragma unroll
                for (int e = 0; e < J / 2; ++e) {
                    const uint4 v = gload_nt(reinterpret_cast<const uint4*>(br) + e);
                    base[i][4 * e] = v.x, base[i][4 * e + 1] = v.y, base[i][4 * e + 2] = v.z, base[i][4 * e + 3] = v.w;
                }
            } else {
#pragma unroll
                for (int e = 0; e < J; ++e) {
                    const uint2 v = gload_u2(reinterpret_cast<const uint2*>(br) + e);
                    base[i][2 * e] = v.x, base[i][2 * e + 1] = v.y;
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4 * J; ++e)
                if (nl + e < seg_hi) base[i][e >> 1] |= (uint32_t)*gptr(br + e) << (16 * (e & 1));
        }
    }

    // h: the ranges' sums added in order, scaled by a power of two, in two halves
    {
        const int r = tid / TPR, q = tid % TPR;
        const int id = r < rows ? *gptr(a.ids + r0 + r) : -1;
        const bool on = (unsigned)id < (unsigned)a.count;
        const int rank = on ? rank_of(a, id) : 0;
        const float* hr = a.h + ((int64_t)(r0 + r) * a.nseg + seg) * a.R;
        const int64_t range = (int64_t)a.b * a.nseg * a.R;
        uint32_t* row = hp + r * ldh;
        uint32_t big = 0;
        for (int j = 4 * q; j < Rp; j += 4 * TPR) {
            f4 v = {0.f, 0.f, 0.f, 0.f};
            if (j < rank) {
                for (int s = 0; s < a.splits; ++s) v += *(__attribute__((address_space(1))) const f4*)(hr + s * range + j);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (j + e >= rank) v[e] = 0.f;
                    big = max(big, __float_as_uint(v[e]) & 0x7FFFFFFFu);
                }
            }
            *(f4*)(row + j) = v;
        }
#pragma unroll
        for (int d = 1; d < TPR; d <<= 1) big = max(big, (uint32_t)__shfl_xor((int)big, d));
        // a row that is not finite is left as it is: every output of it is lost
        const int ex = big == 0 || big >= 0x7F800000u ? 0 : 14 - __builtin_amdgcn_frexp_expf(__uint_as_float(big));
        for (int j = 4 * q; j < Rp; j += 4 * TPR) {
            const f4 v = *(const f4*)(row + j);
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float t = ldexpf(v[e], ex);
                const uint16_t hi = f_to_h(t);
                const float rest = t - h_to_f(hi);
                w[e] = (uint32_t)hi | (uint32_t)((hi & 0x7C00u) == 0x7C00u ? 0 : f_to_h(rest)) << 16;
            }
            *(u32x4*)(row + j) = u32x4{w[0], w[1], w[2], w[3]};
        }
        if (q == 0) {
            sid[r] = on ? id : -1;
            sexp[r] = -ex;
        }
    }
    __syncthreads();

    const int mine = lane < TM ? sid[lane] : -1;
    u64 left = __ballot(mine >= 0);
    const uint32_t sel = c < 2 ? 0x05040100u : 0x07060302u;   // the hi or the lo halves of two values
    auto put = [&](int i, const f4 (&d)[J], bool plain, float s, int ex) {
        const int r = 16 * i + m;
        uint16_t* yr = a.y + (int64_t)(r0 + r) * a.ldy + nl;
        uint32_t o[2 * J];
#pragma unroll
        for (int e = 0; e < 2 * J; ++e) {
            const h2 bv = as_h2(base[i][e]);
            const float v0 = fmaf(ldexpf(d[e >> 1][2 * (e & 1)], ex), s, (float)bv[0]);
            const float v1 = fmaf(ldexpf(d[e >> 1][2 * (e & 1) + 1], ex), s, (float)bv[1]);
            o[e] = plain ? base[i][e] : (uint32_t)f_to_h(v0) | (uint32_t)f_to_h(v1) << 16;
        }
        if (whole) {
            if constexpr (J % 2 == 0) {
#pragma unroll
                for (int e = 0; e < J / 2; ++e)
                    gstore_u4(reinterpret_cast<uint4*>(yr) + e, make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]));
            } else {
#pragma unroll
                for (int e = 0; e < J; ++e) *(__attribute__((address_space(1))) u32x2*)(yr + 4 * e) = u32x2{o[2 * e], o[2 * e + 1]};
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4 * J; ++e)
                if (nl + e < seg_hi) *gptr(yr + e) = (uint16_t)(o[e >> 1] >> (16 * (e & 1)));
        }
    };
    while (left) {
        int id[ID], rank[ID], most = 0;
        u64 of[ID];
#pragma unroll
        for (int k = 0; k < ID; ++k) {
            // past the last adapter the first is repeated, for no rows
            id[k] = k && !left ? id[0] : __builtin_amdgcn_readlane(mine, __ffsll(left) - 1);
            of[k] = k && !left ? 0 : __ballot(mine == id[k]);
            left &= ~of[k];
            rank[k] = rank_of(a, id[k]);
            most = max(most, rank[k]);
        }
        f4 acc[ID][MU][J];
#pragma unroll
        for (int k = 0; k < ID; ++k)
#pragma unroll
            for (int i = 0; i < MU; ++i)
#pragma unroll
                for (int j = 0; j < J; ++j) acc[k][i][j] = f4{0.f, 0.f, 0.f, 0.f};
        for (int t = 0; t < most; t += 16) {
            uint4 bv[ID][J];
#pragma unroll
            for (int k = 0; k < ID; ++k)
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const int n = min(nw + (m >> 2) * 4 * J + 4 * j + (m & 3), seg_hi - 1), f = t + 8 * (c & 1);
                    const uint16_t* br = a.B + ((int64_t)id[k] * a.N + n) * a.R;
                    bv[k][j] = f < rank[k] ? load8_until(br, f, rank[k]) : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
            for (int i = 0; i < MU; ++i) {
                const uint32_t* row = hp + (16 * i + m) * ldh + t + 8 * (c & 1);
                const u32x4 p0 = *(const u32x4*)row, p1 = *(const u32x4*)(row + 4);
                const h8 hv = as_h8(make_uint4(__builtin_amdgcn_perm(p0[1], p0[0], sel), __builtin_amdgcn_perm(p0[3], p0[2], sel),
                                               __builtin_amdgcn_perm(p1[1], p1[0], sel), __builtin_amdgcn_perm(p1[3], p1[2], sel)));
#pragma unroll
                for (int k = 0; k < ID; ++k)
#pragma unroll
                    for (int j = 0; j < J; ++j)
                        acc[k][i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(as_h8(bv[k][j]), hv, acc[k][i][j], 0, 0, 0);
            }
        }
        if (nl < seg_hi) {
#pragma unroll
            for (int k = 0; k < ID; ++k) {
                const float s = *gptr(a.scale + id[k]);
#pragma unroll
                for (int i = 0; i < MU; ++i)
                    if (of[k] >> (16 * i + m) & 1) put(i, acc[k][i], false, s, sexp[16 * i + m]);
            }
        }
    }
    // rows without an adapter
    if (nl < seg_hi && (a.base != a.y || a.ldbase != a.ldy)) {
        const f4 none[J] = {};
#pragma unroll
        for (int i = 0; i < MU; ++i)
            if (16 * i + m < rows && sid[16 * i + m] < 0) put(i, none, true, 0.f, 0);
    }
}

// Rows up to which a workgroup per row looks for its adapter's other rows.
constexpr int LEADER_ROWS = 256;
// Partial sums of a row: at most so many K ranges, in each of the two forms.
constexpr int LEADER_SPLITS = 16, WINDOW_SPLITS = 4;

int rank_tiles(int b, int R) { return b <= LEADER_ROWS ? 1 : R <= 16 ? 1 : R <= 32 ? 2 : 4; }

int k_ranges(int b, int K, int R, int nseg) {
    const bool leader = b <= LEADER_ROWS;
    const int rt = rank_tiles(b, R), waves = leader ? 4 : 8;
    const int64_t units = woq::ceil_div(b, leader ? 1 : 32) * nseg * woq::ceil_div(R, 16 * rt);
    const int64_t want = woq::ceil_div(1024, units), most = std::max<int64_t>(1, K / (waves * 64));
    return (int)std::min<int64_t>(std::min(want, most), leader ? LEADER_SPLITS : WINDOW_SPLITS);
}

template <int W, int RT, bool LEADER>
hipError_t launch_down(const LoraArgs& a, hipStream_t s) {
    LoraArgs args = a;
    void* argv[] = {&args};
    const int groups = (int)woq::ceil_div(a.R, 16 * RT);
    return hipLaunchKernel(reinterpret_cast<const void*>(&lora_down_kernel<W, RT, LEADER>),
                           dim3((unsigned)(LEADER ? a.b : woq::ceil_div(a.b, 32)), (unsigned)(a.nseg * groups), (unsigned)a.splits),
                           dim3(64 * W), argv, 0, s);
}

template <int MU, int J, int ID>
hipError_t launch_up(LoraArgs a, hipStream_t s) {
    a.tile0[0] = 0;
    for (int i = 0; i < a.nseg; ++i)
        a.tile0[i + 1] = a.tile0[i] + (int)woq::ceil_div(a.seg_end[i] - (i ? a.seg_end[i - 1] : 0), 64 * J);
    void* argv[] = {&a};
    const size_t lds = (size_t)16 * MU * (woq::round_up(a.R, 16) + 4) * 4;
    if (lds > 60 * 1024) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&lora_up_kernel<MU, J, ID>),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess) return e;
    }
    return hipLaunchKernel(reinterpret_cast<const void*>(&lora_up_kernel<MU, J, ID>),
                           dim3((unsigned)a.tile0[a.nseg], (unsigned)woq::ceil_div(a.b, 16 * MU)), dim3(256), argv, lds, s);
}

int check_lora_w(const woq_lora_w* w) {
    if (!w || w->N < 0 || w->K < 1 || w->R < 1 || w->count < 0 || w->lda < w->K) return WOQ_EINVAL;
    if (w->nseg < 1 || w->nseg > WOQ_MAX_SEGMENTS || w->seg_end[w->nseg - 1] != w->N) return WOQ_EINVAL;
    for (int i = 0; i < w->nseg; ++i)
        if (w->seg_end[i] < (i ? w->seg_end[i - 1] : 0)) return WOQ_EINVAL;
    return WOQ_OK;
}

}  // namespace

extern "C" {

int64_t woq_lora_workspace(const woq_lora_w* w, int64_t b) {
    if (check_lora_w(w) != WOQ_OK || b < 0) return WOQ_EINVAL;
    if ((w->R & 7) || w->R > WOQ_LORA_MAX_R || b > WOQ_LORA_MAX_ROWS) return WOQ_EUNSUPPORTED;
    // no less for more rows, so that one workspace serves every smaller batch
    const int64_t rows = std::min<int64_t>(LEADER_SPLITS * b, std::max<int64_t>(LEADER_SPLITS * LEADER_ROWS, WINDOW_SPLITS * b));
    return std::max<int64_t>(16, rows * w->nseg * w->R * 4);
}

int woq_lora_add(const woq_lora_w* w, const uint16_t* x, int64_t ldx, const int32_t* ids, int64_t b,
                 const uint16_t* base, int64_t ldbase, uint16_t* y, int64_t ldy, void* workspace,
                 int64_t workspace_bytes, void* stream) {
    const int rc = check_lora_w(w);
    if (rc != WOQ_OK) return rc;
    if (b < 0 || ldx < w->K || ldy < w->N || (base && ldbase < w->N)) return WOQ_EINVAL;
    if (b == 0 || w->N == 0) return WOQ_OK;
    if (!x || !ids || !y || !workspace || (w->count > 0 && (!w->A || !w->B || !w->scale))) return WOQ_EINVAL;
    if (!woq::aligned16(x) || (ldx & 7) || ((uintptr_t)ids & 3u) || ((uintptr_t)y & 1u) || ((uintptr_t)base & 1u) ||
        !woq::aligned16(workspace) || !woq::aligned16(w->A) || !woq::aligned16(w->B) || (w->lda & 7) ||
        ((uintptr_t)w->scale & 3u) || ((uintptr_t)w->rank & 3u))
        return WOQ_EALIGN;
    if ((w->R & 7) || w->R > WOQ_LORA_MAX_R || w->N > (int64_t)INT32_MAX - 512 || w->K > (int64_t)INT32_MAX - 512 ||
        b > WOQ_LORA_MAX_ROWS)
        return WOQ_EUNSUPPORTED;
    if (workspace_bytes < woq_lora_workspace(w, b)) return WOQ_EINVAL;
    LoraArgs a;
    a.A = w->A;
    a.B = w->B;
    a.scale = w->scale;
    a.rank = w->rank;
    a.x = x;
    a.ids = ids;
    a.base = base;
    a.y = y;
    a.h = static_cast<float*>(workspace);
    a.ldx = ldx;
    a.ldbase = ldbase;
    a.ldy = ldy;
    a.lda = w->lda;
    a.b = (int)b;
    a.N = (int)w->N;
    a.K = (int)w->K;
    a.R = w->R;
    a.count = w->count;
    a.nseg = w->nseg;
    a.splits = k_ranges(a.b, a.K, a.R, a.nseg);
    a.vec = woq::aligned16(y) && (ldy & 7) == 0 && (!base || (woq::aligned16(base) && (ldbase & 7) == 0));
    for (int i = 0; i < WOQ_MAX_SEGMENTS; ++i) a.seg_end[i] = i < w->nseg ? (int)w->seg_end[i] : (int)w->N;
    hipStream_t s = (hipStream_t)stream;
    hipError_t e;
    if (b <= LEADER_ROWS) e = launch_down<4, 1, true>(a, s);
    else if (rank_tiles(a.b, a.R) == 1) e = launch_down<8, 1, false>(a, s);
    else if (rank_tiles(a.b, a.R) == 2) e = launch_down<8, 2, false>(a, s);
    else e = launch_down<8, 4, false>(a, s);
    if (e == hipSuccess) e = b <= 64 ? launch_up<1, 1, 8>(a, s) : launch_up<4, 4, 1>(a, s);
    if (e != hipSuccess) {
        woq::set_hip_error((int)e);
        return WOQ_EHIP;
    }
    return WOQ_OK;
}

}  // extern "C"
