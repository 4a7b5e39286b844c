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

// One wave: 16 weight rows x 16 activation rows.
__global__ __launch_bounds__(64) void qgemm_int8_a8_tile(A8Args a) {
    const int lane = threadIdx.x, m = lane & 15, c = lane >> 4;
    const int n4 = (a.N + 3) & ~3, k16 = (a.K + 15) & ~15;
    const int n0 = blockIdx.x * 16;
    const int64_t r0 = (int64_t)blockIdx.y * 16;
    const int wrow = n0 + m < n4 ? n0 + m : 0;
    const int64_t xrow = r0 + m < a.b ? r0 + m : 0;
    const uint8_t* wp = a.codes + (int64_t)wrow * a.Kd + 16 * c;
    const int8_t* xp = a.q + xrow * a.ldq + 16 * c;
    i32x4 acc = {0, 0, 0, 0};
    for (int k = 0; k < a.Kd; k += 64) {
        uint4 w = gload_u4(reinterpret_cast<const uint4*>(wp + k));
        const bool in = k + 16 * c < k16;
        uint4 x = gload_u4(reinterpret_cast<const uint4*>(in ? xp + k : xp - 16 * c));
        if (!in) x = make_uint4(0, 0, 0, 0);
        const i32x4 wf = {(int)(w.x ^ 0x80808080u), (int)(w.y ^ 0x80808080u), (int)(w.z ^ 0x80808080u),
                          (int)(w.w ^ 0x80808080u)};
        const i32x4 xf = {(int)x.x, (int)x.y, (int)x.z, (int)x.w};
        acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf, xf, acc, 0, 0, 0);
    }
    // lane: activation row m, weight rows 4c .. 4c + 3
    if (r0 + m >= a.b) return;
    const float sx = *gptr(a.qs + r0 + m);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int n = n0 + 4 * c + i;
        if (n < a.N) *gptr(a.y + (r0 + m) * a.ldy + n) = f_to_h((float)acc[i] * (sx * row_scale(a, n)));
    }
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
    void* argv[] = {&a};
    const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(&qgemm_int8_a8_tile),
                                         dim3((unsigned)woq::ceil_div(a.N, 16), (unsigned)woq::ceil_div(b, 16)),
                                         dim3(64), argv, 0, (hipStream_t)stream);
    if (e != hipSuccess) {
        woq::set_hip_error((int)e);
        return WOQ_EHIP;
    }
    return WOQ_OK;
}
