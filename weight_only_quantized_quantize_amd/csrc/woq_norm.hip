// The residual's addition, the RMS norm and the 8-bit rows between two
// products: one pass over an activation row.
//
//   s = x + res,  r = 1 / sqrt(mean(s^2) + eps),  v = s (w + offset) r,
//   scale = max|v| / 127,  q = rne(v / scale)   (the INT8 scheme, per row).
//
// Bound by HBM at many rows (2 + 2 bytes in and up to 2 + 2 + 1 out per
// channel) and by launch and one memory round trip at few.  A row is held in
// registers by one workgroup, so every value is read once and written once;
// the sum of squares and the maximum share one reduction, because max|v| is
// max|s (w + offset)| times r (multiplying by r > 0 and rounding keep the
// order), so there is one barrier between the loads and the stores.  4096 rows of
// 8192 with a residual, all outputs: 58 us, 5.2 TB/s; one row 3.0 us.
#include <hip/hip_runtime.h>

#include <cmath>

#include "woq_gemv.h"
#include "woq_internal.h"

namespace {

using namespace woqk;

struct NormArgs {
    const uint16_t* x;
    const uint16_t* res;      // null: no residual
    const uint16_t* weight;   // null: no norm, v = s
    uint16_t* sum_out;        // null where not asked for, like y and q
    uint16_t* y;
    int8_t* q;
    float* q_scale;
    int64_t ldx, ldres, ldsum, ldy, ldq;
    float offset, eps, inv_k;
    int K;
};

// Channels 8c .. 8c + 7 of a row as fp32; channels past K read as zero and
// are not loaded.
__device__ __forceinline__ void load8(const uint16_t* row, int c, int K, float (&v)[8]) {
    if (8 * c + 8 <= K) {
        const uint4 p = gload_u4(reinterpret_cast<const uint4*>(row) + c);
        const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = (float)as_h2(w[j])[0];
            v[2 * j + 1] = (float)as_h2(w[j])[1];
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 8 * c + j < K ? h_to_f(*gptr(row + 8 * c + j)) : 0.0f;
    }
}

// fp16 of eight values, rounded to nearest even, to channels 8c .. 8c + 7.
__device__ __forceinline__ void store8(uint16_t* row, int c, int K, const float (&v)[8]) {
    if (8 * c + 8 <= K) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = (uint32_t)f_to_h(v[2 * j]) | (uint32_t)f_to_h(v[2 * j + 1]) << 16;
        gstore_u4(reinterpret_cast<uint4*>(row) + c, make_uint4(w[0], w[1], w[2], w[3]));
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (8 * c + j < K) *gptr(row + 8 * c + j) = f_to_h(v[j]);
    }
}

// One workgroup of T threads per row, P 8-channel chunks per thread.
template <int T, int P>
__global__ __launch_bounds__(T) void add_rmsnorm_kernel(NormArgs a) {
    constexpr int W = T / 64;
    __shared__ float red_s[W];
    __shared__ uint32_t red_m[W];
    const int64_t r = blockIdx.x;
    const int tid = threadIdx.x;
    const uint16_t* xr = a.x + r * a.ldx;
    const uint16_t* rr = a.res ? a.res + r * a.ldres : nullptr;

    // v holds s, then s (w + offset)
    float v[P][8];
    float ss = 0.0f;
    uint32_t m = 0;           // max|v| as ordered bits: a NaN orders above every number
#pragma unroll
    for (int p = 0; p < P; ++p) load8(xr, tid + p * T, a.K, v[p]);
    if (rr) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            float t[8];
            load8(rr, tid + p * T, a.K, t);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[p][j] += t[j];
        }
    }
    if (a.sum_out) {
#pragma unroll
        for (int p = 0; p < P; ++p) store8(a.sum_out + r * a.ldsum, tid + p * T, a.K, v[p]);
    }
    if (a.weight) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            float t[8];
            load8(a.weight, tid + p * T, a.K, t);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                ss = fmaf(v[p][j], v[p][j], ss);
                // past K both factors read as zero, but the offset is not
                v[p][j] *= t[j] + a.offset;
            }
        }
    }
    if (a.q) {
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[p][j]) & 0x7FFFFFFFu);
    }
    if (a.weight || a.q) {
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            ss += __shfl_xor(ss, d);
            m = max(m, (uint32_t)__shfl_xor((int)m, d));
        }
        if constexpr (W > 1) {
            if ((tid & 63) == 0) {
                red_s[tid >> 6] = ss;
                red_m[tid >> 6] = m;
            }
            __syncthreads();
            ss = red_s[0];
            m = red_m[0];
#pragma unroll
            for (int w = 1; w < W; ++w) {
                ss += red_s[w];
                m = max(m, red_m[w]);
            }
        }
    }
    float vmax = __uint_as_float(m);
    if (a.weight) {
        const float rstd = 1.0f / sqrtf(fmaf(ss, a.inv_k, a.eps));
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[p][j] *= rstd;
        vmax *= rstd;
    }
    if (a.y) {
#pragma unroll
        for (int p = 0; p < P; ++p) store8(a.y + r * a.ldy, tid + p * T, a.K, v[p]);
    }
    if (a.q) {
        // a row with a NaN or an infinity: scale NaN, codes 0; a scale that
        // underflows to 0: codes 0
        const bool bad = !(vmax < __builtin_huge_valf());
        const float scale = bad ? __builtin_nanf("") : vmax / 127.0f;
        const bool zero = bad || scale == 0.0f;
        // v / scale by a reciprocal is off by less than 127 * 2^-22; where that
        // could decide the rounding, the division decides (and where the
        // reciprocal overflows)
        const float inv = zero ? 0.0f : 1.0f / scale;
        const bool exact = !(inv < __builtin_huge_valf());
        int8_t* qr = a.q + r * a.ldq;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int c = tid + p * T;
            uint32_t w[2] = {0, 0};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float f = v[p][j] * inv;
                float d = rintf(f);
                if (exact || fabsf(f - d) > 0.4999f) d = rintf(v[p][j] / scale);
                d = zero ? 0.0f : fminf(fmaxf(d, -127.0f), 127.0f);
                w[j >> 2] |= ((uint32_t)(int)d & 0xFFu) << (8 * (j & 3));
            }
            // whole 16-byte pieces of the row are written, zeros past K
            if (8 * c < ((a.K + 15) & ~15))
                *(__attribute__((address_space(1))) u32x2*)(qr + 8 * c) = u32x2{w[0], w[1]};
        }
        if (tid == 0) *gptr(a.q_scale + r) = scale;
    }
}

template <int T, int P>
hipError_t launch(const NormArgs& a, int64_t b, hipStream_t s) {
    NormArgs args = a;
    void* argv[] = {&args};
    return hipLaunchKernel(reinterpret_cast<const void*>(&add_rmsnorm_kernel<T, P>), dim3((unsigned)b), dim3(T), argv,
                           0, s);
}

bool half_rows_ok(const void* p, int64_t ld) { return woq::aligned16(p) && (ld & 7) == 0; }

}  // namespace

extern "C" int woq_add_rmsnorm(const uint16_t* x, int64_t ldx, const uint16_t* res, int64_t ldres,
                               const uint16_t* weight, float offset, float eps, int64_t b, int64_t K,
                               uint16_t* sum_out, int64_t ldsum, uint16_t* y, int64_t ldy, int8_t* q, int64_t ldq,
                               float* q_scale, void* stream) {
    if (b < 0 || K < 1 || ldx < K || (res && ldres < K) || (sum_out && ldsum < K) || (y && ldy < K) ||
        (q && (ldq < K || !q_scale)))
        return WOQ_EINVAL;
    if (weight && !(eps > 0.0f && std::isfinite(eps) && std::isfinite(offset))) return WOQ_EINVAL;
    if (!sum_out && !y && !q) return WOQ_EINVAL;
    if (b == 0) return WOQ_OK;
    if (!x) return WOQ_EINVAL;
    if (!half_rows_ok(x, ldx) || (res && !half_rows_ok(res, ldres)) || (weight && !woq::aligned16(weight)) ||
        (sum_out && !half_rows_ok(sum_out, ldsum)) || (y && !half_rows_ok(y, ldy)) ||
        (q && (!woq::aligned16(q) || (ldq & 15) || ((uintptr_t)q_scale & 3u))))
        return WOQ_EALIGN;
    if (K > WOQ_NORM_MAX_K || b > WOQ_NORM_MAX_ROWS) return WOQ_EUNSUPPORTED;
    NormArgs a;
    a.x = x;
    a.res = res;
    a.weight = weight;
    a.sum_out = sum_out;
    a.y = y;
    a.q = q;
    a.q_scale = q_scale;
    a.ldx = ldx;
    a.ldres = ldres;
    a.ldsum = ldsum;
    a.ldy = ldy;
    a.ldq = ldq;
    a.offset = offset;
    a.eps = eps;
    a.inv_k = 1.0f / (float)K;
    a.K = (int)K;
    const int chunks = (int)woq::ceil_div(K, 16) * 2;    // whole 16-byte pieces of the codes
    hipStream_t s = (hipStream_t)stream;
    hipError_t e;
    // one chunk to a thread as long as a row fits a workgroup: 4096 rows of 8192,
    // all outputs, 57.9 us (5.2 TB/s, the rate of a large copy) with 1024 threads,
    // 61.2 and 65.3 with two and four chunks to a thread; 1021 rows of 3584 9.1 us
    // with 512, 11.7 with 1024; 2048 rows of 16384 51.5 us with 1024, 53.6 with 512
    if (chunks <= 64) e = launch<64, 1>(a, b, s);
    else if (chunks <= 128) e = launch<128, 1>(a, b, s);
    else if (chunks <= 256) e = launch<256, 1>(a, b, s);
    else if (chunks <= 512) e = launch<512, 1>(a, b, s);
    else if (chunks <= 1024) e = launch<1024, 1>(a, b, s);
    else if (chunks <= 2048) e = launch<1024, 2>(a, b, s);
    else if (chunks <= 4096) e = launch<1024, 4>(a, b, s);
    else e = launch<1024, 8>(a, b, s);
    if (e != hipSuccess) {
        woq::set_hip_error((int)e);
        return WOQ_EHIP;
    }
    return WOQ_OK;
}
