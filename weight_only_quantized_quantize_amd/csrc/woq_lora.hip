// Low-rank adapters of many requests beside a shared projection:
//
//   y[r, n] = fp16(base[r, n] + scale[a] sum_j B[a][n, j] h[r, seg(n) R + j]),
//   h[r, i] = sum_k A[a][i, k] x[r, k],   a = ids[r],
//
// with y = base on rows without an adapter.
#include <hip/hip_runtime.h>

#include "woq_gemv.h"
#include "woq_internal.h"

namespace {

using namespace woqk;

struct LoraArgs {
    const uint16_t* A;        // [count][nseg R][lda]
    const uint16_t* B;        // [count][N][R]
    const float* scale;       // [count]
    const int32_t* rank;      // [count], or null
    const uint16_t* x;
    const int32_t* ids;
    const uint16_t* base;     // null: zeros
    uint16_t* y;
    float* h;                 // [b][nseg R]
    int64_t ldx, ldbase, ldy, lda, b;
    int N, K, R, count, nseg;
    int seg_end[WOQ_MAX_SEGMENTS];
};

__device__ __forceinline__ int segment_of(const LoraArgs& a, int n) {
    int s = 0;
#pragma unroll
    for (int i = 1; i < WOQ_MAX_SEGMENTS; ++i)
        if (i < a.nseg && n >= a.seg_end[i - 1]) s = i;
    return s;
}

__device__ __forceinline__ int rank_of(const LoraArgs& a, int id) {
    return a.rank ? min(max(*gptr(a.rank + id), 0), a.R) : a.R;
}

// One wave per row and inner product.
__global__ __launch_bounds__(64) void lora_down_kernel(LoraArgs a) {
    const int64_t r = blockIdx.y;
    const int i = blockIdx.x, j = i % a.R;
    const int id = *gptr(a.ids + r);
    if ((unsigned)id >= (unsigned)a.count || j >= rank_of(a, id)) return;
    const uint16_t* Ar = a.A + ((int64_t)id * a.nseg * a.R + i) * a.lda;
    const uint16_t* xr = a.x + r * a.ldx;
    float s = 0.0f;
    for (int k = threadIdx.x; k < a.K; k += 64) s = fmaf(h_to_f(*gptr(Ar + k)), h_to_f(*gptr(xr + k)), s);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) s += __shfl_xor(s, d);
    if (threadIdx.x == 0) *gptr(a.h + r * a.nseg * a.R + i) = s;
}

// One thread per output.
__global__ __launch_bounds__(256) void lora_up_kernel(LoraArgs a) {
    const int64_t r = blockIdx.y;
    const int n = blockIdx.x * 256 + threadIdx.x;
    if (n >= a.N) return;
    const int id = *gptr(a.ids + r);
    float v = a.base ? h_to_f(*gptr(a.base + r * a.ldbase + n)) : 0.0f;
    if ((unsigned)id < (unsigned)a.count) {
        const uint16_t* Br = a.B + ((int64_t)id * a.N + n) * a.R;
        const float* h = a.h + (r * a.nseg + segment_of(a, n)) * a.R;
        const int rank = rank_of(a, id);
        float d = 0.0f;
        for (int j = 0; j < rank; ++j) d = fmaf(h_to_f(*gptr(Br + j)), *gptr(h + j), d);
        v = fmaf(d, *gptr(a.scale + id), v);
    }
    *gptr(a.y + r * a.ldy + n) = f_to_h(v);
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
    if ((w->R & 7) || w->R > WOQ_LORA_MAX_R || b > INT32_MAX) return WOQ_EUNSUPPORTED;
    return woq::round_up(b * w->nseg * w->R * 4, 16);
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
        b > 65535)
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
    a.b = b;
    a.N = (int)w->N;
    a.K = (int)w->K;
    a.R = w->R;
    a.count = w->count;
    a.nseg = w->nseg;
    for (int i = 0; i < WOQ_MAX_SEGMENTS; ++i) a.seg_end[i] = i < w->nseg ? (int)w->seg_end[i] : (int)w->N;
    hipStream_t s = (hipStream_t)stream;
    void* argv[] = {&a};
    hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(&lora_down_kernel),
                                   dim3((unsigned)(a.nseg * a.R), (unsigned)b), dim3(64), argv, 0, s);
    if (e == hipSuccess)
        e = hipLaunchKernel(reinterpret_cast<const void*>(&lora_up_kernel),
                            dim3((unsigned)woq::ceil_div(a.N, 256), (unsigned)b), dim3(256), argv, 0, s);
    if (e != hipSuccess) {
        woq::set_hip_error((int)e);
        return WOQ_EHIP;
    }
    return WOQ_OK;
}

}  // extern "C"
