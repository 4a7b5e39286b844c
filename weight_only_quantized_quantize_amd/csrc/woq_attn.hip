// Attention of one new token per row over a paged cache.
//
//   z[t] = scale (q . k[t]), or softcap tanh(scale (q . k[t]) / softcap),
//   y = sum_t e^(z[t] - m) v[t] / sum_t e^(z[t] - m),   m = max_t z[t].
//
// One wave per row and query head: a lane takes every 64th token for the scores,
// then every 64th value of the head for the sums.
#include <hip/hip_runtime.h>

#include <cmath>

#include "woq_gemv.h"
#include "woq_internal.h"

namespace {

using namespace woqk;

struct AttnArgs {
    const uint8_t* k;
    const uint8_t* v;
    const float* ks;          // null for fp16
    const float* vs;
    const uint16_t* q;
    const int32_t* pages;
    const int32_t* lens;
    uint16_t* y;
    int64_t ldq, ldpages, ldy, n_pages, capacity;
    float scale, softcap;
    int heads, group, page, dim, window;
};

__global__ __launch_bounds__(64) void attn_decode_kernel(AttnArgs a) {
    __shared__ float qs[WOQ_CACHE_MAX_DIM];
    const int lane = threadIdx.x, hq = blockIdx.x % (a.heads * a.group), r = blockIdx.x / (a.heads * a.group);
    const int h = hq / a.group;
    for (int d = lane; d < a.dim; d += 64) qs[d] = h_to_f(a.q[r * a.ldq + (int64_t)hq * a.dim + d]);
    __syncthreads();
    const int64_t len = min((int64_t)max(a.lens[r], 0), a.capacity);
    const int64_t first = a.window > 0 ? max((int64_t)0, len - a.window) : 0;
    float m = -INFINITY, total = 0.0f, acc[4] = {};
    for (int64_t t0 = first; t0 < len; t0 += 64) {
        const int64_t t = t0 + lane;
        float z = -INFINITY;
        int64_t at = -1;
        if (t < len) {
            const int64_t page = a.pages[r * a.ldpages + t / a.page];
            if (page >= 0 && page < a.n_pages) at = (page * a.heads + h) * a.page + t % a.page;
        }
        if (at >= 0) {
            float s = 0.0f;
            for (int d = 0; d < a.dim; ++d)
                s += qs[d] * (a.ks ? (float)((int)a.k[at * a.dim + d] - 128)
                                   : h_to_f(reinterpret_cast<const uint16_t*>(a.k)[at * a.dim + d]));
            z = s * a.scale * (a.ks ? a.ks[at] : 1.0f);
            if (a.softcap > 0.0f) z = a.softcap * tanhf(z / a.softcap);
        }
        // a NaN score stays: the row becomes NaN
        float top = z;
        for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
        const float next = fmaxf(m, top), base = next == -INFINITY ? 0.0f : next;
        const float keep = expf(m - base);
        const float p = at >= 0 ? expf(z - base) : 0.0f;
        total = total * keep + p;
        const float pv = p * (a.vs && at >= 0 ? a.vs[at] : 1.0f);
        for (int i = 0; i < 4; ++i) acc[i] *= keep;
        for (int j = 0; j < 64 && t0 + j < len; ++j) {
            const float pj = __shfl(pv, j);
            const int64_t aj = __shfl(at, j);
            if (aj < 0) continue;
            for (int i = 0; i < 4; ++i)
                if (lane + 64 * i < a.dim)
                    acc[i] += pj * (a.ks ? (float)((int)a.v[aj * a.dim + lane + 64 * i] - 128)
                                         : h_to_f(reinterpret_cast<const uint16_t*>(a.v)[aj * a.dim + lane + 64 * i]));
        }
        m = next;
    }
    for (int d = 1; d < 64; d <<= 1) total += __shfl_xor(total, d);
    for (int i = 0; i < 4; ++i)
        if (lane + 64 * i < a.dim)
            a.y[r * a.ldy + (int64_t)hq * a.dim + lane + 64 * i] = f_to_h(total == 0.0f ? 0.0f : acc[i] / total);
}

bool half_rows_ok(const void* p, int64_t ld) { return woq::aligned16(p) && (ld & 7) == 0; }

}  // namespace

namespace woq {

int attn_check(const woq_cache* c, const uint16_t* q, int64_t ldq, int32_t q_heads, const int32_t* pages,
               int64_t ldpages, int64_t max_pages, const int32_t* lens, int64_t b, float scale, float softcap,
               int32_t window, const uint16_t* y, int64_t ldy, const void* workspace, int64_t workspace_bytes) {
    const int rc = cache_check(c);
    if (rc == WOQ_EINVAL || b < 0 || q_heads < 1 || q_heads % c->heads || max_pages < 1 || ldpages < max_pages ||
        window < 0 || !std::isfinite(scale) || !std::isfinite(softcap) || softcap < 0.0f)
        return WOQ_EINVAL;
    const int64_t width = (int64_t)q_heads * c->dim;
    if (ldq < width || ldy < width || (q == y && q && ldq != ldy)) return WOQ_EINVAL;
    if (b > 0 && (!q || !pages || !lens || !y || !workspace)) return WOQ_EINVAL;
    if (rc) return rc;
    if (b == 0) return WOQ_OK;
    if (!half_rows_ok(q, ldq) || !half_rows_ok(y, ldy) || ((uintptr_t)pages & 3u) || ((uintptr_t)lens & 3u) ||
        !aligned16(workspace))
        return WOQ_EALIGN;
    if (q_heads > WOQ_ATTN_MAX_HEADS || b > WOQ_ATTN_MAX_ROWS || max_pages > INT32_MAX / c->page)
        return WOQ_EUNSUPPORTED;
    if (workspace_bytes < woq_attn_decode_workspace(c, q_heads, b)) return WOQ_EINVAL;
    return WOQ_OK;
}

}  // namespace woq

extern "C" int64_t woq_attn_decode_workspace(const woq_cache* c, int32_t q_heads, int64_t b) {
    const int rc = woq::cache_check(c);
    if (rc == WOQ_EINVAL || b < 0 || q_heads < 1 || q_heads % c->heads) return WOQ_EINVAL;
    if (rc) return rc;
    if (q_heads > WOQ_ATTN_MAX_HEADS || b > WOQ_ATTN_MAX_ROWS) return WOQ_EUNSUPPORTED;
    return 16;
}

extern "C" int woq_attn_decode(const woq_cache* c, const uint16_t* q, int64_t ldq, int32_t q_heads,
                               const int32_t* pages, int64_t ldpages, int64_t max_pages, const int32_t* lens,
                               int64_t b, float scale, float softcap, int32_t window, uint16_t* y, int64_t ldy,
                               void* workspace, int64_t workspace_bytes, void* stream) {
    const int rc = woq::attn_check(c, q, ldq, q_heads, pages, ldpages, max_pages, lens, b, scale, softcap, window, y,
                                   ldy, workspace, workspace_bytes);
    if (rc || b == 0) return rc;
    AttnArgs a;
    a.k = static_cast<const uint8_t*>(c->k);
    a.v = static_cast<const uint8_t*>(c->v);
    a.ks = c->k_scale;
    a.vs = c->v_scale;
    a.q = q;
    a.pages = pages;
    a.lens = lens;
    a.y = y;
    a.ldq = ldq;
    a.ldpages = ldpages;
    a.ldy = ldy;
    a.n_pages = c->n_pages;
    a.capacity = max_pages * c->page;
    a.scale = scale;
    a.softcap = softcap;
    a.heads = c->heads;
    a.group = q_heads / c->heads;
    a.page = c->page;
    a.dim = c->dim;
    a.window = window;
    void* argv[] = {&a};
    const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(&attn_decode_kernel),
                                         dim3((unsigned)(b * q_heads)), dim3(64), argv, 0, (hipStream_t)stream);
    if (e != hipSuccess) {
        woq::set_hip_error((int)e);
        return WOQ_EHIP;
    }
    return WOQ_OK;
}
