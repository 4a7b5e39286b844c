// The paged cache of keys and values: new tokens rotated, quantised and written
// into their slots, and tokens read back as fp16 rows.
//
//   rotation  (a, b) -> (a cos - b sin, b cos + a sin) for each pair of a head,
//   INT8      scale = max|v| / 127, byte = rne(v / scale) + 128 per token and head.
//
// Bound by memory at many tokens (2047 rows of 16 + 2 x 8 heads of 256 in 15.5 us, 3.9
// TB/s; 16381 tokens of 8 heads of 128 read back in 22-25 us, 4.1-4.6 TB/s) and by one
// launch and two dependent round trips (slot and position with the row, then the
// angles) at few (one row of 64 + 2 x 8 heads of 128 3.3 us).  A head is held by 4, 8 or
// 16 lanes, 16 values each, so a wave takes several heads, its maximum is a reduction
// of two to four steps inside the lanes that hold it, and no value passes through LDS.
// Four heads to a group of lanes, the angles read once for them, were no faster (17.1
// us where this then took 17) and slower for few rows (4.9).
#include <hip/hip_runtime.h>

#include "woq_gemv.h"
#include "woq_internal.h"

namespace {

using namespace woqk;

struct WriteArgs {
    uint8_t* kc;              // cache, codes or fp16
    uint8_t* vc;
    float* ks;                // null for fp16
    float* vs;
    const uint16_t* k;
    const uint16_t* v;
    const uint16_t* q;        // null: no queries
    uint16_t* q_out;
    const int32_t* slots;
    const float* rope;        // null: no rotation
    const int32_t* pos;
    int64_t ldk, ldv, ldq, ldqo, n_slots, n_pos;
    uint32_t items, per_row;  // heads over all rows, heads of a row (k, v, then q)
    int heads, page, dim, rot, interleaved;
};

__device__ __forceinline__ void load8h(const uint16_t* p, float (&v)[8]) {
    const uint4 w = gload_u4(reinterpret_cast<const uint4*>(p));
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[2 * j] = (float)as_h2(u[j])[0];
        v[2 * j + 1] = (float)as_h2(u[j])[1];
    }
}

__device__ __forceinline__ void store8h(uint16_t* p, const float (&v)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) u[j] = (uint32_t)f_to_h(v[2 * j]) | (uint32_t)f_to_h(v[2 * j + 1]) << 16;
    gstore_u4(reinterpret_cast<uint4*>(p), make_uint4(u[0], u[1], u[2], u[3]));
}

__device__ __forceinline__ void load8f(const float* p, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint4 w = gload_u4(reinterpret_cast<const uint4*>(p) + i);
        v[4 * i] = __uint_as_float(w.x);
        v[4 * i + 1] = __uint_as_float(w.y);
        v[4 * i + 2] = __uint_as_float(w.z);
        v[4 * i + 3] = __uint_as_float(w.w);
    }
}

// The bytes of eight codes, rne(v / scale) + 128, by a reciprocal: 1.5 2^23 + 128
// added to v / scale leaves the byte in the sum's low bits.  v times the reciprocal is
// off by less than 127 2^-22; near is set where that could decide the rounding.
constexpr float MAGIC = 12583040.0f;
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float inv, bool& near) {
    uint32_t u[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float t = fmaf(v[j], inv, MAGIC);
        near |= !(fabsf(fmaf(v[j], inv, MAGIC - t)) <= 0.4999f);
        u[j] = __float_as_uint(t);
    }
    auto four = [&](int j) {
        return __builtin_amdgcn_perm(__builtin_amdgcn_perm(u[j + 3], u[j + 2], 0x0c0c0400u),
                                     __builtin_amdgcn_perm(u[j + 1], u[j], 0x0c0c0400u), 0x05040100u);
    };
    return make_uint2(four(0), four(4));
}
// The same by the division, bit for bit the host's.
__device__ __forceinline__ uint2 codes8_exact(const float (&v)[8], float scale) {
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float d = fminf(fmaxf(rintf(v[j] / scale), -127.0f), 127.0f);
        w[j >> 2] |= (uint32_t)((int)d + 128) << (8 * (j & 3));
    }
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void gstore_u2(void* p, uint2 v) {
    *(__attribute__((address_space(1))) u32x2*)p = u32x2{v.x, v.y};
}

// L lanes to a head (a power of two with 16 L >= dim).
template <int L>
__global__ __launch_bounds__(256) void cache_write_kernel(WriteArgs a) {
    const uint32_t item = blockIdx.x * (256 / L) + threadIdx.x / L;
    if (item >= a.items) return;               // whole groups of L lanes leave together
    const int l = threadIdx.x % L;
    const uint32_t r = item / a.per_row;
    const int h = (int)(item - r * a.per_row);
    const int kind = h < a.heads ? 0 : h < 2 * a.heads ? 1 : 2;     // k, v, q
    const bool active = 16 * l < a.dim;
    const bool turn = a.rope && kind != 1 && 16 * l < a.rot;
    // two chunks of eight values per lane: a rotated pair meets in one lane
    const bool apart = a.rope && kind != 1 && !a.interleaved && 16 * l < a.rot;
    const int o0 = apart ? 8 * l : 16 * l, o1 = apart ? a.rot / 2 + 8 * l : 16 * l + 8;

    // the row, its slot and its position are asked for together, then the angles
    const int64_t slot = kind != 2 ? *gptr(a.slots + r) : 0, p = turn ? *gptr(a.pos + r) : 0;
    float x0[8] = {}, x1[8] = {}, c[8], s[8];
    if (active) {
        const uint16_t* row = kind == 0   ? a.k + r * a.ldk + (int64_t)h * a.dim
                              : kind == 1 ? a.v + r * a.ldv + (int64_t)(h - a.heads) * a.dim
                                          : a.q + r * a.ldq + (int64_t)(h - 2 * a.heads) * a.dim;
        load8h(row + o0, x0);
        load8h(row + o1, x1);
    }
    if (slot < 0 || slot >= a.n_slots) return;
    if (turn) {
        if (p >= 0 && p < a.n_pos) {
            load8f(a.rope + p * a.rot + 8 * l, c);
            load8f(a.rope + p * a.rot + a.rot / 2 + 8 * l, s);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) c[j] = s[j] = __builtin_nanf("");
        }
        if (a.interleaved) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float e0 = x0[2 * j], f0 = x0[2 * j + 1], e1 = x1[2 * j], f1 = x1[2 * j + 1];
                x0[2 * j] = e0 * c[j] - f0 * s[j];
                x0[2 * j + 1] = f0 * c[j] + e0 * s[j];
                x1[2 * j] = e1 * c[j + 4] - f1 * s[j + 4];
                x1[2 * j + 1] = f1 * c[j + 4] + e1 * s[j + 4];
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float e = x0[j], f = x1[j];
                x0[j] = e * c[j] - f * s[j];
                x1[j] = f * c[j] + e * s[j];
            }
        }
    }
    if (kind == 2) {
        if (active) {
            uint16_t* out = a.q_out + r * a.ldqo + (int64_t)(h - 2 * a.heads) * a.dim;
            store8h(out + o0, x0);
            store8h(out + o1, x1);
        }
        return;
    }
    const int head = kind == 0 ? h : h - a.heads;
    const uint32_t page = (uint32_t)slot / (uint32_t)a.page;
    const int64_t at = ((int64_t)page * a.heads + head) * a.page + ((uint32_t)slot - page * (uint32_t)a.page);
    if (!a.ks) {
        if (active) {
            uint16_t* out = reinterpret_cast<uint16_t*>(kind == 0 ? a.kc : a.vc) + at * a.dim;
            store8h(out + o0, x0);
            store8h(out + o1, x1);
        }
        return;
    }
    uint32_t m = 0;           // max|v| as ordered bits: a NaN orders above every number
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        m = max(m, __float_as_uint(x0[j]) & 0x7FFFFFFFu);
        m = max(m, __float_as_uint(x1[j]) & 0x7FFFFFFFu);
    }
#pragma unroll
    for (int d = 1; d < L; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
    const float vmax = __uint_as_float(m);
    const bool bad = !(vmax < __builtin_huge_valf());
    const float scale = bad ? __builtin_nanf("") : vmax / 127.0f;
    const bool zero = bad || scale == 0.0f;
    if (active) {
        uint8_t* out = (kind == 0 ? a.kc : a.vc) + at * a.dim;
        uint2 w0 = make_uint2(0x80808080u, 0x80808080u), w1 = w0;
        if (!zero) {
            const float inv = 1.0f / scale;
            bool near = false;
            w0 = codes8(x0, inv, near);
            w1 = codes8(x1, inv, near);
            if (near) {       // also where the reciprocal overflows
                w0 = codes8_exact(x0, scale);
                w1 = codes8_exact(x1, scale);
            }
        }
        gstore_u2(out + o0, w0);
        gstore_u2(out + o1, w1);
    }
    if (l == 0) *gptr((kind == 0 ? a.ks : a.vs) + at) = scale;
}

struct ReadArgs {
    const uint8_t* c[2];      // keys, values
    const float* s[2];
    uint16_t* out[2];         // null: not asked for
    int64_t ld[2];
    const int32_t* slots;
    int64_t n_slots;
    uint32_t items, per_row;
    int heads, page, dim, first;
};

template <int L>
__global__ __launch_bounds__(256) void cache_read_kernel(ReadArgs a) {
    const uint32_t item = blockIdx.x * (256 / L) + threadIdx.x / L;
    const int l = threadIdx.x % L;
    if (item >= a.items || 16 * l >= a.dim) return;
    const uint32_t r = item / a.per_row;
    const int h = (int)(item - r * a.per_row);
    const int kind = a.first + (h >= a.heads), head = h >= a.heads ? h - a.heads : h;
    const int64_t slot = *gptr(a.slots + r);
    uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
    if (slot >= 0 && slot < a.n_slots) {
        const uint32_t page = (uint32_t)slot / (uint32_t)a.page;
        const int64_t at = ((int64_t)page * a.heads + head) * a.page + ((uint32_t)slot - page * (uint32_t)a.page);
        const uint8_t* c = kind ? a.c[1] : a.c[0];
        const float* sp = kind ? a.s[1] : a.s[0];
        if (sp) {
            const float scale = *gptr(sp + at);
            const uint4 w = gload_u4(reinterpret_cast<const uint4*>(c + at * a.dim + 16 * l));
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
            uint32_t o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t p = u[j >> 1] >> (16 * (j & 1));
                const float e = (float)((int)(p & 0xFFu) - 128) * scale, f = (float)((int)(p >> 8 & 0xFFu) - 128) * scale;
                o[j] = (uint32_t)f_to_h(e) | (uint32_t)f_to_h(f) << 16;
            }
            lo = make_uint4(o[0], o[1], o[2], o[3]);
            hi = make_uint4(o[4], o[5], o[6], o[7]);
        } else {
            const uint4* p = reinterpret_cast<const uint4*>(c + (at * a.dim + 16 * l) * 2);
            lo = gload_u4(p);
            hi = gload_u4(p + 1);
        }
    }
    uint4* out = reinterpret_cast<uint4*>((kind ? a.out[1] : a.out[0]) + r * (kind ? a.ld[1] : a.ld[0]) +
                                          (int64_t)head * a.dim + 16 * l);
    gstore_u4(out, lo);
    gstore_u4(out + 1, hi);
}

int lanes_of(int dim) { return dim <= 64 ? 4 : dim <= 128 ? 8 : 16; }

// A launch has fewer than 2^32 threads, whole workgroups of 256.
int64_t max_items(int dim) { return (int64_t)(UINT32_MAX / 256) * (256 / lanes_of(dim)); }

template <class K, class A>
int launch(K k4, K k8, K k16, int dim, uint32_t items, A& args, void* stream) {
    const int L = lanes_of(dim);
    const void* f = reinterpret_cast<const void*>(L == 4 ? k4 : L == 8 ? k8 : k16);
    void* argv[] = {&args};
    const uint32_t per = 256 / L;
    const hipError_t e = hipLaunchKernel(f, dim3(items / per + (items % per != 0)), dim3(256), argv, 0,
                                         (hipStream_t)stream);
    if (e != hipSuccess) {
        woq::set_hip_error((int)e);
        return WOQ_EHIP;
    }
    return WOQ_OK;
}

bool half_rows_ok(const void* p, int64_t ld) { return woq::aligned16(p) && (ld & 7) == 0; }

}  // namespace

namespace woq {

int cache_check(const woq_cache* c) {
    if (!c || (c->fmt != WOQ_CACHE_FP16 && c->fmt != WOQ_CACHE_INT8) || c->n_pages < 1 || c->heads < 1 ||
        c->page < 1 || c->dim < 1)
        return WOQ_EINVAL;
    if (!c->k || !c->v || ((c->fmt == WOQ_CACHE_INT8) != (c->k_scale != nullptr)) ||
        ((c->fmt == WOQ_CACHE_INT8) != (c->v_scale != nullptr)))
        return WOQ_EINVAL;
    if (!aligned16(c->k) || !aligned16(c->v) || !aligned16(c->k_scale) || !aligned16(c->v_scale))
        return WOQ_EALIGN;
    if ((c->dim & 15) || c->dim > WOQ_CACHE_MAX_DIM || (c->page & 15) || c->page > WOQ_CACHE_MAX_PAGE ||
        c->heads > WOQ_CACHE_MAX_HEADS || c->n_pages > INT32_MAX / c->page)
        return WOQ_EUNSUPPORTED;
    return WOQ_OK;
}

}  // namespace woq

namespace woq {

int cache_write_check(const woq_cache* c, const uint16_t* k, int64_t ldk, const uint16_t* v, int64_t ldv,
                      const int32_t* slots, int64_t b, const uint16_t* q, int64_t ldq, int32_t q_heads,
                      const uint16_t* q_out, int64_t ldq_out, const float* rope, int64_t n_pos, int32_t rot,
                      int32_t interleaved, const int32_t* pos) {
    const int rc = cache_check(c);
    if (rc == WOQ_EINVAL || b < 0) return WOQ_EINVAL;
    const int64_t width = (int64_t)c->heads * c->dim;
    if (ldk < width || ldv < width) return WOQ_EINVAL;
    if (q && (q_heads < 1 || !rope || !q_out || ldq < (int64_t)q_heads * c->dim ||
              ldq_out < (int64_t)q_heads * c->dim || (q == q_out && ldq != ldq_out)))
        return WOQ_EINVAL;
    if (rope && (n_pos < 1 || rot < 1 || rot > c->dim || (interleaved != 0 && interleaved != 1))) return WOQ_EINVAL;
    if (b > 0 && (!k || !v || !slots || (rope && !pos))) return WOQ_EINVAL;
    if (rc) return rc;
    if (b == 0) return WOQ_OK;
    if (!half_rows_ok(k, ldk) || !half_rows_ok(v, ldv) || ((uintptr_t)slots & 3u) ||
        (q && (!half_rows_ok(q, ldq) || !half_rows_ok(q_out, ldq_out))) ||
        (rope && (!aligned16(rope) || ((uintptr_t)pos & 3u))))
        return WOQ_EALIGN;
    const int64_t per_row = 2 * (int64_t)c->heads + (q ? q_heads : 0);
    if ((rope && (rot & 15)) || b > max_items(c->dim) / per_row) return WOQ_EUNSUPPORTED;
    return WOQ_OK;
}

}  // namespace woq

extern "C" int woq_cache_write(const woq_cache* c, const uint16_t* k, int64_t ldk, const uint16_t* v, int64_t ldv,
                               const int32_t* slots, int64_t b, const uint16_t* q, int64_t ldq, int32_t q_heads,
                               uint16_t* q_out, int64_t ldq_out, const float* rope, int64_t n_pos, int32_t rot,
                               int32_t interleaved, const int32_t* pos, void* stream) {
    const int rc = woq::cache_write_check(c, k, ldk, v, ldv, slots, b, q, ldq, q_heads, q_out, ldq_out, rope, n_pos,
                                          rot, interleaved, pos);
    if (rc || b == 0) return rc;
    const int64_t per_row = 2 * (int64_t)c->heads + (q ? q_heads : 0);
    WriteArgs a;
    a.kc = static_cast<uint8_t*>(c->k);
    a.vc = static_cast<uint8_t*>(c->v);
    a.ks = c->k_scale;
    a.vs = c->v_scale;
    a.k = k;
    a.v = v;
    a.q = q;
    a.q_out = q_out;
    a.slots = slots;
    a.rope = rope;
    a.pos = pos;
    a.ldk = ldk;
    a.ldv = ldv;
    a.ldq = ldq;
    a.ldqo = ldq_out;
    a.n_slots = c->n_pages * c->page;
    a.n_pos = n_pos;
    a.items = (uint32_t)(b * per_row);
    a.per_row = (uint32_t)per_row;
    a.heads = c->heads;
    a.page = c->page;
    a.dim = c->dim;
    a.rot = rot;
    a.interleaved = interleaved;
    return launch(&cache_write_kernel<4>, &cache_write_kernel<8>, &cache_write_kernel<16>, c->dim, a.items, a, stream);
}

extern "C" int woq_cache_read(const woq_cache* c, const int32_t* slots, int64_t n, uint16_t* k_out, int64_t ldk,
                              uint16_t* v_out, int64_t ldv, void* stream) {
    int rc = woq::cache_check(c);
    if (rc == WOQ_EINVAL || n < 0 || (!k_out && !v_out)) return WOQ_EINVAL;
    const int64_t width = (int64_t)c->heads * c->dim;
    if ((k_out && ldk < width) || (v_out && ldv < width) || (n > 0 && !slots)) return WOQ_EINVAL;
    if (rc) return rc;
    if (n == 0) return WOQ_OK;
    if ((k_out && !half_rows_ok(k_out, ldk)) || (v_out && !half_rows_ok(v_out, ldv)) || ((uintptr_t)slots & 3u))
        return WOQ_EALIGN;
    if (n > max_items(c->dim) / (2 * (int64_t)c->heads)) return WOQ_EUNSUPPORTED;
    ReadArgs a;
    a.c[0] = static_cast<const uint8_t*>(c->k);
    a.c[1] = static_cast<const uint8_t*>(c->v);
    a.s[0] = c->k_scale;
    a.s[1] = c->v_scale;
    a.out[0] = k_out;
    a.out[1] = v_out;
    a.ld[0] = ldk;
    a.ld[1] = ldv;
    a.slots = slots;
    a.n_slots = c->n_pages * c->page;
    a.per_row = (uint32_t)(k_out && v_out ? 2 * c->heads : c->heads);
    a.items = (uint32_t)n * a.per_row;
    a.heads = c->heads;
    a.page = c->page;
    a.dim = c->dim;
    a.first = k_out ? 0 : 1;
    return launch(&cache_read_kernel<4>, &cache_read_kernel<8>, &cache_read_kernel<16>, c->dim, a.items, a, stream);
}
