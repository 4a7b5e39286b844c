// Attention of one new token per row over a paged cache.
//
//   z[t] = scale (q . k[t]), or softcap tanh(scale (q . k[t]) / softcap),
//   y = sum_t e^(z[t] - m) v[t] / sum_t e^(z[t] - m),   m = max_t z[t].
//
// Bound by the cache's bytes at many tokens (64 rows of up to 8192, 64 queries over 8
// heads of 128, INT8: 99 us, 5.6 TB/s of 6.84 that a bare read reaches; 37 rows of a
// window of 4096 over fp16 heads of 256: 134 us, 5.8 TB/s; one row of 131072: 51 us,
// 5.5 TB/s) and by dependent round trips at few (lengths, pages, keys; one row of 509:
// 9.0 us).  One pass over the tokens, a wave 32 of them at a time with the running
// maximum and sum of the softmax, every query head of a key head at once: the scores of
// 16 tokens are one tile of the fp16 matrix cores, tokens as rows, and leave each lane
// with eight tokens of one head, the operand of the values' product as it stands.
// Nothing passes through LDS but the joining of waves.  The keys of the next 32 tokens
// are asked for behind the scores, their values behind the sums; with two workgroups a
// compute unit about 50 KB are in flight there (three workgroups were slower, 102 us
// for 97 with one fp16 number a weight).
//
// Roundings: scores, maxima and sums are fp32.  Weights meet the values as two fp16
// numbers, the nearest and what it leaves, 22 bits of a weight together (2^-40 of the
// largest at least): one more product of an operand that is there, for 0.7% of the time
// at 128 channels and 4% at 64 and 256, and results as near to the exact ones as fp32
// throughout would give, where one fp16 number alone was 1.4 times as far.
#include <hip/hip_runtime.h>

#include <cmath>
#include <type_traits>

#include "woq_gemv.h"
#include "woq_internal.h"

namespace {

using namespace woqk;

constexpr float NONE = -__builtin_huge_valf();
constexpr int TOP = 15;             // weights are at most 2^15, so that fp16 holds what is 2^-40 of that

// A cache's bytes u = code + 128 become the fp16 numbers code 2^-9, exactly: v_perm_b32
// puts two bytes, from anywhere in two words, into the low bytes of two fp16 numbers,
// the subnormals u 2^-24, and one packed fused multiply-add makes u 2^-9 - 128 2^-9 of
// them.  The bytes as they are would do for the matrix instructions too, with the 128
// taken off the sums (64 rows of up to 8192 97.7 us for 98.3, one row of 131072 51.0 for
// 51.2, one row of 509 8.7 for 9.0, but 64 rows of up to 8000 of heads of 256 199 for 180),
// but sums of u are three and more times as large as what is left of them, and the matrix
// cores keep fewer bits of a sum whose operands are subnormal: over 131072 tokens 8.6% of
// the results then were not the nearest fp16 number to the exact ones, 1.6% with
// subnormal codes, and 0.25% as it is, where fp32 throughout has 0.28%.
constexpr int STEP = 9;
__device__ __forceinline__ uint32_t codes2(uint32_t u) {
    const h2 up = {(f16)0x1p15f, (f16)0x1p15f}, offset = {(f16)-0.25f, (f16)-0.25f};
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(as_h2(u), up, offset));
}

// Two fp16 numbers with +-65504 in place of infinities and NaN, for the product with the
// second half of a weight: that half may be 0 or negative, and infinity times it would
// make NaN of what the first half's product has right.  37 rows of up to 6001 over a window
// of 4096 of fp16 heads of 256 133.7 us without, 134.9 with it.
__device__ __forceinline__ uint32_t finite2(uint32_t v) {
    typedef short s2 __attribute__((ext_vector_type(2)));
    typedef unsigned short us2 __attribute__((ext_vector_type(2)));
    const s2 most = {0x7BFF, 0x7BFF};
    const us2 least = {0xFBFF, 0xFBFF};
    const s2 w = __builtin_elementwise_min(__builtin_bit_cast(s2, v), most);
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_min(__builtin_bit_cast(us2, w), least));
}

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// tanh(t ln 2 / 2).  1 - 2 / (1 + 2^t) is off by 2^-24 of 1, which near 0 is not little of
// the result; up to 1.5 there is the odd polynomial that is nearest in relative terms
// (2^-25.6).  Both are within 2^-22.5 of the result with their roundings.
__device__ __forceinline__ float tanh_of(float t) {
    const float u = t * t;
    float p = fmaf(u, 0x1.458fecp-20f, -0x1.0a33f4p-15f);
    p = fmaf(u, p, 0x1.5d40cap-11f);
    p = fmaf(u, p, -0x1.c6af52p-7f);
    p = fmaf(u, p, 0x1.62e43p-2f);
    const float far = fmaf(-2.0f, __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(t)), 1.0f);
    return fabsf(t) <= 1.5f ? t * p : far;
}

// The largest of the four lanes m, m + 16, m + 32 and m + 48, in all of them.
__device__ __forceinline__ float max_over_rows(float v) {
    const uint32_t x = __float_as_uint(v);
    const auto p = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    const float a = fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
    const uint32_t y = __float_as_uint(a);
    const auto s = __builtin_amdgcn_permlane32_swap(y, y, false, false);
    return fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
}

struct AttnArgs {
    const uint8_t* k;
    const uint8_t* v;
    const float* ks;          // null for fp16
    const float* vs;
    const uint16_t* q;
    const int32_t* pages;
    const int32_t* lens;
    uint16_t* y;
    int4* cuts;               // workspace, of every workgroup: row, key head and tile, and how many parts the span
                              // has that it begins and others go on with (0: there is none)
    float* sums;              // [2 * workgroups][heads of a tile][dim]
    float* stats;             // [2 * workgroups][16][2]: the reference of the weights, their sum
    int64_t ldq, ldpages, ldy, n_pages, capacity;
    float factor, cap;        // of the scores in powers of two, see the launch
    int heads, group, page, dim, window, b, tiles, per_tile, groups;
};

// Sum over the lanes up to this one: in rows of 16, then from row to row.
__device__ __forceinline__ int wave_upto(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, true);
    return v;
}

// What row r sees: tokens first .. len - 1, in sixteens s0 .. s1 - 1 and units of
// two of them.
struct Span {
    int len, first, s0, s1, units;
};
__device__ __forceinline__ Span span_from(const AttnArgs& a, int len) {
    Span s;
    s.len = (int)min((int64_t)max(len, 0), a.capacity);
    s.first = a.window > 0 ? max(0, s.len - a.window) : 0;
    s.s0 = s.first >> 4;
    s.s1 = (int)(((uint32_t)s.len + 15) >> 4);
    s.units = (s.s1 - s.s0 + 1) >> 1;
    return s;
}
__device__ __forceinline__ Span span_of(const AttnArgs& a, int r) { return span_from(a, *gptr(a.lens + r)); }

// Positions of a workgroup of the split: an equal share, a unit to each of four waves at
// least.
constexpr int FLAT_WAVES = 4;
__device__ __forceinline__ int per_group(int positions, int groups) {
    return max(FLAT_WAVES, (int)(((uint32_t)positions + groups - 1) / (uint32_t)groups));
}

// The bytes that a lane loads of a sixteen of tokens: of the keys 16 bytes of one
// token's row at a time (token lane % 16), of the values its E = DP / 16 channels of
// four tokens (4 (lane / 16) ..), as the matrix instructions want them.
template <int DP, bool INT8>
struct Tile {
    static constexpr int E = DP / 16;
    static constexpr int NK = INT8 ? DP / 64 : DP / 32;        // 16-byte pieces of a key
    static constexpr int WV = INT8 ? E / 4 : E / 2;            // words of a token's values
    uint4 k[2][NK];
    uint32_t v[8][WV];
    f4 ks[2], vs[2];
};

template <int W>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&v)[W]) {
    if constexpr (W == 1) {
        v[0] = *gptr(reinterpret_cast<const uint32_t*>(p));
    } else if constexpr (W == 2) {
        const uint2 w = gload_u2(reinterpret_cast<const uint2*>(p));
        v[0] = w.x, v[1] = w.y;
    } else {
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
            const uint4 w = gload_u4(reinterpret_cast<const uint4*>(p) + i);
            v[4 * i] = w.x, v[4 * i + 1] = w.y, v[4 * i + 2] = w.z, v[4 * i + 3] = w.w;
        }
    }
}

// The parts that the waves of a workgroup leave of spans they do not hold whole: the
// first and the last of each, in order.
template <int N>
struct Parts {
    int row[N], head[N];                      // row -1: none; key head and tile
    int begins[N], ends[N];                   // whether the part holds the span's first and last unit
    int stop[N];                              // the position behind the span
    float ref[N][16], sum[N][16];
};

// Outputs of one span (or part of one): lane (g, m) has channels E (4 g + i) + e of
// head m in acc[e][i].
template <int E>
__device__ __forceinline__ void store_lane(uint16_t* out, const f4 (&acc)[E], float inv, int g, int dim) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int d = E * (4 * g + i);
        if (d >= dim) continue;
        uint32_t w[E / 2];
#pragma unroll
        for (int e = 0; e < E / 2; ++e)
            w[e] = (uint32_t)f_to_h(acc[2 * e][i] * inv) | (uint32_t)f_to_h(acc[2 * e + 1][i] * inv) << 16;
        if constexpr (E == 4) {
            *(__attribute__((address_space(1))) u32x2*)(out + d) = u32x2{w[0], w[1]};
        } else {
#pragma unroll
            for (int e = 0; e < E / 2; e += 4)
                gstore_u4(reinterpret_cast<uint4*>(out + d + 2 * e), make_uint4(w[e], w[e + 1], w[e + 2], w[e + 3]));
        }
    }
}

// All positions (row, key head, tile of 16 query heads, unit of 32 tokens) in order, an
// equal count of them to every workgroup and in it to every wave (FLAT); or a span, all
// units of a row, head and tile, to every workgroup.  What a wave holds of a span that
// it does not hold whole goes through LDS to its neighbours, and of a span that the
// workgroup does not hold whole through the workspace to the joining launch.
template <int DP, bool INT8, bool EXACT, int WAVES, bool FLAT>
__global__ __launch_bounds__(64 * WAVES, DP == 256 && !(INT8 && FLAT) ? 1 : 2) void attn_split_kernel(AttnArgs a) {
    using Mem = Tile<DP, INT8>;
    constexpr int T = 64 * WAVES, E = Mem::E, NK = Mem::NK, WV = Mem::WV, SIZE = INT8 ? 1 : 2;
    constexpr int PARTS = FLAT ? 2 * WAVES : WAVES;
    constexpr int ROW = DP + 4;               // floats of a head in LDS: 16 heads in different banks
    extern __shared__ __align__(16) float join[];              // [PARTS][per_tile][ROW]
    __shared__ Parts<PARTS> parts;
    __shared__ int scan[WAVES], found[WAVES][2];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int m = lane & 15, g = lane >> 4, HH = a.heads * a.tiles;

    int pos, end, base, per = 0;              // this wave's positions (fewer than 2^31); where its row's begin
    int r, hh = 0, ub = 0;                    // its row, key head and tile, and first unit there
    Span sp;
    // lengths of up to 64 rows stay in the wave's lanes
    const int lane_len = FLAT && a.b <= 64 ? *gptr(a.lens + min(lane, a.b - 1)) : 0;
    auto span = [&](int r) {
        return span_from(a, a.b <= 64 ? __builtin_amdgcn_readlane(lane_len, r)
                                      : __builtin_amdgcn_readfirstlane(*gptr(a.lens + r)));
    };
    if constexpr (FLAT) {
        const int groups = (int)gridDim.x;
        int first, last, share;
        auto divide = [&](int total) {        // false: nothing is left for this workgroup
            const int positions = total * HH;
            per = per_group(positions, groups);
            first = (int)min((int64_t)positions, (int64_t)blockIdx.x * per);
            last = min(positions - first, per) + first;
            share = (last - first + WAVES - 1) / WAVES;
            pos = min(last, first + wave * share);
            end = min(last, pos + share);
            if (first == last && tid == 0) a.cuts[blockIdx.x] = make_int4(0, 0, 0, 0);
            return first < last;
        };
        if (a.b <= 64) {                      // a row to a lane: nothing to exchange between waves
            const int n = lane < a.b ? span_from(a, lane_len).units : 0, upto = wave_upto(n);
            if (!divide(__builtin_amdgcn_readlane(upto, 63))) return;
            r = pos < end ? (int)__builtin_popcountll(__ballot(upto * HH <= pos)) : 0;
            base = r ? __builtin_amdgcn_readlane(upto, r - 1) * HH : 0;
        } else {
            int mine = 0, total = 0;
            const int each = (a.b + T - 1) / T, lo = min(a.b, tid * each), hi = min(a.b, lo + each);
            for (int i = lo; i < hi; ++i) mine += span_of(a, i).units;
            const int upto = wave_upto(mine);
            if (lane == 63) scan[wave] = upto;
            __syncthreads();
            int before = upto - mine;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) {
                if (w < wave) before += scan[w];
                total += scan[w];
            }
            if (!divide(total)) return;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) {
                const int p = first + w * share;
                if (p >= last || p < before * HH || p >= (before + mine) * HH) continue;
                int at = before, i = lo;
                for (; i < hi - 1; ++i) {
                    const int n = span_of(a, i).units;
                    if (p < (at + n) * HH) break;
                    at += n;
                }
                found[w][0] = i, found[w][1] = at;
            }
            __syncthreads();
            r = pos < end ? __builtin_amdgcn_readfirstlane(found[wave][0]) : 0;
            base = pos < end ? __builtin_amdgcn_readfirstlane(found[wave][1]) * HH : 0;
        }
        sp = span(r);
        if (pos < end) {
            const int rel = pos - base;
            hh = __builtin_amdgcn_readfirstlane((int)((uint32_t)rel / (uint32_t)sp.units));
            ub = rel - hh * sp.units;
        }
    } else {
        r = blockIdx.x / HH;
        hh = blockIdx.x - r * HH;
        base = pos = 0;
    }
    if (lane < PARTS / WAVES) parts.row[PARTS / WAVES * wave + lane] = -1;

    // where a lane's pieces of a sixteen stand in bytes; channels past dim are read
    // from the row's start and meet a query of zero
    const int dim = EXACT ? DP : a.dim;
    uint32_t ko[NK], vo[4];
    bool kin[NK];
#pragma unroll
    for (int i = 0; i < NK; ++i) {
        const int d = INT8 ? 64 * i + 16 * g : 32 * i + 8 * g;
        kin[i] = EXACT || d < dim;
        ko[i] = (uint32_t)(m * dim + (kin[i] ? d : 0)) * SIZE;
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) vo[t] = (uint32_t)((4 * g + t) * dim + (EXACT || E * m < dim ? E * m : 0)) * SIZE;
    const uint32_t so = 4 * g;                // scales
    const int spp = a.page >> 4;              // sixteens of a page
    // page of a lane's sixteen s and its place there; -1 where it is not
    int pg = -1, po = 0;
    auto fetch = [&](int s, int stop) {
        pg = -1;
        po = 0;
        if (s < stop) {
            const int p = (int)((uint32_t)s / (uint32_t)spp);
            pg = *gptr(a.pages + r * a.ldpages + p);
            po = s - p * spp;
            if (pg < 0 || pg >= a.n_pages) pg = -1;
        }
    };
    if constexpr (!FLAT) {
        // unit wave + WAVES i of the span: without a window its pages are asked for before the length is there
        const int s = 2 * (wave + WAVES * (lane >> 1)) + (lane & 1), stop = (int)(a.capacity >> 4);
        if (a.window > 0) {
            sp = span_of(a, r);
            fetch(sp.s0 + s, stop);
        } else {
            fetch(s, stop);
            sp = span_of(a, r);
        }
        if (sp.units == 0) {
            const int h = hh / a.tiles, tile = hh - h * a.tiles, n = min(16, a.group - 16 * tile) * a.dim;
            uint16_t* out = a.y + r * a.ldy + (int64_t)(h * a.group + 16 * tile) * a.dim;
            for (int d = tid; d < n; d += T) *gptr(out + d) = 0;
            return;
        }
        end = wave < sp.units;                // one turn of the loop, or none
    }

    int part = 0;
    for (; pos < end; ++hh, ub = 0) {
        const int ue = FLAT ? min(sp.units, ub + (end - pos)) : 0;
        const int n = FLAT ? ue - ub : (sp.units - wave + WAVES - 1) / WAVES;      // units of this wave here
        const int h = hh / a.tiles, tile = hh - h * a.tiles;
        const int heads = min(16, a.group - 16 * tile);          // query heads of this tile
        const int q0 = h * a.group + 16 * tile;

        h8 q[DP / 32];
        {
            const uint16_t* row = a.q + r * a.ldq + (int64_t)(q0 + m) * dim;
#pragma unroll
            for (int i = 0; i < DP / 32; ++i) {
                const int d = INT8 ? 64 * (i / 2) + 16 * g + 8 * (i & 1) : 32 * i + 8 * g;
                uint4 w = make_uint4(0, 0, 0, 0);
                if (m < heads && (EXACT || d < dim)) w = gload_u4(reinterpret_cast<const uint4*>(row + d));
                q[i] = __builtin_bit_cast(h8, w);
            }
        }
        f4 acc[E];
#pragma unroll
        for (int i = 0; i < E; ++i) acc[i] = f4{0, 0, 0, 0};
        float top = NONE, sum = 0.0f;
        int power = -90;                      // INT8: weights times their values' scales are below 2^power

        Mem t;
        bool there[2];
        int64_t at[2];                        // first token of the two sixteens
        int sb = sp.s0 + 2 * ub;              // FLAT: pg and po are of sixteens sb ..
        if constexpr (FLAT) fetch(sb + lane, sp.s1);
        auto place = [&](int i) {
            int l = 2 * i;                    // the lane that holds it
            if constexpr (FLAT) {
                l = sp.s0 + 2 * (ub + i) - sb;
                if (l >= 64) {
                    sb += 64;
                    fetch(sb + lane, sp.s1);
                    l = 0;
                }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int p = __builtin_amdgcn_readlane(pg, l + j), o = __builtin_amdgcn_readlane(po, l + j);
                there[j] = p >= 0;
                at[j] = (((int64_t)max(p, 0) * a.heads + h) * spp + o) * 16;
            }
        };
        auto load_k = [&] {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint8_t* p = a.k + at[j] * dim * SIZE;
#pragma unroll
                for (int i = 0; i < NK; ++i) t.k[j][i] = gload_nt(reinterpret_cast<const uint4*>(p + ko[i]));
                if constexpr (INT8)
                    t.ks[j] = *reinterpret_cast<__attribute__((address_space(1))) const f4*>(gptr(a.ks + at[j]) + so);
            }
        };
        auto load_v = [&] {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint8_t* p = a.v + at[j] * dim * SIZE;
#pragma unroll
                for (int i = 0; i < 4; ++i) load_words<WV>(p + vo[i], t.v[4 * j + i]);
                if constexpr (INT8)
                    t.vs[j] = *reinterpret_cast<__attribute__((address_space(1))) const f4*>(gptr(a.vs + at[j]) + so);
            }
        };

        place(0);
        load_k();
        load_v();
        for (int it = 0; it < n; ++it) {
            const int t0 = 16 * sp.s0 + 32 * (FLAT ? ub + it : wave + WAVES * it);
            const bool seen0 = there[0], seen1 = there[1];
            const bool whole = seen0 && seen1 && t0 >= sp.first && t0 + 32 <= sp.len;
            // scores: lane (g, m) gets tokens 4 g .. 4 g + 3 of both sixteens for head m
            float z[8];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                f4 s = {0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < NK; ++i) {
                    const uint32_t w[4] = {t.k[j][i].x, t.k[j][i].y, t.k[j][i].z, t.k[j][i].w};
                    if constexpr (INT8) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            uint4 c;
                            c.x = codes2(__builtin_amdgcn_perm(w[2 * e], w[2 * e], 0x0c010c00u));
                            c.y = codes2(__builtin_amdgcn_perm(w[2 * e], w[2 * e], 0x0c030c02u));
                            c.z = codes2(__builtin_amdgcn_perm(w[2 * e + 1], w[2 * e + 1], 0x0c010c00u));
                            c.w = codes2(__builtin_amdgcn_perm(w[2 * e + 1], w[2 * e + 1], 0x0c030c02u));
                            s = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, c), q[2 * i + e], s, 0, 0, 0);
                        }
                    } else {
                        uint4 c = t.k[j][i];
                        if (!EXACT && !kin[i]) c = make_uint4(0, 0, 0, 0);
                        s = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, c), q[i], s, 0, 0, 0);
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    z[4 * j + i] = s[i] * a.factor;
                    if constexpr (INT8) z[4 * j + i] *= t.ks[j][i];
                }
            }
            if (a.cap > 0.0f) {
                // factor holds 2 log2(e) / cap
#pragma unroll
                for (int i = 0; i < 8; ++i) z[i] = a.cap * tanh_of(z[i]);
            }
            float vs[8];                      // of the values' scales
            if constexpr (INT8) {
#pragma unroll
                for (int i = 0; i < 8; ++i) vs[i] = t.vs[i >> 2][i & 3];
            }
            if (!whole) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int tok = t0 + 16 * (i >> 2) + 4 * g + (i & 3);
                    if ((i < 4 ? seen0 : seen1) && tok >= sp.first && tok < sp.len) continue;
                    z[i] = NONE;
                    if constexpr (INT8) {
                        vs[i] = 0.0f;
                    } else {
#pragma unroll
                        for (int w = 0; w < WV; ++w) t.v[i][w] = 0;
                    }
                }
            }
            if (it + 1 < n) {
                place(it + 1);
                load_k();
            }
            float most = z[0];
#pragma unroll
            for (int i = 1; i < 8; ++i) most = fmaxf(most, z[i]);
            most = max_over_rows(most);
            if (__any(most > top)) {
                // INT8: what the weights lose the power loses too, in whole steps, so that it goes by the
                // largest product of weight and scale that still counts, not by a scale whose weight is gone
                // (64 rows of up to 8192 99.2 us for 99.6 by the largest scale alone, over one head of 64, 64 rows of
                // up to 16000, 46.4 for 45.2)
                const float next = fmaxf(top, most), fall = top - (next == NONE ? 0.0f : next);
                const int lower = INT8 ? max(-90, power + (int)fmaxf(fall, -300.0f)) : power;
                const float keep = __builtin_amdgcn_exp2f(fall + (float)(power - lower));
                top = next;
                power = lower;
                sum *= INT8 ? __builtin_amdgcn_exp2f(fall) : keep;
#pragma unroll
                for (int i = 0; i < E; ++i) acc[i] *= keep;
            }
            const float ref = (top == NONE ? 0.0f : top) - (INT8 ? 0 : TOP);
            float x[8];                       // weights, times their values' scales
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[i] = __builtin_amdgcn_exp2f(z[i] - ref);
                sum += x[i];
                if constexpr (INT8) x[i] *= vs[i];
            }
            if constexpr (INT8) {
                float large = x[0];
#pragma unroll
                for (int i = 1; i < 8; ++i) large = fmaxf(large, x[i]);
                if (__any(large >= pow2i(power))) {
                    large = max_over_rows(large);
                    const int next = max(power, min(110, (int)(__float_as_uint(large) >> 23) - 126));
                    const float keep = pow2i(max(-126, power - next));
                    power = next;
#pragma unroll
                    for (int i = 0; i < E; ++i) acc[i] *= keep;
                }
                const float raise = pow2i(TOP - power);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] *= raise;
            }
            h8 weights, rests;                // a weight's fp16 and what that leaves of it
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                weights[i] = (f16)x[i];
                rests[i] = (f16)(x[i] - (float)weights[i]);
            }
            // sums: rows of the product are the channels E (lane % 16) + i
#pragma unroll
            for (int c = 0; c < WV; ++c) {
                constexpr int N = INT8 ? 4 : 2;               // channels of a word
                constexpr uint32_t SEL[4] = {INT8 ? 0x0c040c00u : 0x05040100u, INT8 ? 0x0c050c01u : 0x07060302u, 0x0c060c02u,
                                             0x0c070c03u};
#pragma unroll
                for (int x = 0; x < N; ++x) {
                    uint4 v;
                    v.x = __builtin_amdgcn_perm(t.v[1][c], t.v[0][c], SEL[x]);
                    v.y = __builtin_amdgcn_perm(t.v[3][c], t.v[2][c], SEL[x]);
                    v.z = __builtin_amdgcn_perm(t.v[5][c], t.v[4][c], SEL[x]);
                    v.w = __builtin_amdgcn_perm(t.v[7][c], t.v[6][c], SEL[x]);
                    if constexpr (INT8) v = make_uint4(codes2(v.x), codes2(v.y), codes2(v.z), codes2(v.w));
                    f4& o = acc[N * c + x];
                    o = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, v), weights, o, 0, 0, 0);
                    if constexpr (!INT8) v = make_uint4(finite2(v.x), finite2(v.y), finite2(v.z), finite2(v.w));
                    o = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, v), rests, o, 0, 0, 0);
                }
            }
            if (it + 1 < n) load_v();
        }
        if constexpr (INT8) {
            const float unit = pow2i(power - TOP + STEP);
#pragma unroll
            for (int i = 0; i < E; ++i) acc[i] *= unit;
        }

        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        const bool begins = !FLAT || ub == 0, ends = !FLAT || ue == sp.units;
        if (FLAT ? begins && ends : sp.units == 1) {
            if (m < heads)
                store_lane<E>(a.y + r * a.ldy + (int64_t)(q0 + m) * dim, acc, sum == 0.0f ? 0.0f : 1.0f / sum, g, dim);
        } else {
            const int at = PARTS / WAVES * wave + part++;
            if (lane == 0) {
                parts.row[at] = r, parts.head[at] = hh;
                parts.begins[at] = begins, parts.ends[at] = ends;
                parts.stop[at] = base + (hh + 1) * sp.units;
            }
            if (g == 0) parts.ref[at][m] = top, parts.sum[at][m] = sum;
            if (m < heads) {
                float* o = join + (at * a.per_tile + m) * ROW + 4 * E * g;
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int e = 0; e < E; e += 4)
                        *reinterpret_cast<f4*>(o + E * i + e) = f4{acc[e][i], acc[e + 1][i], acc[e + 2][i], acc[e + 3][i]};
            }
        }
        pos += FLAT ? n : 1;
        if (FLAT && pos < end && hh == HH - 1) {
            base = pos;
            hh = -1;
            do {
                ++r;
                sp = span(r);
            } while (sp.units == 0);
        }
    }

    // the parts of one span after another, an output or a part of the workgroup's;
    // lane k looks at part k
    __syncthreads();
    int4 cut = make_int4(0, 0, 0, 0);         // the span that this workgroup begins and others end
    const int at = min(lane, PARTS - 1), row_k = parts.row[at], head_k = parts.head[at];
    uint64_t rest = __ballot(lane < PARTS && row_k >= 0);
    while (rest) {
        const int k0 = __builtin_ctzll(rest);
        const int row = __builtin_amdgcn_readlane(row_k, k0), hh = __builtin_amdgcn_readlane(head_k, k0);
        const uint64_t these = rest & __ballot(row_k == row && head_k == hh);
        rest &= ~these;
        const int h = hh / a.tiles, tile = hh - h * a.tiles, heads = min(16, a.group - 16 * tile);
        const bool begins = parts.begins[k0], ends = parts.ends[63 - __builtin_clzll(these)];
        const int64_t slot = 2 * (int64_t)blockIdx.x + begins;
        if (FLAT && begins && !ends) cut = make_int4(row, hh, parts.stop[k0], 0);
        for (int i = tid; i < heads * (DP / 4); i += T) {
            const int hq = i / (DP / 4), d = 4 * (i - hq * (DP / 4));
            if (!EXACT && d >= dim) continue;
            // every place is read, whether or not a part of this span is there: the reads then wait for each other
            // once, not one by one
            float ref = NONE, l = 0.0f, refs[PARTS], sums[PARTS];
            f4 v[PARTS], o = {0, 0, 0, 0};
#pragma unroll
            for (int k = 0; k < PARTS; ++k) {
                refs[k] = parts.ref[k][hq];
                sums[k] = parts.sum[k][hq];
                v[k] = *reinterpret_cast<const f4*>(join + (k * a.per_tile + hq) * ROW + d);
            }
#pragma unroll
            for (int k = 0; k < PARTS; ++k) ref = these >> k & 1 ? fmaxf(ref, refs[k]) : ref;
            const float zero = ref == NONE ? 0.0f : ref;
#pragma unroll
            for (int k = 0; k < PARTS; ++k) {
                const float keep = __builtin_amdgcn_exp2f(refs[k] - zero);
                const bool in = these >> k & 1;
                l += in ? sums[k] * keep : 0.0f;
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] += in ? v[k][e] * keep : 0.0f;
            }
            if (begins && ends) {
                const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                uint16_t* out = a.y + row * a.ldy + (int64_t)(h * a.group + 16 * tile + hq) * dim + d;
                *(__attribute__((address_space(1))) u32x2*)out =
                    u32x2{(uint32_t)f_to_h(o[0] * inv) | (uint32_t)f_to_h(o[1] * inv) << 16,
                          (uint32_t)f_to_h(o[2] * inv) | (uint32_t)f_to_h(o[3] * inv) << 16};
            } else {
                *(__attribute__((address_space(1))) f4*)(a.sums + (slot * a.per_tile + hq) * dim + d) = o;
                if (d == 0) {
                    *gptr(a.stats + (slot * 16 + hq) * 2) = ref;
                    *gptr(a.stats + (slot * 16 + hq) * 2 + 1) = l;
                }
            }
        }
    }
    if (FLAT && tid == 0) {
        if (cut.z) cut.z = (cut.z - 1) / per - (int)blockIdx.x + 1;       // workgroups up to the one that ends it
        a.cuts[blockIdx.x] = cut;
    }
}

// Joins the parts of the spans that were cut, in order, each under the power of two of
// its own, and writes the zeros of rows that see nothing.  Few spans (FEW) are long and
// have many parts: a workgroup for every span and head.  Otherwise a workgroup for every
// one of the split: it joins the span that that one began and others went on with, all
// heads at once as far as the threads go.  (A workgroup for every cut and head: 6 us
// where this takes 4, and 16 where it takes 6, most of it for those that find nothing.)
template <bool FEW>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a) {
    __shared__ __align__(16) float red[16][WOQ_CACHE_MAX_DIM];
    __shared__ float red_l[16], red_m[16];
    const int tid = threadIdx.x, lane = tid & 63, q_heads = a.heads * a.group, HH = a.heads * a.tiles;
    int wg = blockIdx.x, only = -1;           // whose cut this is, and the one head of it
    if constexpr (FEW) {
        const int span = blockIdx.x / a.per_tile, r = span / HH, hh = span - r * HH;
        const int tile = hh % a.tiles, h = hh / a.tiles;
        only = blockIdx.x - span * a.per_tile;
        if (only >= min(16, a.group - 16 * tile)) return;
        // as the split divides: at most 64 rows
        const int len = *gptr(a.lens + min(lane, a.b - 1));
        const int n = lane < a.b ? span_from(a, len).units : 0, upto = wave_upto(n);
        const int positions = __builtin_amdgcn_readlane(upto, 63) * HH, units = __builtin_amdgcn_readlane(n, r);
        if (units == 0) {
            for (int d = tid; d < a.dim; d += 256)
                *gptr(a.y + r * a.ldy + (int64_t)(h * a.group + 16 * tile + only) * a.dim + d) = 0;
            return;
        }
        const int per = per_group(positions, a.groups);
        const int p0 = (__builtin_amdgcn_readlane(upto, r) - units) * HH + hh * units;
        wg = p0 / per;
        if (wg == (p0 + units - 1) / per) return;
    } else {
        for (int r = wg; r < a.b; r += a.groups) {
            if (span_of(a, r).units) continue;
            for (int d = tid; d < q_heads * a.dim; d += 256) *gptr(a.y + r * a.ldy + d) = 0;
        }
    }
    const int4 cut = a.cuts[wg];
    if (cut.z == 0) return;
    const int h = cut.y / a.tiles, tile = cut.y - h * a.tiles, heads = min(16, a.group - 16 * tile);
    uint16_t* out = a.y + cut.x * a.ldy + (int64_t)(h * a.group + 16 * tile) * a.dim;
    // four channels to a thread
    const int lanes = a.dim <= 64 ? 16 : a.dim <= 128 ? 32 : 64, parts = 256 / lanes;
    const int part = tid / lanes, d = 4 * (tid - part * lanes);
    float ref, l;
    f4 o;
    // N parts of head hq in flight: i0, i0 + step, ...
    auto some = [&](auto count, int hq, int i0, int step) {
        constexpr int N = decltype(count)::value;
        u32x2 st[N];
        f4 v[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            // the first workgroup's part is its second, the others' their first
            const int i = min(i0 + j * step, cut.z - 1);
            const int64_t slot = 2 * ((int64_t)wg + i) + (i == 0);
            st[j] = *(g_u32x2*)(a.stats + (slot * 16 + hq) * 2);
            v[j] = *(__attribute__((address_space(1))) const f4*)(a.sums + (slot * a.per_tile + hq) * a.dim + min(d, a.dim - 4));
        }
        float next = ref;
#pragma unroll
        for (int j = 0; j < N; ++j) next = fmaxf(next, __uint_as_float(st[j][0]));
        const float zero = next == NONE ? 0.0f : next, old = __builtin_amdgcn_exp2f(ref - zero);
        l *= old;
        o *= old;
        ref = next;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if (i0 + j * step >= cut.z) continue;
            const float keep = __builtin_amdgcn_exp2f(__uint_as_float(st[j][0]) - zero);
            l = fmaf(__uint_as_float(st[j][1]), keep, l);
            o += v[j] * keep;
        }
    };
    if (!FEW && cut.z <= 16) {
        for (int hq = part; hq < heads; hq += parts) {
            ref = NONE, l = 0.0f, o = f4{0, 0, 0, 0};
            for (int i = 0; i < cut.z; i += 4) some(std::integral_constant<int, 4>{}, hq, i, 1);
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            if (d < a.dim)
                *(__attribute__((address_space(1))) u32x2*)(out + hq * a.dim + d) =
                    u32x2{(uint32_t)f_to_h(o[0] * inv) | (uint32_t)f_to_h(o[1] * inv) << 16,
                          (uint32_t)f_to_h(o[2] * inv) | (uint32_t)f_to_h(o[3] * inv) << 16};
        }
        return;
    }
    for (int hq = FEW ? only : 0; hq < (FEW ? only + 1 : heads); ++hq) {
        ref = NONE, l = 0.0f, o = f4{0, 0, 0, 0};
        for (int i = part; i < cut.z; i += 8 * parts) some(std::integral_constant<int, 8>{}, hq, i, parts);
        if (d < a.dim) *reinterpret_cast<f4*>(&red[part][d]) = o;
        if (d == 0) red_l[part] = l, red_m[part] = ref;
        __syncthreads();
        if (tid < a.dim) {
            float all = NONE, s = 0.0f, t = 0.0f;
            for (int i = 0; i < parts; ++i) all = fmaxf(all, red_m[i]);
            if (all == NONE) all = 0.0f;
            for (int i = 0; i < parts; ++i) {
                const float keep = __builtin_amdgcn_exp2f(red_m[i] - all);
                s = fmaf(red[i][tid], keep, s);
                t = fmaf(red_l[i], keep, t);
            }
            *gptr(out + hq * a.dim + tid) = f_to_h(t == 0.0f ? 0.0f : s / t);
        }
        if (!FEW) __syncthreads();
    }
}

// Workgroups of a split: as many as keep two on a compute unit.
int workgroups() { return 2 * woq::compute_units(); }

// Where the capacity is no more than this and the spans are no more than the
// workgroups, each takes one whole and there is nothing to join; twice as much where
// the spans are a quarter to a half of the workgroups.  64 queries over 8 heads of 128,
// rows of up to 1024: 4 rows 13.8 us against 8.3 + 4.2 and a launch between them, 32
// rows 14.8 against 15.4 + 3.9, 64 rows 26.6 against 22.3 + 4.8; of up to 2048: 16 rows
// 22.5 against 14.7 + 4.0, 32 rows 23.4 against 19.8 + 4.2, 64 rows 43 against 34.5 +
// 4.8; 256 rows of up to 512 (2048 spans) 57 against 43.5 + 4.8.  (From a graph, calls
// one behind the other: 4 rows 11.9 against 10.5, 32 rows 14.6 against 18.0.)
constexpr int64_t DIRECT = 1024;

struct Layout {
    int64_t sums, stats, bytes;
    int tiles, per_tile;
};
Layout layout(const woq_cache* c, int32_t q_heads) {
    Layout l;
    const int group = q_heads / c->heads, n = 2 * workgroups();
    l.tiles = (group + 15) / 16;
    l.per_tile = std::min(group, 16);
    l.sums = workgroups() * 16;
    l.stats = l.sums + (int64_t)n * l.per_tile * c->dim * 4;
    l.bytes = l.stats + (int64_t)n * 16 * 2 * 4;
    return l;
}

struct Kernel {
    const void* f;
    int waves, dim;           // dim: that of its registers
};
template <int DP, bool INT8>
Kernel split_kernel(int dim, bool flat) {
#define WOQ_ATTN(E, W, F) Kernel{reinterpret_cast<const void*>(&attn_split_kernel<DP, INT8, E, W, F>), W, DP}
    if (flat) return dim == DP ? WOQ_ATTN(true, FLAT_WAVES, true) : WOQ_ATTN(false, FLAT_WAVES, true);
    constexpr int W = DP == 256 ? 4 : 8;
    return dim == DP ? WOQ_ATTN(true, W, false) : WOQ_ATTN(false, W, false);
#undef WOQ_ATTN
}
template <bool INT8>
Kernel split_kernel(int dim, bool flat) {
    return dim <= 64    ? split_kernel<64, INT8>(dim, flat)
           : dim <= 128 ? split_kernel<128, INT8>(dim, flat)
                        : split_kernel<256, INT8>(dim, flat);
}

// Scores are in units of log2: factor s, or cap tanh(factor s ln 2 / 2), with s the
// product of a query and a key's numbers as they enter the matrix instructions.
constexpr double LOG2E = 1.4426950408889634;
float score_factor(const woq_cache* c, float scale, float softcap, int step = STEP) {
    return (float)(std::ldexp(1.0, c->fmt == WOQ_CACHE_INT8 ? step : 0) * LOG2E * scale * (softcap > 0.0f ? 2.0 / softcap : 1.0));
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
    // tokens and positions are 32 bits wide, with room for sums of two
    if (q_heads > WOQ_ATTN_MAX_HEADS || b > WOQ_ATTN_MAX_ROWS || max_pages > WOQ_ATTN_MAX_TOKENS / c->page)
        return WOQ_EUNSUPPORTED;
    const int64_t units = max_pages * c->page / 32 + 1, spans = (int64_t)c->heads * ceil_div(q_heads / c->heads, 16);
    if (units > WOQ_ATTN_MAX_TOKENS / (b * spans)) return WOQ_EUNSUPPORTED;
    if (softcap > WOQ_ATTN_MAX_SOFTCAP) return WOQ_EUNSUPPORTED;
    if (!std::isfinite(score_factor(c, scale, softcap, 24))) return WOQ_EUNSUPPORTED;      // with room above what is used
    if (workspace_bytes < woq_attn_decode_workspace(c, q_heads, b)) return WOQ_EINVAL;
    return WOQ_OK;
}

}  // namespace woq

extern "C" int64_t woq_attn_decode_workspace(const woq_cache* c, int32_t q_heads, int64_t b) {
    const int rc = woq::cache_check(c);
    if (rc == WOQ_EINVAL || b < 0 || q_heads < 1 || q_heads % c->heads) return WOQ_EINVAL;
    if (rc) return rc;
    if (q_heads > WOQ_ATTN_MAX_HEADS || b > WOQ_ATTN_MAX_ROWS) return WOQ_EUNSUPPORTED;
    return layout(c, q_heads).bytes;
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
    a.factor = score_factor(c, scale, softcap);
    a.cap = (float)(LOG2E * softcap);
    a.heads = c->heads;
    a.group = q_heads / c->heads;
    a.page = c->page;
    a.dim = c->dim;
    a.window = window;
    a.b = (int)b;
    const Layout l = layout(c, q_heads);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    a.cuts = reinterpret_cast<int4*>(ws);
    a.sums = reinterpret_cast<float*>(ws + l.sums);
    a.stats = reinterpret_cast<float*>(ws + l.stats);
    a.tiles = l.tiles;
    a.per_tile = l.per_tile;
    a.groups = workgroups();
    void* argv[] = {&a};
    hipStream_t s = (hipStream_t)stream;
    const int64_t spans = b * c->heads * l.tiles;
    const bool flat = spans > workgroups() || a.capacity > (spans * 4 > workgroups() && spans * 2 <= workgroups() ? 2 * DIRECT : DIRECT);
    const Kernel k = c->fmt == WOQ_CACHE_INT8 ? split_kernel<true>(c->dim, flat) : split_kernel<false>(c->dim, flat);
    const size_t lds = (size_t)(flat ? 2 : 1) * k.waves * l.per_tile * (k.dim + 4) * 4;
    const unsigned grid = flat ? (unsigned)workgroups() : (unsigned)spans;
    hipError_t e = hipSuccess;
    if (lds > 64 << 10) e = hipFuncSetAttribute(k.f, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e == hipSuccess) e = hipLaunchKernel(k.f, dim3(grid), dim3(64 * k.waves), argv, lds, s);
    if (e == hipSuccess && flat) {
        const bool few = b <= 64 && spans * 8 <= workgroups();
        e = hipLaunchKernel(few ? reinterpret_cast<const void*>(&attn_join_kernel<true>)
                                : reinterpret_cast<const void*>(&attn_join_kernel<false>),
                            dim3(few ? (unsigned)(spans * l.per_tile) : grid), dim3(256), argv, 0, s);
    }
    if (e != hipSuccess) {
        woq::set_hip_error((int)e);
        return WOQ_EHIP;
    }
    return WOQ_OK;
}
