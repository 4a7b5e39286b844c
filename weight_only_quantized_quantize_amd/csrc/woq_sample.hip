// The next token of every row from its logits and a given random number.
//
// An fp16 logit has fewer than 65536 values, so a histogram over them takes the
// place of a sort: bin e holds how many of a row's logits have the e-th largest
// fp16 value.  Going through the bins from the first is going through the tokens
// from the largest logit down; a bin's mass is its count times one exponential,
// in 64 bits; top-k, min-p and top-p each end the kept tokens at some bin and some
// number of its tokens, and the draw falls on a bin and a number in it.  Only then
// are the logits read again, for the index of that many-th token of that value.
//
// One workgroup per row.  The counts are 16 bits wide (65536 of them are 128 KB of
// LDS); a count that passes 65535 loses 65535 or 65536 of the sum of all, so a sum
// that is not the number of logits tells that some did, and the row then counts in
// 32 bits, one half of the bins at a time.
#include <hip/hip_runtime.h>

#include "woq_gemv.h"
#include "woq_internal.h"

namespace {

using namespace woqk;

constexpr int T = 1024, WAVES = T / 64;
constexpr int CHUNK = 256, CHUNKS = 65536 / CHUNK;     // bins a wave takes at once, four to a lane
constexpr uint32_t DEAD = 0xFFFFu;                     // the bin of NaN and -infinity, of which none is counted

struct SampleArgs {
    const uint16_t* logits;
    const float* temperature; // null where not given, like top_k, top_p, min_p
    const int32_t* top_k;
    const float* top_p;
    const float* min_p;
    const float* u;
    int32_t* token;
    float* prob;              // null: not asked for
    int64_t ld;
    uint32_t N;
};

// The bin of a logit: 0 for the largest fp16 bit pattern, rising as values fall;
// both zeros have the same.
__device__ __forceinline__ uint32_t bin_of(uint32_t h) {
    if ((h & 0x7FFFu) > 0x7C00u || h == 0xFC00u) return DEAD;
    if (h == 0x8000u) h = 0;
    return h & 0x8000u ? h : 0x7FFFu - h;
}

__device__ __forceinline__ double value_of(uint32_t e) {
    return (double)h_to_f((uint16_t)(e & 0x8000u ? e : 0x7FFFu - e));
}

struct Row {
    uint32_t hist[32768];     // two counts to a word, or one count of half of the bins
    double mass[CHUNKS];
    uint32_t count[CHUNKS];
    uint32_t wave[WAVES];
    uint32_t live, first, wide, half;     // logits counted, the first bin of any; counts of 32 bits, of which half
    uint32_t chunk, bin, rank, limit, left;
    double before, kept;
};

__device__ __forceinline__ uint32_t wave_sum(uint32_t v) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v += (uint32_t)__shfl_xor((int)v, d);
    return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
    return v;
}
// Sum over the lanes before this one.
template <class V>
__device__ __forceinline__ V wave_before(V v) {
    const int lane = threadIdx.x & 63;
    V s = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const V o = __shfl_up(s, d);
        if (lane >= d) s += o;
    }
    const V o = __shfl_up(s, 1);
    return lane ? o : V(0);
}

// f(bin) for every logit of the row, in no order.
template <class F>
__device__ __forceinline__ void each(const uint16_t* x, uint32_t N, F f) {
    for (uint32_t c = threadIdx.x; c < N / 8; c += T) {
        const uint4 w = gload_u4(reinterpret_cast<const uint4*>(x) + c);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) f(bin_of(u[j >> 1] >> (16 * (j & 1)) & 0xFFFFu));
    }
    if (threadIdx.x < (N & 7)) f(bin_of(*gptr(x + (N & ~7u) + threadIdx.x)));
}

// Bins half * 32768 ... of a row whose counts are 32 bits wide; called by every thread.
__device__ void count_half(Row& s, const uint16_t* x, uint32_t N, uint32_t half) {
    __syncthreads();
    for (int i = threadIdx.x; i < 32768; i += T) s.hist[i] = 0;
    __syncthreads();
    each(x, N, [&](uint32_t e) {
        if (e != DEAD && e >> 15 == half) atomicAdd(&s.hist[e & 0x7FFFu], 1u);
    });
    if (threadIdx.x == 0) s.half = half;
    __syncthreads();
}

// Sees to it that a chunk's counts are there; called by every thread.
__device__ __forceinline__ void need(Row& s, const uint16_t* x, uint32_t N, uint32_t chunk) {
    if (s.wide && s.half != chunk >> 7) count_half(s, x, N, chunk >> 7);
}

// Counts of the four bins of this lane in a chunk.
__device__ __forceinline__ void counts4(const Row& s, uint32_t chunk, uint32_t (&n)[4]) {
    const int lane = threadIdx.x & 63;
    if (s.wide) {
#pragma unroll
        for (int j = 0; j < 4; ++j) n[j] = s.hist[(chunk & 127) * CHUNK + 4 * lane + j];
    } else {
        const uint32_t a = s.hist[chunk * (CHUNK / 2) + 2 * lane], b = s.hist[chunk * (CHUNK / 2) + 2 * lane + 1];
        n[0] = a & 0xFFFFu, n[1] = a >> 16, n[2] = b & 0xFFFFu, n[3] = b >> 16;
    }
}

struct Weight {
    double top, inv;
    // e^((value - top) / T); what lies 60 below the top weighs less than 2^-86 and
    // counts as nothing: 2^24 such tokens would not move the last bit of a sum
    __device__ __forceinline__ double operator()(uint32_t e) const {
        const double v = value_of(e);
        if (v == top) return 1.0;
        const double z = (v - top) * inv;
        return z >= -60.0 ? exp(z) : 0.0;      // no infinity less infinity
    }
};

// The counts that are kept: all of the bins before the limit, `left` of that bin.
__device__ __forceinline__ uint32_t kept(const Row& s, uint32_t e, uint32_t n) {
    return e < s.limit ? n : e == s.limit ? s.left : 0;
}

// Masses of the kept tokens of every chunk; called by every thread.
__device__ void weigh(Row& s, const uint16_t* x, uint32_t N, const Weight& w) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (uint32_t h = 0; h < (s.wide ? 2u : 1u); ++h) {
        const uint32_t lo = s.wide ? 128 * h : 0, hi = s.wide ? lo + 128 : CHUNKS;
        need(s, x, N, lo);
        for (uint32_t c = lo + wave; c < hi; c += WAVES) {
            double m = 0.0;
            if (s.count[c] && c * CHUNK <= s.limit) {
                uint32_t n[4];
                counts4(s, c, n);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t e = c * CHUNK + 4 * lane + j, k = kept(s, e, n[j]);
                    if (k) m += (double)k * w(e);
                }
                m = wave_sum(m);
            }
            if (lane == 0) s.mass[c] = m;
        }
    }
    __syncthreads();
}

// The first chunk whose running sum exceeds t (or reaches it: REACH), the sum
// before it in s.before; the last chunk with anything where none does, and
// s.kept the sum of all.  Called by the first wave.
template <bool REACH, class F>
__device__ void find_chunk(Row& s, F t_of) {
    const int lane = threadIdx.x;
    double m[CHUNKS / 64], sum = 0.0;
#pragma unroll
    for (int j = 0; j < CHUNKS / 64; ++j) sum += m[j] = s.mass[CHUNKS / 64 * lane + j];
    double before = wave_before(sum);
    const double total = __shfl(before + sum, 63);
    const double t = t_of(total);
    if (lane == 0) s.kept = total;
    int last = -1, hit = -1;
    double at = 0.0, at_last = 0.0;
#pragma unroll
    for (int j = 0; j < CHUNKS / 64; ++j) {
        if (m[j] > 0.0) last = j, at_last = before;
        if (hit < 0 && m[j] > 0.0 && (REACH ? before + m[j] >= t : before + m[j] > t)) hit = j, at = before;
        before += m[j];
    }
    const uint64_t hits = __ballot(hit >= 0), any = __ballot(last >= 0);
    if (hits ? lane == __ffsll((unsigned long long)hits) - 1 : lane == 63 - __clzll(any)) {
        s.chunk = CHUNKS / 64 * lane + (hits ? hit : last);
        s.before = hits ? at : at_last;
    }
}

// In that chunk the first bin likewise: s.bin, its mass's number of tokens that
// reach (or do not exceed) t in s.rank, the sum before it in s.before.  Called by
// the first wave.
template <bool REACH>
__device__ void find_bin(Row& s, const Weight& w, double t) {
    const int lane = threadIdx.x;
    const uint32_t c = s.chunk;
    uint32_t n[4], k[4];
    double each[4], sum = 0.0;
    counts4(s, c, n);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t e = c * CHUNK + 4 * lane + j;
        k[j] = kept(s, e, n[j]);
        each[j] = k[j] ? w(e) : 0.0;
        sum += (double)k[j] * each[j];
    }
    double before = s.before + wave_before(sum);
    int last = -1, hit = -1;
    double at = 0.0, at_last = 0.0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const double m = (double)k[j] * each[j];
        if (m > 0.0) last = j, at_last = before;
        if (hit < 0 && m > 0.0 && (REACH ? before + m >= t : before + m > t)) hit = j, at = before;
        before += m;
    }
    const uint64_t hits = __ballot(hit >= 0), any = __ballot(last >= 0);
    const bool mine = hits ? lane == __ffsll((unsigned long long)hits) - 1 : lane == 63 - __clzll(any);
    if (!mine) return;
    const int j = hits ? hit : last;
    uint32_t kj = k[0];
    double ej = each[0];
#pragma unroll
    for (int i = 1; i < 4; ++i)
        if (i == j) kj = k[i], ej = each[i];
    const double b = hits ? at : at_last, part = (t - b) / ej;
    // REACH: how many tokens it takes; else how many lie before the drawn one
    const double want = REACH ? fmin(fmax(ceil(part), 1.0), (double)kj) : fmin(fmax(floor(part), 0.0), (double)(kj - 1));
    s.bin = c * CHUNK + 4 * lane + j;
    s.rank = hits ? (uint32_t)want : REACH ? kj : kj - 1;
    s.before = b;
    if (REACH) s.kept = b + (double)s.rank * ej;
}

__global__ __launch_bounds__(T) void sample_kernel(SampleArgs a) {
    __shared__ Row s;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t r = blockIdx.x;
    const uint16_t* x = a.logits + r * a.ld;
    float temp = a.temperature ? *gptr(a.temperature + r) : 1.0f;
    int64_t k = a.top_k ? *gptr(a.top_k + r) : 0;
    const float p = a.top_p ? *gptr(a.top_p + r) : 1.0f;
    float min_p = a.min_p ? *gptr(a.min_p + r) : 0.0f;
    if (min_p > 1.0f) min_p = 1.0f;
    const float u = fminf(fmaxf(*gptr(a.u + r), 0.0f), 0x1.fffffep-1f);     // a NaN is 0
    if (!(temp > 0.0f)) temp = 1.0f, k = 1;

    for (int i = tid; i < 32768 / 4; i += T) reinterpret_cast<uint4*>(s.hist)[i] = make_uint4(0, 0, 0, 0);
    if (tid == 0) s.live = 0, s.first = DEAD, s.wide = 0, s.half = 2, s.limit = 65536, s.left = 0;
    __syncthreads();
    {
        uint32_t live = 0, first = DEAD;
        each(x, a.N, [&](uint32_t e) {
            if (e != DEAD) {
                atomicAdd(&s.hist[e >> 1], e & 1 ? 65536u : 1u);
                ++live;
                first = min(first, e);
            }
        });
        live = wave_sum(live);
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) first = min(first, (uint32_t)__shfl_xor((int)first, d));
        if (lane == 0) {
            atomicAdd(&s.live, live);
            atomicMin(&s.first, first);
        }
    }
    __syncthreads();
    const uint32_t live = s.live;
    if (live == 0) {
        if (tid == 0) {
            *gptr(a.token + r) = -1;
            if (a.prob) *gptr(a.prob + r) = 0.0f;
        }
        return;
    }
    auto sums = [&](uint32_t lo, uint32_t hi) {
        for (uint32_t c = lo + wave; c < hi; c += WAVES) {
            uint32_t n[4];
            counts4(s, c, n);
            const uint32_t t = wave_sum(n[0] + n[1] + n[2] + n[3]);
            if (lane == 0) s.count[c] = t;
        }
        __syncthreads();
    };
    sums(0, CHUNKS);
    auto all_counts = [&] {
        uint32_t t = 0;
#pragma unroll
        for (int j = 0; j < CHUNKS / 64; ++j) t += s.count[CHUNKS / 64 * lane + j];
        return t;
    };
    if (wave_sum(all_counts()) != live) {
        __syncthreads();
        if (tid == 0) s.wide = 1;
        count_half(s, x, a.N, 1);
        sums(128, CHUNKS);
        count_half(s, x, a.N, 0);
        sums(0, 128);
    }
    const Weight w{value_of(s.first), 1.0 / (double)temp};
    // top-k: the bin at which the count reaches k
    if (k > 0 && k < live) {
        if (wave == 0) {
            uint32_t before = wave_before(all_counts());
#pragma unroll
            for (int j = 0; j < CHUNKS / 64; ++j) {
                const uint32_t n = s.count[CHUNKS / 64 * lane + j];
                if (before < k && k <= before + n) s.chunk = CHUNKS / 64 * lane + j, s.left = before;
                before += n;
            }
        }
        __syncthreads();
        need(s, x, a.N, s.chunk);
        if (wave == 0) {
            uint32_t n[4];
            counts4(s, s.chunk, n);
            uint32_t before = s.left + wave_before(n[0] + n[1] + n[2] + n[3]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (before < k && k <= before + n[j])
                    s.limit = s.chunk * CHUNK + 4 * lane + j, s.left = (uint32_t)k - before;
                before += n[j];
            }
        }
        __syncthreads();
    }
    // min-p: weights fall from bin to bin, so the first that is too small ends the rest
    if (min_p > 0.0f && wave == 0) {
        uint32_t lo = s.first, hi = 65536;     // the weight of bin lo suffices, that of hi does not
        while (hi - lo > 1) {
            const uint32_t step = (hi - lo + 63) / 64, e = lo + (lane + 1) * step;
            const bool ok = e < hi && e <= 0xFBFFu && w(e) >= (double)min_p;
            const uint32_t n = (uint32_t)__popcll(__ballot(ok));
            const uint32_t up = lo + (n + 1) * step;
            lo += n * step;
            hi = min(hi, up);
        }
        if (lane == 0 && hi <= s.limit) s.limit = hi, s.left = 0;
    }
    __syncthreads();
    weigh(s, x, a.N, w);
    // top-p, then the draw
    if (p < 1.0f) {
        double t = 0.0;
        if (wave == 0)
            find_chunk<true>(s, [&](double total) {
                t = (double)p * total;
                return t;
            });
        __syncthreads();
        need(s, x, a.N, s.chunk);
        if (wave == 0) find_bin<true>(s, w, t);
        __syncthreads();
        if (tid == 0) s.limit = s.bin, s.left = s.rank;
        __syncthreads();
    } else if (wave == 0) {
        find_chunk<false>(s, [&](double total) { return total; });
    }
    __syncthreads();
    double t = 0.0;
    if (wave == 0) {
        const double total = s.kept;
        t = (double)u * total;
        find_chunk<false>(s, [&](double) { return t; });
        if (lane == 0) s.kept = total;
    }
    __syncthreads();
    need(s, x, a.N, s.chunk);
    if (wave == 0) find_bin<false>(s, w, t);
    __syncthreads();
    const uint32_t bin = s.bin, rank = s.rank;
    if (tid == 0 && a.prob) *gptr(a.prob + r) = (float)((double)w(bin) / s.kept);
    // the rank-th token of that bin: each wave counts a range of the row, the one
    // that holds it counts again
    const uint32_t steps = (a.N + 511) / 512, per = (steps + WAVES - 1) / WAVES;
    auto matches = [&](uint32_t step) {
        uint32_t m = 0;
        const uint32_t i0 = step * 512 + 8 * lane;
        if (i0 + 8 <= a.N) {
            const uint4 q = gload_u4(reinterpret_cast<const uint4*>(x + i0));
            const uint32_t v[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) m |= (uint32_t)(bin_of(v[j >> 1] >> (16 * (j & 1)) & 0xFFFFu) == bin) << j;
        } else {
            for (int j = 0; j < 8 && i0 + j < a.N; ++j) m |= (uint32_t)(bin_of(*gptr(x + i0 + j)) == bin) << j;
        }
        return m;
    };
    const uint32_t s0 = wave * per, s1 = min(steps, s0 + per);
    uint32_t n = 0;
    for (uint32_t i = s0; i < s1; ++i) n += __popc(matches(i));
    n = wave_sum(n);
    if (lane == 0) s.wave[wave] = n;
    __syncthreads();
    uint32_t before = 0;
    for (int i = 0; i < wave; ++i) before += s.wave[i];
    if (rank < before || rank >= before + n) return;
    for (uint32_t i = s0; i < s1; ++i) {
        uint32_t m = matches(i);
        const uint32_t c = __popc(m), all = wave_sum(c);
        if (rank >= before + all) {
            before += all;
            continue;
        }
        uint32_t mine = before + wave_before(c);
        if (mine <= rank && rank < mine + c) {
            for (; mine < rank; ++mine) m &= m - 1;
            *gptr(a.token + r) = (int32_t)(i * 512 + 8 * lane + __ffs(m) - 1);
        }
        return;
    }
}

}  // namespace

extern "C" int woq_sample(const uint16_t* logits, int64_t ld, int64_t N, int64_t b, const float* temperature,
                          const int32_t* top_k, const float* top_p, const float* min_p, const float* u,
                          int32_t* token, float* prob, void* stream) {
    if (b < 0 || N < 1 || ld < N) return WOQ_EINVAL;
    if (b == 0) return WOQ_OK;
    if (!logits || !u || !token) return WOQ_EINVAL;
    if (!woq::aligned16(logits) || (ld & 7) ||
        (((uintptr_t)temperature | (uintptr_t)top_k | (uintptr_t)top_p | (uintptr_t)min_p | (uintptr_t)u |
          (uintptr_t)token | (uintptr_t)prob) &
         3u))
        return WOQ_EALIGN;
    if (N > WOQ_SAMPLE_MAX_N || b > INT32_MAX) return WOQ_EUNSUPPORTED;
    SampleArgs a;
    a.logits = logits;
    a.temperature = temperature;
    a.top_k = top_k;
    a.top_p = top_p;
    a.min_p = min_p;
    a.u = u;
    a.token = token;
    a.prob = prob;
    a.ld = ld;
    a.N = (uint32_t)N;
    void* argv[] = {&a};
    const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(&sample_kernel), dim3((unsigned)b), dim3(T),
                                         argv, 0, (hipStream_t)stream);
    if (e != hipSuccess) {
        woq::set_hip_error((int)e);
        return WOQ_EHIP;
    }
    return WOQ_OK;
}
