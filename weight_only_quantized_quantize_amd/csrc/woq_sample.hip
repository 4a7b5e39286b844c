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
// Bound by one compute unit's phases for few rows (one row of 128256 23.6 us: the
// histogram 8, sums of its bins 2.5, limits 2.8, masses 2.5 to 6, searches 2.9, the
// place 2.8), by HBM and those in turn for many (256 rows of 256000 52 us, the
// histogram 26 of them at 5.2 TB/s).  A sort would move the row several times, a
// threshold found in rounds read it several times.
//
// One workgroup per row.  The counts are 16 bits wide (65536 of them are 128 KB of
// LDS, a value and its negative's neighbour to a word); one that passes 65535 loses
// 65535 or 65536 of the sum of all, so a sum that is not the number of logits tells
// that some did, and the row then counts in 32 bits, one half of the bins at a time.
#include <hip/hip_runtime.h>

#include "woq_gemv.h"
#include "woq_internal.h"

namespace {

using namespace woqk;

constexpr int T = 1024, WAVES = T / 64;
constexpr int B = 8, CHUNK = 64 * B, CHUNKS = 65536 / CHUNK;      // bins a wave takes at once, eight to a lane
constexpr int BATCH = 8;                               // loads of a thread in flight
constexpr uint32_t FIRST = 0x3FF, DEAD = 0xFC00;       // +infinity's bin; from DEAD on -infinity and NaN, as before FIRST
constexpr uint32_t ZERO = 0x7FFF;                      // the bin of both zeros
constexpr int LIST = 1024;                             // places of a drawn value that are ranked in one step

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

typedef unsigned short us2 __attribute__((ext_vector_type(2)));
typedef short ss2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ us2 as_us2(uint32_t v) { return __builtin_bit_cast(us2, v); }
__device__ __forceinline__ uint32_t as_u32(us2 v) { return __builtin_bit_cast(uint32_t, v); }

// Bins of a word's two logits: 0x7FFF - h for positive h, h for the others, so they
// rise as values fall; -0 is 0x8000 here, which is added to ZERO later.
__device__ __forceinline__ uint32_t bins_of(uint32_t h, uint32_t& negative) {
    negative = __builtin_bit_cast(uint32_t, __builtin_bit_cast(ss2, h) >> (short)15);
    return h ^ (~negative & 0x7FFF7FFFu);
}
__device__ __forceinline__ uint32_t bin_of(uint32_t h) { return h == 0x8000u ? ZERO : h & 0x8000u ? h : 0x7FFFu - h; }
__device__ __forceinline__ bool alive(uint32_t e) { return e - FIRST < DEAD - FIRST; }

__device__ __forceinline__ double value_of(uint32_t e) {
    return (double)h_to_f((uint16_t)(e & 0x8000u ? e : 0x7FFFu - e));
}

struct Row {
    uint32_t hist[32768];     // bins e and e + 32768, or in 32 bits one half of the bins
    double mass[CHUNKS];
    uint32_t count[CHUNKS];
    uint32_t wave[WAVES], list[LIST];
    uint32_t all, dead, places, wide, half;       // counts of 32 bits, of which half
    uint32_t chunk, bin, rank, limit, left;
    double before, kept;
};

// A lane's value of CTRL (a data-parallel primitive's control), 0 where there is none.
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ uint32_t lanes(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, true);
}
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ double lanes(double v) {
    const u32x2 w = __builtin_bit_cast(u32x2, v);
    return __builtin_bit_cast(double, u32x2{lanes<CTRL, ROWS>(w[0]), lanes<CTRL, ROWS>(w[1])});
}
__device__ __forceinline__ uint32_t last_lane(uint32_t v) { return (uint32_t)__builtin_amdgcn_readlane((int)v, 63); }
__device__ __forceinline__ double last_lane(double v) {
    const u32x2 w = __builtin_bit_cast(u32x2, v);
    return __builtin_bit_cast(double, u32x2{last_lane(w[0]), last_lane(w[1])});
}
// Sum over the lanes up to this one: in rows of 16, then from row to row.
template <class V>
__device__ __forceinline__ V wave_upto(V v) {
    v += lanes<0x111>(v);
    v += lanes<0x112>(v);
    v += lanes<0x114>(v);
    v += lanes<0x118>(v);
    v += lanes<0x142, 0xA>(v);
    v += lanes<0x143, 0xC>(v);
    return v;
}
template <class V>
__device__ __forceinline__ V wave_sum(V v) {
    return last_lane(wave_upto(v));
}

// f(word, index of its first logit) for every whole word of eight logits, several in
// flight, then g(logit, index) for those behind the last.
template <class F, class G>
__device__ __forceinline__ void each(const uint16_t* x, uint32_t N, F f, G g) {
    const uint32_t words = N / 8;
    uint4 w[BATCH];
    for (uint32_t c0 = 0; c0 < words; c0 += T * BATCH) {
#pragma unroll
        for (int i = 0; i < BATCH; ++i)
            w[i] = gload_u4(reinterpret_cast<const uint4*>(x) + min(c0 + i * T + threadIdx.x, words - 1));
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const uint32_t c = c0 + i * T + threadIdx.x;
            if (c < words) f(w[i], 8 * c);
        }
    }
    if (threadIdx.x < (N & 7)) g((uint32_t)*gptr(x + (N & ~7u) + threadIdx.x), (N & ~7u) + threadIdx.x);
}

// Bins half * 32768 ... in 32 bits; called by every thread.
__device__ void count_half(Row& s, const uint16_t* x, uint32_t N, uint32_t half) {
    __syncthreads();
    for (int i = threadIdx.x; i < 32768; i += T) s.hist[i] = 0;
    __syncthreads();
    auto one = [&](uint32_t h, uint32_t) {
        const uint32_t e = bin_of(h);
        if (alive(e) && e >> 15 == half) atomicAdd(&s.hist[e & 0x7FFFu], 1u);
    };
    each(x, N, [&](uint4 q, uint32_t i) {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) one(w[j >> 1] >> (16 * (j & 1)) & 0xFFFFu, i + j);
    }, one);
    if (threadIdx.x == 0) s.half = half;
    __syncthreads();
}

// Sees to it that a chunk's counts are there; called by every thread.
__device__ __forceinline__ void need(Row& s, const uint16_t* x, uint32_t N, uint32_t chunk) {
    if (s.wide && s.half != chunk / (CHUNKS / 2)) count_half(s, x, N, chunk / (CHUNKS / 2));
}

// Counts of this lane's bins of a chunk, -infinity and NaN left out.
__device__ __forceinline__ void counts_of(const Row& s, uint32_t chunk, uint32_t (&n)[B]) {
    const uint32_t e = chunk * CHUNK + B * (threadIdx.x & 63);
    const bool upper = chunk >= CHUNKS / 2, edge = chunk <= FIRST / CHUNK || chunk >= DEAD / CHUNK;
#pragma unroll
    for (int i = 0; i < B; i += 4) {
        const uint4 w = *reinterpret_cast<const uint4*>(s.hist + (e & 0x7FFFu) + i);
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            n[i + j] = s.wide ? v[j] : upper ? v[j] >> 16 : v[j] & 0xFFFFu;
            if (edge && !alive(e + i + j)) n[i + j] = 0;
        }
    }
}

// e^((value - top) / T).  With z = k ln 2 + r, |r| <= ln 2 / 2, the series of e^r to
// r^13 is off by less than 2^-57.  What lies 60 below the top weighs less than 2^-86
// and counts as nothing: 2^24 such tokens would not move the last bit of a sum.
struct Weight {
    double top, inv;
    uint32_t first;           // the bin of top
    __device__ __forceinline__ double exp_of(double z) const {
        const double k = rint(z * 1.4426950408889634);
        const double r = fma(-k, 2.3190468138462996e-17, fma(-k, 0.6931471805599453, z));
        double p = 1.0 / 6227020800.0;
        p = fma(p, r, 1.0 / 479001600.0);
        p = fma(p, r, 1.0 / 39916800.0);
        p = fma(p, r, 1.0 / 3628800.0);
        p = fma(p, r, 1.0 / 362880.0);
        p = fma(p, r, 1.0 / 40320.0);
        p = fma(p, r, 1.0 / 5040.0);
        p = fma(p, r, 1.0 / 720.0);
        p = fma(p, r, 1.0 / 120.0);
        p = fma(p, r, 1.0 / 24.0);
        p = fma(p, r, 1.0 / 6.0);
        p = fma(p, r, 0.5);
        p = fma(p, r, 1.0);
        p = fma(p, r, 1.0);
        const double w = __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, p) + ((uint64_t)(int64_t)(int)k << 52));
        return z >= -60.0 ? w : 0.0;
    }
    __device__ __forceinline__ double operator()(uint32_t e) const {
        const double v = value_of(e);
        return v == top ? 1.0 : exp_of((v - top) * inv);      // an infinity less itself is none
    }
};

// What each value of a chunk weighs of the one before.
__device__ __forceinline__ double step_of(const Weight& w, uint32_t chunk) {
    return w.exp_of((value_of(chunk * CHUNK + 1) - value_of(chunk * CHUNK)) * w.inv);
}

// Weights of this lane's bins of a chunk.  Neighbouring values of a chunk are equally
// far apart, so each weighs the same part of the one before; only the chunks up to
// +infinity's have values one by one.
__device__ __forceinline__ void weights_of(const Weight& w, uint32_t chunk, double (&v)[B]) {
    const uint32_t e = chunk * CHUNK + B * (threadIdx.x & 63);
    if (chunk <= FIRST / CHUNK) {
#pragma unroll
        for (int j = 0; j < B; ++j) v[j] = alive(e + j) ? w(e + j) : 0.0;
        return;
    }
    const double step = step_of(w, chunk);
    double next = w(max(e, w.first));         // bins before the first of all hold nothing
#pragma unroll
    for (int j = 0; j < B; ++j) {
        const bool in = e + j >= w.first;
        v[j] = in ? next : 0.0;
        next = in ? next * step : next;
    }
}

// The counts that are kept: all of the bins before the limit, `left` of that bin.
__device__ __forceinline__ uint32_t kept(const Row& s, uint32_t e, uint32_t n) {
    return e < s.limit ? n : e == s.limit ? s.left : 0;
}

// Masses of the kept tokens of every chunk; called by every thread.
__device__ void weigh(Row& s, const uint16_t* x, uint32_t N, const Weight& w) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (uint32_t h = 0; h < (s.wide ? 2u : 1u); ++h) {
        const uint32_t lo = s.wide ? CHUNKS / 2 * h : 0, hi = s.wide ? lo + CHUNKS / 2 : CHUNKS;
        need(s, x, N, lo);
        for (uint32_t c = lo + wave; c < hi; c += WAVES) {
            double m = 0.0;
            if (s.count[c] && c * CHUNK <= s.limit) {
                uint32_t n[B];
                counts_of(s, c, n);
                if (c > FIRST / CHUNK && c * CHUNK > w.first && (c + 1) * CHUNK <= s.limit) {
                    // all kept: the first weight times a polynomial in what each weighs of the one before
                    // (61 rows of 128256 30.6 -> 28.0 us)
                    const double step = step_of(w, c);
                    m = (double)n[B - 1];
#pragma unroll
                    for (int j = B - 2; j >= 0; --j) m = fma(m, step, (double)n[j]);
                    m *= w(c * CHUNK + B * lane);
                } else {
                    double v[B];
                    weights_of(w, c, v);
#pragma unroll
                    for (int j = 0; j < B; ++j) m = fma((double)kept(s, c * CHUNK + B * lane + j, n[j]), v[j], m);
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
    const double upto = wave_upto(sum), total = last_lane(upto), t = t_of(total);
    double before = upto - sum;
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
    if (hits ? lane == __builtin_ctzll(hits) : lane == 63 - __builtin_clzll(any)) {
        s.chunk = CHUNKS / 64 * lane + (hits ? hit : last);
        s.before = hits ? at : at_last;
    }
}

// In that chunk the first bin likewise: s.bin, how many of its tokens reach t (or lie
// before the one that exceeds it) in s.rank.  Called by the first wave.
template <bool REACH>
__device__ void find_bin(Row& s, const Weight& w, double t) {
    const int lane = threadIdx.x;
    const uint32_t c = s.chunk;
    uint32_t k[B];
    double each[B], sum = 0.0;
    counts_of(s, c, k);
    weights_of(w, c, each);
#pragma unroll
    for (int j = 0; j < B; ++j) {
        k[j] = kept(s, c * CHUNK + B * lane + j, k[j]);
        sum = fma((double)k[j], each[j], sum);
    }
    double before = s.before + (wave_upto(sum) - sum);
    int last = -1, hit = -1;
    double at = 0.0, at_last = 0.0;
#pragma unroll
    for (int j = 0; j < B; ++j) {
        const double m = (double)k[j] * each[j];
        if (m > 0.0) last = j, at_last = before;
        if (hit < 0 && m > 0.0 && (REACH ? before + m >= t : before + m > t)) hit = j, at = before;
        before += m;
    }
    const uint64_t hits = __ballot(hit >= 0), any = __ballot(last >= 0);
    const bool mine = hits ? lane == __builtin_ctzll(hits) : lane == 63 - __builtin_clzll(any);
    if (!mine) return;
    const int j = hits ? hit : last;
    uint32_t kj = k[0];
    double ej = each[0];
#pragma unroll
    for (int i = 1; i < B; ++i)
        if (i == j) kj = k[i], ej = each[i];
    const double b = hits ? at : at_last, part = (t - b) / ej;
    const double want = REACH ? fmin(fmax(ceil(part), 1.0), (double)kj) : fmin(fmax(floor(part), 0.0), (double)(kj - 1));
    s.bin = c * CHUNK + B * lane + j;
    s.rank = hits ? (uint32_t)want : REACH ? kj : kj - 1;
    if (REACH) s.kept = b + (double)s.rank * ej;
}

__global__ __launch_bounds__(T) void sample_kernel(SampleArgs a) {
    __shared__ __align__(16) Row s;
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
    if (tid == 0) s.all = 0, s.dead = 0, s.places = 0, s.wide = 0, s.half = 2, s.limit = 65536, s.left = 0;
    __syncthreads();
    // -infinity, which a mask may have put in most places, goes to a bin of the lane's
    // own behind DEAD, not to one word for all
    const us2 aside = {(unsigned short)lane, (unsigned short)lane};
    auto two = [&](uint32_t h) {
        uint32_t negative;
        us2 e = as_us2(bins_of(h, negative));
        const us2 limit = {(unsigned short)(DEAD - 1), (unsigned short)(DEAD - 1)}, one = {1, 1};
        e = __builtin_elementwise_add_sat(e, (us2)(__builtin_elementwise_min(__builtin_elementwise_sub_sat(e, limit), one) * aside));
        const uint32_t at = as_u32(e) & 0x7FFF7FFFu;
        atomicAdd(&s.hist[at & 0xFFFFu], (negative & 0xFFFFu) + 1u);        // 1, or 65536 in the upper half
        atomicAdd(&s.hist[at >> 16], (negative >> 16) + 1u);
    };
    each(x, a.N, [&](uint4 q, uint32_t) {
        two(q.x);
        two(q.y);
        two(q.z);
        two(q.w);
    }, [&](uint32_t h, uint32_t) {
        const uint32_t e = h & 0x8000u ? h : 0x7FFFu - h;
        atomicAdd(&s.hist[e & 0x7FFFu], e & 0x8000u ? 65536u : 1u);
    });
    __syncthreads();
    if (tid == 0) {
        const uint32_t zeros = s.hist[0] >> 16;
        s.hist[0] &= 0xFFFFu;
        s.hist[ZERO] += zeros;
    }
    __syncthreads();
    // counts of all chunks: of the lower and the upper half of a word at once, and s.all
    // with -infinity and NaN
    {
        uint32_t all = 0;
        for (uint32_t c = wave; c < CHUNKS / 2; c += WAVES) {
            uint32_t lower = 0, upper = 0;
#pragma unroll
            for (int i = 0; i < B; i += 4) {
                const uint32_t e = c * CHUNK + B * lane + i;
                const uint4 w = *reinterpret_cast<const uint4*>(s.hist + e);
                const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    all += (v[j] & 0xFFFFu) + (v[j] >> 16);
                    if (c > FIRST / CHUNK || e + j >= FIRST) lower += v[j] & 0xFFFFu;
                    upper += v[j] >> 16;
                }
            }
            lower = wave_sum(lower);
            upper = c + CHUNKS / 2 < DEAD / CHUNK ? wave_sum(upper) : 0;
            if (lane == 0) s.count[c] = lower, s.count[c + CHUNKS / 2] = upper;
        }
        all = wave_sum(all);
        if (lane == 0) atomicAdd(&s.all, all);
    }
    __syncthreads();
    auto sums = [&](uint32_t half) {          // of a row that counts in 32 bits
        for (uint32_t c = half * (CHUNKS / 2) + wave; c < (half + 1) * (CHUNKS / 2); c += WAVES) {
            uint32_t n[B], t = 0;
            counts_of(s, c, n);
#pragma unroll
            for (int j = 0; j < B; ++j) t += n[j];
            t = wave_sum(t);
            if (lane == 0) s.count[c] = t;
        }
        __syncthreads();
    };
    auto all_counts = [&] {
        uint32_t t = 0;
#pragma unroll
        for (int j = 0; j < CHUNKS / 64; ++j) t += s.count[CHUNKS / 64 * lane + j];
        return t;
    };
    uint32_t live = wave_sum(all_counts());
    if (s.all != a.N) {       // some count was too small, which matters unless it was of -infinity or NaN
        uint32_t dead = 0;
        auto one = [&](uint32_t h, uint32_t) { dead += !alive(bin_of(h)); };
        each(x, a.N, [&](uint4 q, uint32_t i) {
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int j = 0; j < 8; ++j) one(w[j >> 1] >> (16 * (j & 1)) & 0xFFFFu, i);
        }, one);
        dead = wave_sum(dead);
        if (lane == 0 && dead) atomicAdd(&s.dead, dead);
        __syncthreads();
        const uint32_t true_live = a.N - s.dead;
        if (live != true_live) {
            if (tid == 0) s.wide = 1;
            count_half(s, x, a.N, 1);
            sums(1);
            count_half(s, x, a.N, 0);
            sums(0);
        }
        live = true_live;
    }
    if (live == 0) {
        if (tid == 0) {
            *gptr(a.token + r) = -1;
            if (a.prob) *gptr(a.prob + r) = 0.0f;
        }
        return;
    }
    // the first bin of all
    uint32_t first;
    {
        uint32_t c = CHUNKS;
#pragma unroll
        for (int j = CHUNKS / 64 - 1; j >= 0; --j)
            if (s.count[CHUNKS / 64 * lane + j]) c = CHUNKS / 64 * lane + j;
        c = (uint32_t)__builtin_amdgcn_readlane((int)c, __builtin_ctzll(__ballot(c < CHUNKS)));
        need(s, x, a.N, c);
        uint32_t n[B], e = DEAD;
        counts_of(s, c, n);
#pragma unroll
        for (int j = B - 1; j >= 0; --j)
            if (n[j]) e = c * CHUNK + B * lane + j;
        first = (uint32_t)__builtin_amdgcn_readlane((int)e, __builtin_ctzll(__ballot(e < DEAD)));
    }
    uint32_t bin = first, rank = 0;
    if (k == 1) {             // the largest logit, the first of several
        if (tid == 0 && a.prob) *gptr(a.prob + r) = 1.0f;
    } else {
        const Weight w{value_of(first), 1.0 / (double)temp, first};
        // top-k: the bin at which the count reaches k
        if (k > 0 && k < live) {
            if (wave == 0) {
                const uint32_t mine = all_counts();
                uint32_t before = wave_upto(mine) - mine;
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
                uint32_t n[B], mine = 0;
                counts_of(s, s.chunk, n);
#pragma unroll
                for (int j = 0; j < B; ++j) mine += n[j];
                uint32_t before = s.left + wave_upto(mine) - mine;
#pragma unroll
                for (int j = 0; j < B; ++j) {
                    if (before < k && k <= before + n[j])
                        s.limit = s.chunk * CHUNK + B * lane + j, s.left = (uint32_t)k - before;
                    before += n[j];
                }
            }
            __syncthreads();
        }
        // min-p: weights fall from bin to bin, so the first that is too small ends the rest
        if (min_p > 0.0f && wave == 0) {
            uint32_t lo = first, hi = 65536;     // the weight of bin lo suffices, that of hi does not
            while (hi - lo > 1) {
                const uint32_t step = (hi - lo + 63) / 64, e = lo + (lane + 1) * step;
                const bool ok = e < hi && e < DEAD && w(e) >= (double)min_p;
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
        }
        double t = 0.0;
        if (wave == 0) {
            const double kept = p < 1.0f ? s.kept : 0.0;       // top-p leaves less than the chunks' masses
            find_chunk<false>(s, [&](double total) {
                t = (double)u * (p < 1.0f ? kept : total);
                return t;
            });
            if (p < 1.0f && lane == 0) s.kept = kept;
        }
        __syncthreads();
        need(s, x, a.N, s.chunk);
        if (wave == 0) find_bin<false>(s, w, t);
        __syncthreads();
        bin = s.bin, rank = s.rank;
        if (tid == 0 && a.prob) *gptr(a.prob + r) = (float)((double)w(bin) / s.kept);
    }
    // the rank-th token of that bin.  A zero's sign does not matter.
    const uint32_t mask = bin == ZERO ? 0x7FFF7FFFu : 0xFFFFFFFFu;
    const uint32_t value = bin == ZERO ? 0 : (bin & 0x8000u ? bin : 0x7FFFu - bin) * 0x10001u;
    auto differ = [&](uint32_t h) { return as_us2((h & mask) ^ value); };      // 0 for each that is it
    need(s, x, a.N, bin / CHUNK);
    const uint32_t there = s.wide                 ? s.hist[bin & 0x7FFFu]
                           : bin & 0x8000u ? s.hist[bin & 0x7FFFu] >> 16 : s.hist[bin] & 0xFFFFu;
    if (there <= LIST) {
        // all of their places, in any order; each then looks how many lie before it
        auto put = [&](uint32_t i) { s.list[atomicAdd(&s.places, 1u)] = i; };
        each(x, a.N, [&](uint4 q, uint32_t i) {
            const us2 d[4] = {differ(q.x), differ(q.y), differ(q.z), differ(q.w)};
            const us2 least = __builtin_elementwise_min(__builtin_elementwise_min(d[0], d[1]),
                                                        __builtin_elementwise_min(d[2], d[3]));
            if (least[0] && least[1]) return;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (d[j >> 1][j & 1] == 0) put(i + j);
        }, [&](uint32_t h, uint32_t i) {
            if (differ(h)[0] == 0) put(i);
        });
        __syncthreads();
        if (tid < there) {
            const uint32_t mine = s.list[tid];
            uint32_t before = 0;
            for (uint32_t i = 0; i < there; ++i) before += s.list[i] < mine;
            if (before == rank) *gptr(a.token + r) = (int32_t)mine;
        }
        return;
    }
    // many of one value: each wave counts a range of the row, the one that holds it
    // counts again
    const uint32_t steps = (a.N + 511) / 512, per = (steps + WAVES - 1) / WAVES;
    auto matches = [&](uint32_t step) {
        uint32_t m = 0;
        const uint32_t i0 = step * 512 + 8 * lane;
        if (i0 + 8 <= a.N) {
            const uint4 q = gload_u4(reinterpret_cast<const uint4*>(x + i0));
            const us2 d[4] = {differ(q.x), differ(q.y), differ(q.z), differ(q.w)};
#pragma unroll
            for (int j = 0; j < 8; ++j) m |= (uint32_t)(d[j >> 1][j & 1] == 0) << j;
        } else {
            for (int j = 0; j < 8 && i0 + j < a.N; ++j) m |= (uint32_t)(differ(*gptr(x + i0 + j))[0] == 0) << j;
        }
        return m;
    };
    const uint32_t s0 = wave * per, s1 = min(steps, s0 + per);
    uint32_t n = 0;
#pragma unroll 4
    for (uint32_t i = s0; i < s1; ++i) n += __popc(matches(i));
    n = wave_sum(n);
    if (lane == 0) s.wave[wave] = n;
    __syncthreads();
    uint32_t before = 0;
    for (int i = 0; i < wave; ++i) before += s.wave[i];
    if (rank < before || rank >= before + n) return;
    for (uint32_t i = s0; i < s1; ++i) {
        uint32_t m = matches(i);
        const uint32_t c = __popc(m), upto = wave_upto(c), all = last_lane(upto);
        if (rank >= before + all) {
            before += all;
            continue;
        }
        uint32_t mine = before + upto - c;
        if (mine <= rank && rank < mine + c) {
            for (; mine < rank; ++mine) m &= m - 1;
            *gptr(a.token + r) = (int32_t)(i * 512 + 8 * lane + __builtin_ctz(m));
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
    // a launch has fewer than 2^32 threads
    if (N > WOQ_SAMPLE_MAX_N || b > WOQ_SAMPLE_MAX_ROWS) return WOQ_EUNSUPPORTED;
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
