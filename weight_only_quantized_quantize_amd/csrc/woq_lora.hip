// Low-rank adapters of many requests beside a shared projection:
//
//   y[r, n] = fp16(base[r, n] + scale[a] sum_j B[a][n, j] h[r, seg(n) R + j]),
//   h[r, i] = sum_k A[a][i, k] x[r, k],   a = ids[r],
//
// with y = base on rows without an adapter.  Two launches: the inner products
// h into the workspace, and the outer ones added to the base; before them, in
// batches of many rows and adapters, one that puts the rows in order.
//
// Both run on the fp16 matrix cores with 16 ranks (or 16 outputs) of ONE
// adapter against 16 rows: rows that share an adapter share its bytes, and a
// result column belongs to one row, so rows never mix.  h is not rounded to
// fp16 on the way: the ranks of a row are scaled by a power of two, the largest
// to [2^13, 2^14), and split into two fp16 halves, hi + lo; one 16x16x32 step
// multiplies 16 ranks of B with both.  What that loses of a rank is at most 2^-23
// of it (two roundings to 11 bits) or, where lo is subnormal, 2^-25 after
// scaling: 2^-38 of the row's largest.  (fp32 matrix instructions, which would
// lose nothing, have a sixteenth of the fp16 rate.)
//
// A decode batch is bound by the bytes of the adapters that its rows name, or,
// at a few rows, by two launches of a few memory round trips each.  The inner
// kernel has the ids, then every load of a wave together, and no barrier before
// the sums meet; the outer one has three dependent rounds, the ids with base and
// h, the first operands of B, the rest of them; ranks per adapter add a wait to
// each of its loads (64 rows of rank 16: 22.1 us, with a rank array 26.8).  One row beside 8192 x 8192, rank 16: 4.2 + 4.8 us; 64 rows beside
// 10240 x 8192 in three segments, an adapter of rank 16 each: 10.4 + 9.8 us,
// 75 MB at 3.7 TB/s.  (Both products in one launch, each workgroup computing h
// for its 1024 outputs: 11.2 and 36 us.)  A prompt is bound by the base and the
// output: 3001 rows beside 28672 x 3584 in two segments, 8 adapters of rank 64:
// 5 + 20 + 90 us, 402 MB at 3.5 TB/s; every tile of the outer kernel waits for the
// stores of the one before and for its own base.  Ranks above 64 go through h and B
// in groups and spill 12 registers: rank 72 takes 237 us there, 128 244.
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
    float* h;                 // few rows: sums [splits][b][nseg R]; else halves [b][nseg][groups][hi, lo][16 RT]
    int32_t* exps;            // else: the halves' exponents [b][nseg][groups]
    int32_t* order;           // else: the rows, those of one adapter side by side; null: as they are
    int64_t ldx, ldbase, ldy, lda;
    int b, N, K, R, count, nseg, splits, groups, per;
    int vec;                  // rows of base and y may be read and written in 16-byte pieces
    int seg_end[WOQ_MAX_SEGMENTS];
    int tile0[WOQ_MAX_SEGMENTS + 1];   // output tiles before each segment
};

__device__ __forceinline__ int rank_of(const LoraArgs& a, int id) {
    return a.rank ? min(max(*gptr(a.rank + id), 0), a.R) : a.R;
}

__device__ __forceinline__ h8 as_h8(uint4 v) { return __builtin_bit_cast(h8, v); }
__device__ __forceinline__ uint4 load16(const uint16_t* p) { return gload_u4(reinterpret_cast<const uint4*>(p)); }

// Values k .. k + 7 of a row, zero from `end` on (where nothing is read).
__device__ __forceinline__ uint4 load8_until(const uint16_t* row, int k, int end) {
    if (k + 8 <= end) return load16(row + k);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (k + j < end) w[j >> 1] |= (uint32_t)*gptr(row + k + j) << (16 * (j & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The power of two that brings a row's largest |h| (as bits) to [2^13, 2^14).  A row that
// is not finite is left as it is: every output of it is lost.
__device__ __forceinline__ int scale_exponent(uint32_t big) {
    return big == 0 || big >= 0x7F800000u ? 0 : 14 - __builtin_amdgcn_frexp_expf(__uint_as_float(big));
}
// hi | lo << 16 of v 2^ex
__device__ __forceinline__ uint32_t split_halves(float v, int ex) {
    const float s = ldexpf(v, ex);
    const uint16_t hi = f_to_h(s);
    return (uint32_t)hi | (uint32_t)((hi & 0x7C00u) == 0x7C00u ? 0 : f_to_h(s - h_to_f(hi))) << 16;
}
// v_perm selectors: the hi, or the lo, halves of two such words
constexpr uint32_t HI = 0x05040100u, LO = 0x07060302u;

// The adapters of a window of up to 64 NW positions, found by each wave for itself:
// a lane holds the ids of positions lane, 64 + lane, ...
// ORDER: positions in the order of the rows, if there is one; else rows.
template <int NW, bool ORDER>
struct Window {
    int row[NW], ids[NW];
    __device__ __forceinline__ void read(const LoraArgs& a, int first, int rows, int lane) {
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            row[w] = min(first + 64 * w + lane, a.b - 1);
            if (ORDER && a.order) row[w] = *gptr(a.order + row[w]);
            ids[w] = 64 * w + lane < rows ? *gptr(a.ids + row[w]) : -1;
            if ((unsigned)ids[w] >= (unsigned)a.count) ids[w] = -1;
        }
    }
};

// The order in which a prompt's or a large batch's rows are taken: those of one adapter
// side by side (of adapters that are equal modulo 1024: only speed depends on
// it), those without one last.  One workgroup counts and places them; the rows
// of one adapter come in any order, which no result depends on.
constexpr int BINS = 1024;
__global__ __launch_bounds__(BINS) void lora_order_kernel(LoraArgs a) {
    __shared__ int next[BINS + 1], sums[BINS / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    next[tid] = 0;
    if (tid == 0) next[BINS] = 0;
    __syncthreads();
    // four turns of rows at a time, which for most batches is all of them
    constexpr int TURNS = 4;
    int bin[TURNS];
    auto read = [&](int first) {
#pragma unroll
        for (int t = 0; t < TURNS; ++t) bin[t] = *gptr(a.ids + min(first + t * BINS + tid, a.b - 1));
#pragma unroll
        for (int t = 0; t < TURNS; ++t)
            bin[t] = first + t * BINS + tid >= a.b ? -1 : (unsigned)bin[t] < (unsigned)a.count ? bin[t] & (BINS - 1) : BINS;
    };
    // the next place in a row's bin; one atomic where a wave's rows agree
    auto take = [&](int to) {
        const int first = __builtin_amdgcn_readfirstlane(to);
        if (__ballot(to == first) == ~0ull) {
            int at = 0;
            if (lane == 0 && first >= 0) at = atomicAdd(&next[first], 64);
            return __builtin_amdgcn_readfirstlane(at) + lane;
        }
        return to < 0 ? 0 : atomicAdd(&next[to], 1);
    };
    read(0);
    for (int first = 0;; read(first)) {
#pragma unroll
        for (int t = 0; t < TURNS; ++t) take(bin[t]);
        first += TURNS * BINS;
        if (first >= a.b) break;
    }
    __syncthreads();
    const int mine = next[tid];
    int sum = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(sum, d);
        if (lane >= d) sum += o;
    }
    if (lane == 63) sums[wave] = sum;
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < BINS / 64; ++w) {
        before += w < wave ? sums[w] : 0;
        all += sums[w];
    }
    next[tid] = before + sum - mine;
    if (tid == 0) next[BINS] = all;
    __syncthreads();
    if (a.b > TURNS * BINS) read(0);
    for (int first = 0;; read(first)) {
#pragma unroll
        for (int t = 0; t < TURNS; ++t) {
            const int at = take(bin[t]);
            if (bin[t] >= 0) *gptr(a.order + at) = first + t * BINS + tid;
        }
        first += TURNS * BINS;
        if (first >= a.b) break;
    }
}

// The inner products of RT rank tiles of 16 in one segment (blockIdx.y).  The
// W waves split the K range and add their sums in LDS in a fixed order.
//   LEADER: one workgroup per row and K range (blockIdx.z); it works
//     if its row is the 1st, 17th, 33rd .. of its adapter, for it and the next 15,
//     so distinct adapters, and the parts of one that many rows share, run side by
//     side.  The ranges' sums go to the workspace as they are.  Rows turn with the
//     other indexes: workgroups go round the eight XCDs, so of requests of 16 rows
//     each the working ones would all fall to one (256 rows of 10696, rank 56, 16
//     adapters: 115 us instead of 34).
//   otherwise: a window of 32 rows, side by side or in order of their adapters; the
//     workgroups of a window (blockIdx.z) take its adapters in turn.  h is written
//     scaled and split, ready to be multiplied.
// A wave reads 64 channels of its rows of A and x at a time, eight adjacent lanes
// a row, D such pieces ahead, and turns them into operand order in a part of
// LDS of its own (no barrier): read a lane per row straight into the operands,
// the address unit bound this kernel (3001 rows of 3584, two segments of rank 64:
// 25 us instead of 20).
template <int W, int RT, int D, bool LEADER>
__global__ __launch_bounds__(64 * W) void lora_down_kernel(LoraArgs a) {
    constexpr int NW = LEADER ? 4 : 1, WIN = LEADER ? 256 : 32, KC = 64;
    constexpr int CT = LEADER ? 1 : 2;                 // column tiles of 16 rows of x at a time
    constexpr int AP = 2 * RT, XP = 2 * CT;            // pieces of a lane: eight rows each
    constexpr int AREA = 16 * (RT + CT) * 2 * KC;      // bytes of a wave: the operands, then its sums
    static_assert(AREA >= RT * CT * 1024, "the sums fit where the operands were");
    __shared__ uint8_t list[W][WIN];
    __shared__ __align__(16) uint8_t lds[W][AREA];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int m = lane & 15, c = lane >> 4;
    const int seg = blockIdx.y / a.groups, group = blockIdx.y % a.groups, j0 = group * 16 * RT;
    const int w0 = LEADER ? 0 : blockIdx.x * WIN;
    const int nwin = min(a.b - w0, WIN);
    Window<NW, !LEADER> win;
    win.read(a, w0, nwin, lane);
    auto row_of = [&](int at) { return LEADER ? at : __shfl(win.row[0], at); };
    uint8_t* mem = lds[wave];
    auto place = [](int row, int ch) { return row * 2 * KC + 16 * (ch ^ (row & 7)); };
    const int pr = lane >> 3, pc = lane & 7;           // row and chunk of this lane in a piece

    // this wave's pieces of K
    const int chunks = (a.K + KC - 1) / KC;
    const int units = LEADER ? a.splits * W : W, unit = LEADER ? blockIdx.z * W + wave : wave;
    const int lo = (int)((int64_t)chunks * unit / units), hi = (int)((int64_t)chunks * (unit + 1) / units);

    u64 left = LEADER ? 1ull : __ballot(win.ids[0] >= 0);
    for (int turn = 0; left; ++turn) {
        int id, start = 0;                             // the first of the adapter's rows to take
        u64 of[NW];
        if constexpr (LEADER) {
            left = 0;
            const int r = (blockIdx.x + blockIdx.y + gridDim.y * blockIdx.z) % (unsigned)a.b;
            id = -1;
#pragma unroll
            for (int w = 0; w < NW; ++w)
                if (r >> 6 == w) id = __builtin_amdgcn_readlane(win.ids[w], r & 63);
            if (id < 0) return;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                of[w] = __ballot(win.ids[w] == id);
                start += __popcll(of[w] & (r >> 6 > w ? ~0ull : r >> 6 == w ? (1ull << (r & 63)) - 1 : 0));
            }
            if (start & 15) return;
        } else {
            id = __builtin_amdgcn_readlane(win.ids[0], __ffsll(left) - 1);
            of[0] = __ballot(win.ids[0] == id);
            left &= ~of[0];
            if (turn % (int)gridDim.z != (int)blockIdx.z) continue;
        }
        const int rank = rank_of(a, id);
        if (j0 >= rank) continue;
        int total = 0;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            if (of[w] >> lane & 1) list[wave][total + __popcll(of[w] & ((1ull << lane) - 1))] = (uint8_t)(64 * w + lane);
            total += __popcll(of[w]);
        }
        __builtin_amdgcn_wave_barrier();

        const uint16_t* ap[AP];
#pragma unroll
        for (int i = 0; i < AP; ++i)
            ap[i] = a.A + (((int64_t)id * a.nseg + seg) * a.R + min(j0 + 8 * i + pr, a.R - 1)) * a.lda + 8 * pc;
        for (int c0 = start; c0 < total; c0 += LEADER ? WIN : 16 * CT) {
            // columns past the list repeat its first row, or hold anything; their
            // results are dropped
            const bool two = CT == 2 && total - c0 > 16;
            const uint16_t* xp[XP];
#pragma unroll
            for (int i = 0; i < XP; ++i) {
                const int col = c0 + 8 * i + pr;
                xp[i] = a.x + (int64_t)row_of(list[wave][col < total ? col : c0]) * a.ldx + 8 * pc;
            }
            uint4 av[D][AP], xv[D][XP];
            auto load = [&](int d, int chunk) {
                if (chunk >= hi) return;
                const int k = chunk * KC;
                if (k + KC <= a.K) {
#pragma unroll
                    for (int i = 0; i < AP; ++i) av[d][i] = load16(ap[i] + k);
#pragma unroll
                    for (int i = 0; i < XP; ++i)
                        if (c0 + 8 * i < total) xv[d][i] = load16(xp[i] + k);
                } else {                               // the row's last piece, zero past its end
                    const int end = a.K - 8 * pc;
#pragma unroll
                    for (int i = 0; i < AP; ++i) av[d][i] = load8_until(ap[i], k, end);
#pragma unroll
                    for (int i = 0; i < XP; ++i) xv[d][i] = load8_until(xp[i], k, end);
                }
            };
            f4 acc[RT][CT];
#pragma unroll
            for (int t = 0; t < RT; ++t) acc[t][0] = acc[t][CT - 1] = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int d = 0; d < D; ++d) load(d, lo + d);
            for (int s = lo; s < hi; s += D) {
#pragma unroll
                for (int d = 0; d < D; ++d) {
                    if (s + d >= hi) break;
                    auto put = [&](int row, uint4 v) {
                        *(__attribute__((address_space(3))) u32x4*)(mem + place(row, pc)) = u32x4{v.x, v.y, v.z, v.w};
                    };
#pragma unroll
                    for (int i = 0; i < AP; ++i) put(8 * i + pr, av[d][i]);
#pragma unroll
                    for (int i = 0; i < XP; ++i)
                        if (c0 + 8 * i < total) put(16 * RT + 8 * i + pr, xv[d][i]);
                    load(d, s + d + D);
                    auto get = [&](int row, int step) {
                        return __builtin_bit_cast(h8, *(const __attribute__((address_space(3))) u32x4*)(mem + place(row, 4 * step + c)));
                    };
#pragma unroll
                    for (int step = 0; step < KC / 32; ++step) {
                        h8 af[RT];
#pragma unroll
                        for (int t = 0; t < RT; ++t) af[t] = get(16 * t + m, step);
                        const h8 x0 = get(16 * RT + m, step);
#pragma unroll
                        for (int t = 0; t < RT; ++t) acc[t][0] = __builtin_amdgcn_mfma_f32_16x16x32_f16(af[t], x0, acc[t][0], 0, 0, 0);
                        if (two) {
                            const h8 x1 = get(16 * RT + 16 + m, step);
#pragma unroll
                            for (int t = 0; t < RT; ++t) acc[t][CT - 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(af[t], x1, acc[t][CT - 1], 0, 0, 0);
                        }
                    }
                }
            }
            auto red = [&](int w, int i) { return (__attribute__((address_space(3))) f4*)lds[w] + i * 64 + lane; };
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                *red(wave, CT * t) = acc[t][0];
                if (CT == 2) *red(wave, CT * t + 1) = acc[t][CT - 1];
            }
            __syncthreads();
            // a wave finishes a column tile: a lane has ranks 4c .. 4c + 3
            // of every rank tile of one row
            const int col = c0 + 16 * wave + m;
            if (wave == 0 || (wave == 1 && two)) {
                f4 v[RT];
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    v[t] = *red(0, CT * t + wave);
#pragma unroll
                    for (int w = 1; w < W; ++w) v[t] += *red(w, CT * t + wave);
                }
                const int64_t row = row_of(list[wave][col < total ? col : c0]);
                if constexpr (LEADER) {
#pragma unroll
                    for (int t = 0; t < RT; ++t) {
                        const int j = j0 + 16 * t + 4 * c;
                        if (col < total && j < a.R)
                            *(__attribute__((address_space(1))) f4*)(a.h + (((int64_t)blockIdx.z * a.b + row) * a.nseg + seg) * a.R + j) = v[t];
                    }
                } else {
                    uint32_t big = 0;
#pragma unroll
                    for (int t = 0; t < RT; ++t)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if (j0 + 16 * t + 4 * c + e >= rank) v[t][e] = 0.f;
                            big = max(big, __float_as_uint(v[t][e]) & 0x7FFFFFFFu);
                        }
                    big = max(big, (uint32_t)__shfl_xor((int)big, 16));
                    big = max(big, (uint32_t)__shfl_xor((int)big, 32));
                    const int ex = scale_exponent(big);
                    if (col < total) {
                        const int64_t at = (row * a.nseg + seg) * a.groups + group;
                        uint16_t* out = reinterpret_cast<uint16_t*>(a.h) + at * 32 * RT;
#pragma unroll
                        for (int t = 0; t < RT; ++t) {
                            uint32_t w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) w[e] = split_halves(v[t][e], ex);
                            *(__attribute__((address_space(1))) u32x2*)(out + 16 * t + 4 * c) =
                                u32x2{__builtin_amdgcn_perm(w[1], w[0], HI), __builtin_amdgcn_perm(w[3], w[2], HI)};
                            *(__attribute__((address_space(1))) u32x2*)(out + 16 * RT + 16 * t + 4 * c) =
                                u32x2{__builtin_amdgcn_perm(w[1], w[0], LO), __builtin_amdgcn_perm(w[3], w[2], LO)};
                        }
                        if (c == 0) *gptr(a.exps + at) = -ex;
                    }
                }
            }
            __syncthreads();
        }
    }
}

// The columns of a wave's J output tiles, 16 J adjacent ones of one segment.
// The four results that a lane has of a tile are adjacent columns; two tiles
// side by side give a lane eight, and the four lanes of a row 64 adjacent bytes.
template <int J>
struct Cols {
    // first column of the results of lane group c in tile j
    static __device__ __forceinline__ constexpr int at(int c, int j) {
        return j < (J & ~1) ? 32 * (j >> 1) + 8 * c + 4 * (j & 1) : 16 * j + 4 * c;
    }
    // column of row mm of tile j's matrix operand
    static __device__ __forceinline__ int row(int mm, int j) { return at(mm >> 2, j) + (mm & 3); }
    // whole: 16-byte aligned, all columns inside the segment (else the first `left`)
    static __device__ __forceinline__ void load(uint32_t (&v)[2 * J], const uint16_t* p, int c, int left, bool whole) {
        if (whole) {
#pragma unroll
            for (int j = 0; j + 1 < J; j += 2) {
                const uint4 q = load16(p + at(c, j));
                v[2 * j] = q.x, v[2 * j + 1] = q.y, v[2 * j + 2] = q.z, v[2 * j + 3] = q.w;
            }
            if constexpr (J % 2) {
                const uint2 q = gload_u2(reinterpret_cast<const uint2*>(p + at(c, J - 1)));
                v[2 * J - 2] = q.x, v[2 * J - 1] = q.y;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4 * J; ++e) {
                const int n = at(c, e >> 2) + (e & 3);
                const uint32_t t = n < left ? (uint32_t)*gptr(p + n) << (16 * (e & 1)) : 0;
                v[e >> 1] = e & 1 ? v[e >> 1] | t : t;
            }
        }
    }
    static __device__ __forceinline__ void store(const uint32_t (&v)[2 * J], uint16_t* p, int c, int left, bool whole) {
        if (whole) {
#pragma unroll
            for (int j = 0; j + 1 < J; j += 2)
                gstore_u4(reinterpret_cast<uint4*>(p + at(c, j)), make_uint4(v[2 * j], v[2 * j + 1], v[2 * j + 2], v[2 * j + 3]));
            if constexpr (J % 2)
                *(__attribute__((address_space(1))) u32x2*)(p + at(c, J - 1)) = u32x2{v[2 * J - 2], v[2 * J - 1]};
        } else {
#pragma unroll
            for (int e = 0; e < 4 * J; ++e) {
                const int n = at(c, e >> 2) + (e & 3);
                if (n < left) *gptr(p + n) = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
            }
        }
    }
    // fp16(base + s d) of a row's results
    static __device__ __forceinline__ void add(uint32_t (&v)[2 * J], const f4 (&d)[J], float s) {
#pragma unroll
        for (int e = 0; e < 2 * J; ++e) {
            const h2 b = as_h2(v[e]);
            v[e] = (uint32_t)f_to_h(fmaf(d[e >> 1][2 * (e & 1)], s, (float)b[0])) |
                   (uint32_t)f_to_h(fmaf(d[e >> 1][2 * (e & 1) + 1], s, (float)b[1])) << 16;
        }
    }
};

// Segment and first output column of this workgroup's tile (blockIdx.x).
__device__ __forceinline__ int tile_segment(const LoraArgs& a, int width, int& n0) {
    int seg = 0;
#pragma unroll
    for (int i = 1; i < WOQ_MAX_SEGMENTS; ++i)
        if (i < a.nseg && (int)blockIdx.x >= a.tile0[i]) seg = i;
    n0 = (seg ? a.seg_end[seg - 1] : 0) + ((int)blockIdx.x - a.tile0[seg]) * width;
    return seg;
}

// The outer products of few rows: 16 rows x 64 outputs of one segment per
// workgroup of four waves, one output tile a wave.  Each adapter of the 16 rows
// gives a tile of results, of which its rows keep theirs.  A step is 16 ranks of
// one adapter; the operands of the next 2 U steps are always on their way.
// ONE: no adapter has more ranks than a step (R <= 16); then all rows' steps are
// independent and run four at a time without a branch between them (64 rows of 64
// adapters of rank 16 beside 10240 outputs: 9.6 us against 11.4).
template <bool ONE>
__global__ __launch_bounds__(256, 4) void lora_up_rows_kernel(LoraArgs a) {
    constexpr int TM = 16, U = 8;
    using C = Cols<1>;
    extern __shared__ __align__(16) uint32_t hp[];     // [TM][Rp + 4]: hi | lo << 16
    __shared__ int sexp[TM];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int m = lane & 15, c = lane >> 4;
    const int Rp = (a.R + 15) & ~15, ldh = Rp + 4;
    int n0;
    const int seg = tile_segment(a, 64, n0), r0 = blockIdx.y * TM, rows = min(a.b - r0, TM);
    const int nw = n0 + 16 * wave, left = a.seg_end[seg] - nw;      // this wave's columns
    const bool whole = a.vec && (n0 & 7) == 0 && left >= 16;
    Window<1, false> win;
    win.read(a, r0, rows, lane);
    uint32_t v[2] = {0, 0};
    if (a.base && m < rows) C::load(v, a.base + (int64_t)(r0 + m) * a.ldbase + nw, c, left, whole);

    // h, 16 threads a row: the K ranges' sums of four ranks, added in order.
    // They are read before it is known what the row's adapter has of them (a
    // row without one has none in the workspace): what it has not is dropped.
    const int r = tid >> 4, q = tid & 15;
    uint32_t* row = hp + r * ldh;
    const float* hr = a.h + ((int64_t)(r0 + min(r, rows - 1)) * a.nseg + seg) * a.R;
    const int64_t range = (int64_t)a.b * a.nseg * a.R;
    for (int j = 4 * q; j < a.R; j += 64) {
        f4 s = {0.f, 0.f, 0.f, 0.f};
        for (int z = 0; z < a.splits; z += 8) {        // eight loads in flight
            f4 p[8];
#pragma unroll
            for (int u = 0; u < 8; ++u)
                p[u] = *(__attribute__((address_space(1))) const f4*)(hr + min(z + u, a.splits - 1) * range + j);
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (z + u < a.splits) s += p[u];
        }
        *(f4*)(row + j) = s;
    }

    // the distinct adapters of the rows, the k-th in lane k
    int list = 0, count = 0, most = 0;
    for (u64 rest = __ballot(win.ids[0] >= 0); rest; ++count) {
        const int id = __builtin_amdgcn_readlane(win.ids[0], __ffsll(rest) - 1);
        rest &= ~__ballot(win.ids[0] == id);
        if (lane == count) list = id;
        most = max(most, rank_of(a, id));
    }
    const int groups = (most + 15) >> 4, steps = left > 0 ? count * groups : 0;
    // B in the order it lies in memory: one load has the 32 pieces of 16 bytes of
    // one step in the lower lanes and those of the next in the upper ones
    const int brow = min((lane & 31) >> 1, left - 1);
    const uint16_t* bp = a.B + ((int64_t)nw + brow) * a.R + 8 * (lane & 1);
    int lk = 0, lt = 0;                                // the next step to load
    auto load_b = [&](uint4& to) {
        int id[2], tt[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            id[e] = __builtin_amdgcn_readlane(list, lk);
            tt[e] = lt;
            if (++lt == groups) lt = 0, ++lk;
            lk = min(lk, count - 1);                   // past the end the last adapter again
        }
        const bool up = lane >= 32;
        const int left_k = (up ? rank_of(a, id[1]) - 16 * tt[1] : rank_of(a, id[0]) - 16 * tt[0]) - 8 * (lane & 1);
        const int64_t at = (int64_t)(up ? id[1] : id[0]) * a.N * a.R + 16 * (up ? tt[1] : tt[0]);
        to = make_uint4(0, 0, 0, 0);
        if (left_k > 0) to = load16(bp + at);
        if (left_k < 8) {                              // ranks that the adapter has not
            uint32_t w[4] = {to.x, to.y, to.z, to.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] &= (left_k > 2 * e ? 0xFFFFu : 0u) | (left_k > 2 * e + 1 ? 0xFFFF0000u : 0u);
            to = make_uint4(w[0], w[1], w[2], w[3]);
        }
    };
    uint4 bv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        bv[u] = make_uint4(0, 0, 0, 0);
        if (2 * u < steps) load_b(bv[u]);
    }
    const int mine = __shfl(win.ids[0], m);
    const float scale = mine >= 0 ? *gptr(a.scale + mine) : 0.f;

    {   // what the row has of h, scaled by a power of two, in two halves
        const int own = __shfl(win.ids[0], r);
        const int rk = own >= 0 ? rank_of(a, own) : 0;
        uint32_t big = 0;
        for (int j = 4 * q; j < Rp; j += 64) {
            f4 s = *(const f4*)(row + j);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (j + e >= rk) s[e] = 0.f;
                big = max(big, __float_as_uint(s[e]) & 0x7FFFFFFFu);
            }
            *(f4*)(row + j) = s;
        }
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) big = max(big, (uint32_t)__shfl_xor((int)big, d));
        const int ex = scale_exponent(big);
        for (int j = 4 * q; j < Rp; j += 64) {
            const f4 s = *(const f4*)(row + j);
            *(u32x4*)(row + j) = u32x4{split_halves(s[0], ex), split_halves(s[1], ex), split_halves(s[2], ex), split_halves(s[3], ex)};
        }
        if (q == 0) sexp[r] = -ex;
    }
    __syncthreads();

    f4 acc = {0.f, 0.f, 0.f, 0.f}, d[1] = {acc};
    int k = 0, t = 0;
    const uint32_t sel = c < 2 ? HI : LO;
    // the operand of lane (m, c) in a step: row m, piece c & 1
    auto operand = [&](uint4 pair, int e) {
        const int from = 32 * e + 2 * m + (c & 1);
        return as_h8(make_uint4(__shfl((int)pair.x, from), __shfl((int)pair.y, from), __shfl((int)pair.z, from),
                                __shfl((int)pair.w, from)));
    };
    auto halves = [&](int t) {
        const uint32_t* hw = hp + m * ldh + 16 * t + 8 * (c & 1);
        const u32x4 p0 = *(const u32x4*)hw, p1 = *(const u32x4*)(hw + 4);
        return as_h8(make_uint4(__builtin_amdgcn_perm(p0[1], p0[0], sel), __builtin_amdgcn_perm(p0[3], p0[2], sel),
                                __builtin_amdgcn_perm(p1[1], p1[0], sel), __builtin_amdgcn_perm(p1[3], p1[2], sel)));
    };
    if constexpr (ONE) {
        const h8 hv = halves(0);
#pragma unroll
        for (int u = 0; u < U; u += 2) {
            if (2 * u >= steps) continue;
            // (steps past the last adapter: no row takes their results)
            f4 r4[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                r4[e] = __builtin_amdgcn_mfma_f32_16x16x32_f16(operand(bv[u + e / 2], e & 1), hv, f4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (2 * u + e < steps && mine == __builtin_amdgcn_readlane(list, 2 * u + e)) d[0] = r4[e];
        }
    }
    for (int s = 0; !ONE && s < steps; s += 2 * U) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s + 2 * u >= steps) continue;
            const uint4 pair = bv[u];
            if (s + 2 * u + 2 * U < steps) load_b(bv[u]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (s + 2 * u + e >= steps) continue;
                acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(operand(pair, e), halves(t), acc, 0, 0, 0);
                if (++t == groups) {
                    if (mine == __builtin_amdgcn_readlane(list, k)) d[0] = acc;
                    acc = f4{0.f, 0.f, 0.f, 0.f};
                    t = 0, ++k;
                }
            }
        }
    }
    if (left <= 0 || m >= rows || (mine < 0 && a.base == a.y && a.ldbase == a.ldy)) return;
    if (mine >= 0) {
        const int ex = sexp[m];
#pragma unroll
        for (int e = 0; e < 4; ++e) d[0][e] = ldexpf(d[0][e], ex);
        C::add(v, d, scale);
    }
    C::store(v, a.y + (int64_t)(r0 + m) * a.ldy + nw, c, left, whole);
}

// The outer products of windows: 64 rows, 16 to each of four waves, x 64
// outputs at a time, over a.per such tiles; h comes scaled and split and stays in
// registers.  One adapter of the rows after another, each writing its own rows.
//
// h is the first matrix operand and B the second, with column m of its tile j
// the output 4 m + j: a lane then has four adjacent outputs of four rows, and
// the 16 lanes of a row 128 adjacent bytes.  B is read in the order it lies in
// memory, once for the four waves, and passes through LDS into operand order.
// (A lane-per-row access costs the address unit a lookup per lane: with it for
// B, base and y this kernel took 125 us, 3001 rows, 28672 outputs, rank 64; with
// 32 rows and a B of its own to each wave, and so only two waves on a SIMD, 110;
// now 90, where copying base to y takes 65.  Two adapters of a window in one pass
// measured 114: the registers cost more than the second pass.)
template <int RT, bool MULTI>
__global__ __launch_bounds__(256, 4) void lora_up_wide_kernel(LoraArgs a) {
    constexpr int J = 4, TM = 64, TN = 16 * J;
    constexpr int NB = RT == 1 ? 1 : RT / 2;           // steps of 32 ranks (of 16: one, both halves at once)
    constexpr int CH = 2 * RT, NP = (TN * CH + 255) / 256;   // 16-byte pieces of a row of B, of a thread
    __shared__ __align__(16) uint8_t lds[2][TN * 32 * RT];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int m = lane & 15, c = lane >> 4;
    int n_first;
    const int seg = tile_segment(a, TN * a.per, n_first), hi = a.seg_end[seg];
    const int r0 = blockIdx.y * TM, rows = min(a.b - r0, TM);
    const int tiles = min(a.per, (hi - n_first + TN - 1) / TN), groups = MULTI ? a.groups : 1;
    const bool vec = a.vec && (n_first & 3) == 0;
    Window<1, true> win;
    win.read(a, r0, rows, lane);

    // a lane's rows 16 wave + 4 c + e, its columns 4 m .. 4 m + 3 of the tile
    const int row0 = 16 * wave + 4 * c, hrow = __shfl(win.row[0], 16 * wave + m);
    int row[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) row[e] = __shfl(win.row[0], row0 + e);
    // a row's offset is worked out at each use (the empty asm): kept, the offsets
    // of four rows of base and y cost the registers that the loads ahead need
    auto at = [](const uint16_t* p, int r, int64_t ld, int n) {
        asm("" : "+v"(r));
        return p + r * ld + n;
    };
    const int n_lane = n_first + 4 * m;
    uint2 v[4];
    auto load_base = [&](int i, uint32_t of) {         // bit e of `of`: row[e]
        const int left = hi - n_first - i * TN - 4 * m;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] = make_uint2(0, 0);
            if (!a.base || !(of >> e & 1)) continue;
            const uint16_t* p = at(a.base, row[e], a.ldbase, n_lane + i * TN);
            if (vec && left >= 4) {
                v[e] = gload_u2(reinterpret_cast<const uint2*>(p));
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < left) (j < 2 ? v[e].x : v[e].y) |= (uint32_t)*gptr(p + j) << (16 * (j & 1));
            }
        }
    };
    auto store = [&](int i, uint32_t of) {
        const int left = hi - n_first - i * TN - 4 * m;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (!(of >> e & 1)) continue;
            uint16_t* p = const_cast<uint16_t*>(at(a.y, row[e], a.ldy, n_lane + i * TN));
            if (vec && left >= 4) {
                *(__attribute__((address_space(1))) u32x2*)p = u32x2{v[e].x, v[e].y};
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < left) *gptr(p + j) = (uint16_t)((j < 2 ? v[e].x : v[e].y) >> (16 * (j & 1)));
            }
        }
    };
    // position of piece ch of row `row` of B in LDS: eight lanes that read together
    // (rows 4 m + j, one piece) fall on different banks
    auto place = [](int row, int ch) {
        return row * 32 * RT + 16 * (ch ^ (RT == 4 ? row >> 2 & 7 : RT == 2 ? row >> 2 & 3 : row >> 2 & 1));
    };
    const int ch = tid % CH, brow = tid / CH;          // this thread's piece of B, and those 256 / CH rows apart

    // what the workspace holds of a row's h: rows of other adapters, or without
    // one, may hold anything (their results are dropped)
    h8 hv[RT];
    int ex[4];
    auto load_h = [&](int g) {
        const uint16_t* p = reinterpret_cast<const uint16_t*>(a.h) + (((int64_t)hrow * a.nseg + seg) * groups + g) * 32 * RT + 8 * c;
#pragma unroll
        for (int t = 0; t < RT; ++t) hv[t] = as_h8(load16(p + 32 * t));
#pragma unroll
        for (int e = 0; e < 4; ++e)
            ex[e] = *gptr(a.exps + ((int64_t)row[e] * a.nseg + seg) * groups + g);
    };
    // neither of these waits for the adapters to be known
    load_h(0);
    load_base(0, (uint32_t)(~0ull >> (64 - rows) >> row0) & 15u);
    bool once = true;
    u64 rest = __ballot(win.ids[0] >= 0);
    const u64 plain = __ballot(lane < rows) & ~rest;
    int turn = 0;
    while (rest) {
        const int id = __builtin_amdgcn_readlane(win.ids[0], __ffsll(rest) - 1);
        const u64 all = __ballot(win.ids[0] == id);
        rest &= ~all;
        const bool mine = all >> (16 * wave) & 0xFFFF;  // this wave has rows of it
        const uint32_t of = (uint32_t)(all >> row0) & 15u;
        const int rank = rank_of(a, id), used = MULTI ? max(1, (rank + 16 * RT - 1) / (16 * RT)) : 1;
        const float scale = *gptr(a.scale + id);

        uint4 bq[NP];
        auto load_b = [&](int i, int g) {
            // whole pieces of the rows that there are; ranks that the adapter has not
            // are cut off when the pieces are staged
            const int k = 16 * g * RT;
            const bool some = k + 8 * ch < rank && brow < TN;
#pragma unroll
            for (int q = 0; q < NP; ++q) {
                const int n = min(n_first + i * TN + brow + 256 / CH * q, hi - 1);
                bq[q] = load16(some ? a.B + ((int64_t)id * a.N + n) * a.R + k + 8 * ch : a.B);
            }
        };
        auto stage_b = [&](uint8_t* mem, int g) {
            const int left = rank - 16 * g * RT - 8 * ch;
            if (left < 8) {
#pragma unroll
                for (int q = 0; q < NP; ++q) {
                    uint32_t w[4] = {bq[q].x, bq[q].y, bq[q].z, bq[q].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[e] &= (left > 2 * e ? 0xFFFFu : 0u) | (left > 2 * e + 1 ? 0xFFFF0000u : 0u);
                    bq[q] = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            if (brow < TN) {
#pragma unroll
                for (int q = 0; q < NP; ++q)
                    *(__attribute__((address_space(3))) u32x4*)(mem + place(brow + 256 / CH * q, ch)) =
                        u32x4{bq[q].x, bq[q].y, bq[q].z, bq[q].w};
            }
        };
        load_b(0, 0);
        if (MULTI || !once) load_h(0);
        if (!once) load_base(0, of);
        once = false;
        float s[4];                                    // scale and the power of two of a lane's rows
        auto scales = [&]() {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[e] = ldexpf(scale, rank ? ex[e] : 0);
                // a finite scale stays finite: sums of zero have to stay zero
                if (__builtin_isinf(s[e]) && !__builtin_isinf(scale)) s[e] = copysignf(3.4028235e38f, scale);
            }
            // an adapter of rank 0 left nothing there
            if (rank == 0) {
#pragma unroll
                for (int t = 0; t < RT; ++t) hv[t] = h8{};
            }
        };
        scales();
        for (int i = 0; i < tiles; ++i) {
            f4 sum[J];
            for (int g = 0; g < used; ++g, turn ^= 1) {
                uint8_t* mem = lds[turn];
                stage_b(mem, g);
                const bool last = g + 1 == used;
                load_b(last ? min(i + 1, tiles - 1) : i, last ? 0 : g + 1);
                __syncthreads();
                if (mine) {
#pragma unroll
                    for (int j = 0; j < J; ++j) {
                        f4 acc = {0.f, 0.f, 0.f, 0.f};
                        h8 bv[NB];
#pragma unroll
                        for (int t = 0; t < NB; ++t)
                            bv[t] = __builtin_bit_cast(h8, *(const __attribute__((address_space(3))) u32x4*)(mem + place(4 * m + j, RT == 1 ? c & 1 : 4 * t + c)));
#pragma unroll
                        for (int t = 0; t < RT; ++t)   // the hi halves of all ranks, then the lo
                            acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(hv[t], bv[t % NB], acc, 0, 0, 0);
                        if constexpr (MULTI) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) sum[j][e] = g ? fmaf(acc[e], s[e], sum[j][e]) : acc[e] * s[e];
                        } else {
                            sum[j] = acc;
                        }
                    }
                }
                if constexpr (MULTI) {
                    load_h(last ? 0 : g + 1);
                    scales();
                }
            }
            if (mine) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const h2 b0 = as_h2(v[e].x), b1 = as_h2(v[e].y);
                    const float f = MULTI ? 1.f : s[e];
                    v[e].x = (uint32_t)f_to_h(fmaf(sum[0][e], f, (float)b0[0])) | (uint32_t)f_to_h(fmaf(sum[1][e], f, (float)b0[1])) << 16;
                    v[e].y = (uint32_t)f_to_h(fmaf(sum[2][e], f, (float)b1[0])) | (uint32_t)f_to_h(fmaf(sum[3][e], f, (float)b1[1])) << 16;
                }
                store(i, of);
                if (i + 1 < tiles) load_base(i + 1, of);
            }
        }
    }
    // rows without an adapter
    const uint32_t bare = (uint32_t)(plain >> row0) & 15u;
    if (!(plain >> (16 * wave) & 0xFFFF) || (a.base == a.y && a.ldbase == a.ldy)) return;
    for (int i = 0; i < tiles; ++i) {
        load_base(i, bare);
        store(i, bare);
    }
}

// Rows that a workgroup per row may serve: as many as its waves look over.
constexpr int LEADER_ROWS = 256;

// A workgroup per row (which reads an adapter's A once for 16 of its rows, wherever
// they are, and its B once for each 16 rows of the batch that have one of it)
// or windows of rows (which read each of their adapters once, but with the long K
// of few windows on few compute units).  Both launches, us, row by row | windows, 1
// to 16 adapters, rows of one side by side or not:
//   64 rows:  12-18 | 16-35 (10240 x 8192, rank 16), 17-51 | 21-48 (28672 x 3584, rank 64)
//   128 rows: 15-22 | 16-27, 27-87 | 22-41, and 20-31 | 15-28 (28672 x 3584, rank 16)
//   192 rows: 21-29 | 19-26, 36-125 | 25-47, 26-40 | 18-33; 19-31 | 28-34 (3584 x 14336)
//   256 rows: 23-34 | 19-24, 41-163 | 26-43, 31-51 | 19-29; 23-36 | 28-34, 12-21 | 12-18 (1024 x 1024)
// so wide outputs make windows of 97 rows and more; with fewer than eight rows to an
// adapter they lose again (128 rows, 64 adapters: 25-34 | 62-66, 28672 x 3584, rank 16).
bool row_by_row(const LoraArgs& a) {
    if (a.b > LEADER_ROWS) return false;
    return a.b <= 96 || (int64_t)a.b * a.N <= 1 << 21 || 8 * (int64_t)a.count > a.b;
}

// K ranges of a row's inner products, at most, in that form.
constexpr int LEADER_SPLITS = 16;

// Whether windows take the rows in order of their adapters: one more launch, 3.3 us
// at 256 rows, 5 at 4096 and 10 at 16384, against windows that go through every adapter of a batch
// whose rows lie mixed (4096 rows beside 28672 x 3584, rank 64: 16 adapters 910 -> 159 us,
// 8 487 -> 149, 4 274 -> 142; 1021 rows: 254 -> 65, 138 -> 58, 78 -> 56; 384 rows: 133 ->
// 52, 71 -> 37, 42 -> 33).  Packed prompts, whose rows lie in order, gain nothing: below
// this bound they are left as they are.
bool in_order(const LoraArgs& a) { return (int64_t)(a.count - 1) * a.b >= 4096; }

// 16-rank tiles that a window's workgroup takes together.
int rank_tiles(int64_t R) { return R <= 16 ? 1 : R <= 32 ? 2 : 4; }

// K ranges that leave every wave of a few rows' workgroups one round of loads, four
// pieces of 64 channels; fewer where the workgroups that find work would be over three
// to a compute unit, which is what their registers leave room for (64 rows of 8192,
// three segments, an adapter each: 12.3 -> 11.5 us).
int k_ranges(const LoraArgs& a) {
    const int64_t units = (int64_t)std::min(a.b, a.count + a.b / 16 + 1) * a.nseg * a.groups;
    const int64_t room = std::max<int64_t>(1, 3 * woq::compute_units() / units);
    return (int)std::min<int64_t>(std::min<int64_t>(woq::ceil_div(a.K, 4 * 4 * 64), LEADER_SPLITS), room);
}

hipError_t launch(const void* kernel, dim3 grid, int threads, size_t lds, hipStream_t s, LoraArgs a) {
    void* argv[] = {&a};
    return hipLaunchKernel(kernel, grid, dim3((unsigned)threads), argv, lds, s);
}

// Output tiles of `width` columns, counted segment by segment.
unsigned count_tiles(LoraArgs& a, int width) {
    a.tile0[0] = 0;
    for (int i = 0; i < a.nseg; ++i)
        a.tile0[i + 1] = a.tile0[i] + (int)woq::ceil_div(a.seg_end[i] - (i ? a.seg_end[i - 1] : 0), width);
    return (unsigned)a.tile0[a.nseg];
}

hipError_t launch_few(LoraArgs a, hipStream_t s) {
    a.groups = (int)woq::ceil_div(a.R, 16);
    a.splits = k_ranges(a);
    hipError_t e = launch(reinterpret_cast<const void*>(&lora_down_kernel<4, 1, 4, true>),
                          dim3((unsigned)a.b, (unsigned)(a.nseg * a.groups), (unsigned)a.splits), 256, 0, s, a);
    if (e != hipSuccess) return e;
    const unsigned tiles = count_tiles(a, 64);
    return launch(a.R <= 16 ? reinterpret_cast<const void*>(&lora_up_rows_kernel<true>)
                            : reinterpret_cast<const void*>(&lora_up_rows_kernel<false>), dim3(tiles, (unsigned)woq::ceil_div(a.b, 16)), 256,
                  (size_t)16 * (woq::round_up(a.R, 16) + 4) * 4, s, a);
}

template <int RT, int D>
hipError_t launch_many(LoraArgs a, hipStream_t s) {
    a.groups = (int)woq::ceil_div(a.R, 16 * RT);
    a.exps = reinterpret_cast<int32_t*>(a.h) + (int64_t)a.b * a.nseg * a.groups * 16 * RT;
    hipError_t e = hipSuccess;
    if (in_order(a)) {
        a.order = a.exps + (int64_t)a.b * a.nseg * a.groups;
        e = launch(reinterpret_cast<const void*>(&lora_order_kernel), dim3(1), BINS, 0, s, a);
        if (e != hipSuccess) return e;
    }
    // workgroups of a window, which take its adapters in turn, as long as that is two
    // to a compute unit; those that find none left cost their start.  Eight against one,
    // beside 1024 x 1024, rank 16, 8 adapters: 2048 rows 14.6 us and 15.1 (two 14.1),
    // 16384 rows 56 and 36; 2048 rows beside 8192 x 3584 in three segments 35 and 29
    const int64_t windows = woq::ceil_div(a.b, 32), each = windows * a.nseg * a.groups;
    const int slots = (int)std::max<int64_t>(1, std::min<int64_t>({8, a.count, 2 * woq::compute_units() / each}));
    e = launch(reinterpret_cast<const void*>(&lora_down_kernel<8, RT, D, false>),
                          dim3((unsigned)windows, (unsigned)(a.nseg * a.groups), (unsigned)slots), 512, 0, s, a);
    if (e != hipSuccess) return e;
    // tiles a workgroup goes through: more where there is work enough for the device
    const int64_t rows = woq::ceil_div(a.b, 64);
    a.per = (int)std::max<int64_t>(1, std::min<int64_t>(4, rows * woq::ceil_div(a.N, 64) / 1024));
    // counted before the call: the launch takes a copy of a, tile0 included, and the
    // order in which arguments are made is not defined
    const unsigned tiles = count_tiles(a, 64 * a.per);
    return launch(a.groups > 1 ? reinterpret_cast<const void*>(&lora_up_wide_kernel<RT, RT == 4>)
                               : reinterpret_cast<const void*>(&lora_up_wide_kernel<RT, false>),
                  dim3(tiles, (unsigned)rows), 256, 0, s, a);
}

int check_lora_w(const woq_lora_w* w) {
    if (!w || w->N < 0 || w->K < 1 || w->R < 1 || w->count < 0 || w->lda < w->K) return WOQ_EINVAL;
    if (w->nseg < 1 || w->nseg > WOQ_MAX_SEGMENTS || w->seg_end[w->nseg - 1] != w->N) return WOQ_EINVAL;
    for (int i = 0; i < w->nseg; ++i)
        if (w->seg_end[i] < (i ? w->seg_end[i - 1] : 0)) return WOQ_EINVAL;
    return WOQ_OK;
}

}  // namespace

namespace woq {

int lora_check(const woq_lora_w* w, const uint16_t* x, int64_t ldx, const int32_t* ids, int64_t b,
               const uint16_t* base, int64_t ldbase, const uint16_t* y, int64_t ldy, const void* workspace,
               int64_t workspace_bytes) {
    const int rc = check_lora_w(w);
    if (rc != WOQ_OK) return rc;
    if (b < 0 || ldx < w->K || ldy < w->N || (base && ldbase < w->N)) return WOQ_EINVAL;
    if (b == 0 || w->N == 0) return WOQ_OK;
    if (!x || !ids || !y || !workspace || (w->count > 0 && (!w->A || !w->B || !w->scale))) return WOQ_EINVAL;
    if (!aligned16(x) || (ldx & 7) || ((uintptr_t)ids & 3u) || ((uintptr_t)y & 1u) || ((uintptr_t)base & 1u) ||
        !aligned16(workspace) || !aligned16(w->A) || !aligned16(w->B) || (w->lda & 7) ||
        ((uintptr_t)w->scale & 3u) || ((uintptr_t)w->rank & 3u))
        return WOQ_EALIGN;
    if ((w->R & 7) || w->R > WOQ_LORA_MAX_R || w->N > WOQ_LORA_MAX_N || w->K > (int64_t)INT32_MAX - 512 ||
        b > WOQ_LORA_MAX_ROWS)
        return WOQ_EUNSUPPORTED;
    return workspace_bytes < woq_lora_workspace(w, b) ? WOQ_EINVAL : WOQ_OK;
}

}  // namespace woq

extern "C" {

int64_t woq_lora_workspace(const woq_lora_w* w, int64_t b) {
    if (check_lora_w(w) != WOQ_OK || b < 0) return WOQ_EINVAL;
    if ((w->R & 7) || w->R > WOQ_LORA_MAX_R || b > WOQ_LORA_MAX_ROWS) return WOQ_EUNSUPPORTED;
    // row by row: the K ranges' sums; windows: halves, an exponent for each group of
    // ranks, and the order.  No less for more rows, so that one workspace serves
    // smaller batches.
    const int64_t few = std::min<int64_t>(b, LEADER_ROWS) * LEADER_SPLITS * w->nseg * w->R * 4;
    const int64_t width = 16 * rank_tiles(w->R), many = b * (w->nseg * woq::ceil_div(w->R, width) * (width * 4 + 4) + 4);
    return std::max<int64_t>(16, std::max(few, many));
}

int woq_lora_add(const woq_lora_w* w, const uint16_t* x, int64_t ldx, const int32_t* ids, int64_t b,
                 const uint16_t* base, int64_t ldbase, uint16_t* y, int64_t ldy, void* workspace,
                 int64_t workspace_bytes, void* stream) {
    const int rc = woq::lora_check(w, x, ldx, ids, b, base, ldbase, y, ldy, workspace, workspace_bytes);
    if (rc != WOQ_OK || b == 0 || w->N == 0) return rc;
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
    a.splits = a.groups = a.per = 1;
    a.exps = a.order = nullptr;
    a.vec = woq::aligned16(y) && (ldy & 7) == 0 && (!base || (woq::aligned16(base) && (ldbase & 7) == 0));
    for (int i = 0; i < WOQ_MAX_SEGMENTS; ++i) a.seg_end[i] = i < w->nseg ? (int)w->seg_end[i] : (int)w->N;
    hipStream_t s = (hipStream_t)stream;
    hipError_t e;
    if (row_by_row(a)) e = launch_few(a, s);
    else if (rank_tiles(a.R) == 1) e = launch_many<1, 4>(a, s);
    else if (rank_tiles(a.R) == 2) e = launch_many<2, 2>(a, s);
    else e = launch_many<4, 2>(a, s);
    if (e != hipSuccess) {
        woq::set_hip_error((int)e);
        return WOQ_EHIP;
    }
    return WOQ_OK;
}

}  // extern "C"
