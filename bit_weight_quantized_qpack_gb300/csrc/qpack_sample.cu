// qpack_sample.cu — the draw of the next token from its logits: temperature, top-k, top-p, min-p and a given random number.
//
// The mathematics. With m the row's maximum, w_i = e^{(x_i - m) / T}. Tokens are ordered by falling logit, the lowest index
// first among equals. Kept are: of the first k tokens, the shortest run from the top whose weights reach p of the sum over
// those k; of these, the ones with w_i >= min_p. The token drawn is the first one in order of index where the sum of kept
// weights passes u times their total.
//
// A token is told from its neighbour by the last place of a sum, so weights are integers: W_i = round(w_i 2^S), S = 46 or
// as many bits fewer as keep the sum of a row below 2^63. Sums of integers do not depend on their order: the same row
// gives the same token whatever the blocks do, and a draw differs from the one in exact arithmetic only where u lies
// within some 2^-44 of a border between two tokens. w itself comes from 2^y by a table of 2^(j / 256) and a polynomial in two-float
// arithmetic (a pair of fp32 whose sum is the value), to about 2^-43: fp64 would take some 20 operations of a unit that does
// 1/64 of fp32's rate.
//
// The kept tokens are found without sorting: a histogram of counts and weights over 2048 intervals of m - x shows the interval
// in which the k-th token or the p-th part of the sum lies, its tokens are gathered and ranked among each other; an
// interval of too many tokens is divided again by the bits of the logits, until its tokens are few or all equal.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "qpack_dev.cuh"
#include "qpack_launch.h"

namespace qpack {
namespace {

__device__ int g_fault_sample = 0;

constexpr int THREADS = 1024, WARPS = THREADS / 32;
constexpr int BINS = 2048;      // two a thread
constexpr int CAP = 1024;       // tokens ranked among each other

// ------------------------------------------------------------------------------------------------------------
// Weights
// ------------------------------------------------------------------------------------------------------------
constexpr int STEPS = 256;
struct Pow2Table {
    float hi[STEPS], lo[STEPS];
};
// 2^(j / 256), -128 <= j < 128, at j & 255: the exponential series in fp64, split into two fp32.
constexpr Pow2Table make_pow2_table() {
    Pow2Table t = {};
    for (int j = -STEPS / 2; j < STEPS / 2; ++j) {
        const double x = 0.6931471805599453094172321 * j / STEPS;
        double sum = 1.0, term = 1.0;
        for (int n = 1; n < 24; ++n) term = term * x / n, sum += term;
        const float hi = float(sum);
        t.hi[j & (STEPS - 1)] = hi;
        t.lo[j & (STEPS - 1)] = float(sum - double(hi));
    }
    return t;
}
__device__ const Pow2Table g_pow2 = make_pow2_table();

// log2(e) / T in two fp32, the row's maximum, and the binary places of a weight.
struct Heat {
    float hi, lo, top;
    int places;
};
// round(2^places e^{(x - top) / T}) for x <= top.
__device__ __forceinline__ unsigned long long weight(const Heat &h, const float2 *pow2, float x) {
    // d = x - top in two floats, exactly; y = d log2(e) / T. Products and sums are written out, so that none is contracted.
    const float d = __fsub_rn(x, h.top), v = __fsub_rn(d, x);
    const float d_lo = __fsub_rn(__fsub_rn(x, __fsub_rn(d, v)), __fadd_rn(h.top, v));
    const float y = __fmul_rn(d, h.hi);
    if (!(y > -48.0f)) return 0;                           // below half of a weight's last place; x = -inf
    const float y_lo = __fadd_rn(__fmaf_rn(d, h.hi, -y), __fmaf_rn(d, h.lo, __fmul_rn(d_lo, h.hi)));
    // y = n + j / 256 + r
    constexpr float magic = 12582912.0f / STEPS;           // 1.5 2^23 / 256: its last place is 1 / 256
    const float shifted = __fadd_rn(y, magic);
    const float r = __fsub_rn(y, __fsub_rn(shifted, magic));
    const int nj = __float_as_int(shifted) - __float_as_int(magic);
    const float2 t = pow2[nj & (STEPS - 1)];
    const int n = (nj + STEPS / 2) >> 8;
    // 2^(r + y_lo) - 1 = a + b: ln2 z + ln2^2 / 2 z^2 + ln2^3 / 6 z^3, |z| < 2^-8.9; the next term is below 2^-42
    constexpr float ln2_hi = 0.693147182464599609375f, ln2_lo = -1.904654299957767e-9f;
    const float z = __fadd_rn(r, y_lo);
    const float a = __fmul_rn(ln2_hi, r);
    const float square = __fmul_rn(__fmul_rn(z, z), __fmaf_rn(z, __fmaf_rn(z, 0.009618129107628477f, 0.05550410866482158f),
                                                              0.2402265069591007f));
    const float b = __fadd_rn(__fmaf_rn(ln2_hi, y_lo, __fmaf_rn(ln2_lo, r, __fmaf_rn(ln2_hi, r, -a))), square);
    // t (1 + a + b)
    const float c = __fmul_rn(t.x, a), sum = __fadd_rn(t.x, c);
    const float low = __fadd_rn(__fmaf_rn(t.x, a, -c), __fmaf_rn(t.x, b, __fmaf_rn(t.y, a, t.y)));
    const float rest = __fadd_rn(__fsub_rn(c, __fsub_rn(sum, t.x)), low);
    // in units of 2^-48: sum has 24 bits from 2^-1 or 2^0 on, |rest| < 2^-17
    const long long fixed = (static_cast<long long>(__float2int_rn(sum * 0x1p30f)) << 18) + __float2int_rn(rest * 0x1p48f);
    const int shift = 48 - h.places - n;                   // >= 2
    if (shift >= 50) return 0;
    return static_cast<unsigned long long>((fixed + (1ll << (shift - 1))) >> shift);
}

// Logits as unsigned numbers of the same order (-0 counts as +0).
__device__ __forceinline__ unsigned key_of(float x) {
    const unsigned u = __float_as_uint(x + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float of_key(unsigned k) { return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k); }

// floor(f * s) and ceil(f * s), 0 <= f < 1.
__device__ __forceinline__ unsigned long long part_of(float f, unsigned long long s, bool up) {
    const unsigned bits = __float_as_uint(f), e = bits >> 23;
    const unsigned long long mant = e ? (bits & 0x7FFFFFu) | 0x800000u : bits & 0x7FFFFFu;
    const int shift = 150 - int(e ? e : 1);                // f = mant 2^-shift, shift >= 24
    const unsigned __int128 prod = static_cast<unsigned __int128>(mant) * s;
    if (shift >= 127) return up && prod ? 1 : 0;
    const unsigned __int128 q = prod >> shift;
    return static_cast<unsigned long long>(q) + (up && (q << shift) != prod ? 1 : 0);
}

// ------------------------------------------------------------------------------------------------------------
// A row: vectors of 16 bytes, those at its ends element by element; what is not of the row reads as -inf.
// ------------------------------------------------------------------------------------------------------------
template <int DT> struct Logits {
    static constexpr int VE = DT == DT_F32 ? 4 : 8, ES = DT == DT_F32 ? 4 : 2;
    const unsigned char *base;  // aligned to 16 bytes, at or below the row's first element
    int skew, count, vectors;   // elements between base and the row, of the row, vectors that hold them

    __device__ __forceinline__ Logits(const void *row, int n) {
        const uintptr_t p = reinterpret_cast<uintptr_t>(row);
        base = reinterpret_cast<const unsigned char *>(p & ~uintptr_t(15));
        skew = int(p & 15) / ES, count = n, vectors = (skew + n + VE - 1) / VE;
    }
    __device__ __forceinline__ int index(int vec) const { return vec * VE - skew; }     // of its first element
    __device__ __forceinline__ void load(int vec, float (&x)[VE]) const {
        const int i0 = index(vec);
        if (vec < vectors && i0 >= 0 && i0 + VE <= count) {
            const uint4 v = *reinterpret_cast<const uint4 *>(base + int64_t(vec) * 16);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < VE; ++e) x[e] = value(w[e * ES / 4], e);
            return;
        }
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            x[e] = -INFINITY;
            if (vec < vectors && i0 + e >= 0 && i0 + e < count) {
                const unsigned char *p = base + int64_t(vec) * 16 + e * ES;
                x[e] = DT == DT_F32 ? *reinterpret_cast<const float *>(p) : value(*reinterpret_cast<const uint16_t *>(p), 0);
            }
        }
    }
    // element e of the word that holds it
    static __device__ __forceinline__ float value(uint32_t w, int e) {
        if (DT == DT_F32) return __uint_as_float(w);
        if (DT == DT_F16) return h2f_bits(uint16_t(e & 1 ? w >> 16 : w & 0xFFFFu));
        return __uint_as_float(e & 1 ? w & 0xFFFF0000u : w << 16);
    }
};

// ------------------------------------------------------------------------------------------------------------
// The kernel: a block a row
// ------------------------------------------------------------------------------------------------------------
struct Shared {
    float2 pow2[STEPS];
    unsigned count[BINS];
    unsigned w_lo[BINS], w_hi[BINS];
    unsigned keys[CAP];
    unsigned long long weights[CAP];
    unsigned long long scan64[WARPS], scan64b[WARPS];
    unsigned scan32[WARPS];
    unsigned long long best;
    int bad;
    unsigned listed, lo_key, hi_key;
    int bin;
    unsigned bin_count, found_key, found_ties;
    unsigned long long before_weight, sum_weight, goal;
    unsigned before_count;
};

// Exclusive sums over the block; *total: the sum. Every thread calls it.
template <class V> __device__ __forceinline__ V block_sum(V v, V *space, V *total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    V x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const V y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) space[w] = x;
    __syncthreads();
    if (w == 0) {
        V y = space[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const V z = __shfl_up_sync(0xffffffffu, y, o);
            if (lane >= o) y += z;
        }
        space[lane] = y;
    }
    __syncthreads();
    *total = space[WARPS - 1];
    return (w ? space[w - 1] : 0) + x - v;
}

// How a pass of the selection tells a token's interval: by m - x, or by key. Out of range: -1.
struct Intervals {
    float top, per;             // by distance: (top - x) per, the last interval takes the rest
    unsigned lo, hi;            // by key: lo <= key <= hi
    int shift;                  // < 0: by distance
    __device__ __forceinline__ int of(float x) const {
        if (x == -INFINITY) return -1;
        if (shift < 0) return int(fminf((top - x) * per, float(BINS - 1)));
        const unsigned k = key_of(x);
        return k < lo || k > hi ? -1 : int((hi - k) >> shift);
    }
};

template <int DT, bool WEIGH>
__device__ __forceinline__ void fill(Shared &s, const Logits<DT> &row, const Intervals &iv, const Heat &heat) {
    for (int i = threadIdx.x; i < BINS; i += THREADS) s.count[i] = s.w_lo[i] = s.w_hi[i] = 0;
    __syncthreads();
    for (int v = threadIdx.x; v < row.vectors; v += THREADS) {
        float x[Logits<DT>::VE];
        row.load(v, x);
#pragma unroll
        for (int e = 0; e < Logits<DT>::VE; ++e) {
            const int b = iv.of(x[e]);
            if (b < 0) continue;
            atomicAdd(&s.count[b], 1u);
            if (WEIGH) {
                const unsigned long long w = weight(heat, s.pow2, x[e]);
                const unsigned lo = unsigned(w), old = atomicAdd(&s.w_lo[b], lo);
                const unsigned carry = unsigned(w >> 32) + (old + lo < old);
                if (carry) atomicAdd(&s.w_hi[b], carry);
            }
        }
    }
    __syncthreads();
}

// Finds the token at which the running count (or weight) from the top reaches `goal`: its key, and how many of the tokens of
// that key are kept. before_*: what lies above the intervals of `iv`, which the histogram holds.
template <int DT, bool WEIGH>
__device__ __forceinline__ void select(Shared &s, const Logits<DT> &row, Intervals iv, const Heat &heat,
                                       unsigned long long goal) {
    const int tid = threadIdx.x;
    unsigned long long above = 0;                          // counts or weights above the intervals
    for (;;) {
        // the interval that reaches the goal
        unsigned long long mine[2], total;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            mine[i] = WEIGH ? (static_cast<unsigned long long>(s.w_hi[2 * tid + i]) << 32) + s.w_lo[2 * tid + i]
                            : s.count[2 * tid + i];
        unsigned long long at = above + block_sum(mine[0] + mine[1], s.scan64, &total);
        if (tid == 0) s.listed = 0, s.lo_key = 0xFFFFFFFFu, s.hi_key = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (at < goal && goal <= at + mine[i]) s.bin = 2 * tid + i, s.bin_count = s.count[2 * tid + i], s.before_weight = at;
            at += mine[i];
        }
        __syncthreads();
        const int bin = s.bin;
        const unsigned n = s.bin_count;
        above = s.before_weight;
        // its tokens
        unsigned lo = 0xFFFFFFFFu, hi = 0;
        for (int v = tid; v < row.vectors; v += THREADS) {
            float x[Logits<DT>::VE];
            row.load(v, x);
#pragma unroll
            for (int e = 0; e < Logits<DT>::VE; ++e) {
                if (iv.of(x[e]) != bin) continue;
                const unsigned k = key_of(x[e]);
                lo = min(lo, k), hi = max(hi, k);
                if (n <= CAP) s.keys[atomicAdd(&s.listed, 1u)] = k;
            }
        }
        lo = __reduce_min_sync(0xffffffffu, lo), hi = __reduce_max_sync(0xffffffffu, hi);
        if ((tid & 31) == 0) atomicMin(&s.lo_key, lo), atomicMax(&s.hi_key, hi);
        __syncthreads();
        lo = s.lo_key, hi = s.hi_key;
        if (lo == hi) {                                    // all alike
            if (tid == 0) {
                const unsigned long long w = WEIGH ? weight(heat, s.pow2, of_key(lo)) : 1;
                s.found_key = lo, s.found_ties = unsigned((goal - above + w - 1) / w);
            }
            break;
        }
        if (n <= CAP) {
            if (WEIGH && tid < n) s.weights[tid] = weight(heat, s.pow2, of_key(s.keys[tid]));
            __syncthreads();
            if (tid < n) {
                const unsigned k = s.keys[tid];
                unsigned long long over = above;
                unsigned same = 0;
                for (int i = 0; i < int(n); ++i) {
                    const unsigned o = s.keys[i];
                    if (o > k) over += WEIGH ? s.weights[i] : 1;
                    same += o == k;
                }
                const unsigned long long w = WEIGH ? s.weights[tid] : 1;
                if (over < goal && goal <= over + same * w)
                    s.found_key = k, s.found_ties = unsigned((goal - over + w - 1) / w);
            }
            break;
        }
        // too many: divide the interval by keys
        iv.lo = lo, iv.hi = hi;
        const int bits = 32 - __clz(hi - lo);
        iv.shift = max(0, bits - 11);
        fill<DT, WEIGH>(s, row, iv, heat);
    }
    __syncthreads();
}

template <int DT> __global__ void __launch_bounds__(THREADS, 1) sample_kernel(SampleArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    Shared &s = *reinterpret_cast<Shared *>(smem);
    constexpr int VE = Logits<DT>::VE;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int64_t b = blockIdx.x;
    if (tid < STEPS) s.pow2[tid] = make_float2(g_pow2.hi[tid], g_pow2.lo[tid]);
    if (tid == 0) s.best = 0, s.bad = 0;
    pdl_launch_dependents();
    pdl_wait();
    const Logits<DT> row(static_cast<const unsigned char *>(a.logits) + b * a.ld * Logits<DT>::ES, int(a.vocab));
    __syncthreads();

    // -- the maximum, at its lowest index --------------------------------------------------------------------
    unsigned long long best = 0;                           // key, then the index inverted
    bool bad = false;
    for (int v = tid; v < row.vectors; v += THREADS) {
        float x[VE];
        row.load(v, x);
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            bad |= !(x[e] < INFINITY);                     // NaN or +inf
            const unsigned long long k = static_cast<unsigned long long>(key_of(x[e])) << 32 | unsigned(~(row.index(v) + e));
            best = x[e] > -INFINITY && k > best ? k : best;
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) {
        if (best) atomicMax(&s.best, best);
        if (bad) s.bad = 1;
    }
    __syncthreads();
    best = s.best;
    const float given = a.temperature ? a.temperature[b] : 1.0f, heat_t = given > 0x1p64f ? 0x1p64f : given;
    if (s.bad || best == 0 || !(heat_t >= 0x1p-64f)) {
        if (tid == 0) {
            if (s.bad) atomicOr(&g_fault_sample, FAULT_NONFINITE_X);
            a.tokens[b] = s.bad || best == 0 ? -1 : int(~unsigned(best));
            if (a.probs) a.probs[b] = s.bad ? __int_as_float(0x7FC00000) : best == 0 ? 0.0f : 1.0f;
        }
        return;
    }
    Heat heat;
    {
        const double c = 1.4426950408889634 / double(heat_t);
        heat.hi = float(c), heat.lo = float(c - double(heat.hi));
        heat.top = of_key(unsigned(best >> 32));
        heat.places = a.places;
    }

    // -- the last token kept by top-k and top-p ---------------------------------------------------------------
    const int k = a.top_k ? a.top_k[b] : 0;
    const float p = a.top_p ? a.top_p[b] : 1.0f, min_p = a.min_p ? a.min_p[b] : 0.0f;
    bool cut_k = k > 0 && k < a.vocab;
    const bool cut_p = p < 1.0f;
    unsigned last_key = 0, last_ties = 0;                  // kept: keys above, and so many of this one (0: nothing cut)
    if (cut_k || cut_p) {
        Intervals iv;
        iv.top = heat.top, iv.per = BINS / fmaxf(32.0f, 32.0f * heat_t), iv.shift = -1;
        unsigned long long sum;
        if (cut_p) fill<DT, true>(s, row, iv, heat);
        else fill<DT, false>(s, row, iv, heat);
        if (cut_k) {
            unsigned total;
            block_sum(s.count[2 * tid] + s.count[2 * tid + 1], s.scan32, &total);
            cut_k = unsigned(k) < total;                   // masked tokens do not count
        }
        if (cut_k) {
            select<DT, false>(s, row, iv, heat, unsigned(k));
            last_key = s.found_key, last_ties = s.found_ties;
        }
        if (cut_p) {
            // the sum over the k tokens
            unsigned long long mine = 0;
            for (int v = tid; v < row.vectors; v += THREADS) {
                float x[VE];
                row.load(v, x);
#pragma unroll
                for (int e = 0; e < VE; ++e)
                    if (key_of(x[e]) > last_key) mine += weight(heat, s.pow2, x[e]);
            }
            block_sum(mine, s.scan64, &sum);
            if (cut_k) {
                sum += last_ties * weight(heat, s.pow2, of_key(last_key));
                fill<DT, true>(s, row, iv, heat);
            }
            const unsigned long long goal = max(1ull, part_of(fmaxf(p, 0.0f), sum, true));
            select<DT, true>(s, row, iv, heat, goal);
            last_key = s.found_key, last_ties = s.found_ties;
        }
    }
    const unsigned long long one = 1ull << heat.places;
    const unsigned long long least = min_p >= 1.0f ? one : min_p > 0.0f ? max(1ull, part_of(min_p, one, true)) : 1ull;
    const unsigned long long last_weight = last_ties ? weight(heat, s.pow2, of_key(last_key)) : 0;
    const bool ties_count = last_weight >= least;

    // -- sums of kept weights by warps' shares of the row, in order of index ---------------------------------------
    const int per = (row.vectors + WARPS - 1) / WARPS, v0 = w * per, v1 = min(v0 + per, row.vectors);
    auto kept = [&](float x, unsigned &ties) -> unsigned long long {
        const unsigned key = key_of(x);
        if (last_ties && key <= last_key) {
            ties += key == last_key;
            return 0;
        }
        const unsigned long long y = weight(heat, s.pow2, x);
        return y >= least ? y : 0;
    };
    unsigned long long sum = 0;
    unsigned ties = 0;
    for (int v = v0 + lane; v < v1; v += 32) {
        float x[VE];
        row.load(v, x);
#pragma unroll
        for (int e = 0; e < VE; ++e) sum += kept(x[e], ties);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    ties = __reduce_add_sync(0xffffffffu, ties);
    __syncthreads();
    if (lane == 0) s.scan64[w] = sum, s.scan32[w] = ties;
    __syncthreads();
    unsigned long long before = 0, total = 0;
    unsigned ties_before = 0, all_ties = 0;
    for (int i = 0; i < WARPS; ++i) {
        const unsigned here = min(s.scan32[i], last_ties - min(all_ties, last_ties));
        const unsigned long long add = s.scan64[i] + (ties_count ? here * last_weight : 0);
        if (i < w) before += add, ties_before += s.scan32[i];
        total += add, all_ties += s.scan32[i];
        if (i == w) sum = add;
    }
    const float u = fminf(fmaxf(a.u[b], 0.0f), 0x1.fffffep-1f);
    const unsigned long long goal = part_of(u, total, false);
    if (goal < before || goal >= before + sum) return;     // another warp's

    // -- the token -----------------------------------------------------------------------------------------------
    unsigned left = last_ties - min(ties_before, last_ties);
    unsigned long long run = before;
    for (int v = v0; v < v1; v += 32) {
        float x[VE];
        row.load(v + lane < v1 ? v + lane : row.vectors, x);
        unsigned t = 0;
        unsigned long long mine = 0;
#pragma unroll
        for (int e = 0; e < VE; ++e) mine += kept(x[e], t);
        unsigned t_scan = t;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned y = __shfl_up_sync(0xffffffffu, t_scan, o);
            if (lane >= o) t_scan += y;
        }
        unsigned may = left - min(left, t_scan - t);       // ties that this lane may keep
        mine += ties_count ? min(t, may) * last_weight : 0;
        unsigned long long scan = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long y = __shfl_up_sync(0xffffffffu, scan, o);
            if (lane >= o) scan += y;
        }
        const unsigned long long end = run + scan;
        if (goal >= end - mine && goal < end) {
            unsigned long long at = end - mine;
            for (int e = 0; e < VE; ++e) {
                unsigned tie = 0;
                unsigned long long y = kept(x[e], tie);
                if (tie && may) y = ties_count ? last_weight : 0, --may;
                if (goal < at + y) {
                    a.tokens[b] = row.index(v + lane) + e;
                    if (a.probs) a.probs[b] = float(double(y) / double(total));
                    break;
                }
                at += y;
            }
        }
        run += __shfl_sync(0xffffffffu, scan, 31);
        left -= min(left, __shfl_sync(0xffffffffu, t_scan, 31));
        if (goal < run) return;
    }
}

template <int DT> cudaError_t run(const SampleArgs &a, cudaStream_t s) {
    static int opted[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!opted[dev]) {
        e = cudaFuncSetAttribute(sample_kernel<DT>, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Shared));
        if (e != cudaSuccess) return e;
        opted[dev] = 1;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(a.rows));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = sizeof(Shared);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, sample_kernel<DT>, a);
}

}  // namespace

cudaError_t launch_sample(SampleArgs a, cudaStream_t s) {
    int bits = 0;
    while ((int64_t(1) << bits) < a.vocab) ++bits;
    a.places = 62 - bits < 46 ? 62 - bits : 46;
    return a.dt == DT_F32 ? run<DT_F32>(a, s) : a.dt == DT_F16 ? run<DT_F16>(a, s) : run<DT_BF16>(a, s);
}

cudaError_t fault_word_sample(int **word) {
    return cudaGetSymbolAddress(reinterpret_cast<void **>(word), g_fault_sample);
}

}  // namespace qpack
