// qpack_sample.cu — the draw of the next token from its logits: temperature, top-k, top-p, min-p and a given random
// number.
//
// The mathematics. With m the row's maximum, w_i = e^{(x_i - m) / T}. Tokens are ordered by falling logit, the lowest
// index first among equals. Kept are: of the first k tokens, the shortest run from the top whose weights reach p of
// the sum over those k; of these, the ones with w_i >= min_p. The token drawn is the first one in order of index
// where the sum of kept weights passes u times their total.
//
// A token is told from its neighbour by the last place of a sum, so weights are integers: W_i = round(w_i 2^S), S =
// 46 or as many bits fewer as keep the sum of a row below 2^63. Sums of integers do not depend on their order: the
// same row gives the same token whatever the blocks do, and a draw differs from the one in exact arithmetic only
// where u lies within some 2^-44 of a border between two tokens. w itself comes from 2^y by a table of 2^(j / 256)
// and a polynomial in two-float arithmetic (a pair of fp32 whose sum is the value), to about 2^-43: fp64 would take
// some 20 operations of a unit that does 1/64 of fp32's rate.
//
// The kept tokens are found without sorting: a histogram of counts and weights over 2048 intervals of m - x shows the
// interval in which the k-th token or the p-th part of the sum lies, its tokens are gathered and ranked among each
// other; an interval of too many tokens is divided again by the bits of the logits, until its tokens are few or all
// equal.
//
// What bounds it. A row is read from HBM once and from L2 some four times more (maximum, histogram, gathering, the
// sums of the draw), 64 rows of 128256 fp32 logits 33 MB (156 MB through L2): 5 us at the copy rate, 70 to 86 us as
// it is, by how many tokens the temperatures leave of weight. Schedulers are 57% busy, with some 220
// thread-instructions a token, of which a weight is some 50; the rest are passes over the tokens, shared atomics, two
// barriers of the row's blocks a pass, sums over 2048 intervals, and a launch's cold instruction cache. One row of
// 32000 is all latency: 25 us.
//
// A row is split over up to 8 blocks of a cluster, of 1024 threads, which read each other's totals in shared memory,
// as long as there are no more blocks than SMs; other rows take one block of 512 threads, two of which fit an SM (us
// for one row of 32000 / 64 of 128256 / 256 of 32000 unfiltered / 33 of 50257 of all kinds: a block of 1024 a row 48
// / 213 / 64 / 78, split 29 / 90 / 55 / 43, as it is 25 / 70 / 33 / 31; as it is but with twice the blocks, of 512
// threads, where a row is split 25 / 73 / 33 / 61). The rule has steps. us for rows of 32000 / 128256 without a
// filter: 38 rows 30 / 41 and 39 rows 15 / 32 (152 blocks in clusters of four seem not to find their SMs all at once;
// 78 in pairs do); 76 rows 16 / 33 and 77 rows 20 / 82 (from there on half of the SMs have a block of 512 until rows
// fill them all); 304 rows 31 / 123 and 305 rows 45 / 164.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cfloat>

#include "qpack_dev.cuh"
#include "qpack_launch.h"

namespace qpack {
namespace {

__device__ int g_fault_sample = 0;

constexpr int BINS = 2048;
constexpr int CAP = 1024;       // tokens ranked among each other
constexpr int MOST_BLOCKS = 8;  // a row's

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
__device__ const __align__(16) Pow2Table g_pow2 = make_pow2_table();

// log2(e) / T in two fp32, the row's maximum, and the binary places of a weight.
struct Heat {
    float hi, lo, top;
    int places;
};
// round(2^places e^{(x - top) / T}) for x <= top.
__device__ __forceinline__ unsigned long long weight(const Heat &h, const float *pow2, float x) {
    // d = x - top in two floats, exactly; y = d log2(e) / T. Products and sums are written out, so that none is
    // contracted.
    const float d = __fsub_rn(x, h.top);
    const float full = __fmul_rn(d, h.hi), y = fmaxf(full, -60.0f);
    float tail = __fmul_rn(d, h.lo);
    const float v = __fsub_rn(d, x);
    tail = __fmaf_rn(__fsub_rn(__fsub_rn(x, __fsub_rn(d, v)), __fadd_rn(h.top, v)), h.hi, tail);
    const float y_lo = __fadd_rn(__fmaf_rn(d, h.hi, -y), tail);
    // y = n + j / 256 + r
    constexpr float magic = 12582912.0f / STEPS;           // 1.5 2^23 / 256: its last place is 1 / 256
    const float shifted = __fadd_rn(y, magic);
    const float r = __fsub_rn(y, __fsub_rn(shifted, magic));
    const int nj = __float_as_int(shifted) - __float_as_int(magic);
    const float *entry = pow2 + (nj & (STEPS - 1)) * 32;
    const float2 t = make_float2(entry[0], entry[STEPS * 32]);
    const int n = (nj + STEPS / 2) >> 8;
    // 2^(r + y_lo) - 1 = a + b: ln2 z + ln2^2 / 2 z^2 + ln2^3 / 6 z^3 + ln2^4 / 24 z^4, |z| < 2^-8.9; the next term
    // is below 2^-54, and the limit is the rounding of the square and what follows it, together below 2^-19, to fp32:
    // some 2^-43
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
    // (sum + rest) 2^e: sum's 24 bits (from 2^-1 or 2^0 on) are a whole number where e is 24 or more, |rest| 2^e is
    // below 2^30; where e is less the sum of both is rounded at once
    const int e = h.places + n;
    const bool whole = e >= 24;
    const float part = (whole ? 0.0f : sum) + rest;
    // (below half of a weight's last place, x = -inf too: 0, since a NaN converts to it)
    const int low_part = __float2int_rn(part * (full > -48.0f ? __int_as_float((e + 127) << 23) : __int_as_float(0x7FC00000)));
    const unsigned high = whole ? unsigned(__float2int_rn(sum * 0x1p24f)) : 0u;
    return static_cast<unsigned long long>(high) * (1u << (max(e, 24) - 24)) + static_cast<long long>(low_part);
}

// The same by a call, where few tokens are weighed: the kernel's code is read cold by every launch.
__device__ __noinline__ unsigned long long weight_call(float hi, float lo, float top, int places, const float *pow2, float x) {
    const Heat h = {hi, lo, top, places};
    return weight(h, pow2, x);
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
    __device__ __forceinline__ bool inside(int vec) const { return vec >= (skew > 0) && vec < (skew + count) / VE; }
    // A vector's words: loaded where all of it is the row's, -inf else; `patch` puts in what there is of the ends.
    __device__ __forceinline__ uint4 words(int vec) const {
        constexpr uint32_t none = DT == DT_F32 ? 0xFF800000u : DT == DT_F16 ? 0xFC00FC00u : 0xFF80FF80u;
        uint4 v = make_uint4(none, none, none, none);
        if (inside(vec)) v = *reinterpret_cast<const uint4 *>(base + int64_t(vec) * 16);
        return v;
    }
    __device__ __forceinline__ void patch(int vec, float (&x)[VE]) const {
        if (inside(vec) || vec >= vectors) return;
        const int i0 = index(vec);
        for (int e = 0; e < VE; ++e)
            if (i0 + e >= 0 && i0 + e < count) {
                const float y = element(vec, e);
#pragma unroll
                for (int k = 0; k < VE; ++k) x[k] = k == e ? y : x[k];
            }
    }
    __device__ __forceinline__ float element(int vec, int e) const {           // one of the row's
        const unsigned char *p = base + int64_t(vec) * 16 + e * ES;
        return DT == DT_F32 ? *reinterpret_cast<const float *>(p) : value(*reinterpret_cast<const uint16_t *>(p), 0);
    }
    static __device__ __forceinline__ void widen(const uint4 &v, float (&x)[VE]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < VE; ++e) x[e] = value(w[e * ES / 4], e);
    }
    __device__ __forceinline__ void load(int vec, float (&x)[VE]) const {
        widen(words(vec), x);
        patch(vec, x);
    }
    // element e of the word that holds it
    static __device__ __forceinline__ float value(uint32_t w, int e) {
        if (DT == DT_F32) return __uint_as_float(w);
        if (DT == DT_F16) return h2f_bits(uint16_t(e & 1 ? w >> 16 : w & 0xFFFFu));
        return __uint_as_float(e & 1 ? w & 0xFFFF0000u : w << 16);
    }
};

// ------------------------------------------------------------------------------------------------------------
// The kernel: one to eight blocks a row, which read each other's shared memory
// ------------------------------------------------------------------------------------------------------------
struct Shared {
    float pow2[2][STEPS][32];   // high and low parts, once for each lane's bank: lanes ask for entries at random
    alignas(16) unsigned count[BINS];       // of the tokens in an interval,
    alignas(16) uint2 sums[BINS];           // or their weights: low and high words
    unsigned keys[CAP];         // of this block's tokens in the interval
    unsigned all_keys[CAP];     // of all blocks'
    unsigned long long weights[CAP];
    unsigned long long scan64[32];
    unsigned scan32[32];
    // what the blocks tell each other
    unsigned long long sum, kept;
    unsigned best, first, ties, listed, lo_key, hi_key;
    int bad;
    // what a thread tells its block
    int bin, share;
    unsigned found_key, found_ties;
    unsigned long long above;
};

// The largest of three; NaN where one is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

struct Cluster {
    unsigned rank, size;
    __device__ __forceinline__ Cluster() {
        asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
        asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(size));
    }
    __device__ __forceinline__ void sync() const {
        if (size == 1) __syncthreads();
        else asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    __device__ __forceinline__ uint2 read2(const unsigned *p, unsigned r) const {       // aligned to 8 bytes
        uint32_t at;
        uint2 v;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(r));
        asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
        return v;
    }
    // A word of block `lane`, or `none`: a warp asks all blocks at once (a loop over them waits for each).
    template <class V> __device__ __forceinline__ V read_lane(const V *p, V none) const {
        const unsigned r = threadIdx.x & 31;
        return r < size ? read(p, r) : none;
    }
    template <class V> __device__ __forceinline__ V read(const V *p, unsigned r) const {
        uint32_t at;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(r));
        if constexpr (sizeof(V) == 8) {
            unsigned long long v;
            asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(at) : "memory");
            return v;
        } else {
            unsigned v;
            asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
            return V(v);
        }
    }
};

// Exclusive sums over the block; *total: the sum. Every thread calls it.
template <int WARPS, class V> __device__ __forceinline__ V block_sum(V v, V *space, V *total) {
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
    V y = lane < WARPS ? space[lane] : 0;                  // every warp adds up all of them
#pragma unroll
    for (int o = 1; o < WARPS; o <<= 1) {
        const V z = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) y += z;
    }
    *total = __shfl_sync(0xffffffffu, y, WARPS - 1);
    V before = __shfl_sync(0xffffffffu, y, w ? w - 1 : 0);
    if (w == 0) before = 0;
    return before + x - v;
}

// How a pass of the selection tells a token's interval: by m - x, or by key. Out of range: -1.
struct Intervals {
    float top, per;             // by distance: (top - x) per, the last interval takes the rest
    unsigned lo, hi;            // by key: lo <= key <= hi
    int shift;                  // < 0: by distance
    float floor;                // tokens below are in no interval
    __device__ __forceinline__ int of(float x) const {
        if (!(x >= floor) || x == -INFINITY) return -1;
        if (shift < 0) return int(fminf((top - x) * per, float(BINS - 1)));
        const unsigned k = key_of(x);
        return k < lo || k > hi ? -1 : int((hi - k) >> shift);
    }
};

// What a row's passes share.
template <int DT, int THREADS> struct Row {
    static constexpr int VE = Logits<DT>::VE, WARPS = THREADS / 32, PER = BINS / THREADS;
    Shared &s;
    const Cluster &c;
    Logits<DT> logits;
    int v0, v1;                 // this block's vectors
    Heat heat;
    const float *pow2;          // the lane's table

    __device__ __forceinline__ unsigned long long weigh(float x) const { return weight(heat, pow2, x); }
    __device__ __forceinline__ unsigned long long weigh_rare(float x) const {
        return weight_call(heat.hi, heat.lo, heat.top, heat.places, pow2, x);
    }
    // 16 elements a thread and pass, whose loads are under way together: the passes behind the first read L2, and
    // wait for it more than they compute.
    static constexpr int FLIGHT = 16 / VE;
    // batch(first vector, elements): from vector v on, `step` apart, to `end`
    template <class B> __device__ __forceinline__ void batches(int v, int step, int end, B batch) const {
        for (; v < end; v += FLIGHT * step) {
            uint4 raw[FLIGHT];
#pragma unroll
            for (int i = 0; i < FLIGHT; ++i) raw[i] = logits.words(v + i * step < end ? v + i * step : logits.vectors);
            float x[FLIGHT][VE];
#pragma unroll
            for (int i = 0; i < FLIGHT; ++i) {
                Logits<DT>::widen(raw[i], x[i]);
                if (v + i * step < end) logits.patch(v + i * step, x[i]);
            }
            batch(v, x);
        }
    }
    template <class F> __device__ __forceinline__ void each(F f) const {
        batches(v0 + int(threadIdx.x), THREADS, v1, [&](int, const float (&x)[FLIGHT][VE]) {
#pragma unroll
            for (int i = 0; i < 16; ++i) f(x[i / VE][i % VE]);
        });
    }
    // The elements of a batch that are at or above a limit, and not above another, as bits.
    static __device__ __forceinline__ unsigned reach(float limit, const float (&x)[FLIGHT][VE], float most = INFINITY) {
        unsigned m = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) m |= x[i / VE][i % VE] >= limit && x[i / VE][i % VE] <= most ? 1u << i : 0u;
        return m;
    }
    // f(vector, element of it, x) of those elements, one after the other: few of many are looked at, and a branch an
    // element cost more than all else
    template <class F> __device__ __forceinline__ void pick(unsigned m, int v, int step, F f) const {
        while (m) {
            const int i = __ffs(m) - 1, vec = v + i / VE * step;
            m &= m - 1;
            f(vec, i % VE, logits.element(vec, i % VE));
        }
    }

    // Counts the intervals' tokens, or (WEIGH) adds up their weights, of which those below `least` are left out.
    // Returns the thread's sum of all weights above iv.floor.
    template <bool WEIGH> __device__ __forceinline__ unsigned long long fill(const Intervals &iv, unsigned long long least) {
        for (int i = threadIdx.x; i < BINS; i += THREADS) {
            if (WEIGH) s.sums[i] = make_uint2(0, 0);
            else s.count[i] = 0;
        }
        __syncthreads();
        unsigned long long sum = 0;
        auto put = [&](float x, unsigned long long w) {
            const int b = iv.of(x);
            if (b < 0) return;
            const unsigned lo = unsigned(w), old = atomicAdd(&s.sums[b].x, lo);
            const unsigned carry = unsigned(w >> 32) + (old + lo < old);
            if (carry) atomicAdd(&s.sums[b].y, carry);
        };
        if (!WEIGH) {
            each([&](float x) {
                const int b = iv.of(x);
                if (b >= 0) atomicAdd(&s.count[b], 1u);
            });
        } else if (iv.floor == -INFINITY) {
            each([&](float x) {
                const unsigned long long w = weigh(x);
                sum += w;
                if (w >= least) put(x, w);
            });
        } else {                                           // few are left
            batches(v0 + int(threadIdx.x), THREADS, v1, [&](int v, const float (&x)[FLIGHT][VE]) {
                pick(reach(iv.floor, x), v, THREADS, [&](int, int, float y) {
                    const unsigned long long w = weigh_rare(y);
                    if (y > iv.floor) sum += w;
                    if (w >= least) put(y, w);
                });
            });
        }
        return sum;
    }

    // The thread's intervals of all blocks: counts, or weights. All blocks' words are asked for before the first is
    // added.
    __device__ __forceinline__ void counts_of(unsigned long long (&n)[PER]) const {
#pragma unroll
        for (int i = 0; i < PER; i += 2) {
            uint2 x[MOST_BLOCKS];
#pragma unroll
            for (unsigned r = 0; r < MOST_BLOCKS; ++r)
                x[r] = r < c.size ? c.read2(&s.count[PER * threadIdx.x + i], r) : make_uint2(0, 0);
            n[i] = n[i + 1] = 0;
#pragma unroll
            for (unsigned r = 0; r < MOST_BLOCKS; ++r) n[i] += x[r].x, n[i + 1] += x[r].y;
        }
    }
    __device__ __forceinline__ void weights_of(unsigned long long (&n)[PER]) const {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            uint2 x[MOST_BLOCKS];
#pragma unroll
            for (unsigned r = 0; r < MOST_BLOCKS; ++r)
                x[r] = r < c.size ? c.read2(&s.sums[PER * threadIdx.x + i].x, r) : make_uint2(0, 0);
            n[i] = 0;
#pragma unroll
            for (unsigned r = 0; r < MOST_BLOCKS; ++r) n[i] += static_cast<unsigned long long>(x[r].y) << 32 | x[r].x;
        }
    }

    // Finds the token at which the running count (or weight) from the top reaches `goal`: its key, and how many of
    // the tokens of that key are kept (s.found_key, s.found_ties). The intervals are filled. Every thread of all
    // blocks calls it. `apart`: the blocks have not met since.
    template <bool WEIGH>
    __device__ __forceinline__ void select(Intervals iv, unsigned long long goal, unsigned long long least, bool apart) {
        const int tid = threadIdx.x;
        unsigned long long above = 0;                      // counts or weights above the intervals
        for (;; apart = true) {
            if (apart) c.sync();
            // the interval that reaches the goal
            unsigned long long mine[PER], sum = 0, total;
            if (WEIGH) weights_of(mine);
            else counts_of(mine);
#pragma unroll
            for (int i = 0; i < PER; ++i) sum += mine[i];
            unsigned long long at = above + block_sum<WARPS>(sum, s.scan64, &total);
            if (tid == 0) s.listed = 0, s.lo_key = 0xFFFFFFFFu, s.hi_key = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                if (at < goal && goal <= at + mine[i]) s.bin = PER * tid + i, s.above = at;
                at += mine[i];
            }
            __syncthreads();
            const int bin = s.bin;
            above = s.above;
            // its tokens
            unsigned lo = 0xFFFFFFFFu, hi = 0;
            // (a little outside the interval's ends: of() decides)
            const float from = iv.shift >= 0 ? of_key(iv.lo) : bin == BINS - 1 ? -FLT_MAX : iv.top - float(bin + 2) / iv.per;
            const float to = iv.shift >= 0 ? of_key(iv.hi) : iv.top - float(bin - 1) / iv.per;
            batches(v0 + tid, THREADS, v1, [&](int v, const float (&x)[FLIGHT][VE]) {
                pick(reach(fmaxf(from, iv.floor), x, to), v, THREADS, [&](int, int, float y) {
                    if (iv.of(y) != bin || (WEIGH && least > 1 && weigh_rare(y) < least)) return;
                    const unsigned k = key_of(y);
                    lo = min(lo, k), hi = max(hi, k);
                    const unsigned n = atomicAdd(&s.listed, 1u);
                    if (n < CAP) s.keys[n] = k;
                });
            });
            lo = __reduce_min_sync(0xffffffffu, lo), hi = __reduce_max_sync(0xffffffffu, hi);
            if ((tid & 31) == 0) atomicMin(&s.lo_key, lo), atomicMax(&s.hi_key, hi);
            c.sync();
            const unsigned listed = c.read_lane(&s.listed, 0u), n = __reduce_add_sync(0xffffffffu, listed);
            lo = __reduce_min_sync(0xffffffffu, c.read_lane(&s.lo_key, 0xFFFFFFFFu));
            hi = __reduce_max_sync(0xffffffffu, c.read_lane(&s.hi_key, 0u));
            if (lo == hi) {                                // all alike
                if (tid == 0) {
                    const unsigned long long w = WEIGH ? weigh_rare(of_key(lo)) : 1;
                    s.found_key = lo, s.found_ties = unsigned((goal - above + w - 1) / w);
                }
                break;
            }
            if (n <= CAP) {
                unsigned first = 0;
                for (unsigned r = 0; r < c.size; ++r) {
                    const unsigned m = __shfl_sync(0xffffffffu, listed, r);
                    for (unsigned i = tid; i < m; i += THREADS) {
                        const unsigned k = c.read(&s.keys[i], r);
                        s.all_keys[first + i] = k;
                        if (WEIGH) s.weights[first + i] = weigh_rare(of_key(k));
                    }
                    first += m;
                }
                __syncthreads();
                for (unsigned t = tid; t < n; t += THREADS) {
                    const unsigned k = s.all_keys[t];
                    unsigned long long over = above;
                    unsigned same = 0;
#pragma unroll 8
                    for (unsigned i = 0; i < n; ++i) {
                        const unsigned o = s.all_keys[i];
                        if (o > k) over += WEIGH ? s.weights[i] : 1;
                        same += o == k;
                    }
                    const unsigned long long w = WEIGH ? s.weights[t] : 1;
                    if (over < goal && goal <= over + same * w)
                        s.found_key = k, s.found_ties = unsigned((goal - over + w - 1) / w);
                }
                break;
            }
            // too many: divide the interval by keys
            iv.lo = lo, iv.hi = hi;
            iv.shift = max(0, 32 - __clz(hi - lo) - 11);
            fill<WEIGH>(iv, least);
        }
        __syncthreads();
    }
};

// THREADS: 512, two blocks an SM, where a row has one; 1024 where it has more, so that they lie on different SMs.
template <int DT, int THREADS> __global__ void __launch_bounds__(THREADS, 1024 / THREADS) sample_kernel(SampleArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    Shared &s = *reinterpret_cast<Shared *>(smem);
    constexpr int VE = Logits<DT>::VE, WARPS = THREADS / 32, PER = BINS / THREADS;
    const Cluster c;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
    const int64_t b = blockIdx.x / c.size;
    for (int i = w; i < 2 * STEPS / 4; i += WARPS) {       // a warp four entries: a lane a copy
        const float4 t = reinterpret_cast<const float4 *>(&g_pow2)[i];
        float *to = &s.pow2[0][0][0] + i * 128 + lane;
        to[0] = t.x, to[32] = t.y, to[64] = t.z, to[96] = t.w;
    }
    if (tid == 0) s.best = 0, s.bad = 0, s.first = 0xFFFFFFFFu, s.share = -1;
    pdl_launch_dependents();
    pdl_wait();
    const unsigned char *const logits = static_cast<const unsigned char *>(a.logits) + b * a.ld * Logits<DT>::ES;
    Row<DT, THREADS> row = {s, c, Logits<DT>(logits, int(a.vocab)), 0, 0, {}, &s.pow2[0][0][lane]};
    const int share = (row.logits.vectors + int(c.size) - 1) / int(c.size);
    row.v0 = min(int(c.rank) * share, row.logits.vectors), row.v1 = min(row.v0 + share, row.logits.vectors);
    const float given = a.temperature ? a.temperature[b] : 1.0f, heat_t = given > 0x1p64f ? 0x1p64f : given;
    const int k = a.top_k ? a.top_k[b] : 0;
    const float p = a.top_p ? a.top_p[b] : 1.0f, min_p = a.min_p ? a.min_p[b] : 0.0f;
    const float u = fminf(fmaxf(a.u[b], 0.0f), 0x1.fffffep-1f);
    __syncthreads();

    // -- the maximum ----------------------------------------------------------------------------------------------
    float top = -INFINITY;
    row.batches(row.v0 + tid, THREADS, row.v1, [&](int, const float (&x)[Row<DT, THREADS>::FLIGHT][VE]) {
#pragma unroll
        for (int i = 0; i < 16; i += 2) top = max3_nan(top, x[i / VE][i % VE], x[i / VE][i % VE + 1]);
    });
#pragma unroll
    for (int o = 16; o; o >>= 1) top = max3_nan(top, top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) {
        if (!(top < INFINITY)) s.bad = 1;
        else if (top > -INFINITY) atomicMax(&s.best, key_of(top));
    }
    c.sync();
    const unsigned best = __reduce_max_sync(0xffffffffu, c.read_lane(&s.best, 0u));
    const bool bad = __any_sync(0xffffffffu, c.read_lane(&s.bad, 0) != 0);
    top = of_key(best);
    if (bad || best == 0 || !(heat_t >= 0x1p-64f)) {
        // a token without a draw: none, or the lowest index of the maximum
        if (!bad && best) {
            row.batches(row.v0 + tid, THREADS, row.v1, [&](int v, const float (&x)[Row<DT, THREADS>::FLIGHT][VE]) {
                row.pick(row.reach(top, x), v, THREADS, [&](int vec, int e, float) {
                    atomicMin(&s.first, unsigned(row.logits.index(vec) + e));
                });
            });
            c.sync();
        }
        if (tid == 0 && c.rank == 0) {
            unsigned first = 0xFFFFFFFFu;
            for (unsigned r = 0; r < c.size; ++r) first = min(first, c.read(&s.first, r));
            if (bad) atomicOr(&g_fault_sample, FAULT_NONFINITE_X);
            a.tokens[b] = int(first);                      // -1 where there is none
            if (a.probs) a.probs[b] = bad ? __int_as_float(0x7FC00000) : best == 0 ? 0.0f : 1.0f;
        }
        if (c.size > 1) c.sync();                          // none leaves while another reads its memory
        return;
    }
    {                                      // log2(e) / T in two floats: fp64 would take 4 us of a block's threads
        constexpr float log2e_hi = 1.44269502162933349609375f, log2e_lo = 1.925963033500e-8f;
        row.heat.hi = __fdiv_rn(log2e_hi, heat_t);
        row.heat.lo = __fdiv_rn(__fadd_rn(__fmaf_rn(-row.heat.hi, heat_t, log2e_hi), log2e_lo), heat_t);
        row.heat.top = top;
        row.heat.places = a.places;
    }
    const unsigned long long one = 1ull << a.places;

    // -- the last token kept by top-k and top-p ---------------------------------------------------------------
    bool cut_k = k > 0 && k < a.vocab;
    const bool cut_p = p < 1.0f;
    unsigned last_ties = 0;                // kept: logits above the last one, and so many equal to it (0: nothing cut)
    float last = -INFINITY;
    if (cut_k || cut_p) {
        Intervals iv = {row.heat.top, BINS / fmaxf(32.0f, 32.0f * heat_t), 0, 0, -1, -INFINITY};
        if (cut_k) {
            row.template fill<false>(iv, 0);
            unsigned total = 0, mine = 0;
            c.sync();
            unsigned long long each_one[PER];
            row.counts_of(each_one);
#pragma unroll
            for (int i = 0; i < PER; ++i) mine += unsigned(each_one[i]);
            block_sum<WARPS>(mine, s.scan32, &total);
            cut_k = unsigned(k) < total;                   // masked tokens do not count
            if (cut_k) {
                row.template select<false>(iv, unsigned(k), 0, false);
                last = of_key(s.found_key), last_ties = s.found_ties;
                iv.floor = last;
            }
        }
        if (cut_p) {
            // The sum of the tokens kept so far, and their weights by intervals. Tokens whose weight is below (1 - p)
            // / 2 of the largest over their number stay below (1 - p) / 2 of the sum all together: they are behind
            // the last one kept, and are left out.
            const float beyond = fminf((1.0f - fmaxf(p, 0.0f)) * 0.5f, 0.5f);
            const unsigned long long least = max(1ull, part_of(beyond, one, false) / a.vocab);
            unsigned long long sum = row.template fill<true>(iv, least), total;
            block_sum<WARPS>(sum, s.scan64, &total);
            if (tid == 0) s.sum = total;
            c.sync();
            sum = c.read_lane(&s.sum, 0ull);
#pragma unroll
            for (int o = MOST_BLOCKS / 2; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            sum = __shfl_sync(0xffffffffu, sum, 0);
            if (cut_k) sum += last_ties * row.weigh_rare(last);    // of the last one's equals those kept
            row.template select<true>(iv, max(1ull, part_of(fmaxf(p, 0.0f), sum, true)), least, false);
            last = of_key(s.found_key), last_ties = s.found_ties;
        }
    }
    const unsigned long long least = min_p >= 1.0f ? one : min_p > 0.0f ? max(1ull, part_of(min_p, one, true)) : 1ull;
    const unsigned long long last_weight = last_ties ? row.weigh_rare(last) : 0;
    const bool ties_count = last_weight >= least;

    // -- sums of kept weights by warps' shares of the block's vectors, in order of index ------------------------------
    const int per = (row.v1 - row.v0 + WARPS - 1) / WARPS, v0 = min(row.v0 + w * per, row.v1), v1 = min(v0 + per, row.v1);
    auto kept = [&](float x, unsigned &ties) -> unsigned long long {
        if (x <= last) {                                   // (-inf where nothing is cut)
            ties += x == last && last_ties;
            return 0;
        }
        const unsigned long long y = row.weigh_rare(x);
        return y >= least ? y : 0;
    };
    unsigned long long sum = 0;
    unsigned ties = 0;
    const bool all = !last_ties && least == 1;
    row.batches(v0 + lane, 32, v1, [&](int v, const float (&x)[Row<DT, THREADS>::FLIGHT][VE]) {
        const unsigned m = all ? 0xFFFFu : row.reach(last, x);
        if (all || __any_sync(__activemask(), __popc(m) > 4)) {        // many: all of them, without a branch each
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float y = x[i / VE][i % VE];
                const unsigned long long z = row.weigh(y);
                ties += y == last && last_ties;
                sum += (y > last || all) && z >= least ? z : 0;
            }
        } else {
            row.pick(m, v, 32, [&](int, int, float y) { sum += kept(y, ties); });
        }
    });
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    ties = __reduce_add_sync(0xffffffffu, ties);
    __syncthreads();
    if (lane == 0) s.scan64[w] = sum, s.scan32[w] = ties;
    __syncthreads();
    if (tid == 0) {
        unsigned long long all = 0;
        unsigned equal = 0;
        for (int i = 0; i < WARPS; ++i) all += s.scan64[i], equal += s.scan32[i];
        s.kept = all, s.ties = equal;
    }
    c.sync();
    // kept weights before this warp's share, and in all
    unsigned long long before = 0, total = 0, mine = 0;
    unsigned ties_before = 0, all_ties = 0;
    const unsigned long long sums = c.read_lane(&s.kept, 0ull);
    const unsigned equals = c.read_lane(&s.ties, 0u);
    for (unsigned r = 0; r < c.size; ++r) {
        const unsigned here = __shfl_sync(0xffffffffu, equals, r), may = last_ties - min(all_ties, last_ties);
        const unsigned long long add = __shfl_sync(0xffffffffu, sums, r) + (ties_count ? min(here, may) * last_weight : 0);
        if (r == c.rank) {
            before = total, ties_before = all_ties;
            for (int i = 0; i < WARPS; ++i) {
                const unsigned left = last_ties - min(ties_before, last_ties);
                const unsigned long long part = s.scan64[i] + (ties_count ? min(s.scan32[i], left) * last_weight : 0);
                if (i == w) {
                    mine = part;
                    break;
                }
                before += part, ties_before += s.scan32[i];
            }
        }
        total += add, all_ties += here;
    }
    const unsigned long long goal = part_of(u, total, false);
    if (lane == 0 && goal >= before && goal < before + mine)       // one warp's
        s.share = w, s.above = before, s.found_ties = ties_before;
    __syncthreads();
    if (const int holder = s.share; holder >= 0) {         // the block looks through the warp's share together
        unsigned left = last_ties - min(s.found_ties, last_ties);
        unsigned long long run = s.above;
        const int from = row.v0 + holder * per, to = min(from + per, row.v1);
        for (int v = from; v < to; v += THREADS) {
            float x[VE];
            row.logits.load(v + tid < to ? v + tid : row.logits.vectors, x);
            unsigned t = 0, t_all;
            unsigned long long here = 0, all_here;
#pragma unroll
            for (int e = 0; e < VE; ++e) here += kept(x[e], t);
            const unsigned t_before = block_sum<WARPS>(t, s.scan32, &t_all);
            unsigned may = left - min(left, t_before);     // ties that this thread may keep
            here += ties_count ? min(t, may) * last_weight : 0;
            const unsigned long long start = run + block_sum<WARPS>(here, s.scan64, &all_here);
            if (goal >= start && goal < start + here) {
                unsigned long long at = start;
                for (int e = 0; e < VE; ++e) {
                    unsigned tie = 0;
                    unsigned long long y = kept(x[e], tie);
                    if (tie && may) y = ties_count ? last_weight : 0, --may;
                    if (goal < at + y) {
                        a.tokens[b] = row.logits.index(v + tid) + e;
                        if (a.probs) a.probs[b] = float(double(y) / double(total));
                        break;
                    }
                    at += y;
                }
            }
            run += all_here;
            left -= min(left, t_all);
            if (goal < run) break;
        }
    }
    if (c.size > 1) c.sync();                              // none leaves while another reads its memory
}

// Blocks a row: as many as keep the SMs busy, of 4096 tokens or more each.
int blocks_a_row(int64_t rows, int64_t vocab) {
    int n = 1;
    while (n < MOST_BLOCKS && rows * n * 2 <= num_sms() && vocab >= 8192 * n) n *= 2;
    return n;
}

template <int DT, int THREADS> cudaError_t run(const SampleArgs &a, int blocks, cudaStream_t s) {
    static int opted[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!opted[dev]) {
        e = cudaFuncSetAttribute(sample_kernel<DT, THREADS>, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Shared));
        if (e != cudaSuccess) return e;
        opted[dev] = 1;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(a.rows * blocks));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = sizeof(Shared);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(blocks), attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = blocks > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, sample_kernel<DT, THREADS>, a);
}
template <int DT> cudaError_t run_type(const SampleArgs &a, cudaStream_t s) {
    const int blocks = blocks_a_row(a.rows, a.vocab);
    return blocks > 1 ? run<DT, 1024>(a, blocks, s) : run<DT, 512>(a, 1, s);
}

}  // namespace

cudaError_t launch_sample(SampleArgs a, cudaStream_t s) {
    int bits = 0;
    while ((int64_t(1) << bits) < a.vocab) ++bits;
    a.places = 62 - bits < 46 ? 62 - bits : 46;
    return a.dt == DT_F32 ? run_type<DT_F32>(a, s) : a.dt == DT_F16 ? run_type<DT_F16>(a, s) : run_type<DT_BF16>(a, s);
}

cudaError_t fault_word_sample(int **word) {
    return cudaGetSymbolAddress(reinterpret_cast<void **>(word), g_fault_sample);
}

}  // namespace qpack
