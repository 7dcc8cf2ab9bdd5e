// Sampling with temperature, top-k, top-p and min-p from given random numbers.
//
// With z = l / T, the three filters keep a beginning of the row's order each
// (falling z, equal ones by rising index), so together they keep one beginning,
// and the token drawn is the kept one with the largest z - log noise.  No row
// is ever sorted whole:
//
//   1. sample_stats_kernel, S CTAs a row: the row's maximum and sum of
//      exponentials, and, in a call without filters, the race itself: one pass over
//      logits and noise, joined by the row's last CTA;
//   2. sample_pick_kernel, S CTAs a row, where filters may be on: what can be
//      kept is cut down to candidates without knowing the order -- top-k and
//      top-p by the maxima of the first pass's threads, S x 512 tokens of the
//      row: with k of them, or p of the row's weight, at and above a bound, so
//      many of the row's tokens are (the bound lowered by what one quotient
//      spans); min-p by its own bound -- and collected in a list of the row;
//   3. the row's last CTA settles the cuts and the race among up to kWide
//      candidates: a few it sorts; of more it finds the cut's place in bins of
//      their counts or weights and sorts what lies in that bin alone, tokens
//      above it are kept for certain.  Only the kept ones' random numbers are
//      read;
//   4. with more candidates (a flat row, a top-k above 1024) it counts them in
//      bins, which bounds where the cuts fall; tokens above are kept for certain
//      and take part in the race as they are read, their weights summed; only the
//      tokens around the cuts are collected and sorted;
//   5. where even those are more than kList, or the bins do not bound the cut, it
//      finds the cuts by bisection over order-preserving keys: thousands of equal
//      logits, but also a nucleus of many thousand tokens, and a top-k of more
//      tokens than a mask leaves the row.
//
// Steps 4 and 5 are one CTA's walks over the whole row, two or three in step 4
// and some 20 to 50 in step 5.
//
// Bound: HBM for many rows (every logit once; the passes after the first find
// them in L2), launches and the chain of passes for few.  Measured, 151936
// tokens a row: 256 f32 rows without filters 45.4 us, 6.8 TB/s; one bf16 row with
// top-k and top-p 14.7 us (7 k clocks the first kernel, 20 k the second); 64 bf16
// rows with filters of their own 25-31 us, by what the filters leave.  One row,
// and 64 of them: a nucleus of 100 to 4000 tokens 21-28 and 28-37 us (step 3; in
// one of the 64 rows at T = 1.3 and p = 0.99 step 5, 4.5 ms), top-k 2000 to 20000
// 140-200 and 200-300 us (step 4), a nucleus of 15000 tokens 2.9 and 4.6 ms, five
// tokens left by a mask under top-k 50 1.2 and 2.0 ms, 105 of them (the others at
// -1e9) under top-k 500 4.0 and 6.4 ms (step 5).
//
// Sums are added in an order that depends on the sizes alone, and the sort
// makes the order of collection irrelevant, so a row's token and logprob do
// not depend on timing.
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace w4a16 {

constexpr int kStatThreads = 512, kPickThreads = 512;
constexpr int kWide = 8192;   // candidates of a row's list
constexpr int kList = 2048;   // those of them, around a cut, that are sorted
constexpr int kFew = 256;     // those that are sorted by counting
constexpr int kBins = 4096;   // of the histogram of a flat row
constexpr int kTopBins = 2 * kPickThreads;  // of the histogram of the first pass's maxima
constexpr int kMaxSplits = 8;  // CTAs a row, a power of two
constexpr float kBig = 3.402823466e38f;
constexpr float kLog2E = 1.4426950408889634f;
// the rows' arrival counters in the workspace's counter area, behind the attention kernels'
constexpr int kSampleCounters = 4096, kSampleSplitRows = 4096;

// What a CTA leaves of its slice after the first pass, and its part of the race.
struct SliceStats {
    float lmax, sum, best;
    int imax, ibest, pad[3];
};
// A row's part of the workspace; behind it the maxima of the S x kStatThreads threads of the first pass.
struct RowSpace {
    SliceStats stats[kMaxSplits];
    int found, pad[3];            // candidates collected (may exceed kWide)
    uint32_t key[kWide];          // candidates: keys of z, all bits turned (rising key is falling z)
    int index[kWide];
    W4A16_DEVICE float* maxima() { return reinterpret_cast<float*>(this + 1); }
};
__host__ __device__ constexpr size_t row_space(int S) { return sizeof(RowSpace) + (size_t)S * kStatThreads * 4; }
W4A16_DEVICE RowSpace* space_of(void* workspace, int r, int S) {
    return reinterpret_cast<RowSpace*>(static_cast<char*>(workspace) + kCounterBytes + r * row_space(S));
}

// order-preserving map of f32 to unsigned (no NaN): a < b <=> key(a) < key(b)
W4A16_DEVICE uint32_t key_of(float z) {
    const uint32_t u = __float_as_uint(z);
    return (u >> 31) ? ~u : (u | 0x80000000u);
}
W4A16_DEVICE float value_of(uint32_t k) { return __uint_as_float((k >> 31) ? (k & 0x7fffffffu) : ~k); }

// a logit as f32: NaN counts as -inf, +inf as the largest finite value, -0 as 0
W4A16_DEVICE float clean(float x) { return fminf(fmaxf(x, -INFINITY), kBig) + 0.f; }
template <int DT>
W4A16_DEVICE float decode(uint32_t bits) {
    if constexpr (DT == W4A16_F32) return clean(__uint_as_float(bits));
    if constexpr (DT == W4A16_BF16) return clean(__uint_as_float(bits << 16));
    return clean(f16_bits_to_f32((uint16_t)bits));
}
// z of a cleaned logit above -inf: the f32 quotient, finite
W4A16_DEVICE float z_of(float l, float t) { return fmaxf(fminf(__fdiv_rn(l, t), kBig), -kBig) + 0.f; }

W4A16_DEVICE float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
W4A16_DEVICE float lg2(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// One CTA's arrival, by one thread behind a barrier: the CTA's writes are before
// it, the others' after it.  Their number before this one.
W4A16_DEVICE unsigned arrive(unsigned* counter) {
    unsigned n;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(n) : "l"(counter) : "memory");
    return n;
}

// ---- reductions over the CTA, in a fixed order --------------------------------
template <int NT>
W4A16_DEVICE float cta_sum(float x, float* f) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    __syncthreads();
    if (lane == 0) f[threadIdx.x >> 5] = x;
    __syncthreads();
    x = lane < NT / 32 ? f[lane] : 0.f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}
template <int NT>
W4A16_DEVICE int cta_count(int x, int* n) {
    const int lane = threadIdx.x & 31;
    x = __reduce_add_sync(0xffffffffu, x);
    __syncthreads();
    if (lane == 0) n[threadIdx.x >> 5] = x;
    __syncthreads();
    return __reduce_add_sync(0xffffffffu, lane < NT / 32 ? n[lane] : 0);
}
// the largest x (never -0 or NaN) and, of equal ones, the lowest index, over a warp
W4A16_DEVICE void warp_best(float& x, int& i) {
    const uint32_t y = key_of(x), top = __reduce_max_sync(0xffffffffu, y);
    i = __reduce_min_sync(0xffffffffu, y == top ? i : 0x7fffffff);
    x = value_of(top);
}
template <int NT>
W4A16_DEVICE void cta_best(float& x, int& i, float* f, int* n) {
    const int lane = threadIdx.x & 31;
    warp_best(x, i);
    __syncthreads();
    if (lane == 0) {
        f[threadIdx.x >> 5] = x;
        n[threadIdx.x >> 5] = i;
    }
    __syncthreads();
    x = f[lane & (NT / 32 - 1)];
    i = n[lane & (NT / 32 - 1)];
    warp_best(x, i);
}
template <int NT>
W4A16_DEVICE float cta_min(float x, float* f) {
    x = value_of(__reduce_min_sync(0xffffffffu, key_of(x)));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) f[threadIdx.x >> 5] = x;
    __syncthreads();
    return value_of(__reduce_min_sync(0xffffffffu, key_of(f[threadIdx.x & (NT / 32 - 1)])));
}
// sum over the threads before this one, of counts
W4A16_DEVICE uint32_t cta_before(uint32_t x, int* n) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t s = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= d) s += y;
    }
    __syncthreads();
    if (lane == 31) n[warp] = (int)s;
    __syncthreads();
    return s - x + __reduce_add_sync(0xffffffffu, lane < warp ? (uint32_t)n[lane] : 0u);
}
// sum over the threads before this one
W4A16_DEVICE float cta_before(float x, float* f) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float s = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const float y = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= d) s += y;
    }
    __syncthreads();
    if (lane == 31) f[warp] = s;
    __syncthreads();
    float w = lane < warp ? f[lane] : 0.f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) w += __shfl_xor_sync(0xffffffffu, w, d);
    const float before = __shfl_up_sync(0xffffffffu, s, 1);
    return w + (lane ? before : 0.f);
}

// ---- a CTA's slice of a row ----------------------------------------------------
// Tokens that a warp has set aside: fewer than 32, and up to 256 of one load.
struct Aside {
    float l[288];
    int i[288];
};
template <int DT, int NT>
struct Slice {
    static constexpr int VE = DT == W4A16_F32 ? 4 : 8;  // logits of a 16-byte load
    using El = typename std::conditional<DT == W4A16_F32, uint32_t, uint16_t>::type;
    const El* row;
    int V, head, v0, v1, tail;  // [0, head) and [tail, V) one by one; 16-byte loads v0 .. v1 behind head
    bool first, last;

    W4A16_DEVICE Slice(const void* base, int64_t off, int vocab, int rank, int S) {
        row = static_cast<const El*>(base) + off;
        V = vocab;
        head = (int)(((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / sizeof(El));
        if (head > V) head = V;
        const int nv = (V - head) / VE;
        v0 = (int)((int64_t)nv * rank / S);
        v1 = (int)((int64_t)nv * (rank + 1) / S);
        tail = head + nv * VE;
        first = rank == 0;
        last = rank == S - 1;
    }
    W4A16_DEVICE static void split(const uint4& x, float (&l)[VE]) {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (DT == W4A16_F32) {
                l[i] = decode<DT>(w[i]);
            } else {
                l[2 * i] = decode<DT>(w[i] & 0xffffu);
                l[2 * i + 1] = decode<DT>(w[i] >> 16);
            }
        }
    }
    // one(logit, index) for single tokens, many(logits, index of the first) for VE of them: this thread's
    // tokens, by rising index
    template <typename One, typename Many>
    W4A16_DEVICE void each(One one, Many many) const {
        constexpr int U = 4;
        if (first && (int)threadIdx.x < head) one(at((int)threadIdx.x), (int)threadIdx.x);
        const uint4* vec = reinterpret_cast<const uint4*>(row + head);
        int v = v0 + (int)threadIdx.x;
        uint4 x[U];  // U loads in flight all the time: one is issued as one is used
        if (v < v1) {
#pragma unroll
            for (int u = 0; u < U; ++u) x[u] = vec[min(v + u * NT, v1 - 1)];
        }
        for (; v < v1; v += U * NT) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (v + u * NT >= v1) break;
                float l[VE];
                split(x[u], l);
                x[u] = vec[min(v + (u + U) * NT, v1 - 1)];
                many(l, head + (v + u * NT) * VE);
            }
        }
        if (last && tail + (int)threadIdx.x < V) one(at(tail + (int)threadIdx.x), tail + (int)threadIdx.x);
    }
    // one(logit, index) for the tokens with a logit >= low, by the whole CTA.
    template <typename One>
    W4A16_DEVICE void from(float low, Aside* aside, One one) const {
        batches(low, aside, [&](int n, float l, int i) {
            if ((int)(threadIdx.x & 31) < n) one(l, i);
        });
    }
    // The same by warps: some(n, logit, index) with n tokens in the first lanes.
    // They are set aside per warp and handed over 32 at a time, so that `some`,
    // which divides, counts or collects, runs with full warps however rare they
    // are, and is there once and not for every load.
    template <typename Some>
    W4A16_DEVICE void batches(float low, Aside* aside, Some some) const {
        constexpr int U = 4;
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        Aside& own = aside[warp];
        int count = 0;  // set aside, the same in every lane
        auto put = [&](float l, int i) {
            const bool hit = l >= low && l > -INFINITY;
            const unsigned m = __ballot_sync(0xffffffffu, hit);
            if (!m) return;
            if (hit) {
                const int at = count + __popc(m & ((1u << lane) - 1u));
                own.l[at] = l;
                own.i[at] = i;
            }
            count += __popc(m);
        };
        auto hand_over = [&](int least) {
            while (count >= least && count > 0) {
                __syncwarp();
                const int n = count < 32 ? count : 32, at = count - n + lane;
                const float l = lane < n ? own.l[at] : 0.f;
                const int i = lane < n ? own.i[at] : 0;
                count -= n;
                __syncwarp();
                some(n, l, i);
                __syncwarp();
            }
        };
        if (first && warp == 0) put(lane < head ? at(lane) : -INFINITY, lane);
        const uint4* vec = reinterpret_cast<const uint4*>(row + head);
        for (int v = v0 + warp * 32; v < v1; v += U * NT) {
            uint4 x[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int y = v + u * NT + lane;
                x[u] = y < v1 ? vec[y] : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int y = v + u * NT + lane;
                float l[VE];
                split(x[u], l);
                float b = l[0];
#pragma unroll
                for (int z = 1; z < VE; ++z) b = fmaxf(b, l[z]);
                if (!__any_sync(0xffffffffu, y < v1 && b >= low)) continue;
#pragma unroll
                for (int z = 0; z < VE; ++z) put(y < v1 ? l[z] : -INFINITY, head + y * VE + z);
                hand_over(32);
            }
        }
        if (last && warp == 0) put(tail + lane < V ? at(tail + lane) : -INFINITY, tail + lane);
        hand_over(32);
        hand_over(1);
    }
    W4A16_DEVICE float at(int i) const { return decode<DT>(row[i]); }
};

// A row's parameters.
struct RowParams {
    float T, tp, mp, c2;  // temperature, top-p, min-p, log2(e) / T
    int k;
    bool greedy, by_k, by_p, by_m, race;
    W4A16_DEVICE RowParams(const w4a16_sample_args& p, int r) {
        const float t = p.temperature ? p.temperature[r] : 1.f;
        greedy = !(t > 0.f);
        T = greedy ? 1.f : fminf(fmaxf(t, 1e-30f), 1e30f);  // no quotient of usual logits overflows or is subnormal
        c2 = fminf(kLog2E / T, kBig);
        k = p.top_k ? p.top_k[r] : 0;
        tp = p.top_p ? p.top_p[r] : 1.f;
        mp = p.min_p ? p.min_p[r] : 0.f;
        by_k = !greedy && k > 0 && k < p.vocab;
        by_p = !greedy && tp < 1.f;
        by_m = !greedy && mp > 0.f;
        race = !greedy && !by_k && !by_p && !by_m;
    }
};

// The row's token and its log-probability, by one thread.
W4A16_DEVICE void write_token(const w4a16_sample_args& p, int r, int token, float z, float zmax, float sum) {
    p.token[r] = token;
    if (p.logprob) p.logprob[r] = (z - zmax) - logf(sum);
}
// The same where the logit has to be read, or there is none.
template <int DT, int NT>
W4A16_DEVICE void write_row(const w4a16_sample_args& p, int r, const Slice<DT, NT>& row, const RowParams& q, int token,
                            int imax, float lmax, float sum) {
    if (lmax == -INFINITY) {
        p.token[r] = -1;
        if (p.logprob) p.logprob[r] = -INFINITY;
        return;
    }
    if (token < 0 || token >= p.vocab) token = imax;  // the noise of every kept token was infinite or NaN
    write_token(p, r, token, z_of(row.at(token), q.T), z_of(lmax, q.T), sum);
}

// The slices' results as one, the sums added in slice order; by whole warps.
struct RowStats {
    float lmax, sum, best;
    int imax, ibest;
    W4A16_DEVICE RowStats(const SliceStats* s, int S, float c2) {
        s += threadIdx.x & (S - 1);  // (S is a power of two: the slices again and again)
        const float mine = __ldcg(&s->lmax), part = __ldcg(&s->sum);
        lmax = mine;
        best = __ldcg(&s->best);
        imax = __ldcg(&s->imax);
        ibest = __ldcg(&s->ibest);
        warp_best(lmax, imax);
        warp_best(best, ibest);
        const float scaled = mine == -INFINITY ? 0.f : part * ex2((mine - lmax) * c2);
        sum = 0.f;
        for (int i = 0; i < S; ++i) sum += __shfl_sync(0xffffffffu, scaled, i);
    }
};

// ---- 1. maximum, sum, and the race of unfiltered rows ---------------------------
// One thread's part of a pass over a slice: its largest logit and sum of
// exponentials (STATS), and its part of the race (`race`).
//
// The race runs on approximate scores, l / T - log e, with errors below
// 2^-21 |z| + 2^-20 and |z| <= |score| + 104 for any finite noise: a thread
// keeps its two best loads, and the exact scores of the few loads that come
// near the CTA's best decide.
template <int DT, int NT, bool STATS>
struct Pass {
    using Row = Slice<DT, NT>;
    static constexpr int VE = Row::VE;
    const Row& slice;
    const float* noise;
    const RowParams& q;
    float mx = -kBig, sum = 0.f;
    int vmax = -1;  // the load in which mx came first: a token below V, or V + a vector's first token
    float top = -INFINITY, top2 = -INFINITY;
    int vtop = -1;
    float inv_t;
    bool race;

    W4A16_DEVICE float approx(float l, float e) const { return fmaf(l, inv_t, -0.6931471805599453f * lg2(e)); }
    W4A16_DEVICE void enter(float t, int at) {
        top2 = fmaxf(top2, fminf(top, t));
        if (t > top) {
            top = t;
            vtop = at;
        }
    }
    W4A16_DEVICE void maximum(float b, int at) {  // -kBig itself may be the first
        if (b > mx || (vmax < 0 && b == -kBig)) {
            sum *= ex2((mx - b) * q.c2);
            mx = b;
            vmax = at;
        }
    }
    W4A16_DEVICE void one(float l, int i) {
        if constexpr (STATS) {
            maximum(l, i);
            sum += ex2((l - mx) * q.c2);
        }
        if (race && l > -INFINITY) enter(approx(l, noise[i]), i);
    }
    W4A16_DEVICE void many(const float (&l)[VE], int i0) {
        if constexpr (STATS) {
            float b = l[0];
#pragma unroll
            for (int x = 1; x < VE; ++x) b = fmaxf(b, l[x]);
            maximum(b, slice.V + i0);
            float s = 0.f;
#pragma unroll
            for (int x = 0; x < VE; ++x) s += ex2((l[x] - mx) * q.c2);
            sum += s;
        }
    }
    W4A16_DEVICE Pass(const Row& slice_, const float* noise_, const RowParams& q_, bool race_)
        : slice(slice_), noise(noise_), q(q_), race(race_) {
        inv_t = fminf(1.f / q.T, kBig);
        const int V = slice.V;
        const bool noise4 = (reinterpret_cast<uintptr_t>(noise + slice.head) & 15) == 0;
        if (!race) {
            if constexpr (STATS)
                slice.each([&](float l, int i) { one(l, i); }, [&](const float (&l)[VE], int i0) { many(l, i0); });
        } else if (noise4) {
            // logits and their random numbers together, U vectors in flight all the time
            constexpr int U = VE == 4 ? 4 : 3, NE = VE / 4;
            const uint4* vec = reinterpret_cast<const uint4*>(slice.row + slice.head);
            const float4* nv = reinterpret_cast<const float4*>(noise + slice.head);
            if (slice.first && (int)threadIdx.x < slice.head) one(slice.at((int)threadIdx.x), (int)threadIdx.x);
            uint4 x[U];
            float4 e[U][NE];
            auto load = [&](int u, int y) {
                y = min(y, slice.v1 - 1);  // past the end: again, and not counted
                x[u] = __ldcs(vec + y);
#pragma unroll
                for (int z = 0; z < NE; ++z) e[u][z] = __ldcs(nv + y * NE + z);
            };
            int v = slice.v0 + (int)threadIdx.x;
            if (v < slice.v1) {
#pragma unroll
                for (int u = 0; u < U; ++u) load(u, v + u * NT);
            }
            for (; v < slice.v1; v += U * NT) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (v + u * NT >= slice.v1) break;
                    const int i0 = slice.head + (v + u * NT) * VE;
                    float l[VE], t = -INFINITY;
                    slice.split(x[u], l);
#pragma unroll
                    for (int z = 0; z < NE; ++z)
                        t = fmaxf(t, fmaxf(fmaxf(approx(l[4 * z], e[u][z].x), approx(l[4 * z + 1], e[u][z].y)),
                                           fmaxf(approx(l[4 * z + 2], e[u][z].z), approx(l[4 * z + 3], e[u][z].w))));
                    load(u, v + (u + U) * NT);
                    many(l, i0);
                    enter(t, V + i0);
                }
            }
            if (slice.last && slice.tail + (int)threadIdx.x < V)
                one(slice.at(slice.tail + (int)threadIdx.x), slice.tail + (int)threadIdx.x);
        } else {  // a row whose random numbers are not aligned as its logits are
            slice.each([&](float l, int i) { one(l, i); }, [&](const float (&l)[VE], int i0) {
                many(l, i0);
                float t = -INFINITY;
#pragma unroll
                for (int x = 0; x < VE; ++x) t = fmaxf(t, approx(l[x], noise[i0 + x]));
                enter(t, V + i0);
            });
        }
    }
    // the slice's winner, by the whole CTA
    W4A16_DEVICE void winner(float& best, int& ibest, float* rf, int* ri) const {
        const int V = slice.V;
        best = -INFINITY;
        ibest = 0x7fffffff;
        float lead = top;
        int none = 0;
        cta_best<NT>(lead, none, rf, ri);
        const float near = lead - 2e-3f - 8e-6f * fabsf(lead);  // (NaN where lead is infinite: all compare true below)
        auto exact = [&](int i) {
            const float l = slice.at(i);
            const float x = z_of(l, q.T) - logf(noise[i]);
            if (l > -INFINITY && (x > best || (x == best && i < ibest))) {
                best = x;
                ibest = i;
            }
        };
        auto all_of = [&](int at) {  // a load's tokens
            if (at < 0) return;
#pragma unroll 1
            for (int x = 0; x < (at < V ? 1 : VE); ++x) exact((at < V ? at : at - V) + x);
        };
        if (!(top < near)) {
            if (!(top2 < near)) {
                slice.each([&](float, int i) { all_of(i); }, [&](const float (&)[VE], int i0) { all_of(V + i0); });
            } else {
                all_of(vtop);
            }
        }
        cta_best<NT>(best, ibest, rf, ri);
    }
};

template <int DT>
__global__ void __launch_bounds__(kStatThreads, 2) sample_stats_kernel(const w4a16_sample_args p, const int S,
                                                                    const int filters) {
    constexpr int NT = kStatThreads;
    __shared__ float rf[32];
    __shared__ int ri[32];
    __shared__ int last;
    pdl_wait();
    pdl_launch_dependents();
    const int r = (int)blockIdx.y, rank = (int)blockIdx.x, V = p.vocab;
    const Slice<DT, NT> slice(p.logits, r * p.logits_row, V, rank, S);
    const RowParams q(p, r);
    constexpr int VE = Slice<DT, NT>::VE;
    // (with filters the second kernel runs the race of the rows that have none, beside the other rows' cuts)
    const bool race = q.race && !filters;
    const Pass<DT, NT, true> pass(slice, p.noise + r * p.noise_row, q, race);
    const float mx = pass.mx;
    const int vmax = pass.vmax;
    const float mine = vmax >= 0 ? mx : -INFINITY;  // this thread's largest logit
    float lmax = mine;
    int imax = vmax >= 0 ? (vmax < V ? vmax : vmax - V) : 0x7fffffff;  // the first token of its load
    cta_best<NT>(lmax, imax, rf, ri);
    if (lmax > -INFINITY) {  // the token itself: loads rise with the threads' first tokens, so the lowest holds the lowest
        int at = 0;
#pragma unroll
        for (int x = VE - 1; x > 0; --x)
            if (imax + x < V && slice.at(imax + x) == lmax) at = x;
        if (slice.at(imax) != lmax) imax += at;
    }
    const float sum = cta_sum<NT>(mine == -INFINITY ? 0.f : pass.sum * ex2((mine - lmax) * q.c2), rf);
    float best = -INFINITY;
    int ibest = 0x7fffffff;
    if (race) pass.winner(best, ibest, rf, ri);
    RowSpace* space = space_of(p.workspace, r, S);
    const bool settled = race || q.greedy;  // nothing is left for the second kernel
    if (S == 1 && (settled || !filters)) {
        if (threadIdx.x == 0) write_row<DT, NT>(p, r, slice, q, q.greedy ? imax : ibest, imax, lmax, sum);
        if (!filters) return;
    }
    if (threadIdx.x == 0) {
        SliceStats* s = space->stats + rank;
        s->lmax = lmax;
        s->sum = sum;
        s->best = best;
        s->imax = imax;
        s->ibest = ibest;
        if (rank == 0) space->found = 0;
    }
    if (!settled && !q.race) space->maxima()[rank * NT + threadIdx.x] = mine;
    if (S == 1 || !settled) return;
    // the row's last CTA joins the slices
    if (threadIdx.x == 0) {
        unsigned* counter = static_cast<unsigned*>(p.workspace) + kSampleCounters + r;
        last = arrive(counter) == (unsigned)(S - 1);
        if (last) *counter = 0;
    }
    __syncthreads();
    if (last && threadIdx.x < 32) {
        const RowStats a(space->stats, S, q.c2);
        if (threadIdx.x == 0) write_row<DT, NT>(p, r, slice, q, q.greedy ? a.imax : a.ibest, a.imax, a.lmax, a.sum);
    }
}

// The candidate list, by rising key and then by rising index: bitonic, n a
// power of two, 32 at least.  Steps between entries less than 32 apart stay in
// the registers of a warp.
template <int NT>
W4A16_DEVICE void sort_list(uint32_t* key, int* idx, int n) {
    auto in_warp = [&](int k0, int k1) {  // stages k0 .. k1, their steps of 16 and less
        for (int t = threadIdx.x; t < n; t += NT) {
            uint32_t x = key[t];
            int u = idx[t];
            for (int k = k0; k <= k1; k <<= 1)
                for (int j = min(k >> 1, 16); j > 0; j >>= 1) {
                    const uint32_t y = __shfl_xor_sync(0xffffffffu, x, j);
                    const int v = __shfl_xor_sync(0xffffffffu, u, j);
                    const bool less = y < x || (y == x && v < u);
                    if (less == (((t & k) == 0) == ((t & j) == 0))) {
                        x = y;
                        u = v;
                    }
                }
            key[t] = x;
            idx[t] = u;
        }
    };
    __syncthreads();
    in_warp(2, 32);
    for (int k = 64; k <= n; k <<= 1) {
        for (int j = k >> 1; j >= 32; j >>= 1) {
            __syncthreads();
            for (int t = threadIdx.x; t < n / 2; t += NT) {
                const int a = 2 * t - (t & (j - 1)), b = a + j;
                const uint32_t x = key[a], y = key[b];
                const int u = idx[a], v = idx[b];
                if ((x > y || (x == y && u > v)) == ((a & k) == 0)) {
                    key[a] = y;
                    key[b] = x;
                    idx[a] = v;
                    idx[b] = u;
                }
            }
        }
        __syncthreads();
        in_warp(k, k);
    }
    __syncthreads();
}

// The same for up to 256 entries by counting, for each, the entries before it:
// NT / n threads an entry, 4 entries of the list at a time.  `rank` has room
// for n.  (256 entries: 2.6 k clocks against 5 k.)
template <int NT>
W4A16_DEVICE void sort_few(uint32_t* key, int* idx, int* rank, int n) {
    __syncthreads();
    const int e = (int)threadIdx.x & (n - 1), part = (int)threadIdx.x / n, each = n * n / NT;
    const uint32_t x = key[e];
    const int u = idx[e];
    if ((int)threadIdx.x < n) rank[e] = 0;
    int before = 0;
    for (int j = part * each; j < (part + 1) * each; j += 2) {
        const uint2 y = *reinterpret_cast<const uint2*>(key + j);
        const int2 v = *reinterpret_cast<const int2*>(idx + j);
        before += (y.x < x || (y.x == x && v.x < u)) + (y.y < x || (y.y == x && v.y < u));
    }
    __syncthreads();
    if (before) atomicAdd(rank + e, before);
    __syncthreads();
    if ((int)threadIdx.x < n) {
        const int at = rank[e];
        key[at] = x;
        idx[at] = u;
    }
    __syncthreads();
}

// ---- 2. to 5. filtered rows ------------------------------------------------------
template <int DT>
__global__ void __launch_bounds__(kPickThreads, 2) sample_pick_kernel(const w4a16_sample_args p, const int S) {
    constexpr int NT = kPickThreads;
    __shared__ float rf[32];
    __shared__ int ri[32];
    extern __shared__ unsigned char pick_smem[];
    uint32_t* list_z = reinterpret_cast<uint32_t*>(pick_smem);
    int* list_i = reinterpret_cast<int*>(list_z + kList);
    int* hist = list_i + kList;
    Aside* aside = reinterpret_cast<Aside*>(hist + kBins);  // one a warp
    __shared__ int win[8];    // windows of bins (two), tokens above and between, list length, last arrival
    __shared__ float bound[2];
    pdl_wait();
    pdl_launch_dependents();
    const int r = (int)blockIdx.y, rank = (int)blockIdx.x, V = p.vocab;
    const RowParams q(p, r);
    if (q.greedy) return;
    RowSpace* space = space_of(p.workspace, r, S);
    float top[kMaxSplits];  // maxima of the first pass's threads, distinct tokens of the row
#pragma unroll
    for (int i = 0; i < kMaxSplits; ++i)
        top[i] = i < S && (q.by_k || q.by_p) ? __ldcg(space->maxima() + i * NT + threadIdx.x) : -INFINITY;
    const RowStats st(space->stats, S, q.c2);
    const float T = q.T, lmax = st.lmax, sum = st.sum;
    const float* noise = p.noise + r * p.noise_row;
    const Slice<DT, NT> slice(p.logits, r * p.logits_row, V, rank, S), row(p.logits, r * p.logits_row, V, 0, 1);
    if (lmax == -INFINITY) {
        if (rank == 0 && threadIdx.x == 0) write_row<DT, NT>(p, r, row, q, -1, -1, lmax, sum);
        return;
    }
    const float zmax = z_of(lmax, T);
    const float least = q.by_m ? fminf(logf(q.mp), 0.f) : -INFINITY;  // of z - zmax
    float best = -INFINITY, zbest = 0.f;
    int ibest = 0x7fffffff;
    auto score_of = [&](float z, float e, int i) {
        if (!(z - zmax >= least)) return;
        const float x = z - logf(e);
        if (x > best || (x == best && i < ibest)) {
            best = x;
            ibest = i;
            zbest = z;
        }
    };
    auto score = [&](float z, int i) { score_of(z, noise[i], i); };
    auto settle = [&] {  // the CTA's best: the thread that has it writes
        const int mine = ibest;
        cta_best<NT>(best, ibest, rf, ri);
        if (ibest == 0x7fffffff) {
            if (threadIdx.x == 0) write_row<DT, NT>(p, r, row, q, ibest, st.imax, lmax, sum);
        } else if (mine == ibest) {
            write_token(p, r, ibest, zbest, zmax, sum);
        }
    };
    auto weight = [&](float z) { return ex2((z - zmax) * kLog2E); };
    const bool alone = !q.by_k && !q.by_p;  // min-p alone, whose bound is known, or no filter: every CTA for itself

    // ---- 2. candidates: logits >= low
    // top-p: tokens with z < zmax - R weigh less than V e^-R = (1 - p) sum e^-0.02 together
    float R = 40.f;
    if (q.by_p && !q.by_k) R = fminf(fmaxf(logf((float)V / ((1.f - q.tp) * sum)), 0.f) + 0.02f, 80.f);
    float low = lmax - R * T * 1.0001f;
    bool listed = q.by_p && !q.by_k;  // whether the candidates may be few
    bool all = true;                  // whether every token that may be kept is among them
    const float wide = low, unit = 2147483648.f / sum;
    const int most = min(kList / 2, S * NT / 2);  // maxima that make a good list: so many make ~20 % more tokens
    if (V > kList && (q.by_p || (q.by_k && q.k <= most))) {
        // bins of the maxima, their counts (top-k) or their weights' floors in 2^-31 of the sum (top-p): with
        // `target` in the first bins, the lowest maximum in them bounds the candidates
        float least_top = lmax;
#pragma unroll
        for (int i = 0; i < kMaxSplits; ++i)
            if (top[i] > -INFINITY) least_top = fminf(least_top, top[i]);
        least_top = cta_min<NT>(least_top, rf);
        const float scale = (kTopBins - 2) / fmaxf(fminf(lmax - least_top, 40.f * T), 1e-30f);
        // (of top-p a second time by count, where all maxima do not weigh enough: most nuclei still lie
        // within, and their weight will tell)
        for (int turn = q.by_k ? 1 : 0; turn < 2; ++turn) {
            uint2* bins = reinterpret_cast<uint2*>(hist);
            const uint32_t target = q.by_k ? (uint32_t)q.k
                                    : turn ? (uint32_t)min(S * NT * 7 / 8, kWide * 3 / 8)
                                           : (uint32_t)fmaxf(fminf(q.tp * 1.00001f, 1.f) * 2147483648.f, 1.f);
            __syncthreads();
            bins[threadIdx.x] = make_uint2(0u, 0u);
            if (threadIdx.x == 0) win[0] = kTopBins;
            __syncthreads();
            auto bin_of = [&](float l) { return (int)fminf((lmax - l) * scale, (float)(kTopBins - 1)); };
#pragma unroll
            for (int i = 0; i < kMaxSplits; ++i)
                if (top[i] > -INFINITY)
                    atomicAdd(hist + bin_of(top[i]), turn ? 1 : (int)(uint32_t)(ex2((top[i] - lmax) * q.c2) * unit));
            __syncthreads();
            const uint2 mine = bins[threadIdx.x];
            const uint32_t before = cta_before(mine.x + mine.y, ri);
            if (before < target && before + mine.x + mine.y >= target)
                win[0] = 2 * threadIdx.x + (before + mine.x < target);
            __syncthreads();
            const int cut = win[0];
            if (cut >= kTopBins - 1) continue;  // not reached (or in the last bin, which has no end)
            float tau = lmax;
#pragma unroll
            for (int i = 0; i < kMaxSplits; ++i)
                if (top[i] > -INFINITY && bin_of(top[i]) <= cut) tau = fminf(tau, top[i]);
            // The order is that of the quotients: tokens whose z equals tau's may lie below tau by what one z spans,
            // 2^-23 of |l| at most (2^-149 T where z is subnormal).
            tau = cta_min<NT>(tau, rf);
            tau -= fabsf(tau) * 0x1p-21f + T * 0x1p-148f;
            if (q.by_k || tau > low) {
                low = tau;
                all = q.by_k || turn == 0;
            }
            listed = true;
            break;
        }
    }
    // what min-p drops need not be listed, but where top-p counts within what top-k left
    const float floor_l = (zmax + least) * T - fabsf(zmax * T) * 1e-5f - 1e-5f;  // no token below it passes min-p
    if (q.by_m && !(q.by_k && q.by_p) && floor_l >= low) {
        low = floor_l;
        listed = all = true;
    }
    if (V <= kList) {
        low = -kBig;
        listed = all = true;
    }
    if (alone) {
        if (q.race) {
            Pass<DT, NT, false>(slice, noise, q, true).winner(best, ibest, rf, ri);
        } else {
            slice.from(floor_l, aside, [&](float l, int i) { score(z_of(l, T), i); });
            cta_best<NT>(best, ibest, rf, ri);
        }
        if (threadIdx.x == 0) {
            space->stats[rank].best = best;
            space->stats[rank].ibest = ibest;
        }
    } else if (listed) {
        slice.batches(low, aside, [&](int m, float l, int i) {
            const int lane = (int)threadIdx.x & 31;
            int at = lane == 0 ? atomicAdd(&space->found, m) : 0;
            at = __shfl_sync(0xffffffffu, at, 0) + lane;
            if (lane < m && at < kWide) {
                space->key[at] = ~key_of(z_of(l, T));
                space->index[at] = i;
            }
        });
    }
    // ---- the row's last CTA goes on
    if (S > 1) {
        __syncthreads();
        if (threadIdx.x == 0) {
            unsigned* counter = static_cast<unsigned*>(p.workspace) + kSampleCounters + r;
            win[7] = arrive(counter) == (unsigned)(S - 1);
            if (win[7]) *counter = 0;
        }
        __syncthreads();
        if (!win[7]) return;
    } else {
        __syncthreads();
    }
    if (alone) {
        if (threadIdx.x >= 32) return;
        const RowStats a(space->stats, S, q.c2);
        if (threadIdx.x == 0) write_row<DT, NT>(p, r, row, q, a.ibest, a.imax, lmax, sum);
        return;
    }
    // (the first entries with their number, whether they are there or not)
    const uint32_t key0 = __ldcg(space->key + threadIdx.x);
    const int index0 = __ldcg(space->index + threadIdx.x);
    int n = listed ? __ldcg(&space->found) : kWide + 1;
    // (both cuts on a long list: the second is one of what the first leaves)
    const bool in_bins = n > kFew && n <= kWide && q.by_k != q.by_p;
    bool flat = n > kWide || ((n > kList || !all) && !in_bins);
    if (!flat && !in_bins) {
        if ((int)threadIdx.x < n) {
            list_z[threadIdx.x] = key0;
            list_i[threadIdx.x] = index0;
        }
        for (int i = NT + threadIdx.x; i < n; i += NT) {
            list_z[i] = __ldcg(space->key + i);
            list_i[i] = __ldcg(space->index + i);
        }
    }
    const int k = q.k;
    int above = 0, between = 0;        // tokens above the windows around the cuts, and between them
    float mass_a = 0.f, mass_b = 0.f;  // their weights
    bool slow = false;
    if (in_bins) {
        // bins of z, their counts (top-k) or weights in 2^-31 of the sum (top-p, rounded to nearest: a sum
        // of 8192 is off by 2^-19 of it at most): the cut lies in the bin in which `target` is reached
        const float range = fminf(zmax - z_of(fmaxf(low, -kBig), T), 80.f), scale = (kTopBins - 2) / fmaxf(range, 1e-30f);
        auto bin_of = [&](float z) { return (int)fminf((zmax - z) * scale, (float)(kTopBins - 1)); };
        const uint32_t target = q.by_k ? (uint32_t)k : (uint32_t)fmaxf(fminf(q.tp, 1.f) * 2147483648.f, 1.f);
        uint2* bins = reinterpret_cast<uint2*>(hist);
        bins[threadIdx.x] = make_uint2(0u, 0u);
        if (threadIdx.x == 0) {
            win[0] = kTopBins;
            win[1] = win[6] = 0;
        }
        __syncthreads();
#pragma unroll 4
        for (int i = threadIdx.x; i < n; i += NT) {
            const float z = value_of(~__ldcg(space->key + i));
            atomicAdd(hist + bin_of(z), q.by_k ? 1 : (int)__float2uint_rn(weight(z) * unit));
        }
        __syncthreads();
        const uint2 mine = bins[threadIdx.x];
        const uint32_t before = cta_before(mine.x + mine.y, ri);
        if (before < target && before + mine.x + mine.y >= target) {
            const bool second = before + mine.x < target;
            win[0] = 2 * threadIdx.x + second;
            win[1] = (int)(before + (second ? mine.x : 0u));  // in the bins above
        }
        __syncthreads();
        const int cut = win[0];  // kTopBins: all are kept
#pragma unroll 4
        for (int i = threadIdx.x; i < n; i += NT) {
            const uint32_t y = __ldcg(space->key + i);
            const int x = __ldcg(space->index + i), b = bin_of(value_of(~y));
            if (b < cut) {
                score(value_of(~y), x);
            } else if (b == cut) {
                const int at = atomicAdd(&win[6], 1);
                if (at < kList) {
                    list_z[at] = y;
                    list_i[at] = x;
                }
            }
        }
        __syncthreads();
        n = win[6];
        above = q.by_k ? win[1] : win[1] != 0;  // (of top-p only whether there are any)
        mass_a = q.by_k ? 0.f : (float)(uint32_t)win[1] / unit;
        flat = n > kList || (!all && cut == kTopBins);  // too many equals, or the nucleus reaches below the list
        if (flat) {
            above = 0, mass_a = 0.f;
            __syncthreads();
        }
    }
    if (flat) {
        if (!all) low = wide;
        // ---- 4. too many: bins of equal width in l, from the maximum down
        for (int i = threadIdx.x; i < kBins; i += NT) hist[i] = 0;
        if (threadIdx.x == 0) win[6] = 0;
        const float width = fmaxf((lmax - low) * 1.0001f, 1e-30f);
        // no bin narrower than 4 units in the last place of a logit: equal z lie in one bin or in two neighbours
        const float scale = fminf((kBins - 3) / width, 2097152.f / fmaxf(fmaxf(fabsf(lmax), fabsf(low)), 1e-30f));
        // round((lmax - l) scale), by adding 2^23: never rising with l
        auto bin_of = [&](float l) {
            return (int)(__float_as_uint(fminf((lmax - l) * scale, (float)(kBins - 1)) + 8388608.f) & 0x7fffffu);
        };
        __syncthreads();
        row.from(low, aside, [&](float l, int) { atomicAdd(&hist[bin_of(l)], 1); });
        __syncthreads();
        // thread: PB bins; sums of counts, and of least and greatest weights, before them
        constexpr int PB = kBins / NT;
        const int base = threadIdx.x * PB;
        const float step = q.c2 / scale;  // of the exponent, base 2, a bin
        float cnt[PB], lo[PB], up[PB], ct = 0.f, lt = 0.f, ut = 0.f;
#pragma unroll
        for (int i = 0; i < PB; ++i) {
            cnt[i] = (float)hist[base + i];  // at most 2^24: exact
            lo[i] = cnt[i] * ex2(-((float)(base + i) + 0.51f) * step);
            up[i] = cnt[i] * ex2(fminf(-((float)(base + i) - 0.51f) * step, 0.f));
            ct += cnt[i];
            lt += lo[i];
            ut += up[i];
        }
        const float cb = cta_before(ct, rf), lb = cta_before(lt, rf), ub = cta_before(ut, rf);
        if (threadIdx.x == 0) {
            win[0] = win[1] = win[2] = kBins;
            bound[0] = bound[1] = 0.f;
        }
        __syncthreads();
        if (q.by_k) {  // the bin in which the k-th token lies
            float c = cb, a = lb, u = ub;
#pragma unroll
            for (int i = 0; i < PB; ++i) {
                if (c < (float)k && c + cnt[i] >= (float)k) {
                    win[2] = base + i;
                    bound[0] = a;          // the kept weight is at least this
                    bound[1] = u + up[i];  // and at most this
                }
                c += cnt[i], a += lo[i], u += up[i];
            }
        }
        __syncthreads();
        const int bk = win[2];
        if (q.by_p) {
            const float t_lo = q.tp * (q.by_k ? bound[0] : sum) * 0.9999f;
            const float t_up = q.tp * (q.by_k ? bound[1] : sum) * 1.0001f;
            float a = lb, u = ub;
#pragma unroll
            for (int i = 0; i < PB; ++i) {
                u += up[i];
                a += lo[i];
                if (u >= t_lo) atomicMin(&win[0], base + i);  // the cut is in this bin or below
                if (a >= t_up) atomicMin(&win[1], base + i);  // in this bin or above
            }
        }
        __syncthreads();
        int b1 = win[0], b2 = win[1];
        // (a k-th token at the end of a range that the maxima do not bound: its equals may lie below it)
        const int end = q.by_k && low == wide ? min(bin_of(low), kBins) - 1 : kBins - 1;
        slow = (q.by_k && bk >= end) || (q.by_p && (q.by_k ? b1 : b2) >= kBins - 1);
        // equal z may have unequal l, one bin apart at most: a bin more on each side
        if (q.by_k && b2 > bk) b2 = bk;
        if (!q.by_p) b1 = b2 = bk;
        b1 = max(b1 - 1, 0);
        b2 = min(b2 + 1, kBins - 1);
        int bk1 = q.by_k ? max(bk - 1, 0) : kBins, bk2 = q.by_k ? min(bk + 1, kBins - 1) : kBins - 1;
        if (q.by_k && bk1 <= b2 + 1) {  // one window
            b2 = bk2;
            bk1 = kBins;
        }
        const bool apart = bk1 < kBins;
        if (!slow) {
            int ca = 0, cc = 0;
#pragma unroll
            for (int i = 0; i < PB; ++i) {
                const int b = base + i;
                if (b < b1) ca += (int)cnt[i];
                if (apart && b > b2 && b < bk1) cc += (int)cnt[i];
            }
            above = cta_count<NT>(ca, ri);
            between = cta_count<NT>(cc, ri);
            row.from(low, aside, [&](float l, int i) {
                const int b = bin_of(l);
                if (b < b1) {
                    const float z = z_of(l, T);
                    mass_a += weight(z);
                    score(z, i);
                } else if (b <= b2 || (apart && b >= bk1 && b <= bk2)) {
                    const int at = atomicAdd(&win[6], 1);
                    if (at < kList) {
                        list_z[at] = ~key_of(z_of(l, T));
                        list_i[at] = i;
                    }
                } else if (apart && b < bk1) {
                    mass_b += weight(z_of(l, T));
                }
            });
            mass_a = cta_sum<NT>(mass_a, rf);
            mass_b = cta_sum<NT>(mass_b, rf);
            n = win[6];
            slow = n > kList;
        }
    }
    if (!slow) {
        // ---- 3. the list decides
        int size = 32;
        while (size < n) size <<= 1;
        for (int i = n + (int)threadIdx.x; i < size; i += NT) {
            list_z[i] = 0xffffffffu;
            list_i[i] = 0x7fffffff;
        }
        if (size <= kFew)
            sort_few<NT>(list_z, list_i, hist, size);
        else
            sort_list<NT>(list_z, list_i, size);
        constexpr int PL = kList / NT;
        const int per = max(size / NT, 1), base = (int)threadIdx.x * per;  // entries a thread, and its first
        // entries that top-k keeps (a second window lies behind `between` tokens)
        const int kept_k = q.by_k ? min(n, k - above - between) : n;
        float w[PL], wt = 0.f;
#pragma unroll
        for (int i = 0; i < PL; ++i) {
            w[i] = i < per && base + i < kept_k ? weight(value_of(~list_z[base + i])) : 0.f;
            wt += w[i];
        }
        const float before = cta_before(wt, rf), listed_mass = cta_sum<NT>(wt, rf);
        const float total = q.by_k ? mass_a + mass_b + listed_mass : sum;
        const float want = q.by_p ? q.tp * total : INFINITY;
        float at = mass_a + before, z[PL], e[PL];
#pragma unroll
        for (int i = 0; i < PL; ++i) {  // the kept ones' random numbers, all on their way
            const int x = base + i;
            const bool kept = i < per && x < kept_k && (!q.by_p || at < want || (above == 0 && x == 0));
            z[i] = kept ? value_of(~list_z[x]) : 0.f;
            e[i] = kept ? noise[list_i[x]] : NAN;  // (takes no part)
            at += w[i];
        }
#pragma unroll
        for (int i = 0; i < PL; ++i) score_of(z[i], e[i], list_i[min(base + i, kList - 1)]);
    }
    if (slow) {
        // ---- 5. bisection
        best = -INFINITY, ibest = 0x7fffffff;
        uint32_t cut = 0;  // keys above it are kept, and `ties` of those equal to it
        int ties = V;
        auto count = [&](uint32_t c) {
            int m = 0;
            row.from(-INFINITY, aside, [&](float l, int) { m += key_of(z_of(l, T)) >= c; });
            return cta_count<NT>(m, ri);
        };
        if (q.by_k) {
            uint32_t lo = 0, hi = key_of(zmax);
            while (lo < hi) {
                const uint32_t mid = lo + (hi - lo + 1) / 2;
                if (count(mid) >= k) lo = mid; else hi = mid - 1;
            }
            cut = lo;
            ties = k - count(cut + 1);
        }
        if (q.by_p) {
            const bool by_k = q.by_k && cut > 0;  // (0: top-k takes all there are, and no token has that key)
            const float wcut = by_k ? weight(value_of(cut)) : 0.f;
            const uint32_t top = cut;
            const int top_ties = ties;
            auto mass = [&](uint32_t c) {  // weight of the kept tokens with a key >= c
                float s = 0.f;
                row.from(-INFINITY, aside, [&](float l, int) {
                    const float z = z_of(l, T);
                    const uint32_t y = key_of(z);
                    if (y >= c && y > top) s += weight(z);
                });
                return cta_sum<NT>(s, rf) + (by_k && c <= top ? (float)top_ties * wcut : 0.f);
            };
            const float want = q.tp * mass(top);
            uint32_t lo = top, hi = key_of(zmax);
            while (lo < hi) {  // the largest key at and above which the weight reaches `want`
                const uint32_t mid = lo + (hi - lo + 1) / 2;
                if (mass(mid) >= want) lo = mid; else hi = mid - 1;
            }
            const float over = mass(lo + 1), wt = weight(value_of(lo));
            const int here = by_k && lo == top ? top_ties : count(lo) - count(lo + 1);
            cut = lo;
            ties = 1;
            if (wt > 0.f && over + wt < want) {  // tie i stays while over + i wt < want
                int a = 1, b = here;
                while (a < b) {
                    const int mid = (a + b) / 2;
                    if (over + (float)mid * wt < want) a = mid + 1; else b = mid;
                }
                ties = a;
            }
        }
        int lo = 0, hi = V;  // the smallest end with `ties` ties before it
        while (lo < hi) {
            const int mid = (lo + hi) / 2;
            int m = 0;
            row.from(-INFINITY, aside, [&](float l, int i) { m += i < mid && key_of(z_of(l, T)) == cut; });
            if (cta_count<NT>(m, ri) >= ties) hi = mid; else lo = mid + 1;
        }
        row.from(-INFINITY, aside, [&](float l, int i) {
            const float z = z_of(l, T);
            const uint32_t y = key_of(z);
            if (l > -INFINITY && (y > cut || (y == cut && i < lo))) score(z, i);
        });
    }
    settle();
}

// CTAs a row, of slices of 4096 tokens at least.  Two CTAs share an SM, and a
// CTA costs about as much as 6000 tokens beside its slice, so the fewest
// (waves) x (slice + 6000) is taken; with filters 4 at least, whose threads'
// maxima are what the candidates are found by.  (Rows of 151936: 256 f32 rows
// without filters, 1 CTA a row 45.9 us, 2 52.4, 4 58.4; 64 bf16 rows with
// filters, 2 33.0 us, 4 26.2, 8 33.5; one row, 4 16.7 us, 8 15.4.)
static int splits_of(int rows, int vocab, bool filters, int sms) {
    if (rows > kSampleSplitRows) return 1;
    int best = 1;
    int64_t least = INT64_MAX;
    for (int S = 1; S <= kMaxSplits && (S == 1 || vocab / S >= 4096); S <<= 1) {
        const int64_t waves = ((int64_t)rows * S + 2 * sms - 1) / (2 * sms), cost = waves * (vocab / S + 6000);
        if (cost < least || (filters && S <= 4)) {
            best = S;
            least = cost;
        }
    }
    return best;
}

size_t sample_workspace(int rows, int vocab, bool filters, int sms) {
    if (!filters && splits_of(rows, vocab, filters, sms) == 1) return 0;
    return kCounterBytes + rows * row_space(splits_of(rows, vocab, filters, sms));
}

template <int DT>
static cudaError_t launch(const w4a16_sample_args& a, int S, cudaStream_t s) {
    const bool pdl = (a.flags & W4A16_FLAG_PDL) != 0;
    const int filters = a.top_k || a.top_p || a.min_p;
    const dim3 grid((unsigned)S, (unsigned)a.rows);
    cudaError_t e = launch_kernel(sample_stats_kernel<DT>, grid, dim3(kStatThreads), 0, s, pdl, a, S, filters);
    if (e != cudaSuccess) return e;
    note_launch();
    if (!filters) return cudaSuccess;
    constexpr int smem = kList * 8 + kBins * 4 + kPickThreads / 32 * (int)sizeof(Aside);
    static bool set_for[64];
    int dev = 0;
    e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!set_for[dev]) {
        e = cudaFuncSetAttribute(sample_pick_kernel<DT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        set_for[dev] = true;
    }
    e = launch_kernel(sample_pick_kernel<DT>, grid, dim3(kPickThreads), (size_t)smem, s, pdl, a, S);
    if (e == cudaSuccess) note_launch();
    return e;
}

cudaError_t launch_sample(const w4a16_sample_args& a, int sms, cudaStream_t s) {
    const int S = splits_of(a.rows, a.vocab, a.top_k || a.top_p || a.min_p, sms);
    if (a.dtype == W4A16_F32) return launch<W4A16_F32>(a, S, s);
    if (a.dtype == W4A16_BF16) return launch<W4A16_BF16>(a, S, s);
    return launch<W4A16_F16>(a, S, s);
}

}  // namespace w4a16
