// Sampling with temperature, top-k, top-p and min-p from given random numbers:
// one CTA a row.
//
// The three filters keep a beginning of the row's order (falling z, equal ones
// by rising index), so what they keep together is one cut: the tokens whose
// order-preserving key is above the cut's, and the first `ties` of those whose
// key equals it.  Keys and counts are integers, and sums are added in a fixed
// order, so a row's token does not depend on timing.
#include "common.cuh"
#include "kernels.h"

namespace w4a16 {

constexpr int kSampleThreads = 1024;

// order-preserving map of f32 to unsigned (no NaN): a < b <=> key(a) < key(b)
W4A16_DEVICE uint32_t key_of(float z) {
    const uint32_t u = __float_as_uint(z);
    return (u >> 31) ? ~u : (u | 0x80000000u);
}
W4A16_DEVICE float value_of(uint32_t k) { return __uint_as_float((k >> 31) ? (k & 0x7fffffffu) : ~k); }

template <int DT>
W4A16_DEVICE float load_logit(const void* row, int i) {
    if constexpr (DT == W4A16_F32) return __ldg(static_cast<const float*>(row) + i);
    const uint16_t b = __ldg(static_cast<const uint16_t*>(row) + i);
    if constexpr (DT == W4A16_BF16) return __uint_as_float((uint32_t)b << 16);
    return f16_bits_to_f32(b);
}

// z of a logit: NaN counts as -inf, +inf as the largest finite value; -0 as 0
W4A16_DEVICE float z_of(float x, float t) {
    const float z = __fdiv_rn(x, t);
    return z != z ? -INFINITY : fminf(z, 3.402823466e38f) + 0.f;
}

struct Red {
    float f[32];
    int i[32];
};
// sum / maximum over the CTA, the same value in every thread, added in a fixed order
W4A16_DEVICE float cta_sum(float x, Red& r) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) r.f[threadIdx.x >> 5] = x;
    __syncthreads();
    x = r.f[threadIdx.x & 31];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}
W4A16_DEVICE int cta_sum(int x, Red& r) {
    x = __reduce_add_sync(0xffffffffu, x);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) r.i[threadIdx.x >> 5] = x;
    __syncthreads();
    return __reduce_add_sync(0xffffffffu, r.i[threadIdx.x & 31]);
}
// the largest x, and among equal ones the lowest index
W4A16_DEVICE void cta_best(float& x, int& i, Red& r) {
    auto join = [&](float y, int j) {
        if (y > x || (y == x && j < i)) {
            x = y;
            i = j;
        }
    };
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) join(__shfl_xor_sync(0xffffffffu, x, d), __shfl_xor_sync(0xffffffffu, i, d));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) {
        r.f[threadIdx.x >> 5] = x;
        r.i[threadIdx.x >> 5] = i;
    }
    __syncthreads();
    x = r.f[threadIdx.x & 31];
    i = r.i[threadIdx.x & 31];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) join(__shfl_xor_sync(0xffffffffu, x, d), __shfl_xor_sync(0xffffffffu, i, d));
}

template <int DT>
__global__ void __launch_bounds__(kSampleThreads) sample_kernel(const w4a16_sample_args p) {
    __shared__ Red red;
    pdl_launch_dependents();
    pdl_wait();
    const int r = blockIdx.x, V = p.vocab;
    const void* row = DT == W4A16_F32 ? (const void*)(static_cast<const float*>(p.logits) + r * p.logits_row)
                                      : (const void*)(static_cast<const uint16_t*>(p.logits) + r * p.logits_row);
    const float* noise = p.noise + r * p.noise_row;
    const float temp = p.temperature ? p.temperature[r] : 1.f;
    const bool greedy = !(temp > 0.f);
    const float t = greedy ? 1.f : temp;
    auto z_at = [&](int i) { return z_of(load_logit<DT>(row, i), t); };

    float zmax = -INFINITY;
    int imax = V;
    for (int i = threadIdx.x; i < V; i += kSampleThreads) {
        const float z = z_at(i);
        if (z > zmax) {
            zmax = z;
            imax = i;
        }
    }
    cta_best(zmax, imax, red);
    if (zmax == -INFINITY) {
        if (threadIdx.x == 0) {
            p.token[r] = -1;
            if (p.logprob) p.logprob[r] = -INFINITY;
        }
        return;
    }
    float sum = 0.f;
    for (int i = threadIdx.x; i < V; i += kSampleThreads) sum += expf(z_at(i) - zmax);
    sum = cta_sum(sum, red);

    int token = imax;
    if (!greedy) {
        // the cut: keys above `cut` are kept, and `ties` of those equal to it
        uint32_t cut = 0;
        int ties = V;
        const int k = p.top_k ? p.top_k[r] : 0;
        auto count = [&](uint32_t c) {  // tokens with a key >= c
            int n = 0;
            for (int i = threadIdx.x; i < V; i += kSampleThreads) n += key_of(z_at(i)) >= c;
            return cta_sum(n, red);
        };
        if (k > 0 && k < V) {
            for (int b = 31; b >= 0; --b)
                if (count(cut | (1u << b)) >= k) cut |= 1u << b;
            ties = k - (cut == 0xffffffffu ? 0 : count(cut + 1));
        }
        const float tp = p.top_p ? p.top_p[r] : 1.f;
        if (tp < 1.f) {
            // mass of the kept tokens above a key; the ties of the top-k cut share one value
            const float wcut = expf(value_of(cut) - zmax);
            auto mass = [&](uint32_t c) {
                float s = 0.f;
                for (int i = threadIdx.x; i < V; i += kSampleThreads) {
                    const float z = z_at(i);
                    const uint32_t y = key_of(z);
                    if (y >= c && y > cut) s += expf(z - zmax);
                }
                return cta_sum(s, red) + (c <= cut && cut != 0 ? ties * wcut : 0.f);
            };
            const float want = tp * mass(cut);
            // the largest key at and above which the kept mass reaches `want`
            uint32_t lo = cut, hi = key_of(zmax);
            while (lo < hi) {
                const uint32_t mid = lo + (hi - lo + 1) / 2;
                if (mass(mid) >= want) lo = mid; else hi = mid - 1;
            }
            const uint32_t c = lo;
            const float above = c == 0xffffffffu ? 0.f : mass(c + 1), w = expf(value_of(c) - zmax);
            int n = c == cut ? ties : count(c) - count(c + 1);
            int keep = 1;
            while (keep < n && above + keep * w < want) ++keep;
            cut = c;
            ties = keep;
        }
        const float mp = p.min_p ? p.min_p[r] : 0.f;
        const float least = mp > 0.f ? fminf(logf(mp), 0.f) : -INFINITY;
        // the index below which the ties of the cut are kept
        int end = V;
        {
            int lo = 0, hi = V;  // the smallest end with at least `ties` ties before it
            while (lo < hi) {
                const int mid = (lo + hi) / 2;
                int n = 0;
                for (int i = threadIdx.x; i < mid; i += kSampleThreads) n += key_of(z_at(i)) == cut;
                if (cta_sum(n, red) >= ties) hi = mid; else lo = mid + 1;
            }
            end = lo;
        }
        float best = -INFINITY;
        token = V;
        for (int i = threadIdx.x; i < V; i += kSampleThreads) {
            const float z = z_at(i);
            const uint32_t y = key_of(z);
            if (z == -INFINITY || y < cut || (y == cut && i >= end) || !(z - zmax >= least)) continue;
            const float score = z - logf(noise[i]);
            if (score > best || (score == best && i < token)) {
                best = score;
                token = i;
            }
        }
        cta_best(best, token, red);
        if (token >= V) token = imax;  // every noise of the kept tokens was infinite or NaN
    }
    if (threadIdx.x == 0) {
        p.token[r] = token;
        if (p.logprob) p.logprob[r] = (z_at(token) - zmax) - logf(sum);
    }
}

cudaError_t launch_sample(const w4a16_sample_args& a, int, cudaStream_t s) {
    const bool pdl = (a.flags & W4A16_FLAG_PDL) != 0;
    const dim3 grid((unsigned)a.rows), block(kSampleThreads);
    note_launch();
    if (a.dtype == W4A16_F32) return launch_kernel(sample_kernel<W4A16_F32>, grid, block, 0, s, pdl, a);
    if (a.dtype == W4A16_BF16) return launch_kernel(sample_kernel<W4A16_BF16>, grid, block, 0, s, pdl, a);
    return launch_kernel(sample_kernel<W4A16_F16>, grid, block, 0, s, pdl, a);
}

}  // namespace w4a16
