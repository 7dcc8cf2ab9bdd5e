// Attention over 8-bit caches and of trees of drafted tokens: a warp takes one
// token and head and goes through its positions one by one.
#include "codes.cuh"
#include "paged_attn.cuh"

namespace w4a16 {

template <typename Ty, int D, bool Q8>
__global__ void __launch_bounds__(256) paged_simple_kernel(const __grid_constant__ PagedAttnParams p) {
    pdl_wait();
    pdl_launch_dependents();
    const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31, t = (int)(w / p.Hq), h = (int)(w % p.Hq), hk = h / p.G;
    if (t >= p.T || t >= p.q_start[p.B]) return;
    int lo = 0, hi = p.B;  // the last request that begins at t or before it and has a token
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.q_start[mid] <= t) lo = mid; else hi = mid;
    }
    const Request r = request_of(p, lo);
    if (r.n * p.G <= p.small_rows) return;
    constexpr int N = D / 32;
    float q[N], o[N] = {};
    const uint16_t* qp = p.q + t * p.q_token + h * p.q_head + lane * N;
    for (int i = 0; i < N; ++i) q[i] = Ty::lo(qp[i]);
    const int past = r.L - r.n;
    int e = last_seen(p, r, t - r.t0), first = first_seen(p, e);
    const uint32_t* mask = nullptr;
    if (p.tree) {
        mask = p.tree + t * p.tree_token;
        int c = 0;
        for (int k = 0; k < r.n && k < 32 * p.words; ++k) c += (mask[k >> 5] >> (k & 31)) & 1;
        e = r.L - 1;
        first = p.window > 0 ? max(0, past + c - p.window) : 0;
    }
    float m = -INFINITY, l = 0.f;
    const int* table = p.table + (int64_t)lo * p.table_stride;
    for (int j = mask ? 0 : first; j <= e; ++j) {
        if (mask) {
            if (j < past && j < first) continue;
            const int k = j - past;
            if (k >= 0 && (k >= 32 * p.words || !((mask[k >> 5] >> (k & 31)) & 1))) continue;
        }
        const int pg = table[j >> p.shift];
        if (pg < 0 || pg >= p.pages) continue;
        const int64_t sl = j & ((1 << p.shift) - 1);
        float s = 0.f, v[N];
        const int64_t ka = pg * p.kp + hk * p.kh + sl * p.ks + lane * N, va = pg * p.vp + hk * p.vh + sl * p.vs + lane * N;
        float kscale = 1.f, vscale = 1.f;
        if constexpr (Q8) {
            kscale = finite_or_nan(p.k_scale[pg * p.ksp + hk * p.ksh + sl * p.kss]);
            vscale = finite_or_nan(p.v_scale[pg * p.vsp + hk * p.vsh + sl * p.vss]);
            const uint8_t *k8 = reinterpret_cast<const uint8_t*>(p.k) + ka, *v8 = reinterpret_cast<const uint8_t*>(p.v) + va;
            for (int i = 0; i < N; ++i) {
                s = fmaf(q[i], p.e4m3 ? code_value<true>(k8[i]) : code_value<false>(k8[i]), s);
                v[i] = p.e4m3 ? code_value<true>(v8[i]) : code_value<false>(v8[i]);
            }
        } else {
            for (int i = 0; i < N; ++i) {
                s = fmaf(q[i], Ty::lo(p.k[ka + i]), s);
                v[i] = Ty::lo(p.v[va + i]);
            }
        }
        for (int d = 1; d < 32; d <<= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        s *= kscale * p.scale2;
        const float n = fmaxf(m, s), f = n == -INFINITY ? 1.f : exp2f(m - n), x = s == -INFINITY ? 0.f : exp2f(s - n);
        l = l * f + x;
        for (int i = 0; i < N; ++i) o[i] = o[i] * f + (s == -INFINITY ? 0.f : x * vscale * v[i]);
        m = n;
    }
    uint16_t* out = p.out + t * p.o_token + h * p.o_head + lane * N;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    for (int i = 0; i < N; i += 2) *reinterpret_cast<uint32_t*>(out + i) = Ty::pack(o[i] * inv, o[i + 1] * inv);
    if (p.lse && lane == 0) p.lse[(int64_t)t * p.Hq + h] = l == 0.f ? -INFINITY : kLn2 * (m + log2f(l));
}

cudaError_t launch_paged_simple(const PagedAttnParams& p, bool bf16, int d, cudaStream_t s, bool pdl) {
    const dim3 grid((unsigned)(((int64_t)p.T * p.Hq + 7) / 8));
    auto run = [&](auto kernel) { return launch_kernel(kernel, grid, dim3(256), 0, s, pdl, p); };
    if (p.k_scale) {
        if (bf16) return d == 128 ? run(paged_simple_kernel<Bf16, 128, true>) : run(paged_simple_kernel<Bf16, 64, true>);
        return d == 128 ? run(paged_simple_kernel<F16, 128, true>) : run(paged_simple_kernel<F16, 64, true>);
    }
    if (bf16) return d == 128 ? run(paged_simple_kernel<Bf16, 128, false>) : run(paged_simple_kernel<Bf16, 64, false>);
    return d == 128 ? run(paged_simple_kernel<F16, 128, false>) : run(paged_simple_kernel<F16, 64, false>);
}

}  // namespace w4a16
