// Cached keys and values back as 16-bit rows, in one launch.
//
//     x[t][h] = scale * code,  code and scale from slot slot_map[t]
//
// A thread makes a piece of a key and the same piece of the value, of 16 bytes of
// the cache (8 numbers or 16 codes); the pieces of a token are consecutive
// threads.  Bound: HBM, each byte read and written once.  Measured: 32768 tokens, 8
// heads of 128 from int8 (204 MB): 36.6 us, 5.6 TB/s; 300 tokens: the 7.4 us of a call.
#include "codes.cuh"
#include "kernels.h"
#include "paged_attn.cuh"

namespace w4a16 {

constexpr int kReadThreads = 256;

struct KvReadParams {
    w4a16_kv_read_args a;
    int shift, pieces, per_head;  // pieces of a token and of a head
    FastDiv by_head, by_token;
    int64_t slots;
};

template <typename Ty, bool E4M3>
W4A16_DEVICE uint4 values_of(uint32_t lo, uint32_t hi, float scale) {
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w = (i < 2 ? lo : hi) >> (16 * (i & 1));
        r[i] = Ty::pack(code_value<E4M3>(w & 0xffu) * scale, code_value<E4M3>((w >> 8) & 0xffu) * scale);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// CODE: 0 a 16-bit cache, 1 int8, 2 e4m3
template <typename Ty, int CODE>
__global__ void __launch_bounds__(kReadThreads) kv_read_kernel(const KvReadParams p) {
    pdl_wait();
    pdl_launch_dependents();
    const w4a16_kv_read_args& a = p.a;
    const int64_t total = (int64_t)a.tokens * p.pieces, stride = (int64_t)gridDim.x * kReadThreads;
    for (int64_t i = (int64_t)blockIdx.x * kReadThreads + threadIdx.x; i < total; i += stride) {
        const int t = total < (1ll << 31) ? div_by((int)i, p.by_token.m, p.by_token.s) : (int)(i / p.pieces);
        const int r = (int)(i - (int64_t)t * p.pieces), h = div_by(r, p.by_head.m, p.by_head.s);
        const int c = (r - h * p.per_head) * (CODE ? 16 : 8), slot = a.slot_map[t];
        if (slot < 0 || slot >= p.slots) continue;
        const int64_t pg = slot >> p.shift, sl = slot & ((1 << p.shift) - 1);
        const int64_t ka = pg * a.kc_page + h * a.kc_head + sl * a.kc_slot + c, va = pg * a.vc_page + h * a.vc_head + sl * a.vc_slot + c;
        constexpr int size = CODE ? 1 : 2;
        const uint4 k = __ldg(reinterpret_cast<const uint4*>(static_cast<const char*>(a.k_cache) + ka * size));
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(static_cast<const char*>(a.v_cache) + va * size));
        uint4* ko = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.k) + t * a.k_token + h * a.k_head + c);
        uint4* vo = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.v) + t * a.v_token + h * a.v_head + c);
        if constexpr (CODE == 0) {
            *ko = k;
            *vo = v;
        } else {
            const float ks = finite_or_nan(__ldg(a.k_scale + pg * a.ks_page + h * a.ks_head + sl * a.ks_slot));
            const float vs = finite_or_nan(__ldg(a.v_scale + pg * a.vs_page + h * a.vs_head + sl * a.vs_slot));
            ko[0] = values_of<Ty, CODE == 2>(k.x, k.y, ks);
            ko[1] = values_of<Ty, CODE == 2>(k.z, k.w, ks);
            vo[0] = values_of<Ty, CODE == 2>(v.x, v.y, vs);
            vo[1] = values_of<Ty, CODE == 2>(v.z, v.w, vs);
        }
    }
}

cudaError_t launch_kv_read(const w4a16_kv_read_args& a, cudaStream_t s) {
    KvReadParams p;
    p.a = a;
    p.shift = 0;
    while ((1 << p.shift) < a.page_size) ++p.shift;
    p.per_head = a.head_dim / (a.cache_dtype == a.dtype ? 8 : 16);
    p.pieces = p.per_head * a.heads;
    p.by_head = fast_div(p.per_head);
    p.by_token = fast_div(p.pieces);
    p.slots = (int64_t)a.num_pages * a.page_size;
    const int64_t total = (int64_t)a.tokens * p.pieces, ctas = (total + kReadThreads - 1) / kReadThreads;
    auto run = [&](auto kernel) {
        return launch_kernel(kernel, dim3((unsigned)(ctas < 65536 ? ctas : 65536)), dim3(kReadThreads), 0, s,
                             (a.flags & W4A16_FLAG_PDL) != 0, p);
    };
    if (a.cache_dtype == a.dtype) return run(kv_read_kernel<Bf16, 0>);
    const bool e4m3 = a.cache_dtype == W4A16_E4M3;
    if (a.dtype == W4A16_BF16) return e4m3 ? run(kv_read_kernel<Bf16, 2>) : run(kv_read_kernel<Bf16, 1>);
    return e4m3 ? run(kv_read_kernel<F16, 2>) : run(kv_read_kernel<F16, 1>);
}

}  // namespace w4a16
