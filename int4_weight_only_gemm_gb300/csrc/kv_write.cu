// New keys and values into the paged cache, in one launch.
//
//     cache[slot / p][h][slot % p] = x[t][h]   for slot = slot_map[t] in range
//
// A thread moves one 16-byte piece of a key and the same piece of the value,
// for kKvRun tokens (kKvStep apart) with all their loads in flight; the pieces
// of a token are consecutive threads, so reads and writes are whole rows.
// Bound: HBM (each byte read once and written once).
#include "common.cuh"
#include "kernels.h"

namespace w4a16 {

constexpr int kKvThreads = 256;

struct KvWriteParams {
    w4a16_kv_write_args a;
    int shift, pieces, per_head;     // pieces of 8 elements in a token and in a head
    uint32_t pm, hm;                 // divisions by them (FastDiv)
    int ps, hs;
    int64_t slots;                   // num_pages * page_size
};

template <int RUN>
__global__ void __launch_bounds__(kKvThreads) kv_write_kernel(const KvWriteParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const w4a16_kv_write_args& a = p.a;
    const int64_t total = (int64_t)a.tokens * p.pieces, stride = (int64_t)gridDim.x * kKvThreads;
    for (int64_t i0 = (int64_t)blockIdx.x * kKvThreads + threadIdx.x; i0 < total; i0 += stride * RUN) {
        uint4 k[RUN], v[RUN];
        int slot[RUN], h[RUN], c[RUN];
#pragma unroll
        for (int u = 0; u < RUN; ++u) {
            const int64_t i = i0 + u * stride;
            slot[u] = -1;
            if (i < total) {
                const int t = (int)(i / p.pieces), r = (int)(i - (int64_t)t * p.pieces);
                h[u] = div_by(r, p.hm, p.hs);
                c[u] = (r - h[u] * p.per_head) * 8;
                slot[u] = a.slot_map[t];
                k[u] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.k) + t * a.k_token +
                                                            h[u] * a.k_head + c[u]));
                v[u] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.v) + t * a.v_token +
                                                            h[u] * a.v_head + c[u]));
            }
        }
#pragma unroll
        for (int u = 0; u < RUN; ++u) {
            if (slot[u] < 0 || slot[u] >= p.slots) continue;
            const int64_t pg = slot[u] >> p.shift, sl = slot[u] & ((1 << p.shift) - 1);
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.k_cache) + pg * a.kc_page + h[u] * a.kc_head +
                                      sl * a.kc_slot + c[u]) = k[u];
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.v_cache) + pg * a.vc_page + h[u] * a.vc_head +
                                      sl * a.vc_slot + c[u]) = v[u];
        }
    }
}

cudaError_t launch_kv_write(const w4a16_kv_write_args& a, int sms, cudaStream_t s) {
    KvWriteParams p;
    p.a = a;
    p.shift = 0;
    while ((1 << p.shift) < a.page_size) ++p.shift;
    p.per_head = a.head_dim / 8;
    p.pieces = p.per_head * a.heads;
    const FastDiv fh = fast_div(p.per_head), fp = fast_div(p.pieces);
    p.hm = fh.m;
    p.hs = fh.s;
    p.pm = fp.m;
    p.ps = fp.s;
    p.slots = (int64_t)a.num_pages * a.page_size;
    const int64_t total = (int64_t)a.tokens * p.pieces;
    const int64_t ctas = (total + kKvThreads - 1) / kKvThreads;
    return launch_kernel(kv_write_kernel<1>, dim3((unsigned)(ctas < 65536 ? ctas : 65536)), dim3(kKvThreads), 0, s,
                         (a.flags & W4A16_FLAG_PDL) != 0, p);
}

}  // namespace w4a16
