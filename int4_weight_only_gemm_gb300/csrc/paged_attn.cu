// Attention of the new tokens over a paged cache: one warp per query row.
#include "paged_attn.cuh"

namespace w4a16 {

template <typename Ty, int D>
__global__ void __launch_bounds__(128) paged_attn_rows_kernel(const PagedAttnParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int t = (int)(row / p.Hq), h = (int)(row - (int64_t)t * p.Hq);
    if (t >= p.T || t >= p.q_start[p.B]) return;
    int lo = 0, hi = p.B;  // the last request that starts at or before t
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.q_start[mid] <= t) lo = mid; else hi = mid;
    }
    const Request r = request_of(p, lo);
    attn_row<Ty, D>(p, lo, r, t - r.t0, h);
}

size_t paged_attn_workspace(int, int, int, int, int, int, int) { return 0; }

cudaError_t launch_paged_attn(const w4a16_paged_attention_args& a, int, cudaStream_t s) {
    PagedAttnParams p;
    p.q = static_cast<const uint16_t*>(a.q);
    p.k = static_cast<const uint16_t*>(a.k_cache);
    p.v = static_cast<const uint16_t*>(a.v_cache);
    p.table = a.block_table;
    p.q_start = a.q_start;
    p.kv_len = a.kv_len;
    p.out = static_cast<uint16_t*>(a.out);
    p.lse = a.lse;
    p.q_token = a.q_token; p.q_head = a.q_head; p.o_token = a.out_token; p.o_head = a.out_head;
    p.kp = a.kc_page; p.kh = a.kc_head; p.ks = a.kc_slot;
    p.vp = a.vc_page; p.vh = a.vc_head; p.vs = a.vc_slot;
    p.table_stride = a.table_stride;
    p.T = a.tokens; p.B = a.requests; p.Hq = a.q_heads; p.Hkv = a.kv_heads; p.G = a.q_heads / a.kv_heads;
    p.pages = a.num_pages; p.columns = a.columns;
    p.shift = 0;
    while ((1 << p.shift) < a.page_size) ++p.shift;
    p.window = a.window; p.block = a.block;
    p.scale2 = (a.scale == 0.f ? 1.f / sqrtf((float)a.head_dim) : a.scale) * 1.4426950408889634f;
    const bool pdl = (a.flags & W4A16_FLAG_PDL) != 0;
    const int64_t rows = (int64_t)a.tokens * a.q_heads;
    const dim3 grid((unsigned)((rows + 3) / 4)), block(128);
    note_launch();
    if (a.dtype == W4A16_BF16)
        return a.head_dim == 128 ? launch_kernel(paged_attn_rows_kernel<Bf16, 128>, grid, block, 0, s, pdl, p)
                                 : launch_kernel(paged_attn_rows_kernel<Bf16, 64>, grid, block, 0, s, pdl, p);
    return a.head_dim == 128 ? launch_kernel(paged_attn_rows_kernel<F16, 128>, grid, block, 0, s, pdl, p)
                             : launch_kernel(paged_attn_rows_kernel<F16, 64>, grid, block, 0, s, pdl, p);
}

}  // namespace w4a16
