// Attention of the new tokens over a paged cache: tensor maps, workspace, and
// which kernel takes a request -- the small-row kernel (paged_decode.cu) up to
// kSmallRows query rows a key head, the chunk kernel (paged_chunk.cu) above.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "paged_attn.cuh"

namespace w4a16 {

static PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
        return nullptr;
    }();
    return fn;
}

bool paged_tmap(CUtensorMap* m, const PagedAttnParams& p, bool bf16, int d, bool values, int rows) {
    auto encode = encoder();
    if (!encode) return false;
    const uint64_t page = 1ull << p.shift;
    // a dimension of one entry takes any stride: the row's, so that it is a valid one
    const uint64_t ss = (uint64_t)(values ? p.vs : p.ks) * 2;
    const uint64_t hs = p.Hkv == 1 ? ss : (uint64_t)(values ? p.vh : p.kh) * 2;
    const uint64_t ps = p.pages == 1 ? ss : (uint64_t)(values ? p.vp : p.kp) * 2;
    const cuuint64_t dims[4] = {(cuuint64_t)d, page, (cuuint64_t)p.Hkv, (cuuint64_t)p.pages};
    const cuuint64_t strides[3] = {ss, hs, ps};
    const cuuint32_t box[4] = {64, (cuuint32_t)rows, 1, 1}, estr[4] = {1, 1, 1, 1};
    return encode(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                  const_cast<uint16_t*>(values ? p.v : p.k), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool query_tmap(CUtensorMap* m, const PagedAttnParams& p, bool bf16, int d, int tokens) {
    auto encode = encoder();
    if (!encode) return false;
    const uint64_t row = (uint64_t)d * 2;
    const uint64_t hs = p.Hq == 1 ? row : (uint64_t)p.q_head * 2, ts = p.T == 1 ? row : (uint64_t)p.q_token * 2;
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)p.Hq, (cuuint64_t)p.T};
    const cuuint64_t strides[2] = {hs, ts};
    const cuuint32_t box[3] = {64, (cuuint32_t)p.G, (cuuint32_t)tokens}, estr[3] = {1, 1, 1};
    return encode(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
                  const_cast<uint16_t*>(p.q), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The arrival counters, both kernels' partial results (two a CTA, one CTA an SM).
size_t paged_attn_workspace(int, int, int Hq, int Hkv, int d, int max_q, int sms) {
    const bool large = (int64_t)max_q * (Hq / Hkv) > kSmallRows;
    return kCounterBytes + paged_decode_part_bytes(d, sms) + (large ? paged_chunk_part_bytes(d, sms) : 0);
}

cudaError_t launch_paged_attn(const w4a16_paged_attention_args& a, int sms, cudaStream_t s) {
    PagedAttnParams p;
    p.q = static_cast<const uint16_t*>(a.q);
    p.k = static_cast<const uint16_t*>(a.k_cache);
    p.v = static_cast<const uint16_t*>(a.v_cache);
    p.table = a.block_table;
    p.q_start = a.q_start;
    p.kv_len = a.kv_len;
    p.out = static_cast<uint16_t*>(a.out);
    p.lse = a.lse;
    p.q_token = a.q_token, p.q_head = a.q_head, p.o_token = a.out_token, p.o_head = a.out_head;
    p.kp = a.kc_page, p.kh = a.kc_head, p.ks = a.kc_slot;
    p.vp = a.vc_page, p.vh = a.vc_head, p.vs = a.vc_slot;
    p.table_stride = a.table_stride;
    p.T = a.tokens, p.B = a.requests, p.Hq = a.q_heads, p.Hkv = a.kv_heads, p.G = a.q_heads / a.kv_heads;
    p.pages = a.num_pages, p.columns = a.columns;
    p.shift = 0;
    while ((1 << p.shift) < a.page_size) ++p.shift;
    p.window = a.window, p.block = a.block;
    p.counters = static_cast<unsigned*>(a.workspace);
    p.part = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + kCounterBytes);
    p.scale2 = (a.scale == 0.f ? 1.f / sqrtf((float)a.head_dim) : a.scale) * 1.4426950408889634f;
    const bool pdl = (a.flags & W4A16_FLAG_PDL) != 0, bf16 = a.dtype == W4A16_BF16;
    // Which of the two kernels can have requests: all with max_q tokens when T = B max_q.
    const bool even = (int64_t)a.requests * a.max_q == a.tokens;
    const bool large = (int64_t)a.max_q * p.G > kSmallRows, small = !large || !even;
    p.small_rows = small ? kSmallRows : 0;
    p.after_small = small;
    if (small) {
        const cudaError_t e = launch_paged_decode(p, bf16, a.head_dim, sms, s, pdl);
        if (e != cudaSuccess) return e;
        note_launch();
    }
    if (!large) return cudaSuccess;
    p.part = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + kCounterBytes + paged_decode_part_bytes(a.head_dim, sms));
    // (behind the small-row kernel always as its dependent: its CTAs take the SMs as those are done)
    const cudaError_t e = launch_paged_chunk(p, bf16, a.head_dim, (int64_t)a.max_q * p.G <= 128, sms, s, pdl || small);
    if (e == cudaSuccess) note_launch();
    return e;
}

}  // namespace w4a16
