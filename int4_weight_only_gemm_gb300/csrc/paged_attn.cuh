// Shared pieces of the paged-attention kernels: their parameters and the 16-bit
// types.
#pragma once

#include <cuda.h>

#include "common.cuh"
#include "kernels.h"

namespace w4a16 {

struct PagedAttnParams {
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    const int* table;
    const int* q_start;
    const int* kv_len;
    uint16_t* out;
    float* lse;  // or null
    int64_t q_token, q_head, o_token, o_head;
    int64_t kp, kh, ks, vp, vh, vs;  // strides of pages, heads, slots
    int64_t table_stride;
    int T, B, Hq, Hkv, G, pages, shift, columns;
    int window, block;
    int small_rows;  // requests with up to this many query rows a key head go to the small-row kernel
    bool after_small;  // the kernel before in the stream is the same call's small-row kernel
    unsigned* counters;  // arrival counters, zero between calls
    float* part;         // partial results of split work
    float scale2;  // scale * log2(e): scores in the base-2 exponent
    // 8-bit caches: k and v are their codes, strides count bytes
    const float *k_scale, *v_scale;
    int64_t ksp, ksh, kss, vsp, vsh, vss;  // strides of the scales' pages, heads, slots
    bool e4m3;
    // a tree of new tokens, or null
    const uint32_t* tree;
    int64_t tree_token;
    int words;
};

struct Bf16 {
    static constexpr uint32_t idesc_type = 1;  // of kind::f16 operands
    W4A16_DEVICE static float lo(uint32_t v) { return bf16lo(v); }
    W4A16_DEVICE static float hi(uint32_t v) { return bf16hi(v); }
    // bit 15 or 31 is set where that half is an infinity or NaN (its exponent bits are all ones)
    W4A16_DEVICE static uint32_t all_ones(uint32_t v) { return (v & 0x7f807f80u) + 0x00800080u; }
    W4A16_DEVICE static uint32_t pack(float a, float b) {  // a in the low half
        uint32_t r;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
        return r;
    }
};
struct F16 {
    static constexpr uint32_t idesc_type = 0;
    W4A16_DEVICE static float lo(uint32_t v) { return f16_bits_to_f32((uint16_t)v); }
    W4A16_DEVICE static float hi(uint32_t v) { return f16_bits_to_f32((uint16_t)(v >> 16)); }
    W4A16_DEVICE static uint32_t all_ones(uint32_t v) { return (v & 0x7c007c00u) + 0x04000400u; }
    W4A16_DEVICE static uint32_t pack(float a, float b) {
        uint32_t r;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
        return r;
    }
};

// D += A B, 16 x 8 x 16, warp-wide
template <typename Ty>
W4A16_DEVICE void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (Ty::idesc_type == 1)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
W4A16_DEVICE void ldsm_x4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
W4A16_DEVICE void ldsm_x4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

W4A16_DEVICE float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr float kLn2 = 0.6931471805599453f;

// The positions that token i of request b sees: lo <= j <= e.  L and n are the
// request's lengths, already clamped to the table and to the tokens.
struct Request {
    int t0, n, L;
};
// (lengths and table entries are read from L2: the chunk kernel may start without a wait of its own, behind the
// small-row kernel's, and what an SM's first-level cache holds may be older than the kernels before both)
W4A16_DEVICE Request request_of(const PagedAttnParams& p, int b) {
    Request r;
    r.t0 = min(max(__ldcg(p.q_start + b), 0), p.T);
    r.n = min(max(__ldcg(p.q_start + b + 1), r.t0), p.T) - r.t0;
    const int64_t room = (int64_t)p.columns << p.shift;
    r.L = max(__ldcg(p.kv_len + b), 0);
    if (r.L > room) r.L = (int)room;
    return r;
}
W4A16_DEVICE int last_seen(const PagedAttnParams& p, const Request& r, int i) {
    return p.block ? r.L - 1 : r.L - r.n + i;
}
W4A16_DEVICE int first_seen(const PagedAttnParams& p, int e) {
    return p.window > 0 && e >= p.window ? e - p.window + 1 : 0;  // (e may be negative, the window as large as it gets)
}

// What the tokens of a request see, of a tree's nodes or (TREE false) of the
// positions up to their own: from `first` on, all of `lo_all` .. `e_all`, none
// behind `last`.
struct Seen {
    int first, lo_all, e_all, last;
};
template <bool TREE>
W4A16_DEVICE Seen seen_by(const PagedAttnParams& p, const Request& r, int i0, int i1) {  // tokens i0 .. i1
    Seen s;
    if constexpr (TREE) {
        const int past = r.L - r.n;
        s.first = p.window > 0 && past > p.window ? past - p.window : 0;  // (of a node without a bit)
        s.lo_all = p.window > 0 && r.L > p.window ? r.L - p.window : 0;   // (of one that sees them all)
        s.e_all = past - 1;
        s.last = r.L - 1;
    } else {
        s.e_all = last_seen(p, r, i0);
        s.last = last_seen(p, r, i1);
        s.first = first_seen(p, s.e_all);
        s.lo_all = first_seen(p, s.last);
    }
    return s;
}
// Word w of the nodes that token t of a request with n new tokens sees.
W4A16_DEVICE uint32_t tree_word(const PagedAttnParams& p, int t, int n, int w) {
    if (w < 0 || w >= p.words || 32 * w >= n) return 0u;
    const uint32_t x = __ldcg(p.tree + (int64_t)t * p.tree_token + w);
    return n - 32 * w >= 32 ? x : x & ((1u << (n - 32 * w)) - 1u);
}
// The first context position that a token of a tree sees: its place is behind the context by its depth.
W4A16_DEVICE int tree_first(const PagedAttnParams& p, const Request& r, int t) {
    if (p.window == 0) return 0;
    int64_t at = (int64_t)r.L - r.n - p.window;
    for (int w = 0; w < p.words && 32 * w < r.n; ++w) at += __popc(tree_word(p, t, r.n, w));
    return at > 0 ? (int)at : 0;
}

// Tensor map of the key or value cache, (column, slot, head, page), in boxes of
// 64 columns by `rows` slots, 128-byte swizzle; of 8-bit codes in boxes of d
// columns without one (paged_attn.cu).
bool paged_tmap(CUtensorMap* m, const PagedAttnParams& p, bool bf16, bool codes, int d, bool values, int rows);

// Tensor map of the queries, (column, head, token), in boxes of 64 columns by
// the heads of a group by `tokens` tokens, 128-byte swizzle (paged_attn.cu).
bool query_tmap(CUtensorMap* m, const PagedAttnParams& p, bool bf16, int d, int tokens);

// requests of up to 16 query rows a key head (paged_decode.cuh)
constexpr int kSmallRows = 16;
size_t paged_decode_part_bytes(int d, int sms);
template <bool TREE>
cudaError_t launch_paged_decode(const PagedAttnParams& p, bool bf16, int d, int sms, cudaStream_t s, bool pdl);

// and over an 8-bit cache (paged_decode8.cuh); few: none of these has more than 8; no more partial results than there
template <bool TREE>
cudaError_t launch_paged_decode8(const PagedAttnParams& p, bool bf16, int d, bool few, int sms, cudaStream_t s, bool pdl);

// the other requests (paged_chunk.cuh)
size_t paged_chunk_part_bytes(int d, int sms);
// one: no request has more than 128 rows a key head
template <bool TREE, bool Q8>
cudaError_t launch_paged_chunk(const PagedAttnParams& p, bool bf16, int d, bool one, int sms, cudaStream_t s, bool pdl);
template <bool TREE, bool Q8>
int paged_chunk_status();

}  // namespace w4a16
