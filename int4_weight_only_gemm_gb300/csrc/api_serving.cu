// C ABI of the serving operators: argument checks and launch counting.  See
// include/w4a16.h.
#include <cstdint>
#include <initializer_list>

#include "kernels.h"

// the binding packs these structs by position
static_assert(sizeof(w4a16_page_plan_args) == 104 && sizeof(w4a16_kv_write_args) == 152 &&
                  sizeof(w4a16_paged_attention_args) == 224 && sizeof(w4a16_sample_args) == 112,
              "argument structs without padding");

namespace w4a16 {
namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Bytes [lo, hi) that a strided array of `size`-byte elements spans.
struct Span {
    uintptr_t lo, hi;
};
struct Dim {
    int64_t count, stride;
};
Span span(const void* p, int size, Dim a, Dim b = {1, 0}, Dim c = {1, 0}, Dim d = {1, 0}) {
    int64_t last = 1;
    for (const Dim& x : {a, b, c, d}) {
        if (x.count < 1) return {0, 0};
        last += (x.count - 1) * x.stride;
    }
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return {lo, lo + (uintptr_t)(last * size)};
}
bool meet(const Span& a, const Span& b) { return a.lo < b.hi && b.lo < a.hi; }

int check_page_size(int p) {
    if (p < 1) return W4A16_EINVAL;
    return p >= 8 && p <= 256 && (p & (p - 1)) == 0 ? W4A16_OK : W4A16_EUNSUPPORTED;
}

// Strides, in elements, of at least `least`; that of a dimension of one entry
// is not looked at, since nothing goes by it.
int check_strides(int64_t least, std::initializer_list<Dim> dims) {
    for (const Dim& x : dims)
        if (x.count > 1 && x.stride < least) return W4A16_EINVAL;
    for (const Dim& x : dims)
        if (x.count > 1 && x.stride % 8) return W4A16_EALIGN;
    return W4A16_OK;
}

int status_of(cudaError_t e) { return e == cudaSuccess ? W4A16_OK : W4A16_ECUDA; }

}  // namespace
}  // namespace w4a16

using namespace w4a16;

extern "C" {

int w4a16_page_plan(const w4a16_page_plan_args* a, w4a16_stream_t stream) {
    if (!a || (a->flags & ~(unsigned)W4A16_FLAG_PDL)) return W4A16_EINVAL;
    if (a->requests < 0 || a->num_free < 0 || a->columns < 1 || a->tokens < 0 || a->table_stride < a->columns)
        return W4A16_EINVAL;
    int st = check_page_size(a->page_size);
    if (st != W4A16_OK) return st;
    if (a->requests > kPlanMaxRequests) return W4A16_EUNSUPPORTED;
    if (!a->q_start || !a->pages_used || (a->num_free && !a->free_pages) ||
        (a->tokens && (!a->positions || !a->slot_map)) ||
        (a->requests && (!a->past_len || !a->new_len || !a->block_table || !a->kv_len)))
        return W4A16_EINVAL;
    const void* all[] = {a->past_len, a->new_len, a->free_pages, a->block_table, a->q_start,
                         a->kv_len,   a->positions, a->slot_map, a->pages_used};
    for (const void* p : all)
        if (!aligned(p, 4)) return W4A16_EALIGN;
    const Span out[] = {span(a->block_table, 4, {a->requests, a->table_stride}, {a->columns, 1}),
                        span(a->q_start, 4, {a->requests + 1, 1}),
                        span(a->kv_len, 4, {a->requests, 1}),
                        span(a->positions, 4, {a->tokens, 1}),
                        span(a->slot_map, 4, {a->tokens, 1}),
                        span(a->pages_used, 4, {1, 1})};
    const Span in[] = {span(a->past_len, 4, {a->requests, 1}), span(a->new_len, 4, {a->requests, 1}),
                       span(a->free_pages, 4, {a->num_free, 1})};
    for (int i = 0; i < 6; ++i) {
        for (int j = 0; j < i; ++j)
            if (meet(out[i], out[j])) return W4A16_EINVAL;
        for (const Span& x : in)
            if (meet(out[i], x)) return W4A16_EINVAL;
    }
    const int sms = current_sms();
    if (sms <= 0) return W4A16_ECUDA;
    st = status_of(launch_page_plan(*a, sms, reinterpret_cast<cudaStream_t>(stream)));
    if (st == W4A16_OK) note_launch();
    return st;
}

int w4a16_kv_write(const w4a16_kv_write_args* a, w4a16_stream_t stream) {
    if (!a || (a->flags & ~(unsigned)W4A16_FLAG_PDL) || a->reserved) return W4A16_EINVAL;
    if (a->tokens < 0 || a->heads < 1 || a->head_dim < 1 || a->num_pages < 1) return W4A16_EINVAL;
    int st = check_page_size(a->page_size);
    if (st != W4A16_OK) return st;
    if ((a->dtype != W4A16_BF16 && a->dtype != W4A16_F16) || a->head_dim % 8 || a->head_dim > 1024 ||
        a->heads > 1024 || (int64_t)a->num_pages * a->page_size >= (1ll << 31))
        return W4A16_EUNSUPPORTED;
    if (a->tokens == 0) return W4A16_OK;
    if (!a->k || !a->v || !a->slot_map || !a->k_cache || !a->v_cache) return W4A16_EINVAL;
    if (!aligned(a->k, 16) || !aligned(a->v, 16) || !aligned(a->slot_map, 4) || !aligned(a->k_cache, 16) ||
        !aligned(a->v_cache, 16))
        return W4A16_EALIGN;
    st = check_strides(0, {{a->tokens, a->k_token}, {a->heads, a->k_head}, {a->tokens, a->v_token}, {a->heads, a->v_head}});
    if (st == W4A16_OK)
        st = check_strides(1, {{a->num_pages, a->kc_page}, {a->heads, a->kc_head}, {a->page_size, a->kc_slot},
                               {a->num_pages, a->vc_page}, {a->heads, a->vc_head}, {a->page_size, a->vc_slot}});
    if (st != W4A16_OK) return st;
    const Dim d = {a->head_dim, 1};
    const Span kc = span(a->k_cache, 2, {a->num_pages, a->kc_page}, {a->heads, a->kc_head}, {a->page_size, a->kc_slot}, d);
    const Span vc = span(a->v_cache, 2, {a->num_pages, a->vc_page}, {a->heads, a->vc_head}, {a->page_size, a->vc_slot}, d);
    for (const Span& c : {kc, vc})
        for (const Span& x : {span(a->k, 2, {a->tokens, a->k_token}, {a->heads, a->k_head}, d),
                              span(a->v, 2, {a->tokens, a->v_token}, {a->heads, a->v_head}, d),
                              span(a->slot_map, 4, {a->tokens, 1})})
            if (meet(c, x)) return W4A16_EINVAL;
    const int sms = current_sms();
    if (sms <= 0) return W4A16_ECUDA;
    st = status_of(launch_kv_write(*a, sms, reinterpret_cast<cudaStream_t>(stream)));
    if (st == W4A16_OK) note_launch();
    return st;
}

static int check_paged_sizes(int tokens, int requests, int Hq, int Hkv, int d, int max_q) {
    if (tokens < 0 || requests < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv || max_q < 0) return W4A16_EINVAL;
    if ((d != 64 && d != 128) || Hq / Hkv > 64 || Hq > 65535 || requests > kPlanMaxRequests ||
        (int64_t)tokens * Hq >= (1ll << 31))
        return W4A16_EUNSUPPORTED;
    return W4A16_OK;
}

size_t w4a16_paged_attention_workspace_bytes(int tokens, int requests, int Hq, int Hkv, int d, int max_q) {
    if (check_paged_sizes(tokens, requests, Hq, Hkv, d, max_q) != W4A16_OK) return 0;
    const int sms = current_sms();
    return sms > 0 ? paged_attn_workspace(tokens, requests, Hq, Hkv, d, max_q, sms) : 0;
}

int w4a16_paged_attention(const w4a16_paged_attention_args* a, w4a16_stream_t stream) {
    if (!a || (a->flags & ~(unsigned)W4A16_FLAG_PDL)) return W4A16_EINVAL;
    int st = check_paged_sizes(a->tokens, a->requests, a->q_heads, a->kv_heads, a->head_dim, a->max_q);
    if (st != W4A16_OK) return st;
    if (a->num_pages < 1 || a->columns < 1 || a->table_stride < a->columns || a->window < 0 ||
        (a->block != 0 && a->block != 1) || !(a->scale >= 0.f))
        return W4A16_EINVAL;
    st = check_page_size(a->page_size);
    if (st != W4A16_OK) return st;
    if ((a->dtype != W4A16_BF16 && a->dtype != W4A16_F16) || (int64_t)a->num_pages * a->page_size >= (1ll << 31) ||
        (int64_t)a->columns * a->page_size >= (1ll << 31))
        return W4A16_EUNSUPPORTED;
    if (a->tokens == 0 || a->requests == 0 || a->max_q == 0) return W4A16_OK;  // no new token
    if (!a->q || !a->k_cache || !a->v_cache || !a->block_table || !a->q_start || !a->kv_len || !a->out)
        return W4A16_EINVAL;
    if (!aligned(a->q, 16) || !aligned(a->k_cache, 16) || !aligned(a->v_cache, 16) || !aligned(a->out, 16) ||
        !aligned(a->block_table, 4) || !aligned(a->q_start, 4) || !aligned(a->kv_len, 4) || !aligned(a->lse, 4))
        return W4A16_EALIGN;
    st = check_strides(1, {{a->tokens, a->q_token}, {a->q_heads, a->q_head}, {a->tokens, a->out_token},
                           {a->q_heads, a->out_head}, {a->num_pages, a->kc_page}, {a->kv_heads, a->kc_head},
                           {a->page_size, a->kc_slot}, {a->num_pages, a->vc_page}, {a->kv_heads, a->vc_head},
                           {a->page_size, a->vc_slot}});
    if (st != W4A16_OK) return st;
    const Dim d = {a->head_dim, 1};
    const Span in[] = {
        span(a->q, 2, {a->tokens, a->q_token}, {a->q_heads, a->q_head}, d),
        span(a->k_cache, 2, {a->num_pages, a->kc_page}, {a->kv_heads, a->kc_head}, {a->page_size, a->kc_slot}, d),
        span(a->v_cache, 2, {a->num_pages, a->vc_page}, {a->kv_heads, a->vc_head}, {a->page_size, a->vc_slot}, d),
        span(a->block_table, 4, {a->requests, a->table_stride}, {a->columns, 1}),
        span(a->q_start, 4, {a->requests + 1, 1}), span(a->kv_len, 4, {a->requests, 1})};
    const Span out = span(a->out, 2, {a->tokens, a->out_token}, {a->q_heads, a->out_head}, d);
    const Span lse = a->lse ? span(a->lse, 4, {(int64_t)a->tokens * a->q_heads, 1}) : Span{0, 0};
    for (const Span& x : in)
        if (meet(out, x) || meet(lse, x)) return W4A16_EINVAL;
    if (meet(out, lse)) return W4A16_EINVAL;
    const int sms = current_sms();
    if (sms <= 0) return W4A16_ECUDA;
    const size_t need = paged_attn_workspace(a->tokens, a->requests, a->q_heads, a->kv_heads, a->head_dim, a->max_q, sms);
    if (need && (!a->workspace || a->workspace_bytes < need || !aligned(a->workspace, 16))) return W4A16_EWORKSPACE;
    return status_of(launch_paged_attn(*a, sms, reinterpret_cast<cudaStream_t>(stream)));
}

size_t w4a16_sample_workspace_bytes(int rows, int vocab, int filters) {
    if (rows < 1 || rows > 65535 || vocab < 1 || vocab > (1 << 24)) return 0;
    const int sms = current_sms();
    return sms > 0 ? sample_workspace(rows, vocab, filters != 0, sms) : 0;
}

int w4a16_sample(const w4a16_sample_args* a, w4a16_stream_t stream) {
    if (!a || (a->flags & ~(unsigned)W4A16_FLAG_PDL)) return W4A16_EINVAL;
    if (a->rows < 0 || a->vocab < 1 || a->logits_row < 0 || a->noise_row < 0) return W4A16_EINVAL;
    if (a->dtype != W4A16_BF16 && a->dtype != W4A16_F16 && a->dtype != W4A16_F32) return W4A16_EUNSUPPORTED;
    if (a->vocab > (1 << 24) || a->rows > 65535) return W4A16_EUNSUPPORTED;
    if (a->rows == 0) return W4A16_OK;
    if (!a->logits || !a->noise || !a->token) return W4A16_EINVAL;
    const int size = a->dtype == W4A16_F32 ? 4 : 2;
    if (!aligned(a->logits, size) || !aligned(a->noise, 4) || !aligned(a->temperature, 4) || !aligned(a->top_k, 4) ||
        !aligned(a->top_p, 4) || !aligned(a->min_p, 4) || !aligned(a->token, 4) || !aligned(a->logprob, 4))
        return W4A16_EALIGN;
    const Span in[] = {span(a->logits, size, {a->rows, a->logits_row}, {a->vocab, 1}),
                       span(a->noise, 4, {a->rows, a->noise_row}, {a->vocab, 1}),
                       a->temperature ? span(a->temperature, 4, {a->rows, 1}) : Span{0, 0},
                       a->top_k ? span(a->top_k, 4, {a->rows, 1}) : Span{0, 0},
                       a->top_p ? span(a->top_p, 4, {a->rows, 1}) : Span{0, 0},
                       a->min_p ? span(a->min_p, 4, {a->rows, 1}) : Span{0, 0}};
    const Span token = span(a->token, 4, {a->rows, 1});
    const Span lp = a->logprob ? span(a->logprob, 4, {a->rows, 1}) : Span{0, 0};
    for (const Span& x : in)
        if (meet(token, x) || meet(lp, x)) return W4A16_EINVAL;
    if (meet(token, lp)) return W4A16_EINVAL;
    const int sms = current_sms();
    if (sms <= 0) return W4A16_ECUDA;
    const size_t need = sample_workspace(a->rows, a->vocab, a->top_k || a->top_p || a->min_p, sms);
    if (need && (!a->workspace || a->workspace_bytes < need || !aligned(a->workspace, 16))) return W4A16_EWORKSPACE;
    return status_of(launch_sample(*a, sms, reinterpret_cast<cudaStream_t>(stream)));
}

uint64_t w4a16_stream_capture_id(w4a16_stream_t stream) {
    cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
    unsigned long long id = 0;
    if (cudaStreamGetCaptureInfo(reinterpret_cast<cudaStream_t>(stream), &status, &id) != cudaSuccess) {
        (void)cudaGetLastError();  // (the default stream while another one captures)
        return 0;
    }
    return status == cudaStreamCaptureStatusActive ? id : 0;
}

}  // extern "C"
