// C ABI of the serving operators: argument checks and launch counting.  See
// include/w4a16.h.
#include <cstdint>
#include <initializer_list>

#include "kernels.h"

// the binding packs these structs by position
static_assert(sizeof(w4a16_page_plan_args) == 104 && sizeof(w4a16_kv_write_args) == 152 &&
                  sizeof(w4a16_paged_attention_args) == 224 && sizeof(w4a16_sample_args) == 112 &&
                  sizeof(w4a16_paged_attention_ext) == 88 && sizeof(w4a16_rope_args) == 96 &&
                  sizeof(w4a16_kv_store_args) == 296 && sizeof(w4a16_kv_read_args) == 216,
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
int check_strides(int64_t least, std::initializer_list<Dim> dims, int multiple = 8) {
    for (const Dim& x : dims)
        if (x.count > 1 && x.stride < least) return W4A16_EINVAL;
    for (const Dim& x : dims)
        if (x.count > 1 && x.stride % multiple) return W4A16_EALIGN;
    return W4A16_OK;
}

int check_rotary(int d, int rotary, int interleaved) {
    return rotary < 2 || rotary % 2 || rotary > d || (interleaved != 0 && interleaved != 1) ? W4A16_EINVAL : W4A16_OK;
}

// Whether two arrays are one: pointer, and the strides that count.
bool same(const void* p, const void* q, Dim a, Dim b, Dim c, Dim d) {
    return p == q && (a.count < 2 || a.stride == b.stride) && (c.count < 2 || c.stride == d.stride);
}

// Whether the first tokens of two arrays (spans x and y) lie apart within rows of
// one stride, so that all their tokens do.
bool beside(int tokens, int64_t pt, int64_t qt, const Span& x, const Span& y) {
    if (meet(x, y)) return false;
    if (tokens < 2) return true;
    const uintptr_t lo = x.lo < y.lo ? x.lo : y.lo, hi = x.hi > y.hi ? x.hi : y.hi;
    return pt == qt && hi - lo <= (uintptr_t)pt * 2;
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

int w4a16_rope(const w4a16_rope_args* a, w4a16_stream_t stream) {
    if (!a || (a->flags & ~(unsigned)W4A16_FLAG_PDL)) return W4A16_EINVAL;
    if (a->tokens < 0 || a->heads < 1 || a->head_dim < 1) return W4A16_EINVAL;
    int st = check_rotary(a->head_dim, a->rotary_dim, a->interleaved);
    if (st != W4A16_OK) return st;
    if ((a->dtype != W4A16_BF16 && a->dtype != W4A16_F16) || a->head_dim % 8 || a->head_dim > 256 || a->heads > 1024)
        return W4A16_EUNSUPPORTED;
    if (a->tokens == 0) return W4A16_OK;
    if (!a->x || !a->out || !a->positions || !a->frequencies) return W4A16_EINVAL;
    if (!aligned(a->x, 16) || !aligned(a->out, 16) || !aligned(a->positions, 4) || !aligned(a->frequencies, 8))
        return W4A16_EALIGN;
    st = check_strides(0, {{a->tokens, a->x_token}, {a->heads, a->x_head}});
    if (st == W4A16_OK) st = check_strides(1, {{a->tokens, a->out_token}, {a->heads, a->out_head}});
    if (st != W4A16_OK) return st;
    const Dim d = {a->head_dim, 1};
    const Span x = span(a->x, 2, {a->tokens, a->x_token}, {a->heads, a->x_head}, d);
    const Span out = span(a->out, 2, {a->tokens, a->out_token}, {a->heads, a->out_head}, d);
    if (!same(a->x, a->out, {a->tokens, a->x_token}, {a->tokens, a->out_token}, {a->heads, a->x_head},
              {a->heads, a->out_head}) && meet(x, out))
        return W4A16_EINVAL;
    if (meet(out, span(a->positions, 4, {a->tokens, 1})) || meet(out, span(a->frequencies, 8, {a->rotary_dim / 2, 1})))
        return W4A16_EINVAL;
    const int sms = current_sms();
    if (sms <= 0) return W4A16_ECUDA;
    st = status_of(launch_rope(*a, sms, reinterpret_cast<cudaStream_t>(stream)));
    if (st == W4A16_OK) note_launch();
    return st;
}

int w4a16_rope_frequencies(int rotary_dim, double base, int scaling, double factor, double length, double low,
                           double high, double* frequencies, float* magnitude) {
    const double most = 1e300;
    if (!frequencies || !magnitude || rotary_dim < 2 || rotary_dim % 2 || scaling < W4A16_ROPE_NONE ||
        scaling > W4A16_ROPE_WAVELENGTH || !(base > 0 && base < most) || !(factor > 0 && factor < most))
        return W4A16_EINVAL;
    if (scaling == W4A16_ROPE_RAMP && !(base > 1)) return W4A16_EINVAL;  // (pairs have to turn less one after the other)
    if (scaling >= W4A16_ROPE_RAMP && (!(length > 0 && length < most) || !(low > 0 && low < high && high < most)))
        return W4A16_EINVAL;
    rope_frequencies(rotary_dim, base, scaling, factor, length, low, high, frequencies, magnitude);
    return W4A16_OK;
}

int w4a16_kv_store(const w4a16_kv_store_args* a, w4a16_stream_t stream) {
    if (!a || (a->flags & ~(unsigned)W4A16_FLAG_PDL)) return W4A16_EINVAL;
    if (a->tokens < 0 || a->q_heads < 0 || a->heads < 1 || a->head_dim < 1 || a->num_pages < 1) return W4A16_EINVAL;
    int st = check_page_size(a->page_size);
    if (st != W4A16_OK) return st;
    const bool turn = a->frequencies != nullptr;
    if (turn) st = check_rotary(a->head_dim, a->rotary_dim, a->interleaved);
    else if (a->q_heads || a->rotary_dim || a->interleaved) st = W4A16_EINVAL;
    if (st != W4A16_OK) return st;
    const bool codes = a->cache_dtype == W4A16_INT8 || a->cache_dtype == W4A16_E4M3;
    if ((a->dtype != W4A16_BF16 && a->dtype != W4A16_F16) || (!codes && a->cache_dtype != a->dtype) ||
        a->head_dim % (codes ? 16 : 8) || a->head_dim > 256 || a->heads > 1024 || a->q_heads > 1024 ||
        (int64_t)a->num_pages * a->page_size >= (1ll << 31))
        return W4A16_EUNSUPPORTED;
    if (!codes && (a->k_scale || a->v_scale)) return W4A16_EINVAL;
    if (a->tokens == 0) return W4A16_OK;
    if (!a->k || !a->v || !a->slot_map || !a->k_cache || !a->v_cache || (codes && (!a->k_scale || !a->v_scale)) ||
        (a->q_heads && (!a->q || !a->q_out)) || (turn && !a->positions))
        return W4A16_EINVAL;
    if (!aligned(a->k, 16) || !aligned(a->v, 16) || !aligned(a->slot_map, 4) || !aligned(a->k_cache, 16) ||
        !aligned(a->v_cache, 16) || !aligned(a->k_scale, 4) || !aligned(a->v_scale, 4) || !aligned(a->positions, 4) ||
        !aligned(a->frequencies, 8) || (a->q_heads && (!aligned(a->q, 16) || !aligned(a->q_out, 16))))
        return W4A16_EALIGN;
    const Dim T = {a->tokens, 1}, d = {a->head_dim, 1};
    st = check_strides(0, {{a->tokens, a->k_token}, {a->heads, a->k_head}, {a->tokens, a->v_token}, {a->heads, a->v_head}});
    if (st == W4A16_OK && a->q_heads) st = check_strides(0, {{a->tokens, a->q_token}, {a->q_heads, a->q_head}});
    if (st == W4A16_OK && a->q_heads) st = check_strides(1, {{a->tokens, a->out_token}, {a->q_heads, a->out_head}});
    if (st == W4A16_OK)
        st = check_strides(1, {{a->num_pages, a->kc_page}, {a->heads, a->kc_head}, {a->page_size, a->kc_slot},
                               {a->num_pages, a->vc_page}, {a->heads, a->vc_head}, {a->page_size, a->vc_slot}},
                           codes ? 16 : 8);
    if (st == W4A16_OK && codes)
        st = check_strides(1, {{a->num_pages, a->ks_page}, {a->heads, a->ks_head}, {a->page_size, a->ks_slot},
                               {a->num_pages, a->vs_page}, {a->heads, a->vs_head}, {a->page_size, a->vs_slot}}, 1);
    if (st != W4A16_OK) return st;
    const int size = codes ? 1 : 2;
    const Span none = {0, 0};
    const Span q = a->q_heads ? span(a->q, 2, {a->tokens, a->q_token}, {a->q_heads, a->q_head}, d) : none;
    const Span in[] = {span(a->k, 2, {a->tokens, a->k_token}, {a->heads, a->k_head}, d),
                       span(a->v, 2, {a->tokens, a->v_token}, {a->heads, a->v_head}, d),
                       span(a->slot_map, 4, T),
                       turn ? span(a->positions, 4, T) : none,
                       turn ? span(a->frequencies, 8, {a->rotary_dim / 2, 1}) : none,
                       q};
    const Span out[] = {
        span(a->k_cache, size, {a->num_pages, a->kc_page}, {a->heads, a->kc_head}, {a->page_size, a->kc_slot}, d),
        span(a->v_cache, size, {a->num_pages, a->vc_page}, {a->heads, a->vc_head}, {a->page_size, a->vc_slot}, d),
        codes ? span(a->k_scale, 4, {a->num_pages, a->ks_page}, {a->heads, a->ks_head}, {a->page_size, a->ks_slot}) : none,
        codes ? span(a->v_scale, 4, {a->num_pages, a->vs_page}, {a->heads, a->vs_head}, {a->page_size, a->vs_slot}) : none};
    for (const Span& y : out)
        for (const Span& x : in)
            if (meet(y, x)) return W4A16_EINVAL;
    // (keys and values may share an array, page by page; a scale lies in no other output)
    if (meet(out[2], out[0]) || meet(out[2], out[1]) || meet(out[3], out[0]) || meet(out[3], out[1])) return W4A16_EINVAL;
    if (a->q_heads) {
        // q_out may be q itself; it may lie between k and v in the fused projection's rows, so that spans say
        // nothing there: rows of one stride, and heads that do not meet
        const Span o = span(a->q_out, 2, {a->tokens, a->out_token}, {a->q_heads, a->out_head}, d);
        for (const Span& y : out)
            if (meet(o, y)) return W4A16_EINVAL;
        for (int i = 2; i < 5; ++i)
            if (meet(o, in[i])) return W4A16_EINVAL;
        if (!same(a->q, a->q_out, {a->tokens, a->q_token}, {a->tokens, a->out_token}, {a->q_heads, a->q_head},
                  {a->q_heads, a->out_head})) {
            for (int i : {0, 1, 5})
                if (meet(o, in[i])) return W4A16_EINVAL;
        } else {
            const struct { const void* p; int64_t token, head; } kv[] = {{a->k, a->k_token, a->k_head}, {a->v, a->v_token, a->v_head}};
            for (int i = 0; i < 2; ++i)
                if (meet(o, in[i]) && !beside(a->tokens, a->out_token, kv[i].token,
                                              span(a->q_out, 2, {a->q_heads, a->out_head}, d),
                                              span(kv[i].p, 2, {a->heads, kv[i].head}, d)))
                    return W4A16_EINVAL;
        }
    }
    const int sms = current_sms();
    if (sms <= 0) return W4A16_ECUDA;
    st = status_of(launch_kv_store(*a, sms, reinterpret_cast<cudaStream_t>(stream)));
    if (st == W4A16_OK) note_launch();
    return st;
}

int w4a16_kv_read(const w4a16_kv_read_args* a, w4a16_stream_t stream) {
    if (!a || (a->flags & ~(unsigned)W4A16_FLAG_PDL)) return W4A16_EINVAL;
    if (a->tokens < 0 || a->heads < 1 || a->head_dim < 1 || a->num_pages < 1) return W4A16_EINVAL;
    int st = check_page_size(a->page_size);
    if (st != W4A16_OK) return st;
    const bool codes = a->cache_dtype == W4A16_INT8 || a->cache_dtype == W4A16_E4M3;
    if ((a->dtype != W4A16_BF16 && a->dtype != W4A16_F16) || (!codes && a->cache_dtype != a->dtype) ||
        a->head_dim % (codes ? 16 : 8) || a->head_dim > 1024 || a->heads > 1024 ||
        (int64_t)a->num_pages * a->page_size >= (1ll << 31))
        return W4A16_EUNSUPPORTED;
    if (!codes && (a->k_scale || a->v_scale)) return W4A16_EINVAL;
    if (a->tokens == 0) return W4A16_OK;
    if (!a->k || !a->v || !a->slot_map || !a->k_cache || !a->v_cache || (codes && (!a->k_scale || !a->v_scale)))
        return W4A16_EINVAL;
    if (!aligned(a->k, 16) || !aligned(a->v, 16) || !aligned(a->slot_map, 4) || !aligned(a->k_cache, 16) ||
        !aligned(a->v_cache, 16) || !aligned(a->k_scale, 4) || !aligned(a->v_scale, 4))
        return W4A16_EALIGN;
    st = check_strides(1, {{a->tokens, a->k_token}, {a->heads, a->k_head}, {a->tokens, a->v_token}, {a->heads, a->v_head}});
    if (st == W4A16_OK)
        st = check_strides(1, {{a->num_pages, a->kc_page}, {a->heads, a->kc_head}, {a->page_size, a->kc_slot},
                               {a->num_pages, a->vc_page}, {a->heads, a->vc_head}, {a->page_size, a->vc_slot}},
                           codes ? 16 : 8);
    if (st == W4A16_OK && codes)
        st = check_strides(0, {{a->num_pages, a->ks_page}, {a->heads, a->ks_head}, {a->page_size, a->ks_slot},
                               {a->num_pages, a->vs_page}, {a->heads, a->vs_head}, {a->page_size, a->vs_slot}}, 1);
    if (st != W4A16_OK) return st;
    const int size = codes ? 1 : 2;
    const Dim d = {a->head_dim, 1};
    const Span none = {0, 0};
    const Span in[] = {
        span(a->k_cache, size, {a->num_pages, a->kc_page}, {a->heads, a->kc_head}, {a->page_size, a->kc_slot}, d),
        span(a->v_cache, size, {a->num_pages, a->vc_page}, {a->heads, a->vc_head}, {a->page_size, a->vc_slot}, d),
        codes ? span(a->k_scale, 4, {a->num_pages, a->ks_page}, {a->heads, a->ks_head}, {a->page_size, a->ks_slot}) : none,
        codes ? span(a->v_scale, 4, {a->num_pages, a->vs_page}, {a->heads, a->vs_head}, {a->page_size, a->vs_slot}) : none,
        span(a->slot_map, 4, {a->tokens, 1})};
    const Span k = span(a->k, 2, {a->tokens, a->k_token}, {a->heads, a->k_head}, d);
    const Span v = span(a->v, 2, {a->tokens, a->v_token}, {a->heads, a->v_head}, d);
    for (const Span& x : in)
        if (meet(k, x) || meet(v, x)) return W4A16_EINVAL;
    // k and v may be slices of the same rows
    if (meet(k, v) && !beside(a->tokens, a->k_token, a->v_token, span(a->k, 2, {a->heads, a->k_head}, d),
                              span(a->v, 2, {a->heads, a->v_head}, d)))
        return W4A16_EINVAL;
    st = status_of(launch_kv_read(*a, reinterpret_cast<cudaStream_t>(stream)));
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
    return w4a16_paged_attention_ex(a, nullptr, stream);
}

int w4a16_paged_attention_ex(const w4a16_paged_attention_args* a, const w4a16_paged_attention_ext* ext,
                             w4a16_stream_t stream) {
    if (!a || (a->flags & ~(unsigned)W4A16_FLAG_PDL)) return W4A16_EINVAL;
    w4a16_paged_attention_ext x = {};
    x.cache_dtype = a->dtype;
    if (ext) x = *ext;
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
    const bool codes = x.cache_dtype == W4A16_INT8 || x.cache_dtype == W4A16_E4M3;
    if (!codes && x.cache_dtype != a->dtype) return W4A16_EUNSUPPORTED;
    if (!codes && (x.k_scale || x.v_scale)) return W4A16_EINVAL;
    if (x.tree ? x.tree_words < 1 || a->block : x.tree_words != 0) return W4A16_EINVAL;
    if (x.tree_words > 64) return W4A16_EUNSUPPORTED;
    if (a->tokens == 0 || a->requests == 0 || a->max_q == 0) return W4A16_OK;  // no new token
    if (!a->q || !a->k_cache || !a->v_cache || !a->block_table || !a->q_start || !a->kv_len || !a->out ||
        (codes && (!x.k_scale || !x.v_scale)))
        return W4A16_EINVAL;
    if (!aligned(a->q, 16) || !aligned(a->k_cache, 16) || !aligned(a->v_cache, 16) || !aligned(a->out, 16) ||
        !aligned(a->block_table, 4) || !aligned(a->q_start, 4) || !aligned(a->kv_len, 4) || !aligned(a->lse, 4) ||
        !aligned(x.k_scale, 4) || !aligned(x.v_scale, 4) || !aligned(x.tree, 4))
        return W4A16_EALIGN;
    st = check_strides(1, {{a->tokens, a->q_token}, {a->q_heads, a->q_head}, {a->tokens, a->out_token},
                           {a->q_heads, a->out_head}});
    if (st == W4A16_OK)
        st = check_strides(1, {{a->num_pages, a->kc_page}, {a->kv_heads, a->kc_head}, {a->page_size, a->kc_slot},
                               {a->num_pages, a->vc_page}, {a->kv_heads, a->vc_head}, {a->page_size, a->vc_slot}},
                           codes ? 16 : 8);
    if (st == W4A16_OK && codes)
        st = check_strides(0, {{a->num_pages, x.ks_page}, {a->kv_heads, x.ks_head}, {a->page_size, x.ks_slot},
                               {a->num_pages, x.vs_page}, {a->kv_heads, x.vs_head}, {a->page_size, x.vs_slot}}, 1);
    if (st == W4A16_OK && x.tree) st = check_strides(x.tree_words, {{a->tokens, x.tree_token}}, 1);
    if (st != W4A16_OK) return st;
    const Dim d = {a->head_dim, 1};
    const int size = codes ? 1 : 2;
    const Dim P = {a->num_pages, 0}, H = {a->kv_heads, 0}, S = {a->page_size, 0};
    auto at = [](Dim x, int64_t stride) { return Dim{x.count, stride}; };
    const Span in[] = {
        span(a->q, 2, {a->tokens, a->q_token}, {a->q_heads, a->q_head}, d),
        span(a->k_cache, size, at(P, a->kc_page), at(H, a->kc_head), at(S, a->kc_slot), d),
        span(a->v_cache, size, at(P, a->vc_page), at(H, a->vc_head), at(S, a->vc_slot), d),
        span(a->block_table, 4, {a->requests, a->table_stride}, {a->columns, 1}),
        span(a->q_start, 4, {a->requests + 1, 1}), span(a->kv_len, 4, {a->requests, 1}),
        codes ? span(x.k_scale, 4, at(P, x.ks_page), at(H, x.ks_head), at(S, x.ks_slot)) : Span{0, 0},
        codes ? span(x.v_scale, 4, at(P, x.vs_page), at(H, x.vs_head), at(S, x.vs_slot)) : Span{0, 0},
        x.tree ? span(x.tree, 4, {a->tokens, x.tree_token}, {x.tree_words, 1}) : Span{0, 0}};
    const Span out = span(a->out, 2, {a->tokens, a->out_token}, {a->q_heads, a->out_head}, d);
    const Span lse = a->lse ? span(a->lse, 4, {(int64_t)a->tokens * a->q_heads, 1}) : Span{0, 0};
    for (const Span& y : in)
        if (meet(out, y) || meet(lse, y)) return W4A16_EINVAL;
    if (meet(out, lse)) return W4A16_EINVAL;
    const int sms = current_sms();
    if (sms <= 0) return W4A16_ECUDA;
    const size_t need = paged_attn_workspace(a->tokens, a->requests, a->q_heads, a->kv_heads, a->head_dim, a->max_q, sms);
    if (need && (!a->workspace || a->workspace_bytes < need || !aligned(a->workspace, 16))) return W4A16_EWORKSPACE;
    return status_of(launch_paged_attn(*a, x, sms, reinterpret_cast<cudaStream_t>(stream)));
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
