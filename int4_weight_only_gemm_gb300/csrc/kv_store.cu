// Rotary positions of queries and keys, and keys and values into the paged cache
// of 16 or 8 bits, in one launch; w4a16_rope is the same kernel with queries alone.
//
//     (a, b) -> (a cos w - b sin w, a sin w + b cos w) magnitude,  w = position * frequency
//     scale = max |x| / top,  code = round(x * (top / max |x|))
//
// A CTA takes a few tokens.  Its threads first make the cosines and sines of the
// tokens' pairs, in shared memory for all heads, then 16 lanes (32 for heads over
// 128 wide) take a head's row at a time, 8 elements a lane.  Angles: a frequency
// is a 64-bit fraction F of a turn a position, so position * F modulo 2^64 is the
// fraction of a turn, without rounding; its top 32 bits go to sincospi.
//
// Bound: HBM, each row read and written once.
#include <cmath>

#include "codes.cuh"
#include "kernels.h"
#include "paged_attn.cuh"

namespace w4a16 {

constexpr int kRowThreads = 256;
constexpr int kRowTokens = 16;  // most tokens of a CTA

struct RowParams {
    const uint16_t *q, *k, *v;
    uint16_t* q_out;
    const int* positions;
    const double* freq;  // or null: nothing is rotated
    const int* slots;
    void *kc, *vc;
    float *ks, *vs;
    int64_t q_token, q_head, o_token, o_head, k_token, k_head, v_token, v_head;
    int64_t kcp, kch, kcs, vcp, vch, vcs, ksp, ksh, kss, vsp, vsh, vss;
    int64_t total_slots;
    int tokens, q_heads, heads, d, half, interleaved, shift;
    int per_cta;    // tokens of a CTA
    int rows, row0s;  // rows (q heads, k heads, v heads) of a token, and those of one CTA
    bool by_lane;   // a pair's partner is in the same lane, or in the lane `half / 8` on
    float magnitude;
    FastDiv by_rows, by_half;
};

enum { kCode16 = 0, kCodeInt8 = 1, kCodeE4m3 = 2 };

template <typename Ty>
W4A16_DEVICE float half_of(const uint4& v, int i) {
    const uint32_t x = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
    return i & 1 ? Ty::hi(x) : Ty::lo(x);
}

template <typename Ty, int CODE, int LANES>
__global__ void __launch_bounds__(kRowThreads) kv_store_kernel(const __grid_constant__ RowParams p) {
    extern __shared__ float2 turn[];  // [token][pair] cosine and sine
    pdl_wait();
    pdl_launch_dependents();
    const int t0 = (int)blockIdx.x * p.per_cta, nt = min(p.per_cta, p.tokens - t0);
    const int r0 = (int)blockIdx.y * p.row0s, nr = min(p.row0s, p.rows - r0);
    constexpr int GROUPS = kRowThreads / LANES;
    const int lane = threadIdx.x % LANES, col = 8 * lane;
    const bool on = col < p.d;
    // (all lanes of a warp go round together: shuffles)
    const int items = nt * nr, rounds = (items + GROUPS - 1) / GROUPS;
    struct Row {
        int tt, kind, h, slot;  // token of the CTA; 0 query, 1 key, 2 value; head
        bool live;
        const uint16_t* src;
        uint4 raw;
    };
    auto load = [&](int n) {  // the row of round n, on its way
        Row r;
        const int item = n * GROUPS + threadIdx.x / LANES;
        const bool have = item < items;
        r.tt = !have ? 0 : nr == p.rows ? div_by(item, p.by_rows.m, p.by_rows.s) : item / nr;
        const int row = r0 + (have ? item - r.tt * nr : 0), t = t0 + r.tt;
        r.kind = row < p.q_heads ? 0 : row < p.q_heads + p.heads ? 1 : 2;
        r.h = row - (r.kind == 0 ? 0 : r.kind == 1 ? p.q_heads : p.q_heads + p.heads);
        r.slot = r.kind ? p.slots[t] : 0;
        r.live = have && on && (!p.freq || p.positions[t] >= 0) && (r.kind == 0 || (r.slot >= 0 && r.slot < p.total_slots));
        r.src = r.kind == 0   ? p.q + t * p.q_token + r.h * p.q_head
                : r.kind == 1 ? p.k + t * p.k_token + r.h * p.k_head
                              : p.v + t * p.v_token + r.h * p.v_head;
        r.raw = make_uint4(0u, 0u, 0u, 0u);
        if (have && on) r.raw = *reinterpret_cast<const uint4*>(r.src + col);
        return r;
    };
    Row next = load(0);
    if (p.freq) {
        for (int e = threadIdx.x; e < nt * p.half; e += kRowThreads) {
            const int tt = div_by(e, p.by_half.m, p.by_half.s), i = e - tt * p.half;
            const double turns = p.freq[i] * 0.15915494309189533577;  // of 2 pi
            const int64_t f = __double2ll_rn((turns - rint(turns)) * 18446744073709551616.0);
            const uint64_t w = (uint64_t)(int64_t)p.positions[t0 + tt] * (uint64_t)f;
            float s, c;
            sincospif((float)(int32_t)(w >> 32) * 4.656612873077393e-10f, &s, &c);  // 2 / 2^32
            turn[e] = make_float2(c * p.magnitude, s * p.magnitude);
        }
        __syncthreads();
    }
    for (int n = 0; n < rounds; ++n) {
        const Row cur = next;
        if (n + 1 < rounds) next = load(n + 1);
        const int tt = cur.tt, kind = cur.kind, h = cur.h, slot = cur.slot, t = t0 + tt;
        const bool live = cur.live;
        const uint4 raw = cur.raw;
        const uint16_t* src = cur.src;
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = half_of<Ty>(raw, i);
        if (p.freq) {
            const bool turns = kind < 2 && live;
            const float2* cs = turn + tt * p.half;
            if (p.interleaved) {
                if (turns)
#pragma unroll
                    for (int i = 0; i < 8; i += 2)
                        if (col + i < 2 * p.half) {
                            const float2 w = cs[(col + i) >> 1];
                            const float a = x[i], b = x[i + 1];
                            x[i] = a * w.x - b * w.y;
                            x[i + 1] = a * w.y + b * w.x;
                        }
            } else if (p.by_lane) {
                const int gap = p.half >> 3;
                const int from = (threadIdx.x & 31 & ~(LANES - 1)) + (lane < gap ? lane + gap : lane < 2 * gap ? lane - gap : lane);
                const uint4 o = make_uint4(__shfl_sync(0xffffffffu, raw.x, from), __shfl_sync(0xffffffffu, raw.y, from),
                                           __shfl_sync(0xffffffffu, raw.z, from), __shfl_sync(0xffffffffu, raw.w, from));
                if (turns && lane < 2 * gap)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 w = cs[lane < gap ? col + i : col + i - p.half];
                        const float y = half_of<Ty>(o, i);
                        x[i] = lane < gap ? x[i] * w.x - y * w.y : y * w.y + x[i] * w.x;
                    }
            } else {
                // (partners by element, all read before any lane of the row writes: out may be x)
                float y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int at = col + i < p.half ? col + i + p.half : col + i - p.half;
                    y[i] = turns && col + i < 2 * p.half ? Ty::lo(src[at]) : 0.f;
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (turns && col + i < 2 * p.half) {
                        const bool first = col + i < p.half;
                        const float2 w = cs[first ? col + i : col + i - p.half];
                        x[i] = first ? x[i] * w.x - y[i] * w.y : y[i] * w.y + x[i] * w.x;
                    }
            }
        }
        const uint4 packed = make_uint4(Ty::pack(x[0], x[1]), Ty::pack(x[2], x[3]), Ty::pack(x[4], x[5]), Ty::pack(x[6], x[7]));
        if (kind == 0) {
            if (live) *reinterpret_cast<uint4*>(p.q_out + t * p.o_token + h * p.o_head + col) = packed;
        }
        const int64_t pg = slot >> p.shift, sl = slot & ((1 << p.shift) - 1);
        const int64_t at = kind == 1 ? pg * p.kcp + h * p.kch + sl * p.kcs : pg * p.vcp + h * p.vch + sl * p.vcs;
        if constexpr (CODE == kCode16) {
            // (what is not rotated is copied bit for bit)
            if (live && kind) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(kind == 1 ? p.kc : p.vc) + at + col) =
                p.freq && kind == 1 && col < 2 * p.half ? packed : raw;
        } else {
            uint32_t most = 0;  // magnitudes as integers: NaN and infinities are the largest
#pragma unroll
            for (int i = 0; i < 8; ++i) most = max(most, __float_as_uint(x[i]) & 0x7fffffffu);
#pragma unroll
            for (int i = 1; i < LANES; i <<= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, i));
            const float top = CODE == kCodeInt8 ? 127.f : 448.f, amax = __uint_as_float(most);
            const bool none = most < (27u << 23), bad = most >= 0x7f800000u;  // below 2^-100
            const float scale = bad ? __uint_as_float(0x7fffffffu) : none ? 0.f : __fdiv_rn(amax, top);
            const float inv = bad || none ? 0.f : __fdiv_rn(top, amax);
            uint32_t w[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float a = x[4 * i] * inv, b = x[4 * i + 1] * inv, c = x[4 * i + 2] * inv, e = x[4 * i + 3] * inv;
                if constexpr (CODE == kCodeInt8) {
                    w[i] = bad ? 0u
                               : __byte_perm(__byte_perm(__float2int_rn(a), __float2int_rn(b), 0x0040),
                                             __byte_perm(__float2int_rn(c), __float2int_rn(e), 0x0040), 0x5410);
                } else {
                    uint16_t lo, hi;
                    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
                    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(e), "f"(c));
                    w[i] = bad ? 0u : (uint32_t)lo | (uint32_t)hi << 16;
                }
            }
            if (live && kind) {
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(kind == 1 ? p.kc : p.vc) + at + col) = make_uint2(w[0], w[1]);
                if (lane == 0)
                    *(kind == 1 ? p.ks + pg * p.ksp + h * p.ksh + sl * p.kss : p.vs + pg * p.vsp + h * p.vsh + sl * p.vss) = scale;
            }
        }
    }
}

template <typename Ty, int CODE>
static cudaError_t launch_rows(const RowParams& p, dim3 grid, size_t smem, cudaStream_t s, bool pdl) {
    return p.d <= 128 ? launch_kernel(kv_store_kernel<Ty, CODE, 16>, grid, dim3(kRowThreads), smem, s, pdl, p)
                      : launch_kernel(kv_store_kernel<Ty, CODE, 32>, grid, dim3(kRowThreads), smem, s, pdl, p);
}

static cudaError_t launch(RowParams& p, bool bf16, int code, int rot, int sms, cudaStream_t s, bool pdl) {
    p.half = p.freq ? rot / 2 : 1;
    p.by_lane = p.half % 8 == 0;
    p.rows = p.q_heads + 2 * p.heads;
    const int groups = kRowThreads / (p.d <= 128 ? 16 : 32);
    // Tokens of a CTA: as many as its groups of lanes have rows for, up to eight rounds of them while the GPU stays
    // full (cosines for all threads, loads a round ahead); a token's rows over several CTAs where tokens are too few.
    int per = groups / p.rows;
    per = per < 1 ? 1 : per > kRowTokens ? kRowTokens : per;
    while (per * 2 <= kRowTokens && (int64_t)per * 2 * p.rows <= 8 * groups && p.tokens / (per * 2) >= 16 * sms) per *= 2;
    const int ctas = (p.tokens + per - 1) / per;
    int split = 1;
    while (ctas * split * 2 <= 4 * sms && (p.rows + split * 2 - 1) / (split * 2) >= groups) split *= 2;
    p.per_cta = per;
    p.row0s = (p.rows + split - 1) / split;
    p.by_rows = fast_div(p.rows);
    p.by_half = fast_div(p.half);
    const dim3 grid((unsigned)ctas, (unsigned)((p.rows + p.row0s - 1) / p.row0s));
    const size_t smem = p.freq ? (size_t)per * p.half * sizeof(float2) : 0;
    if (bf16)
        return code == kCode16     ? launch_rows<Bf16, kCode16>(p, grid, smem, s, pdl)
               : code == kCodeInt8 ? launch_rows<Bf16, kCodeInt8>(p, grid, smem, s, pdl)
                                   : launch_rows<Bf16, kCodeE4m3>(p, grid, smem, s, pdl);
    return code == kCode16     ? launch_rows<F16, kCode16>(p, grid, smem, s, pdl)
           : code == kCodeInt8 ? launch_rows<F16, kCodeInt8>(p, grid, smem, s, pdl)
                               : launch_rows<F16, kCodeE4m3>(p, grid, smem, s, pdl);
}

cudaError_t launch_kv_store(const w4a16_kv_store_args& a, int sms, cudaStream_t s) {
    RowParams p = {};
    p.q = static_cast<const uint16_t*>(a.q), p.k = static_cast<const uint16_t*>(a.k);
    p.v = static_cast<const uint16_t*>(a.v), p.q_out = static_cast<uint16_t*>(a.q_out);
    p.positions = a.positions, p.freq = a.frequencies, p.slots = a.slot_map;
    p.kc = a.k_cache, p.vc = a.v_cache, p.ks = a.k_scale, p.vs = a.v_scale;
    p.q_token = a.q_token, p.q_head = a.q_head, p.o_token = a.out_token, p.o_head = a.out_head;
    p.k_token = a.k_token, p.k_head = a.k_head, p.v_token = a.v_token, p.v_head = a.v_head;
    p.kcp = a.kc_page, p.kch = a.kc_head, p.kcs = a.kc_slot, p.vcp = a.vc_page, p.vch = a.vc_head, p.vcs = a.vc_slot;
    p.ksp = a.ks_page, p.ksh = a.ks_head, p.kss = a.ks_slot, p.vsp = a.vs_page, p.vsh = a.vs_head, p.vss = a.vs_slot;
    p.total_slots = (int64_t)a.num_pages * a.page_size;
    while ((1 << p.shift) < a.page_size) ++p.shift;
    p.tokens = a.tokens, p.q_heads = a.q_heads, p.heads = a.heads, p.d = a.head_dim;
    p.interleaved = a.interleaved, p.magnitude = a.magnitude;
    return launch(p, a.dtype == W4A16_BF16, a.cache_dtype == W4A16_INT8 ? kCodeInt8 : a.cache_dtype == W4A16_E4M3 ? kCodeE4m3 : kCode16,
                  a.rotary_dim, sms, s, (a.flags & W4A16_FLAG_PDL) != 0);
}

cudaError_t launch_rope(const w4a16_rope_args& a, int sms, cudaStream_t s) {
    RowParams p = {};
    p.q = static_cast<const uint16_t*>(a.x), p.q_out = static_cast<uint16_t*>(a.out);
    p.positions = a.positions, p.freq = a.frequencies;
    p.q_token = a.x_token, p.q_head = a.x_head, p.o_token = a.out_token, p.o_head = a.out_head;
    p.tokens = a.tokens, p.q_heads = a.heads, p.d = a.head_dim;
    p.interleaved = a.interleaved, p.magnitude = a.magnitude;
    return launch(p, a.dtype == W4A16_BF16, kCode16, a.rotary_dim, sms, s, (a.flags & W4A16_FLAG_PDL) != 0);
}

void rope_frequencies(int r, double base, int scaling, double factor, double length, double low, double high, double* f,
                      float* magnitude) {
    const double two_pi = 6.283185307179586476925;
    const double b = scaling == W4A16_ROPE_BASE && r > 2 ? base * std::pow(factor, (double)r / (r - 2)) : base;
    // the pair (not a whole number) that turns `turns` times in `length` positions
    auto pair_of = [&](double turns) { return r * std::log(length / (turns * two_pi)) / (2 * std::log(base)); };
    double lo = 0, hi = 0;
    if (scaling == W4A16_ROPE_RAMP) {
        lo = std::fmax(std::floor(pair_of(high)), 0.0);
        hi = std::fmin(std::ceil(pair_of(low)), r / 2 - 1.0);
    }
    *magnitude = scaling == W4A16_ROPE_RAMP ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
    for (int i = 0; i < r / 2; ++i) {
        f[i] = std::pow(b, -2.0 * i / r);
        double stretched = scaling == W4A16_ROPE_LINEAR ? 1.0 : 0.0;
        if (scaling == W4A16_ROPE_RAMP) stretched = (i - lo) / std::fmax(hi - lo, 0.001);
        if (scaling == W4A16_ROPE_WAVELENGTH) stretched = (high - length * f[i] / two_pi) / (high - low);
        stretched = std::fmin(std::fmax(stretched, 0.0), 1.0);
        f[i] = f[i] * (1.0 - stretched) + f[i] / factor * stretched;
    }
}

}  // namespace w4a16
