// Rotary positions of queries and keys, and keys and values into the paged cache
// of 16 or 8 bits, in one launch; w4a16_rope is the same kernel with queries alone.
//
//     (a, b) -> (a cos w - b sin w, a sin w + b cos w) magnitude,  w = position * frequency
//     scale = max |x| / top,  code = round(x * (top / max |x|))
//
// A CTA takes a few tokens.  Its threads first make the cosines and sines of the
// tokens' pairs, in shared memory for all heads, then 16 lanes (32 for heads over
// 128 wide) take a token's rows one after the other, 8 elements a lane, with the
// cosines and sines of their columns in registers.  Angles: a frequency
// is a 64-bit fraction F of a turn a position, so position * F modulo 2^64 is the
// fraction of a turn, without rounding; its top 32 bits go to sincospi.
//
// Bound: HBM, each row read and written once; what is left to it is the latency of a
// round and, in 8 bits, issue slots (196 instructions a warp for two rows, 62 % of the
// slots).  Queries alone have the loads of three rows on their way (one 73 us, two 61-65,
// three 58.6, four 58.4), a store one (two ahead: a fifth more time with turns, 52 us for 49
// without, stored and read back).
// Measured: 16301 tokens of 40 heads of 128 in bf16 (334 MB), half of each head
// turned: 58.6 us, 5.7 TB/s, the whole head in pairs 59.4; keys and values of 16301
// tokens, 8 heads of 128, to e4m3 (101 MB), with the read-back of the cache
// 49; 64 tokens of 32 + 8 heads, turned and to int8: 6.7 us alone, 9.7 us a call.
// 16301 tokens of 32 + 8 heads and their values, turned and stored: 110 us to int8 (109 to
// e4m3, 107 to 16 bits) for a floor of 54 (59), half the rate of either of its parts: the
// query rows, two in three, take the one load ahead of the others and, in 8 bits, their
// shuffles and products too.  (w4a16_rope over both and w4a16_kv_write: 96, in 16 bits 89.)
#include <cmath>

#include "codes.cuh"
#include "kernels.h"
#include "paged_attn.cuh"

namespace w4a16 {

constexpr int kRowThreads = 256;

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
    int per_shift;  // log2 of the tokens of a CTA
    int rows, cta_rows;  // rows (q heads, k heads, v heads) of a token, and those of one CTA
    bool by_lane;   // a pair's partner is in the same lane, or in the lane `half / 8` on
    float magnitude;
    FastDiv by_half;
};

enum { kCode16 = 0, kCodeInt8 = 1, kCodeE4m3 = 2 };

template <typename Ty>
W4A16_DEVICE float half_of(const uint4& v, int i) {
    const uint32_t x = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
    return i & 1 ? Ty::hi(x) : Ty::lo(x);
}

// KV: keys and values too, else queries alone; TURN: with rotary positions.  CTAs an SM as the registers allow.  Without
// turns, five of 48 registers: 16301 tokens stored in 8 bits and read back 49 us, with four 52, with six 55.
template <typename Ty, int CODE, int LANES, bool KV, bool TURN>
__global__ void __launch_bounds__(kRowThreads, !TURN ? 5 : 3) kv_store_kernel(const __grid_constant__ RowParams p) {
    extern __shared__ float2 turn[];  // [token][pair] cosine and sine
    pdl_wait();
    pdl_launch_dependents();
    constexpr int GROUPS = kRowThreads / LANES;
    const int group = threadIdx.x / LANES, lane = threadIdx.x % LANES, col = 8 * lane;
    // a group of lanes has one token, and every step-th of its rows from `sub` on
    const int tt = group & ((1 << p.per_shift) - 1), sub = group >> p.per_shift, step = GROUPS >> p.per_shift;
    const int t0 = (int)blockIdx.x << p.per_shift, t = t0 + tt, nt = min(1 << p.per_shift, p.tokens - t0);
    const int r0 = (int)blockIdx.y * p.cta_rows, r1 = min(r0 + p.cta_rows, p.rows);
    const bool on = t < p.tokens && col < p.d;
    const bool here = on && (!TURN || p.positions[t] >= 0);
    const int slot = KV && t < p.tokens ? p.slots[t] : -1;
    const bool stored = here && slot >= 0 && slot < p.total_slots;
    // what of an address goes by the token
    const int64_t pg = slot >> p.shift, sl = slot & ((1 << p.shift) - 1);
    const uint16_t *qs = p.q + t * p.q_token + col, *ks = nullptr, *vs = nullptr;
    int64_t kat = 0, vat = 0;
    float *kscale = nullptr, *vscale = nullptr;
    if constexpr (KV) {
        ks = p.k + t * p.k_token + col;
        vs = p.v + t * p.v_token + col;
        kat = pg * p.kcp + sl * p.kcs + col;
        vat = pg * p.vcp + sl * p.vcs + col;
        if constexpr (CODE != kCode16) {
            kscale = p.ks + pg * p.ksp + sl * p.kss;
            vscale = p.vs + pg * p.vsp + sl * p.vss;
        }
    }
    uint16_t* const qo = p.q_out + t * p.o_token + col;

    struct Row {
        int kind, h;  // 0 query, 1 key, 2 value; head
        bool live;
        const uint16_t* src;
    };
    auto where = [&](int row) {
        Row r;
        r.kind = 0;
        r.h = row;
        r.live = here && row < r1;
        if (KV && row >= p.q_heads) {
            r.kind = row < p.q_heads + p.heads ? 1 : 2;
            r.h = row - p.q_heads - (r.kind == 2 ? p.heads : 0);
            r.live = stored && row < r1;
            r.src = (r.kind == 1 ? ks : vs) + r.h * (r.kind == 1 ? p.k_head : p.v_head);
        } else {
            r.src = qs + r.h * p.q_head;
        }
        return r;
    };
    auto load = [&](int row) {  // on its way
        const Row r = where(row);
        return r.live ? *reinterpret_cast<const uint4*>(r.src) : make_uint4(0u, 0u, 0u, 0u);
    };
    constexpr int AHEAD = KV ? 1 : 3;  // rows whose loads are on their way
    uint4 ahead[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) ahead[i] = load(r0 + i * step + sub);

    float2 w[8];  // of the lane's columns (of its pairs, the first four, where these lie together)
    uint32_t turned = 0;  // bit i: w[i] is of a column (of a pair) that turns
    if constexpr (TURN) {
        for (int e = threadIdx.x; e < nt * p.half; e += kRowThreads) {
            const int et = div_by(e, p.by_half.m, p.by_half.s), i = e - et * p.half;
            const double turns = p.freq[i] * 0.15915494309189533577;  // of 2 pi
            const int64_t f = __double2ll_rn((turns - rint(turns)) * 18446744073709551616.0);
            const uint64_t phase = (uint64_t)(int64_t)p.positions[t0 + et] * (uint64_t)f;
            float s, c;
            sincospif((float)(int32_t)(phase >> 32) * 4.656612873077393e-10f, &s, &c);  // 2 / 2^32
            turn[e] = make_float2(c * p.magnitude, s * p.magnitude);
        }
        __syncthreads();
        const float2* cs = turn + tt * p.half;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int at = col + (p.interleaved ? 2 * i : i);
            const bool does = on && at < 2 * p.half && (!p.interleaved || i < 4);
            turned |= does ? 1u << i : 0u;
            w[i] = does ? cs[p.interleaved ? at >> 1 : at < p.half ? at : at - p.half] : make_float2(1.f, 0.f);
        }
    }
    const int gap = p.half >> 3;
    const int partner = (threadIdx.x & 31 & ~(LANES - 1)) + (lane < gap ? lane + gap : lane < 2 * gap ? lane - gap : lane);
    if (TURN && !p.interleaved && lane < gap && p.by_lane)
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i].y = -w[i].y;

    auto turn_and_store = [&](int row, uint4& buffer) {
        const Row cur = where(row);
        const int kind = cur.kind, h = cur.h;
        const bool live = cur.live;
        const uint4 raw = buffer;
        buffer = load(row + AHEAD * step);
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = half_of<Ty>(raw, i);
        if constexpr (TURN) {
            const bool turns = !KV || kind < 2;
            if (p.interleaved) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (turns && ((turned >> i) & 1u)) {
                        const float a = x[2 * i], b = x[2 * i + 1];
                        x[2 * i] = a * w[i].x - b * w[i].y;
                        x[2 * i + 1] = a * w[i].y + b * w[i].x;
                    }
            } else if (p.by_lane) {
                const uint4 o = make_uint4(__shfl_sync(0xffffffffu, raw.x, partner), __shfl_sync(0xffffffffu, raw.y, partner),
                                           __shfl_sync(0xffffffffu, raw.z, partner), __shfl_sync(0xffffffffu, raw.w, partner));
                if (turns && turned)
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = x[i] * w[i].x + half_of<Ty>(o, i) * w[i].y;
            } else {
                // (partners by element, all read before any lane of the row writes: out may be x)
                float y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int at = col + i < p.half ? col + i + p.half : col + i - p.half;
                    y[i] = turns && live && ((turned >> i) & 1u) ? Ty::lo(cur.src[at - col]) : 0.f;
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (turns && ((turned >> i) & 1u))
                        x[i] = col + i < p.half ? x[i] * w[i].x - y[i] * w[i].y : x[i] * w[i].x + y[i] * w[i].y;
            }
        }
        const uint4 packed = make_uint4(Ty::pack(x[0], x[1]), Ty::pack(x[2], x[3]), Ty::pack(x[4], x[5]), Ty::pack(x[6], x[7]));
        if (!KV || kind == 0) {
            if (live) *reinterpret_cast<uint4*>(qo + h * p.o_head) = packed;
            if (!KV || CODE == kCode16) return;
        }
        const int64_t at = (kind == 1 ? kat : vat) + h * (kind == 1 ? p.kch : p.vch);
        if constexpr (CODE == kCode16) {
            // (what is not rotated is copied bit for bit)
            if (live) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(kind == 1 ? p.kc : p.vc) + at) =
                TURN && kind == 1 && col < 2 * p.half ? packed : raw;
        } else {
            uint32_t most = 0;  // magnitudes as integers: NaN and infinities are the largest
#pragma unroll
            for (int i = 0; i < 8; ++i) most = max(most, __float_as_uint(x[i]) & 0x7fffffffu);
#pragma unroll
            for (int i = 1; i < LANES; i <<= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, i));
            const float top = CODE == kCodeInt8 ? 127.f : 448.f, amax = __uint_as_float(most);
            const bool none = most < (27u << 23), bad = most >= 0x7f800000u;  // below 2^-100
            // amax / top: a quotient by a constant, put right by what it leaves (correct in the last place: Markstein, "Computation
            // of elementary functions on the IBM RISC System/6000 processor", 1990; tried for every mantissa)
            const float rcp = CODE == kCodeInt8 ? 1.f / 127.f : 1.f / 448.f, about = amax * rcp;
            const float quotient = __fmaf_rn(__fmaf_rn(-about, top, amax), rcp, about);
            const float scale = bad ? __uint_as_float(0x7fffffffu) : none ? 0.f : quotient;
            const float inv = bad || none ? 0.f : __fdiv_rn(top, amax);
            uint32_t codes[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float a = __fmul_rn(x[4 * i], inv), b = __fmul_rn(x[4 * i + 1], inv);
                const float c = __fmul_rn(x[4 * i + 2], inv), e = __fmul_rn(x[4 * i + 3], inv);
                if constexpr (CODE == kCodeInt8) {
                    // the sum with 1.5 * 2^23 is rounded to a whole number, which is its low bits
                    auto bits = [](float y) { return __float_as_uint(__fadd_rn(y, 12582912.f)); };
                    codes[i] = bad ? 0u : __byte_perm(__byte_perm(bits(a), bits(b), 0x0040), __byte_perm(bits(c), bits(e), 0x0040), 0x5410);
                } else {
                    uint16_t lo, hi;
                    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
                    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(e), "f"(c));
                    codes[i] = bad ? 0u : (uint32_t)lo | (uint32_t)hi << 16;
                }
            }
            if (live && kind) {
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(kind == 1 ? p.kc : p.vc) + at) = make_uint2(codes[0], codes[1]);
                if (lane == 0)
                    *((kind == 1 ? kscale : vscale) + h * (kind == 1 ? p.ksh : p.vsh)) = scale;
            }
        }
    };
    // (all lanes of a warp go round together: shuffles)
#pragma unroll 1
    for (int row = r0; row < r1; row += AHEAD * step)
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (i == 0 || row + i * step < r1) turn_and_store(row + i * step + sub, ahead[i]);
}

template <typename Ty, int CODE>
static cudaError_t launch_rows(const RowParams& p, dim3 grid, size_t smem, cudaStream_t s, bool pdl) {
    auto run = [&](auto kernel) { return launch_kernel(kernel, grid, dim3(kRowThreads), smem, s, pdl, p); };
    const bool narrow = p.d <= 128;
    if constexpr (CODE == kCode16)
        if (p.heads == 0) return narrow ? run(kv_store_kernel<Ty, CODE, 16, false, true>) : run(kv_store_kernel<Ty, CODE, 32, false, true>);
    if (!p.freq) return narrow ? run(kv_store_kernel<Ty, CODE, 16, true, false>) : run(kv_store_kernel<Ty, CODE, 32, true, false>);
    return narrow ? run(kv_store_kernel<Ty, CODE, 16, true, true>) : run(kv_store_kernel<Ty, CODE, 32, true, true>);
}

static cudaError_t launch(RowParams& p, bool bf16, int code, int rot, int sms, cudaStream_t s, bool pdl) {
    p.half = p.freq ? rot / 2 : 1;
    p.by_lane = p.half % 8 == 0;
    p.rows = p.q_heads + 2 * p.heads;
    const int groups = kRowThreads / (p.d <= 128 ? 16 : 32);
    // Tokens of a CTA, a power of two: as many as its groups of lanes have rows for, up to 24 rounds of them while
    // the GPU stays full (a lane's cosines are read once, loads are a round ahead); a token's rows over several CTAs
    // where tokens are too few.
    while ((2 << p.per_shift) <= groups && (p.rows << p.per_shift) * 2 <= groups) ++p.per_shift;
    while ((2 << p.per_shift) <= groups && (p.rows << p.per_shift) * 2 <= 24 * groups &&
           (p.tokens >> (p.per_shift + 1)) >= 12 * sms)
        ++p.per_shift;
    const int per = 1 << p.per_shift, ctas = (p.tokens + per - 1) / per;
    int split = 1;
    while (ctas * split * 2 <= 4 * sms && (p.rows + split * 2 - 1) / (split * 2) >= groups) split *= 2;
    p.cta_rows = (p.rows + split - 1) / split;
    p.by_half = fast_div(p.half);
    const dim3 grid((unsigned)ctas, (unsigned)((p.rows + p.cta_rows - 1) / p.cta_rows));
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
    // the pair (not a whole number, and it may lie outside the head's) that turns `turns` times in `length` positions
    auto pair_of = [&](double turns) { return r * std::log(length / (turns * two_pi)) / (2 * std::log(base)); };
    double lo = 0, hi = 0;
    if (scaling == W4A16_ROPE_RAMP) {
        lo = std::fmax(std::floor(pair_of(high)), 0.0);
        hi = std::fmin(std::ceil(pair_of(low)), r - 1.0);  // (behind the last pair where that turns more than `low` times)
    }
    *magnitude = scaling == W4A16_ROPE_RAMP ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
    for (int i = 0; i < r / 2; ++i) {
        f[i] = std::pow(b, -2.0 * i / r);
        double stretched = scaling == W4A16_ROPE_LINEAR ? 1.0 : 0.0;
        if (scaling == W4A16_ROPE_RAMP) stretched = i >= hi ? 1.0 : (i - lo) / std::fmax(hi - lo, 1.0);
        if (scaling == W4A16_ROPE_WAVELENGTH) stretched = (high - length * f[i] / two_pi) / (high - low);
        stretched = std::fmin(std::fmax(stretched, 0.0), 1.0);
        f[i] = f[i] * (1.0 - stretched) + f[i] / factor * stretched;
    }
}

}  // namespace w4a16
