// What the small-row kernels of the paged attention share (16-bit caches:
// paged_decode.cuh, 8-bit ones: paged_decode8.cuh): how the keys of all requests
// are cut over the CTAs, and how the pieces of a pair are joined.
//
// The 128-key units of all (request, key head) pairs form one line, and CTA c of
// C (one an SM) takes the places [c U / C, (c + 1) U / C).  A pair whose units
// fall to several CTAs is joined by the last of them to arrive, in CTA order, so
// the result does not depend on timing.
#pragma once

#include "paged_attn.cuh"

namespace w4a16 {

constexpr int kDecWarps = 8;
constexpr int kDecThreads = 32 * kDecWarps;
constexpr int kDecTile = 16;                      // keys of a warp's tile
constexpr int kDecUnit = kDecTile * kDecWarps;    // keys of a unit
// What a pair costs beside its units, in units: the rows' first load, the
// warps' meeting and the output, of which the copies ahead hide a part.
constexpr int kDecPair = 2;
template <int D, int ROWS = 16>
constexpr int kDecPart = ROWS * (D + 2);          // floats of a partial result: (maximum, sum) of its rows, the rows

// Units of a request for one key head, and its first key (a multiple of 16).
struct DecSpan {
    int units, j0;
};
template <bool TREE>
W4A16_DEVICE DecSpan dec_span(const PagedAttnParams& p, const Request& r) {
    DecSpan s{0, 0};
    if (r.n == 0 || r.n * p.G > p.small_rows) return s;
    const Seen see = seen_by<TREE>(p, r, 0, r.n - 1);
    s.j0 = see.first & ~(kDecTile - 1);
    const int keys = see.last + 1 - s.j0;
    s.units = keys > 0 ? (keys + kDecUnit - 1) / kDecUnit : 1;  // no key: one unit that writes zeros
    return s;
}

// x / y for 0 <= x and 0 < y: in 32 bits where both fit, a fifth of the time
W4A16_DEVICE int64_t quotient(int64_t x, int64_t y) {
    return (x | y) >> 32 ? x / y : (int64_t)((uint32_t)x / (uint32_t)y);
}
// CTA that holds place u of the line of U places cut over C CTAs
W4A16_DEVICE int owner_of(int64_t u, int64_t U, int C) { return (int)quotient((u + 1) * C - 1, U); }

// This CTA's part of the line, which begins in pair (b, hk) of request r; a pair
// takes kDecPair + units places.
struct DecCut {
    int64_t U, u0, u1, s0;  // the line's places, the CTA's, and the first pair's first
    int C, b, hk;
    Request r;
    DecSpan sp;
};
// False where there is nothing to do.  Every thread of the CTA calls it; warp_sum
// holds kDecWarps numbers, misc 8.
template <bool TREE>
W4A16_DEVICE bool dec_cut(const PagedAttnParams& p, int64_t* warp_sum, volatile int* misc, DecCut& cut) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = (int)blockIdx.x;
    const int per = (p.B + kDecThreads - 1) / kDecThreads;
    const int b0 = min((int)threadIdx.x * per, p.B), b1 = min(b0 + per, p.B);
    Request r{0, 0, 0};
    DecSpan sp{0, 0};
    int64_t mine = 0;
    auto places = [&](int b) {  // of a request, r and sp on the way
        r = request_of(p, b);
        sp = dec_span<TREE>(p, r);
        return sp.units ? (int64_t)(sp.units + kDecPair) * p.Hkv : (int64_t)0;
    };
    for (int b = b0; b < b1; ++b) mine += places(b);
    int64_t before = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, before, d);
        if (lane >= d) before += x;
    }
    if (lane == 31) warp_sum[warp] = before;
    __syncthreads();
    int64_t U = 0;
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) {
        if (w < warp) before += warp_sum[w];
        U += warp_sum[w];
    }
    before -= mine;
    const int C = (int)(U < gridDim.x ? U : gridDim.x);  // every CTA of the C has a place at least
    if (c >= C) return false;
    const int64_t u0 = quotient(c * U, C), u1 = quotient((c + 1) * U, C);
    if (u0 >= before && u0 < before + mine) {
        int64_t at = before;
        for (int b = b0; b < b1; ++b) {
            const int64_t n = per == 1 ? mine : places(b);
            if (u0 < at + n) {
                const int len = sp.units + kDecPair;
                misc[0] = b;
                const int head = (int)quotient(u0 - at, len);
                misc[1] = head;
                misc[2] = (int)(u0 - at - (int64_t)head * len);
                misc[3] = r.t0;
                misc[4] = r.n;
                misc[5] = r.L;
                misc[6] = sp.units;
                misc[7] = sp.j0;
                break;
            }
            at += n;
        }
    }
    __syncthreads();
    cut.U = U;
    cut.u0 = u0;
    cut.u1 = u1;
    cut.C = C;
    cut.b = misc[0];
    cut.hk = misc[1];
    cut.s0 = u0 - misc[2];
    cut.r = Request{misc[3], misc[4], misc[5]};
    cut.sp = DecSpan{misc[6], misc[7]};
    return u1 > cut.s0 + kDecPair;  // else a place before the pair's first unit
}

// The pieces of a pair that CTAs c0 .. c1 hold; the last to arrive joins them in
// CTA order.  Every thread of the CTA calls it behind its stores of the piece.
// With `room` (a float4 and two floats a thread), and where the rows need half of the
// threads at most, groups of threads take every so many-th piece and meet there, in
// an order of their own: 18 pieces of four rows one after the other took 4.2 us.
template <typename Ty, int D, int ROWS = 16>
W4A16_DEVICE void dec_join(const PagedAttnParams& p, const Request& done, int done_hk, int c0, int c1, volatile int* misc,
                           float* room = nullptr) {
    const int R = done.n * p.G, pieces = c1 - c0 + 1;
    __syncthreads();
    if (threadIdx.x == 0) {
        unsigned n;  // releases the CTA's stores, ordered before by the barrier
        asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(n) : "l"(p.counters + c0) : "memory");
        const int last = n == (unsigned)(pieces - 1);
        if (last) p.counters[c0] = 0;
        misc[0] = last;
    }
    __syncthreads();
    if (!misc[0]) return;
    // a thread: four columns of a row, kJoin pieces at a time under a running maximum
    auto piece = [&](int i) { return p.part + (int64_t)(2 * (c0 + i) + (i == 0)) * kDecPart<D, ROWS>; };
    constexpr int kJoin = ROWS == 16 ? 12 : 4;
    const int elements = R * (D / 4);
    int groups = 1;
    if (room)
        while (2 * groups * elements <= kDecThreads && 2 * groups * 2 <= pieces) groups *= 2;
    const int group = groups > 1 ? (int)threadIdx.x / elements : 0;
    for (int e = groups > 1 ? (int)threadIdx.x - group * elements : (int)threadIdx.x;
         e < elements && (groups == 1 || group < groups); e += kDecThreads) {
        const int jr = e / (D / 4), col = (e - jr * (D / 4)) * 4;
        float jm = -INFINITY, js = 0.f;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i0 = group; i0 < pieces; i0 += kJoin * groups) {
            float2 mi[kJoin];
            float4 x[kJoin];
#pragma unroll
            for (int i = 0; i < kJoin; ++i) {
                mi[i] = make_float2(-INFINITY, 0.f);
                if (i0 + i * groups < pieces) {
                    mi[i] = __ldcg(reinterpret_cast<const float2*>(piece(i0 + i * groups)) + jr);
                    x[i] = __ldcg(reinterpret_cast<const float4*>(piece(i0 + i * groups) + 2 * ROWS + jr * D + col));
                }
            }
            float M = jm;
#pragma unroll
            for (int i = 0; i < kJoin; ++i) M = fmaxf(M, mi[i].x);
            const float jb = M == -INFINITY ? 0.f : M;
            const float g = jm == -INFINITY ? 1.f : exp2_approx(jm - jb);
            js *= g;
            y.x *= g;
            y.y *= g;
            y.z *= g;
            y.w *= g;
            jm = M;
#pragma unroll
            for (int i = 0; i < kJoin; ++i) {
                if (mi[i].y == 0.f) continue;  // no piece, or no seen key in it
                const float f = exp2_approx(mi[i].x == -INFINITY ? 0.f : mi[i].x - jb);
                js = fmaf(mi[i].y, f, js);
                y.x = fmaf(x[i].x, f, y.x);
                y.y = fmaf(x[i].y, f, y.y);
                y.z = fmaf(x[i].z, f, y.z);
                y.w = fmaf(x[i].w, f, y.w);
            }
        }
        if (groups > 1) {
            float4* ys = reinterpret_cast<float4*>(room);
            float2* ms = reinterpret_cast<float2*>(room + 4 * kDecThreads);
            ys[threadIdx.x] = y;
            ms[threadIdx.x] = make_float2(jm, js);
            named_bar(4, groups * elements);  // (whole warps: elements are a multiple of 16, groups even)
            if (group > 0) return;
            for (int g = 1; g < groups; ++g) {
                const float2 o = ms[g * elements + e];
                const float4 v = ys[g * elements + e];
                const float M = fmaxf(jm, o.x), b = M == -INFINITY ? 0.f : M;
                const float fa = js == 0.f ? 0.f : exp2_approx(jm == -INFINITY ? 0.f : jm - b);
                const float fb = o.y == 0.f ? 0.f : exp2_approx(o.x == -INFINITY ? 0.f : o.x - b);
                js = js * fa + o.y * fb;
                y = make_float4(y.x * fa + v.x * fb, y.y * fa + v.y * fb, y.z * fa + v.z * fb, y.w * fa + v.w * fb);
                jm = M;
            }
        }
        const int i = jr / p.G, h = done_hk * p.G + jr - i * p.G;
        const float inv = 1.f / js;
        uint2 v = make_uint2(0u, 0u);
        if (js != 0.f) v = make_uint2(Ty::pack(y.x * inv, y.y * inv), Ty::pack(y.z * inv, y.w * inv));
        *reinterpret_cast<uint2*>(p.out + (int64_t)(done.t0 + i) * p.o_token + (int64_t)h * p.o_head + col) = v;
        if (p.lse && col == 0)
            p.lse[(int64_t)(done.t0 + i) * p.Hq + h] = js == 0.f ? -INFINITY : kLn2 * (jm + log2f(js));
    }
}

}  // namespace w4a16
