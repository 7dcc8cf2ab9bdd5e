// Paged attention for few query rows: requests whose new tokens make at most
// 16 rows a key head (one token with up to 16 heads a group, or a few tokens).
//
//     row r = i G + g of (request b, key head hk): token i, head hk G + g
//     out = sum_j 2^(s_j - m) v_j / sum_j 2^(s_j - m),  s_j = scale log2(e) q . k_j
//
// Bound: HBM -- every key and value of every request is read once, and 16 rows
// do 4 x 16 flops a byte at most.  So the work is cut by bytes, not by
// requests: the 128-key units of all (request, key head) pairs form one line,
// and CTA c of C (one an SM) takes the units [c U / C, (c + 1) U / C).  A pair
// whose units fall to several CTAs is joined by the last of them to arrive, in
// CTA order, so the result does not depend on timing.
//
// Inside a CTA eight warps work without meeting: warp w takes the 16-key tiles
// w, w + 8, ... of the range through a ring of its own, filled by tensor
// copies (one 128-byte-swizzled box a page and 64 columns) that its lane 0
// issues, and keeps the rows' maxima, sums and 16 x head_dim outputs in
// registers.  The products are warp-wide 16 x 8 x 16 MMAs: with 16 rows the
// tensor pipe is not what bounds this kernel, and fragments that stay in
// registers need no tensor-memory round trip between the two products.  The
// warps' results meet once per pair, in shared memory.
//
// Positions that a row does not see are masked in the scores; the values of
// positions that no row of the tile sees (stale slots of the last page, slots
// before the window) are cleared in shared memory first, and non-finite values
// that only some rows see are added for those rows alone, so that no row takes
// a NaN from a position outside its own.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "paged_attn.cuh"

namespace w4a16 {

static __device__ int g_decode_status;

constexpr int kDecWarps = 8;
constexpr int kDecThreads = 32 * kDecWarps;
constexpr int kDecTile = 16;                      // keys of a warp's tile
constexpr int kDecUnit = kDecTile * kDecWarps;    // keys of a unit

template <int D>
struct Dec {
    static constexpr int kSlabs = D / 64;                    // 64-column slabs of a tile
    static constexpr int kHalf = kSlabs * kDecTile * 128;    // bytes of a tile's keys (and of its values)
    static constexpr int kSlots = D == 128 ? 3 : 6;          // ring slots a warp
    static constexpr int kRing = kDecWarps * kSlots * 2 * kHalf;
    static constexpr int kRegs = D / 2;                      // output accumulators a thread
    static constexpr int kMergeOff = kRing;
    static constexpr int kMerge = 4 * kRegs * 32 * 4;
    static constexpr int kMlOff = kMergeOff + kMerge;        // [warp][16][2]
    static constexpr int kBarOff = kMlOff + kDecWarps * 16 * 2 * 4;
    static constexpr int kMiscOff = kBarOff + kDecWarps * kSlots * 8;
    static constexpr int kSmem = kMiscOff + 64 + 1024;
    static constexpr int kPart = 16 * (D + 2);               // floats of a partial result
};
static_assert(Dec<128>::kSmem <= 232448 && Dec<64>::kSmem <= 232448, "shared memory");

// Units of a request for one key head, and its first key (a multiple of 16).
struct DecSpan {
    int units, j0;
};
W4A16_DEVICE DecSpan dec_span(const PagedAttnParams& p, const Request& r) {
    DecSpan s{0, 0};
    if (r.n == 0 || r.n * p.G > p.small_rows) return s;
    s.j0 = first_seen(p, last_seen(p, r, 0)) & ~(kDecTile - 1);
    const int keys = last_seen(p, r, r.n - 1) + 1 - s.j0;
    s.units = keys > 0 ? (keys + kDecUnit - 1) / kDecUnit : 1;  // no key: one unit that writes zeros
    return s;
}

// CTA that holds unit u of U over C CTAs
W4A16_DEVICE int owner_of(int64_t u, int64_t U, int C) { return (int)(((u + 1) * C - 1) / U); }

template <typename Ty, int D>
__global__ void __launch_bounds__(kDecThreads, 1)
    paged_decode_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                        const PagedAttnParams p) {
    using L = Dec<D>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem =
        reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    float* merge = reinterpret_cast<float*>(smem + L::kMergeOff);
    float* ml = reinterpret_cast<float*>(smem + L::kMlOff);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
    volatile int* misc = reinterpret_cast<volatile int*>(smem + L::kMiscOff);
    volatile int* abort_flag = misc;  // misc: abort, request, head, offset, last
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = (int)blockIdx.x;

    uint64_t* wbar = bars + warp * L::kSlots;
    unsigned char* ring = smem + warp * (L::kSlots * 2 * L::kHalf);
    if (threadIdx.x == 0) *abort_flag = 0;
    if (lane == 0) {
        for (int i = 0; i < L::kSlots; ++i) mbar_init(wbar + i, 1);
        fence_mbar_init();
        prefetch_tmap(&tmap_k);
        prefetch_tmap(&tmap_v);
    }
    pdl_launch_dependents();
    pdl_wait();

    // ---- this CTA's units: sums over the requests, a run of them a thread ----
    __shared__ int64_t warp_sum[kDecWarps];
    const int per = (p.B + kDecThreads - 1) / kDecThreads;
    const int b0 = min((int)threadIdx.x * per, p.B), b1 = min(b0 + per, p.B);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) mine += (int64_t)dec_span(p, request_of(p, b)).units * p.Hkv;
    int64_t before = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, before, d);
        if (lane >= d) before += x;
    }
    if (lane == 31) warp_sum[warp] = before;
    __syncthreads();
    int64_t U = 0;
    for (int w = 0; w < kDecWarps; ++w) {
        if (w < warp) before += warp_sum[w];
        U += warp_sum[w];
    }
    before -= mine;
    const int C = (int)(U < gridDim.x ? U : gridDim.x);  // every CTA of the C has a unit at least
    if (c >= C) return;
    const int64_t u0 = (int64_t)c * U / C, u1 = (int64_t)(c + 1) * U / C;
    if (u0 >= before && u0 < before + mine) {
        int64_t at = before;
        for (int b = b0; b < b1; ++b) {
            const int64_t n = (int64_t)dec_span(p, request_of(p, b)).units;
            if (u0 < at + n * p.Hkv) {
                misc[1] = b;
                misc[2] = (int)((u0 - at) / n);
                misc[3] = (int)((u0 - at) % n);
                break;
            }
            at += n * p.Hkv;
        }
    }
    __syncthreads();
    int b = misc[1], hk = misc[2], off = misc[3];
    int64_t u = u0;  // the current piece's first unit

    // ---- the warp's ring -------------------------------------------------
    int put = 0, get = 0;          // slots to fill and to read next
    uint32_t parity = 0;           // of `get`
    uint32_t gone = 0;             // 2 bits a slot: pages of the tile that are not there
    const int page = 1 << p.shift, box = page < kDecTile ? page : kDecTile;
    const int boxes = kDecTile / box;  // 1, or 2 for 8-slot pages

    struct Piece {
        Request r;
        int j0, e_last, tile0, tiles;  // first key, last key seen, this warp's first tile and their number
    } w;
    int ent[2];       // table entries of the tiles ent_base + lane
    int ent_base = 0;
    auto open_piece = [&](int take) {
        w.r = request_of(p, b);
        const DecSpan s = dec_span(p, w.r);
        w.j0 = s.j0;
        w.e_last = last_seen(p, w.r, w.r.n - 1);
        w.tile0 = off * kDecWarps + warp;
        const int all = w.e_last < w.j0 ? 0 : (w.e_last - w.j0) / kDecTile + 1;  // tiles that hold a seen key
        const int end = min((off + take) * kDecWarps, all);
        w.tiles = w.tile0 < end ? (end - w.tile0 + kDecWarps - 1) / kDecWarps : 0;
        ent_base = -32;
    };
    auto entries = [&](int base) {  // lane i: the pages of tile base + i
        ent_base = base;
        const int t = base + lane;
        ent[0] = ent[1] = -1;
        if (t < w.tiles) {
            const int j = w.j0 + (w.tile0 + t * kDecWarps) * kDecTile;
            const int* row = p.table + (int64_t)b * p.table_stride;
            for (int i = 0; i < boxes; ++i) {
                const int col = (j + i * box) >> p.shift;
                if (col < p.columns) ent[i] = row[col];
            }
        }
    };
    auto issue = [&](int t) {  // the copies of this piece's tile t
        if (t >= ent_base + 32) entries(t);
        int pg[2];
        uint32_t no = 0;
        for (int i = 0; i < boxes; ++i) {
            pg[i] = __shfl_sync(0xffffffffu, ent[i], t - ent_base);
            if (pg[i] < 0 || pg[i] >= p.pages) {
                pg[i] = p.pages;  // past the tensor: the copy fills with zeros
                no |= 1u << i;
            }
        }
        gone = (gone & ~(3u << (2 * put))) | no << (2 * put);
        __syncwarp();  // every lane has read the slot's last tile
        if (lane == 0) {
            unsigned char* dst = ring + put * 2 * L::kHalf;
            const int j = w.j0 + (w.tile0 + t * kDecWarps) * kDecTile;
            mbar_arrive_expect_tx(wbar + put, 2u * L::kHalf);
            for (int i = 0; i < boxes; ++i) {
                const int slot = (j + i * box) & (page - 1);
#pragma unroll
                for (int s = 0; s < L::kSlabs; ++s)
                    tma_load_4d(dst + s * (kDecTile * 128) + i * box * 128, &tmap_k, 64 * s, slot, hk, pg[i],
                                wbar + put);
#pragma unroll
                for (int s = 0; s < L::kSlabs; ++s)
                    tma_load_4d(dst + L::kHalf + s * (kDecTile * 128) + i * box * 128, &tmap_v, 64 * s, slot, hk,
                                pg[i], wbar + put);
            }
        }
        put = put + 1 == L::kSlots ? 0 : put + 1;
    };

    int64_t left = u1 - u0;
    int units = dec_span(p, request_of(p, b)).units;
    int take = (int)(left < units - off ? left : units - off);
    open_piece(take);
    int issued = 0;
    for (; issued < w.tiles && issued < L::kSlots; ++issued) issue(issued);

    while (true) {
        // ---- the query rows as A fragments -------------------------------
        const int R = w.r.n * p.G;
        const int ra = lane >> 2, rb = ra + 8;  // this thread's two rows
        uint32_t qa[D / 16][4];
        {
            const int ia = ra / p.G, ib = rb / p.G;
            const uint32_t* qpa = reinterpret_cast<const uint32_t*>(
                p.q + (int64_t)(w.r.t0 + ia) * p.q_token + (int64_t)(hk * p.G + ra - ia * p.G) * p.q_head) + (lane & 3);
            const uint32_t* qpb = reinterpret_cast<const uint32_t*>(
                p.q + (int64_t)(w.r.t0 + ib) * p.q_token + (int64_t)(hk * p.G + rb - ib * p.G) * p.q_head) + (lane & 3);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                qa[k][0] = ra < R ? qpa[8 * k] : 0u;
                qa[k][1] = rb < R ? qpb[8 * k] : 0u;
                qa[k][2] = ra < R ? qpa[8 * k + 4] : 0u;
                qa[k][3] = rb < R ? qpb[8 * k + 4] : 0u;
            }
        }
        const int ea = ra < R ? last_seen(p, w.r, ra / p.G) : -1, eb = rb < R ? last_seen(p, w.r, rb / p.G) : -1;
        const int la = first_seen(p, ea), lb = first_seen(p, eb);
        const int e_min = last_seen(p, w.r, 0), lo_min = first_seen(p, e_min);
        const int lo_max = first_seen(p, w.e_last);

        float o[D / 8][4];
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[n][i] = 0.f;
        float ma = -INFINITY, mb = -INFINITY, sa = 0.f, sb = 0.f;

        bool ok = true;
        for (int t = 0; t < issued; ++t) {
            ok = mbar_wait_warp(wbar + get, parity, abort_flag, &g_decode_status) && ok;
            // given up: the copies in flight still have to land, none is added
            if (!ok) (void)mbar_wait_warp(wbar + get, parity, nullptr, &g_decode_status);
            const uint32_t kb = smem_u32(ring + get * 2 * L::kHalf), vb = kb + L::kHalf;
            const uint32_t no = (gone >> (2 * get)) & 3u;
            const int j = w.j0 + (w.tile0 + t * kDecWarps) * kDecTile;
            if (ok) {
                // scores: two accumulators a column tile, even and odd steps
                float s0[4] = {}, s1[4] = {}, s2[4] = {}, s3[4] = {};
                {
                    const int row = (lane & 7) + ((lane & 16) >> 1), ch = (lane >> 3) & 1;
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        uint32_t f[4];
                        const int chunk = 2 * (k & 3) + ch;
                        ldsm_x4(f, kb + (k >> 2) * (kDecTile * 128) + row * 128 + ((chunk ^ (row & 7)) << 4));
                        mma_16816<Ty>(k & 1 ? s2 : s0, qa[k], f[0], f[1]);
                        mma_16816<Ty>(k & 1 ? s3 : s1, qa[k], f[2], f[3]);
                    }
                }
                float x[8];  // row a: keys 2q, 2q+1, 8+2q, 9+2q; row b alike (q = lane % 4)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    x[i] = (s0[i] + s2[i]) * p.scale2;
                    x[2 + i] = (s1[i] + s3[i]) * p.scale2;
                    x[4 + i] = (s0[2 + i] + s2[2 + i]) * p.scale2;
                    x[6 + i] = (s1[2 + i] + s3[2 + i]) * p.scale2;
                }
                const bool edge = j < lo_max || j + kDecTile - 1 > e_min || no;
                uint32_t alone = 0;  // keys of the tile whose values are added row by row
                if (edge) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int key = (i & 1) + 2 * (lane & 3) + 8 * (i >> 1), jj = j + key;
                        const bool there = !((no >> (boxes == 2 ? key >> 3 : 0)) & 1u);
                        if (!(there && jj >= la && jj <= ea)) x[i] = -INFINITY;
                        if (!(there && jj >= lb && jj <= eb)) x[4 + i] = -INFINITY;
                    }
                    // values: a lane looks at half a key's row
                    const int key = lane >> 1, jj = j + key;
                    const bool none = jj < lo_min || jj > w.e_last;  // seen by no row
                    const bool some = !none && (jj < lo_max || jj > e_min);
                    bool odd = false;
                    if (none || some) {
                        for (int s = 0; s < L::kSlabs; ++s)
                            for (int i = 0; i < 4; ++i) {
                                const uint32_t a = vb + s * (kDecTile * 128) + key * 128 + ((((lane & 1) * 4 + i) ^ (key & 7)) << 4);
                                if (none) {
                                    asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(a), "r"(0) : "memory");
                                } else {
                                    const uint4 v = lds_v4(a);
                                    for (uint32_t y : {v.x, v.y, v.z, v.w})
                                        odd |= !(fabsf(Ty::lo(y)) < INFINITY) || !(fabsf(Ty::hi(y)) < INFINITY);
                                }
                            }
                    }
                    const uint32_t lanes = __ballot_sync(0xffffffffu, odd);
                    for (int i = 0; i < kDecTile; ++i)
                        if ((lanes >> (2 * i)) & 3u) alone |= 1u << i;
                    fence_proxy_async_smem();  // the slot's next copy comes after these stores
                    __syncwarp();
                }
                float na = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), nb = fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7]));
#pragma unroll
                for (int d = 1; d < 4; d <<= 1) {
                    na = fmaxf(na, __shfl_xor_sync(0xffffffffu, na, d));
                    nb = fmaxf(nb, __shfl_xor_sync(0xffffffffu, nb, d));
                }
                na = fmaxf(na, ma);
                nb = fmaxf(nb, mb);
                if (__any_sync(0xffffffffu, na > ma || nb > mb)) {
                    const float fa = na == -INFINITY ? 1.f : exp2_approx(ma - na);
                    const float fb = nb == -INFINITY ? 1.f : exp2_approx(mb - nb);
                    sa *= fa;
                    sb *= fb;
#pragma unroll
                    for (int n = 0; n < D / 8; ++n) {
                        o[n][0] *= fa;
                        o[n][1] *= fa;
                        o[n][2] *= fb;
                        o[n][3] *= fb;
                    }
                    ma = na;
                    mb = nb;
                }
                const float ba = ma == -INFINITY ? 0.f : ma, bb = mb == -INFINITY ? 0.f : mb;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[i] = exp2_approx(x[i] - ba);
                    x[4 + i] = exp2_approx(x[4 + i] - bb);
                    sa += x[i];
                    sb += x[4 + i];
                }
                if (alone) {
                    for (int key = 0; key < kDecTile; ++key) {
                        if (!((alone >> key) & 1u)) continue;
                        const int src = (lane & ~3) + ((key & 7) >> 1), i = (key & 1) + ((key >> 3) << 1);
                        const float mine_a = i == 0 ? x[0] : i == 1 ? x[1] : i == 2 ? x[2] : x[3];
                        const float mine_b = i == 0 ? x[4] : i == 1 ? x[5] : i == 2 ? x[6] : x[7];
                        const float wa = __shfl_sync(0xffffffffu, mine_a, src), wb = __shfl_sync(0xffffffffu, mine_b, src);
                        const bool va = j + key >= la && j + key <= ea, vv = j + key >= lb && j + key <= eb;
#pragma unroll
                        for (int n = 0; n < D / 8; ++n) {
                            const uint32_t y = lds_u32(vb + (n >> 3) * (kDecTile * 128) + key * 128 +
                                                       (((n & 7) ^ (key & 7)) << 4) + (lane & 3) * 4);
                            if (va) {
                                o[n][0] = fmaf(wa, Ty::lo(y), o[n][0]);
                                o[n][1] = fmaf(wa, Ty::hi(y), o[n][1]);
                            }
                            if (vv) {
                                o[n][2] = fmaf(wb, Ty::lo(y), o[n][2]);
                                o[n][3] = fmaf(wb, Ty::hi(y), o[n][3]);
                            }
                        }
                    }
                    __syncwarp();
                    const int key = lane >> 1;
                    if ((alone >> key) & 1u)
                        for (int s = 0; s < L::kSlabs; ++s)
                            for (int i = 0; i < 4; ++i)
                                asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(
                                                 vb + s * (kDecTile * 128) + key * 128 +
                                                 ((((lane & 1) * 4 + i) ^ (key & 7)) << 4)),
                                             "r"(0)
                                             : "memory");
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                // the weights in two parts, x = hi + lo to 2^-16 (2^-22 in fp16): a decoding row often
                // hangs on a few positions, whose rounding does not average out, and the tensor pipe is idle
                const uint32_t pa[4] = {Ty::pack(x[0], x[1]), Ty::pack(x[4], x[5]), Ty::pack(x[2], x[3]),
                                        Ty::pack(x[6], x[7])};
                const uint32_t pb[4] = {Ty::pack(x[0] - Ty::lo(pa[0]), x[1] - Ty::hi(pa[0])),
                                        Ty::pack(x[4] - Ty::lo(pa[1]), x[5] - Ty::hi(pa[1])),
                                        Ty::pack(x[2] - Ty::lo(pa[2]), x[3] - Ty::hi(pa[2])),
                                        Ty::pack(x[6] - Ty::lo(pa[3]), x[7] - Ty::hi(pa[3]))};
                const int row = lane & 15, ch = lane >> 4;
#pragma unroll
                for (int n = 0; n < D / 16; ++n) {
                    uint32_t f[4];
                    const int chunk = 2 * (n & 3) + ch;
                    ldsm_x4_t(f, vb + (n >> 2) * (kDecTile * 128) + row * 128 + ((chunk ^ (row & 7)) << 4));
                    mma_16816<Ty>(o[2 * n], pa, f[0], f[1]);
                    mma_16816<Ty>(o[2 * n + 1], pa, f[2], f[3]);
                    mma_16816<Ty>(o[2 * n], pb, f[0], f[1]);
                    mma_16816<Ty>(o[2 * n + 1], pb, f[2], f[3]);
                }
            }
            if (++get == L::kSlots) {
                get = 0;
                parity ^= 1;
            }
            if (ok && issued < w.tiles) issue(issued++);
        }

        // ---- the next piece's first copies, before this one's results meet ----
        const Request r = w.r;
        const int done_hk = hk;
        const int64_t first = u - off, end = first + units;  // the pair's units on the line
        const bool from_start = off == 0, to_end = off + take == units;
        left -= take;
        u += take;
        const bool more = left > 0;
        if (more) {
            off = 0;
            if (++hk == p.Hkv) {
                hk = 0;
                do {
                    ++b;
                    units = dec_span(p, request_of(p, b)).units;
                } while (units == 0);
            }
            take = (int)(left < units ? left : units);
            open_piece(take);
            for (issued = 0; issued < w.tiles && issued < L::kSlots; ++issued) issue(issued);
        }

        // ---- the warps' results ------------------------------------------
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) {
            sa += __shfl_xor_sync(0xffffffffu, sa, d);
            sb += __shfl_xor_sync(0xffffffffu, sb, d);
        }
        if ((lane & 3) == 0) {
            ml[(warp * 16 + ra) * 2] = ma;
            ml[(warp * 16 + ra) * 2 + 1] = sa;
            ml[(warp * 16 + rb) * 2] = mb;
            ml[(warp * 16 + rb) * 2 + 1] = sb;
        }
        __syncthreads();
        float Ma = -INFINITY, Mb = -INFINITY;
#pragma unroll
        for (int i = 0; i < kDecWarps; ++i) {
            Ma = fmaxf(Ma, ml[(i * 16 + ra) * 2]);
            Mb = fmaxf(Mb, ml[(i * 16 + rb) * 2]);
        }
        const float fa = exp2_approx(ma - (Ma == -INFINITY ? 0.f : Ma));
        const float fb = exp2_approx(mb - (Mb == -INFINITY ? 0.f : Mb));
        if (warp >= 4) {
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    merge[(warp - 4) * (L::kRegs * 32) + (4 * n + i) * 32 + lane] = o[n][i] * (i < 2 ? fa : fb);
        }
        __syncthreads();
        if (warp < 4) {
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float* at = merge + warp * (L::kRegs * 32) + (4 * n + i) * 32 + lane;
                    *at = fmaf(o[n][i], i < 2 ? fa : fb, *at);
                }
        }
        __syncthreads();
        // thread: pairs of neighbouring columns of a row
        const bool whole = from_start && to_end;
        float* part = p.part + (int64_t)(2 * c + (from_start ? 1 : 0)) * L::kPart;
        for (int e = threadIdx.x; e < 16 * D / 2; e += kDecThreads) {
            const int ln = e & 31, half = (e >> 5) & 1, n = e >> 6;
            const int row = (ln >> 2) + 8 * half, col = 8 * n + 2 * (ln & 3);
            if (row >= R) continue;
            float y0 = 0.f, y1 = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                y0 += merge[i * (L::kRegs * 32) + (4 * n + 2 * half) * 32 + ln];
                y1 += merge[i * (L::kRegs * 32) + (4 * n + 2 * half + 1) * 32 + ln];
            }
            float M = -INFINITY, S = 0.f;
#pragma unroll
            for (int i = 0; i < kDecWarps; ++i) M = fmaxf(M, ml[(i * 16 + row) * 2]);
            const float base = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int i = 0; i < kDecWarps; ++i) {
                const float s = ml[(i * 16 + row) * 2 + 1];
                const float m = ml[(i * 16 + row) * 2];
                if (s != 0.f) S = fmaf(s, exp2_approx(m == -INFINITY ? 0.f : m - base), S);
            }
            if (whole) {
                const int i = row / p.G, h = done_hk * p.G + row - i * p.G;
                const float inv = 1.f / S;
                *reinterpret_cast<uint32_t*>(p.out + (int64_t)(r.t0 + i) * p.o_token + (int64_t)h * p.o_head + col) =
                    S == 0.f ? 0u : Ty::pack(y0 * inv, y1 * inv);
                if (p.lse && col == 0)
                    p.lse[(int64_t)(r.t0 + i) * p.Hq + h] = S == 0.f ? -INFINITY : kLn2 * (M + log2f(S));
            } else {
                *reinterpret_cast<float2*>(part + 32 + row * D + col) = make_float2(y0, y1);
                if (col == 0) {
                    part[2 * row] = M;
                    part[2 * row + 1] = S;
                }
            }
        }
        if (!whole) {
            // the pieces of CTAs c0 .. c1; the last to arrive joins them in CTA order
            const int c0 = owner_of(first, U, C), c1 = owner_of(end - 1, U, C);
            __threadfence();
            __syncthreads();
            if (threadIdx.x == 0) {
                const unsigned n = atomicAdd(p.counters + c0, 1u);
                const int last = n == (unsigned)(c1 - c0);
                if (last) p.counters[c0] = 0;
                misc[4] = last;
            }
            __syncthreads();
            if (misc[4]) {
                __threadfence();
                for (int e = threadIdx.x; e < R * (D / 4); e += kDecThreads) {
                    const int row = e / (D / 4), col = (e - row * (D / 4)) * 4;
                    float M = -INFINITY;
                    for (int i = c0; i <= c1; ++i)
                        M = fmaxf(M, __ldcg(p.part + (int64_t)(2 * i + (i == c0)) * L::kPart + 2 * row));
                    const float base = M == -INFINITY ? 0.f : M;
                    float S = 0.f;
                    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                    for (int i = c0; i <= c1; ++i) {
                        const float* q = p.part + (int64_t)(2 * i + (i == c0)) * L::kPart;
                        const float2 mi = __ldcg(reinterpret_cast<const float2*>(q + 2 * row));
                        const float4 x = __ldcg(reinterpret_cast<const float4*>(q + 32 + row * D + col));
                        if (mi.y == 0.f) continue;  // no seen key in this piece
                        const float f = exp2_approx(mi.x == -INFINITY ? 0.f : mi.x - base);
                        S = fmaf(mi.y, f, S);
                        y.x = fmaf(x.x, f, y.x);
                        y.y = fmaf(x.y, f, y.y);
                        y.z = fmaf(x.z, f, y.z);
                        y.w = fmaf(x.w, f, y.w);
                    }
                    const int i = row / p.G, h = done_hk * p.G + row - i * p.G;
                    const float inv = 1.f / S;
                    uint2 v = make_uint2(0u, 0u);
                    if (S != 0.f) v = make_uint2(Ty::pack(y.x * inv, y.y * inv), Ty::pack(y.z * inv, y.w * inv));
                    *reinterpret_cast<uint2*>(p.out + (int64_t)(r.t0 + i) * p.o_token + (int64_t)h * p.o_head + col) = v;
                    if (p.lse && col == 0)
                        p.lse[(int64_t)(r.t0 + i) * p.Hq + h] = S == 0.f ? -INFINITY : kLn2 * (M + log2f(S));
                }
            }
        }
        if (!more) break;
        __syncthreads();  // ml and merge are free again
    }
}

template <typename Ty, int D>
static cudaError_t launch(const CUtensorMap& tk, const CUtensorMap& tv, const PagedAttnParams& p, int ctas,
                          cudaStream_t s, bool pdl) {
    static bool set_for[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!set_for[dev]) {
        e = cudaFuncSetAttribute(paged_decode_kernel<Ty, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Dec<D>::kSmem);
        if (e != cudaSuccess) return e;
        set_for[dev] = true;
    }
    return launch_kernel(paged_decode_kernel<Ty, D>, dim3(ctas), dim3(kDecThreads), (size_t)Dec<D>::kSmem, s, pdl, tk,
                         tv, p);
}

size_t paged_decode_part_bytes(int d, int sms) {
    return (size_t)2 * sms * (d == 128 ? Dec<128>::kPart : Dec<64>::kPart) * sizeof(float);
}

cudaError_t launch_paged_decode(const PagedAttnParams& p, bool bf16, int d, int sms, cudaStream_t s, bool pdl) {
    CUtensorMap tk, tv;
    const int box = (1 << p.shift) < kDecTile ? 1 << p.shift : kDecTile;
    if (!paged_tmap(&tk, p, bf16, d, false, box) || !paged_tmap(&tv, p, bf16, d, true, box)) return cudaErrorInvalidValue;
    if (bf16) return d == 128 ? launch<Bf16, 128>(tk, tv, p, sms, s, pdl) : launch<Bf16, 64>(tk, tv, p, sms, s, pdl);
    return d == 128 ? launch<F16, 128>(tk, tv, p, sms, s, pdl) : launch<F16, 64>(tk, tv, p, sms, s, pdl);
}

int decode_read_status() {
    int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_decode_status, sizeof(int)) != cudaSuccess) return W4A16_ECUDA;
    if (cudaMemcpyToSymbol(g_decode_status, &zero, sizeof(int)) != cudaSuccess) return W4A16_ECUDA;
    return v;
}

}  // namespace w4a16
