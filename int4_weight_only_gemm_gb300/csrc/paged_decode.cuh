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
// w, w + 8, ... of the range through a ring of its own and keeps the rows'
// maxima, sums and 16 x head_dim outputs in registers.  The products are
// warp-wide 16 x 8 x 16 MMAs: with 16 rows the tensor pipe is not what bounds
// this kernel, and fragments that stay in registers need no tensor-memory round
// trip between the two products.  The warps' results meet once per pair, in
// shared memory, while the next pair's first tiles are on their way.
//
// The ring is filled by 16-byte asynchronous copies, not by tensor copies: one
// of 16 rows x 128 bytes (all that a 16-slot page gives at once) occupies the
// copy unit of an SM for ~100 clocks, 20 bytes a clock, below what HBM delivers
// to an SM; with them 64 requests took 248 us.
//
// Measured, 32 query heads over 8 key heads of 128, bf16, 16-slot pages: 64
// requests of up to 8448 positions (1.18 GB) 182-185 us, 6.5 TB/s; one request of
// 2304 positions 9.6 us, of which ~3.0 k clocks go to the cut of the line, 2.5 k
// to the first table entries and copies, 1.9 k to the keys and values
// themselves, 2.0 k to the warps' results and 2.4 k to the joining of the 18
// pieces.
//
// Positions that a row does not see are masked in the scores; the values of
// positions that no row of the tile sees (stale slots of the last page, slots
// before the window) are cleared in shared memory first, and non-finite values
// that only some rows see are added for those rows alone, so that no row takes
// a NaN from a position outside its own.
#pragma once

#include "paged_line.cuh"

namespace w4a16 {

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
    static constexpr int kMiscOff = kMlOff + kDecWarps * 16 * 2 * 4;
    static constexpr int kSmem = kMiscOff + 128;
};
static_assert(Dec<128>::kSmem <= 232448 && Dec<64>::kSmem <= 232448, "shared memory");

template <typename Ty, int D, bool TREE>
__global__ void __launch_bounds__(kDecThreads, 1) paged_decode_kernel(const __grid_constant__ PagedAttnParams p) {
    using L = Dec<D>;
    extern __shared__ __align__(128) unsigned char smem[];
    float* merge = reinterpret_cast<float*>(smem + L::kMergeOff);
    float* ml = reinterpret_cast<float*>(smem + L::kMlOff);
    volatile int* misc = reinterpret_cast<volatile int*>(smem + L::kMiscOff);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = (int)blockIdx.x;
    pdl_wait();
    pdl_launch_dependents();  // in this order: the chunk kernel of the same call does not wait for this one to begin

    DecCut cut;
    if (!dec_cut<TREE>(p, reinterpret_cast<int64_t*>(ml), misc, cut)) return;
    const int64_t U = cut.U, u0 = cut.u0, u1 = cut.u1;
    const int C = cut.C;
    int b = cut.b, hk = cut.hk;
    int64_t s0 = cut.s0;  // the pair's first place
    Request r = cut.r;
    DecSpan sp = cut.sp;

    // ---- the warp's ring -------------------------------------------------
    const uint32_t ring = smem_u32(smem) + warp * (L::kSlots * 2 * L::kHalf);
    uint32_t gone = 0;             // 2 bits a slot: pages of the tile that are not there
    const int page = 1 << p.shift, box = page < kDecTile ? page : kDecTile;
    const int boxes = kDecTile / box;  // 1, or 2 for 8-slot pages
    constexpr int kRow = D / 8;        // lanes a row
    const int crow = lane / kRow, cch = lane % kRow;  // this lane's row and 16-byte piece of a copy step
    int j0, e_last, tile0, tiles;      // of the piece: first key, last key seen, this warp's first tile and their number
    int off, take;                     // units of the pair before the piece, and in it
    int ent[2], ent_base;              // table entries of the tiles ent_base + lane
    auto open_piece = [&] {
        off = (int)(u0 > s0 + kDecPair ? u0 - s0 - kDecPair : 0);
        take = (int)(u1 - s0 - kDecPair < sp.units ? u1 - s0 - kDecPair : sp.units) - off;
        j0 = sp.j0;
        e_last = seen_by<TREE>(p, r, 0, r.n - 1).last;
        tile0 = off * kDecWarps + warp;
        const int all = e_last < j0 ? 0 : (e_last - j0) / kDecTile + 1;  // tiles that hold a seen key
        const int end = min((off + take) * kDecWarps, all);
        tiles = tile0 < end ? (end - tile0 + kDecWarps - 1) / kDecWarps : 0;
    };
    auto entries = [&](int t) {  // lane i: the pages of tile t + i
        ent_base = t;
        ent[0] = ent[1] = -1;
        if (t + lane < tiles) {
            const int j = j0 + (tile0 + (t + lane) * kDecWarps) * kDecTile;
            const int* row = p.table + (int64_t)b * p.table_stride;
            for (int i = 0; i < boxes; ++i) {
                const int col = (j + i * box) >> p.shift;
                if (col < p.columns) ent[i] = row[col];
            }
        }
    };
    auto issue = [&](int t, int slot) {  // the copies of the piece's tile t; a group of copies in any case
        if (t < tiles) {
            if (t >= ent_base + 32) entries(t);
            uint32_t no = 0;
            const int j = j0 + (tile0 + t * kDecWarps) * kDecTile;
            const uint32_t dst = ring + slot * 2 * L::kHalf + (cch >> 3) * (kDecTile * 128);
#pragma unroll
            for (int h = 0; h < 2; ++h) {  // rows 0 .. 7 and 8 .. 15
                const int i = boxes == 2 ? h : 0;
                int pg = __shfl_sync(0xffffffffu, ent[i], t - ent_base);
                const bool there = pg >= 0 && pg < p.pages;
                if (!there) {
                    no |= 1u << i;
                    pg = 0;
                }
                const int slot0 = (j + 8 * h) & (page - 1);
                const uint16_t* kp = p.k + pg * p.kp + hk * p.kh + (int64_t)(slot0 + crow) * p.ks + cch * 8;
                const uint16_t* vp = p.v + pg * p.vp + hk * p.vh + (int64_t)(slot0 + crow) * p.vs + cch * 8;
#pragma unroll
                for (int x = 0; x < 8 * kRow / 32; ++x) {
                    const int row = 8 * h + x * (32 / kRow) + crow;
                    const uint32_t a = dst + row * 128 + (((cch & 7) ^ (row & 7)) << 4);
                    cp_async_16_or_zero(a, kp + (int64_t)(x * (32 / kRow)) * p.ks, there);
                    cp_async_16_or_zero(a + L::kHalf, vp + (int64_t)(x * (32 / kRow)) * p.vs, there);
                }
            }
            gone = (gone & ~(3u << (2 * slot))) | no << (2 * slot);
        }
        cp_async_commit();
    };
    // the query rows as A fragments: rows r = lane / 4 and r + 8 of i G + g
    const int ra = lane >> 2, rb = ra + 8, ia = ra / p.G, ib = rb / p.G;
    uint32_t qa[D / 16][4];
    auto load_q = [&] {
        const int R = r.n * p.G;
        const uint32_t* qpa = reinterpret_cast<const uint32_t*>(
            p.q + (int64_t)(r.t0 + ia) * p.q_token + (int64_t)(hk * p.G + ra - ia * p.G) * p.q_head) + (lane & 3);
        const uint32_t* qpb = reinterpret_cast<const uint32_t*>(
            p.q + (int64_t)(r.t0 + ib) * p.q_token + (int64_t)(hk * p.G + rb - ib * p.G) * p.q_head) + (lane & 3);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            qa[k][0] = ra < R ? qpa[8 * k] : 0u;
            qa[k][1] = rb < R ? qpb[8 * k] : 0u;
            qa[k][2] = ra < R ? qpa[8 * k + 4] : 0u;
            qa[k][3] = rb < R ? qpb[8 * k + 4] : 0u;
        }
    };

    open_piece();
    entries(0);
    load_q();
    for (int i = 0; i < L::kSlots; ++i) issue(i, i);

    while (true) {
        const int R = r.n * p.G;
        const Seen see = seen_by<TREE>(p, r, 0, r.n - 1);
        const int e_min = see.e_all, lo_min = see.first, lo_max = see.lo_all;
        int ea = -1, eb = -1, la = 0, lb = 0;  // a row sees la .. ea, and the nodes behind ea that its bits say
        uint32_t ta = 0u, tb = 0u;
        if constexpr (TREE) {
            if (ra < R) ea = e_min, la = tree_first(p, r, r.t0 + ia), ta = tree_word(p, r.t0 + ia, r.n, 0);
            if (rb < R) eb = e_min, lb = tree_first(p, r, r.t0 + ib), tb = tree_word(p, r.t0 + ib, r.n, 0);
        } else {
            if (ra < R) ea = last_seen(p, r, ia);
            if (rb < R) eb = last_seen(p, r, ib);
            la = first_seen(p, ea);
            lb = first_seen(p, eb);
        }
        auto sees = [](int jj, int lo, int e, uint32_t bits) {
            if constexpr (TREE)
                if (jj > e) return (uint32_t)(jj - e - 1) < 32u && ((bits >> (jj - e - 1)) & 1u);
            return jj >= lo && jj <= e;
        };

        float o[D / 8][4];
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[n][i] = 0.f;
        float ma = -INFINITY, mb = -INFINITY, sa = 0.f, sb = 0.f;

        int slot = 0;
        for (int t = 0; t < tiles; ++t) {
            cp_async_wait<L::kSlots - 1>();
            __syncwarp();
            const uint32_t kb = ring + slot * 2 * L::kHalf, vb = kb + L::kHalf;
            const uint32_t no = (gone >> (2 * slot)) & 3u;
            const int j = j0 + (tile0 + t * kDecWarps) * kDecTile;
            {
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
                        if (!(there && sees(jj, la, ea, ta))) x[i] = -INFINITY;
                        if (!(there && sees(jj, lb, eb, tb))) x[4 + i] = -INFINITY;
                    }
                    // values: a lane looks at half a key's row
                    const int key = lane >> 1, jj = j + key;
                    const bool none = jj < lo_min || jj > e_last;  // seen by no row
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
                                    odd |= ((Ty::all_ones(v.x) | Ty::all_ones(v.y) | Ty::all_ones(v.z) |
                                             Ty::all_ones(v.w)) & 0x80008000u) != 0;
                                }
                            }
                    }
                    const uint32_t lanes = __ballot_sync(0xffffffffu, odd);
                    for (int i = 0; i < kDecTile; ++i)
                        if ((lanes >> (2 * i)) & 3u) alone |= 1u << i;
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
                        const bool va = sees(j + key, la, ea, ta), vv = sees(j + key, lb, eb, tb);
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
            __syncwarp();  // every lane has read the tile
            issue(t + L::kSlots, slot);
            slot = slot + 1 == L::kSlots ? 0 : slot + 1;
        }

        // ---- the next pair's first copies and rows, before this one's results meet ----
        const Request done = r;
        const int done_hk = hk;
        const int64_t first = s0 + kDecPair, end = first + sp.units;  // the pair's units on the line
        const bool from_start = off == 0, to_end = off + take == sp.units;
        const bool more = u1 > end + kDecPair;
        if (more) {
            s0 = end;
            if (++hk == p.Hkv) {
                hk = 0;
                do {
                    r = request_of(p, ++b);
                    sp = dec_span<TREE>(p, r);
                } while (sp.units == 0);
            }
            open_piece();
            entries(0);
            load_q();
            for (int i = 0; i < L::kSlots; ++i) issue(i, i);
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
        // With at most 8 rows every warp leaves its own and 8 are added below; the
        // room is for four warps' 16 rows.
        const bool few = R <= 8;
        if (few) {
            float2* at = reinterpret_cast<float2*>(merge) + warp * (L::kRegs / 4 * 32) + lane;
#pragma unroll
            for (int n = 0; n < D / 8; ++n) at[n * 32] = make_float2(o[n][0] * fa, o[n][1] * fa);
        } else {
            float2* at = reinterpret_cast<float2*>(merge) + (warp & 3) * (L::kRegs / 2 * 32) + lane;
            if (warp >= 4) {
#pragma unroll
                for (int n = 0; n < D / 8; ++n) {
                    at[2 * n * 32] = make_float2(o[n][0] * fa, o[n][1] * fa);
                    at[(2 * n + 1) * 32] = make_float2(o[n][2] * fb, o[n][3] * fb);
                }
            }
            __syncthreads();
            if (warp < 4) {
#pragma unroll
                for (int n = 0; n < D / 8; ++n) {
                    float2* x = at + 2 * n * 32;
                    x[0] = make_float2(fmaf(o[n][0], fa, x[0].x), fmaf(o[n][1], fa, x[0].y));
                    x[32] = make_float2(fmaf(o[n][2], fb, x[32].x), fmaf(o[n][3], fb, x[32].y));
                }
            }
        }
        __syncthreads();
        // thread: pairs of neighbouring columns of one row
        const bool whole = from_start && to_end;
        const int row = few ? lane / 4 : lane / 4 + 8 * (warp & 1);
        float M = -INFINITY, S = 0.f;
#pragma unroll
        for (int i = 0; i < kDecWarps; ++i) M = fmaxf(M, ml[(i * 16 + row) * 2]);
        const float base = M == -INFINITY ? 0.f : M;
#pragma unroll
        for (int i = 0; i < kDecWarps; ++i) {
            const float m = ml[(i * 16 + row) * 2], s = ml[(i * 16 + row) * 2 + 1];
            if (s != 0.f) S = fmaf(s, exp2_approx(m == -INFINITY ? 0.f : m - base), S);
        }
        const int ti = row / p.G, th = done_hk * p.G + row - ti * p.G;  // the row's token and head
        uint16_t* out = p.out + (int64_t)(done.t0 + ti) * p.o_token + (int64_t)th * p.o_head;
        float* lse = p.lse ? p.lse + (int64_t)(done.t0 + ti) * p.Hq + th : nullptr;
        float* part = p.part + (int64_t)(2 * c + (from_start ? 1 : 0)) * kDecPart<D>;
        if (row < R) {
            const float inv = 1.f / S;
            // column tiles n of 8: few -- warp, warp + 8; else warp / 2, warp / 2 + 4, ..
            const int step = few ? kDecWarps : kDecWarps / 2;
            const float2* at = reinterpret_cast<const float2*>(merge) + lane + (few ? 0 : (warp & 1) * 32);
            for (int n = few ? warp : warp >> 1; n < D / 8; n += step) {
                const int col = 8 * n + 2 * (lane & 3);
                float y0 = 0.f, y1 = 0.f;
                if (few) {
#pragma unroll
                    for (int i = 0; i < kDecWarps; ++i) {
                        const float2 x = at[(i * (L::kRegs / 4) + n) * 32];
                        y0 += x.x;
                        y1 += x.y;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 x = at[(i * (L::kRegs / 2) + 2 * n) * 32];
                        y0 += x.x;
                        y1 += x.y;
                    }
                }
                if (whole)
                    *reinterpret_cast<uint32_t*>(out + col) = S == 0.f ? 0u : Ty::pack(y0 * inv, y1 * inv);
                else
                    *reinterpret_cast<float2*>(part + 32 + row * D + col) = make_float2(y0, y1);
            }
            if ((few ? warp : warp >> 1) == 0 && (lane & 3) == 0) {
                if (!whole)
                    *reinterpret_cast<float2*>(part + 2 * row) = make_float2(M, S);
                else if (lse)
                    *lse = S == 0.f ? -INFINITY : kLn2 * (M + log2f(S));
            }
        }
        if (!whole) dec_join<Ty, D>(p, done, done_hk, owner_of(first, U, C), owner_of(end - 1, U, C), misc);
        if (!more) break;
        __syncthreads();  // ml and merge are free again
    }
    cp_async_wait<0>();
}

template <typename Ty, int D, bool TREE>
static cudaError_t launch(const PagedAttnParams& p, int ctas, cudaStream_t s, bool pdl) {
    static bool set_for[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!set_for[dev]) {
        e = cudaFuncSetAttribute(paged_decode_kernel<Ty, D, TREE>, cudaFuncAttributeMaxDynamicSharedMemorySize, Dec<D>::kSmem);
        if (e != cudaSuccess) return e;
        set_for[dev] = true;
    }
    return launch_kernel(paged_decode_kernel<Ty, D, TREE>, dim3(ctas), dim3(kDecThreads), (size_t)Dec<D>::kSmem, s, pdl, p);
}

template <bool TREE>
cudaError_t launch_paged_decode(const PagedAttnParams& p, bool bf16, int d, int sms, cudaStream_t s, bool pdl) {
    if (bf16) return d == 128 ? launch<Bf16, 128, TREE>(p, sms, s, pdl) : launch<Bf16, 64, TREE>(p, sms, s, pdl);
    return d == 128 ? launch<F16, 128, TREE>(p, sms, s, pdl) : launch<F16, 64, TREE>(p, sms, s, pdl);
}

}  // namespace w4a16
