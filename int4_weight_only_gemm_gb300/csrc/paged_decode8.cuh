// Paged attention over an 8-bit cache for few query rows (at most 16 a key head).
//
//     s_j = scale log2(e) ks_j (q . kcode_j),  out = sum_j 2^(s_j - m) vs_j vcode_j / sum_j 2^(s_j - m)
//
// Bound: HBM, at half the bytes of a 16-bit cache, with the instructions close
// behind: a 16-key tile of 4.2 KB takes ~540, 240 of them to unpack the codes.  The
// line of units and the joining of pieces are paged_line.cuh's.
//
// Measured, 32 query heads over 8 key heads of 128, bf16, 16-slot pages: 64 requests of
// up to 8448 positions (612 MB) 117 us with int8, 5.2 TB/s (DRAM 67 %, the ALU pipe
// 58 %, issue slots 59 %), 121 with e4m3, 113 in fp16; one request of 2304 positions
// 11.2 us a call, 10.3 in a captured graph.  With one CTA of 252 registers an
// SM it was 226 us, with copies that compute their addresses one by one 146.
//
// Eight warps work without meeting, each with a ring of its own filled by 16-byte
// asynchronous copies: codes, and 4 bytes a key and value for their scales.  The
// products have the keys (and then the columns) as the 16 rows of an MMA and 8
// query rows as its columns, so that one code in a register is used for all query
// rows at once; more than 8 query rows take a second column block.
//
//   * S^T = K Q^T.  Which columns of a head a step of 16 takes is free as long as
//     both operands agree: lane q of four takes the 16 codes that one 16-byte
//     load gives it, four at a step.
//   * O^T = V^T P^T.  The two keys of an operand register sit in two rows of the
//     tile; a byte of either row makes a pair without a transposing load, and
//     which output column a row of the MMA stands for is free again: lane l / 4
//     owns D / 8 columns that follow each other.
//
// A key's scale multiplies its score in f32, a value's its weight, which goes to
// the product in two bf16 parts (16 bits): codes are exact in bf16 and fp16, and
// neither a weight nor a scale leaves bf16's range.  A row's maximum moves only
// when a score passes it by 2^8, so that most tiles need no exchange between lanes.
#pragma once

#include <type_traits>

#include "codes.cuh"
#include "paged_line.cuh"

namespace w4a16 {

// NG: 8-row blocks of query rows, 1 or 2.  With one, a thread needs few enough
// registers for two CTAs an SM.
template <int D, int NG>
struct Dec8 {
    static constexpr int kHalf = kDecTile * D;                 // bytes of a tile's key codes (and of its value codes)
    static constexpr int kSlot = 2 * kHalf + 2 * kDecTile * 4;  // and both scales
    static constexpr int kSlots = (D == 128 ? 5 : 10) / (3 - NG);  // ring slots a warp
    static constexpr int kRing = kDecWarps * kSlots * kSlot;
    static constexpr int kStride = D + 4;                      // floats of a row of results
    static constexpr int kMergeOff = kRing;
    static constexpr int kMerge = kDecWarps * 8 * kStride * 4;
    static constexpr int kMlOff = kMergeOff + kMerge;          // [warp][16][2]
    static constexpr int kMiscOff = kMlOff + kDecWarps * 16 * 2 * 4;
    static constexpr int kLineOff = kMiscOff + 64;
    static constexpr int kSmem = kMiscOff + 128;
};
static_assert(Dec8<128, 2>::kSmem <= 232448 && Dec8<64, 2>::kSmem <= 232448, "shared memory");
static_assert(Dec8<64, 2>::kMerge >= 6 * kDecThreads * 4, "dec_join's room");
static_assert(2 * (Dec8<128, 1>::kSmem + 1024) <= 233472 && 2 * (Dec8<64, 1>::kSmem + 1024) <= 233472, "two CTAs an SM");

// Where a tile's 16-byte piece `chunk` of key `row` lies, so that neither product's loads meet in a bank: four
// lanes on a row and its neighbour (keys), eight on every other row (values).
template <int D>
W4A16_DEVICE uint32_t piece_at(int row, int chunk) {
    if constexpr (D == 128) return row * 128 + ((chunk ^ (((row >> 1) & 3) << 1) ^ ((row & 1) << 2)) << 4);
    return (row >> 1) * 128 + (((row ^ (row >> 2)) & 1) << 6) + ((chunk ^ (((row >> 1) & 1) << 1)) << 4);
}
W4A16_DEVICE uint32_t transposed(uint32_t x) {  // an 8 x 8 block of 16-bit numbers, two a lane
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
W4A16_DEVICE void copy_16(uint32_t smem_dst, const void* gsrc) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_dst), "l"(gsrc) : "memory");
}
W4A16_DEVICE void copy_4(uint32_t smem_dst, const void* gsrc) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_dst), "l"(gsrc) : "memory");
}

template <typename Ty, int D, int NG, bool E4M3, bool TREE>
__global__ void __launch_bounds__(kDecThreads, 3 - NG) paged_decode8_kernel(const __grid_constant__ PagedAttnParams p) {
    using L = Dec8<D, NG>;
    constexpr bool BF = Ty::idesc_type == 1;
    const uint32_t vbase = code_base<true>(), kbase = BF ? vbase : code_base<BF>();
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
    // (the line's numbers wait in shared memory: a piece needs them at its ends alone)
    volatile int64_t* line = reinterpret_cast<volatile int64_t*>(smem + L::kLineOff);
    if (threadIdx.x == 0) line[0] = cut.U, line[1] = cut.u0, line[2] = cut.u1, line[3] = cut.C;
    __syncthreads();
    int b = cut.b, hk = cut.hk;
    int64_t s0 = cut.s0;  // the pair's first place
    Request r = cut.r;
    DecSpan sp = cut.sp;

    // ---- the warp's ring -------------------------------------------------
    const uint32_t ring = smem_u32(smem) + warp * (L::kSlots * L::kSlot);
    uint32_t gone = 0;             // 2 bits a slot: pages of the tile that are not there
    const int page = 1 << p.shift, box = page < kDecTile ? page : kDecTile;
    const int boxes = kDecTile / box;  // 1, or 2 for 8-slot pages
    constexpr int kRow = D / 16;       // lanes a row
    const int crow = lane / kRow, cch = lane % kRow;  // this lane's row and 16-byte piece of a copy step
    int j0, e_last, tile0, tiles;      // of the piece: first key, last key seen, this warp's first tile and their number
    int off, take;                     // units of the pair before the piece, and in it
    int ent[2], ent_base;              // table entries of the tiles ent_base + lane
    const uint8_t *kmine, *vmine;      // this lane's part of a copy: 16 bytes of rows crow, crow + kStep, ..
    const float* smine;                // and a scale of key lane % 16: of the key, in the upper lanes of its value
    auto open_piece = [&] {
        const int64_t u0 = line[1], u1 = line[2];
        kmine = reinterpret_cast<const uint8_t*>(p.k) + hk * p.kh + crow * p.ks + cch * 16;
        vmine = reinterpret_cast<const uint8_t*>(p.v) + hk * p.vh + crow * p.vs + cch * 16;
        const int key = lane & (box - 1);
        smine = lane < 16 ? p.k_scale + hk * p.ksh + key * p.kss : p.v_scale + hk * p.vsh + key * p.vss;
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
    constexpr int kStep = 32 / kRow;   // rows of a copy step
    const uint32_t mine = piece_at<D>(crow, cch);
    const bool dense = p.ks == D && p.vs == D;
    const int64_t spage = lane < 16 ? p.ksp : p.vsp, sslot = lane < 16 ? p.kss : p.vss;
    auto issue = [&](int t, int slot) {  // the copies of the piece's tile t; a group of copies in any case
        if (t < tiles) {
            if (t >= ent_base + 32) entries(t);
            const int slot0 = (j0 + (tile0 + t * kDecWarps) * kDecTile) & (page - 1);
            const uint32_t dst = ring + slot * L::kSlot;
            uint32_t no = 0;
            // rows 8 h .., all of one page; with the slots of a head behind each other (`dense`) the steps' distance is
            // a constant.  Of a page that is not there nothing is copied: any codes stand for numbers, and their
            // weights are zero whatever scales the slot holds.
            auto rows = [&](int h, int steps, auto dense) {
                const int pg = __shfl_sync(0xffffffffu, ent[h], t - ent_base);
                if (pg < 0 || pg >= p.pages) {
                    no |= 1u << h;
                    return;
                }
                const uint8_t* kp = kmine + (pg * p.kp + slot0 * p.ks);
                const uint8_t* vp = vmine + (pg * p.vp + slot0 * p.vs);
                const int64_t kstep = decltype(dense)::value ? kStep * D : kStep * p.ks;
                const int64_t vstep = decltype(dense)::value ? kStep * D : kStep * p.vs;
#pragma unroll
                for (int x = 0; x < 16 / kStep; ++x) {
                    if (x == steps) break;
                    // (piece_at of row x kStep on: 512 bytes behind it, and for D = 128 in the other half of its 128)
                    const uint32_t a = dst + 8 * D * h + x * kStep * D + (D == 128 && (x & 1) ? mine ^ 64u : mine);
                    copy_16(a, kp + x * kstep);
                    copy_16(a + L::kHalf, vp + x * vstep);
                }
                if (steps == 16 / kStep || ((lane >> 3) & 1) == h)
                    copy_4(dst + 2 * L::kHalf + lane * 4, smine + (pg * spage + slot0 * sslot));
            };
            if (boxes == 1) {
                if (dense) rows(0, 16 / kStep, std::true_type{});
                else rows(0, 16 / kStep, std::false_type{});
            } else {  // pages of 8 slots: from slot 0 each
                rows(0, 8 / kStep, std::false_type{});
                rows(1, 8 / kStep, std::false_type{});
            }
            gone = (gone & ~(3u << (2 * slot))) | no << (2 * slot);
        }
        cp_async_commit();
    };
    // the query rows 8 g + lane / 4 as B fragments: lane q of four has the columns 16 (q + 4 c) .. + 15
    const int q = lane & 3, n = lane >> 2;
    uint2 qf[NG][D / 16];  // of four columns, the first and the third, then the others: as codes come in pairs
    auto load_q = [&] {
        const int R = r.n * p.G;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const int row = 8 * g + n, i = row / p.G;
            const uint16_t* at = p.q + (int64_t)(r.t0 + i) * p.q_token + (int64_t)(hk * p.G + row - i * p.G) * p.q_head + 16 * q;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                uint2 x = make_uint2(0u, 0u);
                if (row < R) x = *reinterpret_cast<const uint2*>(at + 64 * (k >> 2) + 4 * (k & 3));
                qf[g][k] = make_uint2(__byte_perm(x.x, x.y, 0x5410), __byte_perm(x.x, x.y, 0x7632));
            }
        }
    };

    open_piece();
    entries(0);
    load_q();
    for (int i = 0; i < L::kSlots; ++i) issue(i, i);

    while (true) {
        const int R = r.n * p.G;
        const bool more_rows = NG == 2 && R > 8;
        const Seen see = seen_by<TREE>(p, r, 0, r.n - 1);
        const int e_min = see.e_all, lo_max = see.lo_all;

        float o[NG][D / 16][4];  // [rows 8 g ..][columns 2 t, 2 t + 1 of the lane's][row 2 q, 2 q + 1 of either column]
        float m[NG][2], l[NG][2];  // of rows 8 g + 2 q, + 1
#pragma unroll
        for (int g = 0; g < NG; ++g) {
#pragma unroll
            for (int t = 0; t < D / 16; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[g][t][i] = 0.f;
            m[g][0] = m[g][1] = -INFINITY;
            l[g][0] = l[g][1] = 0.f;
        }

        int slot = 0;
        for (int t = 0; t < tiles; ++t) {
            cp_async_wait<L::kSlots - 1>();
            __syncwarp();
            const uint32_t kb = ring + slot * L::kSlot, vb = kb + L::kHalf, sb = vb + L::kHalf;
            const uint32_t no = (gone >> (2 * slot)) & 3u;
            const int j = j0 + (tile0 + t * kDecWarps) * kDecTile;
            // scores: keys n and n + 8 by rows 2 q, 2 q + 1
            float s[NG][4] = {};
#pragma unroll
            for (int x = 0; x < D / 64; ++x) {
                const uint4 ka = lds_v4(kb + piece_at<D>(n, q + 4 * x)), kc = lds_v4(kb + piece_at<D>(n + 8, q + 4 * x));
                const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wc[4] = {kc.x, kc.y, kc.z, kc.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t a[4] = {code_pair<E4M3, BF, false>(wa[k], kbase), code_pair<E4M3, BF, false>(wc[k], kbase),
                                           code_pair<E4M3, BF, true>(wa[k], kbase), code_pair<E4M3, BF, true>(wc[k], kbase)};
                    mma_16816<Ty>(s[0], a, qf[0][4 * x + k].x, qf[0][4 * x + k].y);
                    if (more_rows) mma_16816<Ty>(s[NG - 1], a, qf[NG - 1][4 * x + k].x, qf[NG - 1][4 * x + k].y);
                }
            }
            const float ks0 = finite_or_nan(__uint_as_float(lds_u32(sb + 4 * n))) * p.scale2;
            const float ks1 = finite_or_nan(__uint_as_float(lds_u32(sb + 4 * n + 32))) * p.scale2;
            const float vs0 = finite_or_nan(__uint_as_float(lds_u32(sb + 4 * n + 64)));
            const float vs1 = finite_or_nan(__uint_as_float(lds_u32(sb + 4 * n + 96)));
            const bool edge = j < lo_max || j + kDecTile - 1 > e_min || no;
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    s[g][y] *= ks0;
                    s[g][2 + y] *= ks1;
                }
            uint32_t hidden = 0;  // bit 4 g + i: s[g][i] is of a position that the row does not see
            if (edge) {
#pragma unroll
                for (int g = 0; g < NG; ++g)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int row = 8 * g + 2 * q + y, tok = row / p.G;
                        int e = -1, lo = 0;
                        uint32_t bits = 0u;
                        if (row < R) {
                            if constexpr (TREE) {
                                e = e_min;
                                lo = tree_first(p, r, r.t0 + tok);
                                bits = tree_word(p, r.t0 + tok, r.n, 0);
                            } else {
                                e = last_seen(p, r, tok);
                                lo = first_seen(p, e);
                            }
                        }
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const int key = n + 8 * x, jj = j + key;
                            bool sees = jj >= lo && jj <= e;
                            if constexpr (TREE) {
                                const uint32_t node = (uint32_t)(jj - e - 1);
                                if (jj > e) sees = node < 32u && ((bits >> (node & 31u)) & 1u);
                            }
                            if (!sees || ((no >> (boxes == 2 ? x : 0)) & 1u)) {
                                hidden |= 1u << (4 * g + 2 * x + y);
                                s[g][2 * x + y] = -INFINITY;
                            }
                        }
                    }
            }
            bool grew = false;
#pragma unroll
            for (int g = 0; g < NG; ++g)
#pragma unroll
                for (int y = 0; y < 2; ++y) grew |= fmaxf(s[g][y], s[g][2 + y]) > m[g][y] + 8.f;
            if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                for (int g = 0; g < NG; ++g) {
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        float x = fmaxf(s[g][y], s[g][2 + y]);
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
                        x = fmaxf(x, m[g][y]);
                        const float f = x == -INFINITY ? 1.f : exp2_approx(m[g][y] - x);
                        m[g][y] = x;
                        l[g][y] *= f;
#pragma unroll
                        for (int t2 = 0; t2 < D / 16; ++t2) {
                            o[g][t2][y] *= f;
                            o[g][t2][2 + y] *= f;
                        }
                    }
                }
            }
            // weights in two bf16 parts, turned into the second product's operand
            uint32_t ph[NG][2], pl[NG][2];
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                float w[4];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const float base = m[g][y] == -INFINITY ? 0.f : m[g][y];
                    const float a = exp2_approx(s[g][y] - base), d = exp2_approx(s[g][2 + y] - base);
                    l[g][y] += a + d;
                    w[y] = a * vs0;
                    w[2 + y] = d * vs1;
                }
                if (edge)  // (the scale of a position that is not seen may be anything)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if ((hidden >> (4 * g + i)) & 1u) w[i] = 0.f;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const uint32_t hi = Bf16::pack(w[2 * x], w[2 * x + 1]);
                    ph[g][x] = transposed(hi);
                    pl[g][x] = transposed(Bf16::pack(w[2 * x] - Bf16::lo(hi), w[2 * x + 1] - Bf16::hi(hi)));
                }
            }
            // values: keys 2 q, 2 q + 1, 2 q + 8, 2 q + 9, the lane's D / 8 columns of each
            uint32_t v[4][D / 32];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = 2 * q + (i & 1) + 8 * (i >> 1);
                if constexpr (D == 128) {
                    const uint4 x = lds_v4(vb + piece_at<D>(row, n));
                    v[i][0] = x.x, v[i][1] = x.y, v[i][2] = x.z, v[i][3] = x.w;
                } else {
                    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                                 : "=r"(v[i][0]), "=r"(v[i][1])
                                 : "r"(vb + piece_at<D>(row, n >> 1) + (n & 1) * 8));
                }
            }
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {  // four columns: two tiles of two
                uint32_t a[2][4];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const uint32_t lo = __byte_perm(v[0][i], v[1][i], x ? 0x7632 : 0x5410);
                    const uint32_t hi = __byte_perm(v[2][i], v[3][i], x ? 0x7632 : 0x5410);
                    a[x][0] = code_pair<E4M3, true, false>(lo, vbase);
                    a[x][1] = code_pair<E4M3, true, true>(lo, vbase);
                    a[x][2] = code_pair<E4M3, true, false>(hi, vbase);
                    a[x][3] = code_pair<E4M3, true, true>(hi, vbase);
                }
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    if (g && !more_rows) break;
                    mma_16816<Bf16>(o[g][2 * i], a[0], ph[g][0], ph[g][1]);
                    mma_16816<Bf16>(o[g][2 * i + 1], a[1], ph[g][0], ph[g][1]);
                    mma_16816<Bf16>(o[g][2 * i], a[0], pl[g][0], pl[g][1]);
                    mma_16816<Bf16>(o[g][2 * i + 1], a[1], pl[g][0], pl[g][1]);
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
        const bool more = line[2] > end + kDecPair;
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
        for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[g][y] += __shfl_xor_sync(0xffffffffu, l[g][y], d);
                if (n == 0) {
                    ml[(warp * 16 + 8 * g + 2 * q + y) * 2] = m[g][y];
                    ml[(warp * 16 + 8 * g + 2 * q + y) * 2 + 1] = l[g][y];
                }
            }
        __syncthreads();
        // Every warp leaves its rows 0 .. 7 and eight are added; with more rows, warps 4 .. 7 leave all 16 of theirs
        // and warps 0 .. 3 add to them first.  A row's place: even rows first, so that the lanes' stores do not meet.
        auto place = [&](int w, int g, int y) {
            return merge + ((more_rows ? 2 * w + g : w) * 8 + 4 * y + q) * L::kStride + n * (D / 8);
        };
        auto leave = [&](int g, int w, bool add) {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int row = 8 * g + 2 * q + y;
                float M = -INFINITY;
#pragma unroll
                for (int i = 0; i < kDecWarps; ++i) M = fmaxf(M, ml[(i * 16 + row) * 2]);
                const float f = exp2_approx(m[g][y] - (M == -INFINITY ? 0.f : M));
                float4* at = reinterpret_cast<float4*>(place(w, g, y));
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    float4 x = make_float4(o[g][2 * i][y], o[g][2 * i][2 + y], o[g][2 * i + 1][y], o[g][2 * i + 1][2 + y]);
                    const float4 z = add ? at[i] : make_float4(0.f, 0.f, 0.f, 0.f);
                    x = make_float4(fmaf(x.x, f, z.x), fmaf(x.y, f, z.y), fmaf(x.z, f, z.z), fmaf(x.w, f, z.w));
                    at[i] = x;
                }
            }
        };
        if (!more_rows) {
            leave(0, warp, false);
        } else {
            if (warp >= 4) leave(0, warp - 4, false), leave(NG - 1, warp - 4, false);
            __syncthreads();
            if (warp < 4) leave(0, warp, true), leave(NG - 1, warp, true);
        }
        __syncthreads();
        // thread: four columns of a row
        const bool whole = from_start && to_end;
        float* part = p.part + (int64_t)(2 * c + (from_start ? 1 : 0)) * kDecPart<D, 8 * NG>;
        for (int e = threadIdx.x; e < R * (D / 4); e += kDecThreads) {
            const int row = e / (D / 4), col = (e - row * (D / 4)) * 4;
            float M = -INFINITY, S = 0.f;
#pragma unroll
            for (int i = 0; i < kDecWarps; ++i) M = fmaxf(M, ml[(i * 16 + row) * 2]);
            const float base = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int i = 0; i < kDecWarps; ++i) {
                const float mi = ml[(i * 16 + row) * 2], si = ml[(i * 16 + row) * 2 + 1];
                if (si != 0.f) S = fmaf(si, exp2_approx(mi == -INFINITY ? 0.f : mi - base), S);
            }
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            const int blocks = more_rows ? kDecWarps / 2 : kDecWarps;
            for (int i = 0; i < blocks; ++i) {
                const float4 y = *reinterpret_cast<const float4*>(
                    merge + ((more_rows ? 2 * i + (row >> 3) : i) * 8 + 4 * (row & 1) + ((row & 7) >> 1)) * L::kStride + col);
                x.x += y.x;
                x.y += y.y;
                x.z += y.z;
                x.w += y.w;
            }
            const int ti = row / p.G, th = done_hk * p.G + row - ti * p.G;  // the row's token and head
            if (whole) {
                const float inv = 1.f / S;
                *reinterpret_cast<uint2*>(p.out + (int64_t)(done.t0 + ti) * p.o_token + (int64_t)th * p.o_head + col) =
                    S == 0.f ? make_uint2(0u, 0u) : make_uint2(Ty::pack(x.x * inv, x.y * inv), Ty::pack(x.z * inv, x.w * inv));
                if (p.lse && col == 0)
                    p.lse[(int64_t)(done.t0 + ti) * p.Hq + th] = S == 0.f ? -INFINITY : kLn2 * (M + log2f(S));
            } else {
                *reinterpret_cast<float4*>(part + 16 * NG + row * D + col) = x;
                if (col == 0) *reinterpret_cast<float2*>(part + 2 * row) = make_float2(M, S);
            }
        }
        if (!whole) dec_join<Ty, D, 8 * NG>(p, done, done_hk, owner_of(first, line[0], (int)line[3]),
                                             owner_of(end - 1, line[0], (int)line[3]), misc, merge);
        if (!more) break;
        __syncthreads();  // ml and merge are free again
    }
    cp_async_wait<0>();
}

template <typename Ty, int D, int NG, bool E4M3, bool TREE>
static cudaError_t launch(const PagedAttnParams& p, int sms, cudaStream_t s, bool pdl) {
    static bool set_for[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    auto kernel = paged_decode8_kernel<Ty, D, NG, E4M3, TREE>;
    if (!set_for[dev]) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Dec8<D, NG>::kSmem);
        if (e != cudaSuccess) return e;
        set_for[dev] = true;
    }
    return launch_kernel(kernel, dim3((3 - NG) * sms), dim3(kDecThreads), (size_t)Dec8<D, NG>::kSmem, s, pdl, p);
}

template <bool TREE>
cudaError_t launch_paged_decode8(const PagedAttnParams& p, bool bf16, int d, bool few, int sms, cudaStream_t s, bool pdl) {
    auto of = [&](auto ty, auto e4m3) {
        using Ty = decltype(ty);
        constexpr bool E = decltype(e4m3)::value;
        if (few) return d == 128 ? launch<Ty, 128, 1, E, TREE>(p, sms, s, pdl) : launch<Ty, 64, 1, E, TREE>(p, sms, s, pdl);
        return d == 128 ? launch<Ty, 128, 2, E, TREE>(p, sms, s, pdl) : launch<Ty, 64, 2, E, TREE>(p, sms, s, pdl);
    };
    if (bf16) return p.e4m3 ? of(Bf16{}, std::true_type{}) : of(Bf16{}, std::false_type{});
    return p.e4m3 ? of(F16{}, std::true_type{}) : of(F16{}, std::false_type{});
}

}  // namespace w4a16
