// Paged attention for many query rows: prompt chunks, draft blocks, and every
// request whose new tokens make more than 16 rows a key head.  tcgen05 + TMA.
//
//     row r = i G + g of 128: token i of the tile, head hk G + g
//     S = Q K^T,  P = 2^(scale log2(e) S - m),  O = sum over key tiles of P V,  out = O / sum P
//
// An item is up to two 128-row tiles of one (request, key head): the two tiles
// share every key and value tile of 128 positions, and while one tile's softmax
// runs, the tensor cores work on the other's products.  With at most 128 rows
// left (a draft block, the end of a chunk) the two softmax warpgroups take
// turns on the key tiles of the same rows instead, and join their sums.
//
//   * warp 9 copies the pages of the key / value tiles into a ring in shared
//     memory (one 128-byte-swizzled box a page and 64 columns), warp 10 the Q
//     tiles, so that an item's first keys are on their way before the last
//     item's queries are done with;
//   * warp 8 issues the MMAs: S = Q K^T from shared memory (128 x 128 x D, f32
//     in tensor memory), O += P V with P from tensor memory (over S) and V in
//     the layout it has in the cache (its columns are contiguous: MN-major);
//   * warpgroups 0 and 1, a thread a row: mask, row maximum, exponentials, sum,
//     P back to tensor memory.  O is rescaled only when a row's maximum grew by
//     more than 2^8 since the last time: weights up to 2^8 lose nothing in f32
//     sums or in 16-bit floating weights.
//
// The key tiles of all items form one line, cut evenly over the CTAs (one an
// SM); an item whose tiles fall to several CTAs is joined by the last of them
// to arrive, in CTA order.
//
// Precision: weights are rounded to the 16-bit type for the product with V.
// Over hundreds of positions these roundings average out; rows that see fewer
// than 256 positions carry them in two parts (hi + lo, two products).
//
// Positions that no row of an item sees are cleared in the value tile.  Values
// that only some rows see (an item's last tokens' positions, and the window's
// first) and that are not finite are taken out of it and added to the output of
// the rows that see them at the end of the item, so that a NaN stays with
// those.  That costs a pass over these positions, at most 256 at either end
// whatever the context's length, and only in items that have such values.
//
// Bound: the chain softmax -> P -> MMAs -> scores of the two warpgroups, ~3700
// clocks for a key tile of 256 rows, of which the tensor pipe works 2048.
// Measured: a 2048-token chunk of a request of 8448 positions, 32 query heads over
// 8 key heads of 128, bf16 (249 GFLOP): 199.5 us, 1.25 PFLOP/s (the tensor pipe
// active 50 %; pages that are in L2 already make it 1.5 % faster).  16 blocks of
// 16 draft tokens over 4080 positions each (269 MB of keys and values): 51.8 us,
// 5.2 TB/s, 47 us with the pages in L2.  150 tokens behind 8000 positions, 8 heads
// over 2: 70 us, 0.97 ms with a NaN among their values.
//
// Over an 8-bit cache (Q8) tensor copies bring a tile's codes into the upper half
// of its slot, and four more warps turn them into 16-bit numbers over the whole
// slot, exact ones of the queries' type.  A key's scale
// multiplies its score in f32, a value's its weight, which is of the queries' type as
// the codes are (in two parts for rows of fewer than 256 positions).  Bound: as above, with twice the instructions in a
// softmax warp's turn, and with the unpacking of 32768 codes a key tile.  Measured:
// the chunk above 276-283 us with int8 or e4m3, 291-300 in fp16; the 16 blocks 64-73
// (a tile's codes are unpacked for 64 rows, half of what a tile has room for).
//
// For a tree of drafted tokens (TREE) a row sees the positions before the new tokens
// and the nodes that its bits say; the words with a tile's nodes are read at once.
// Measured: 16 trees of 64 nodes over 4080 positions 74.9 us (285 MB, 68 GFLOP; 128
// items on as many of the 152 CTAs, since a cut costs more than it brings by kChJoin); one of
// 13 over 2303 positions 21.7 us, of which ~2.6 go to the cut of the line, 1.8 to the
// first keys, 8 to the five tiles of the longest piece and 6 to the join.
//
// Every wait is bounded: on a timeout the kernel records W4A16_ETIMEOUT, ends
// its copies and MMAs, frees its tensor memory and returns.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>


#include "codes.cuh"
#include "paged_attn.cuh"

namespace w4a16 {

static __device__ int g_chunk_status;

// two softmax warpgroups, the MMA warp, the key / value and the query copy warp; over an 8-bit cache these three have a
// warpgroup (and a warp that idles), and four more warps unpack codes
template <bool Q8>
constexpr int kChThreads = Q8 ? 512 : 352;
constexpr int kChKeys = 128;
constexpr int kChTwo = 256;  // rows that see fewer positions carry their weights in two parts
constexpr int kChSnap = 2, kChJoin = 12;  // key tiles; see the line
constexpr int kChCounters = 1024;  // first arrival counter of this kernel (the small-row kernel's lie below)

// ONE: no request has more rows a key head than one row tile (draft blocks);
// the second tile's place then holds another slot of the ring, and keys come two
// tiles ahead (16 blocks of 16: 55.3 -> 51.9 us).
template <int D, bool ONE, bool Q8 = false>
struct Ch {
    static constexpr int kSlabs = D / 64;
    static constexpr int kTile = kSlabs * 16384;    // bytes of 128 rows of keys, values or queries
    static constexpr int kRows = ONE ? 1 : 2;       // row tiles of an item
    static constexpr int kSlots = (D == 128 ? 7 : 12) - kRows - (Q8 ? 1 : 0);
    static constexpr int kRingOff = kRows * kTile;
    static constexpr int kMlOff = kRingOff + kSlots * kTile;
    static constexpr int kBarOff = kMlOff + 2048;
    static constexpr int kMissOff = kBarOff + 384;            // [8] pages of a tile that are not there
    static constexpr int kMiscOff = kMissOff + 64;
    // Q8: scales of eight tiles [tile][keys', values', values' with 0 for what is not finite][128], 128 ones, and the
    // largest of the values' scales [tile][unpacking warp]
    static constexpr int kScaleOff = kMiscOff + 128;
    static constexpr int kSmem = kScaleOff + (Q8 ? (8 * 3 + 1) * 512 + 128 : 0);  // no static shared memory: the base is 1024-aligned
    static constexpr int kPartHalf = 128 * (D + 2);           // floats of one row tile's partial result
    static constexpr uint32_t kTS = 0, kTO = 256;             // tensor memory: S and P of both tiles, then O
};
static_assert(Ch<128, true>::kSmem <= 232448 && Ch<128, false>::kSmem <= 232448, "shared memory");
static_assert(Ch<64, true>::kSmem <= 232448 && Ch<64, false>::kSmem <= 232448, "shared memory");
static_assert(Ch<128, true, true>::kSmem <= 232448 && Ch<128, false, true>::kSmem <= 232448, "shared memory");
static_assert(Ch<64, true, true>::kSmem <= 232448 && Ch<64, false, true>::kSmem <= 232448, "shared memory");

// Over an 8-bit cache the block is launched with 128 registers a thread, 65536 in all; the two other warpgroups give
// some to the softmax ones: 2 x 184 + 64 + 80 = 4 x 128.
constexpr int kChSoftmaxRegs = 184, kChMmaRegs = 64, kChUnpackRegs = 80;
static_assert(2 * kChSoftmaxRegs + kChMmaRegs + kChUnpackRegs <= 4 * 128, "registers of the launch");
template <int N>
W4A16_DEVICE void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
W4A16_DEVICE void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// ---- instructions ---------------------------------------------------------
// Operand descriptors (K-major and 128-byte swizzle as smem_desc_sw128 has them;
// for V, [128 keys][64 columns] slabs, MN-major: columns contiguous, slabs 16 KB
// apart, 8-key groups 1 KB) differ in the start address alone, in their low
// word.  What they are made of goes through uniform(), so that the compiler
// knows it the same in all lanes and keeps it in uniform registers, which is
// where the instruction wants it: with descriptors built per instruction from
// per-lane values an MMA took ~60 clocks to issue, as long as it runs.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t kDescK = (16u >> 4) << 16, kDescV = (16384u >> 4) << 16;
W4A16_DEVICE uint32_t uniform(uint32_t x) { return __reduce_max_sync(0xffffffffu, x); }
// D[tmem] = A[smem] B[smem] over D columns, issued by one lane of a converged warp; below it D (+)= P[tmem] V[smem]
// over 128 keys
template <int D>
W4A16_DEVICE void score_block(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc) {
    if constexpr (D == 128) asm volatile("{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\t.reg .b32 x, y;\n\t"
        "setp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
        "add.u32 y, %2, 0;\n\tmov.b64 db, {y, %5};\n\t"
        "add.u32 x, %1, 0;\n\t"
        "mov.b64 da, {x, %5};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t"
        "setp.eq.u32 p, 0, 0;\n\t"
        "add.u32 y, %2, 2;\n\tmov.b64 db, {y, %5};\n\t"
        "add.u32 x, %1, 2;\n\t"
        "mov.b64 da, {x, %5};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t"
        "add.u32 y, %2, 4;\n\tmov.b64 db, {y, %5};\n\t"
        "add.u32 x, %1, 4;\n\t"
        "mov.b64 da, {x, %5};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t"
        "add.u32 y, %2, 6;\n\tmov.b64 db, {y, %5};\n\t"
        "add.u32 x, %1, 6;\n\t"
        "mov.b64 da, {x, %5};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t"
        "add.u32 y, %2, 1024;\n\tmov.b64 db, {y, %5};\n\t"
        "add.u32 x, %1, 1024;\n\t"
        "mov.b64 da, {x, %5};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t"
        "add.u32 y, %2, 1026;\n\tmov.b64 db, {y, %5};\n\t"
        "add.u32 x, %1, 1026;\n\t"
        "mov.b64 da, {x, %5};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t"
        "add.u32 y, %2, 1028;\n\tmov.b64 db, {y, %5};\n\t"
        "add.u32 x, %1, 1028;\n\t"
        "mov.b64 da, {x, %5};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t"
        "add.u32 y, %2, 1030;\n\tmov.b64 db, {y, %5};\n\t"
        "add.u32 x, %1, 1030;\n\t"
        "mov.b64 da, {x, %5};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t"
        "}" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(0), "r"(kDescHigh) : "memory");
    else asm volatile("{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\t.reg .b32 x, y;\n\t"
        "setp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
        "add.u32 y, %2, 0;\n\tmov.b64 db, {y, %5};\n\t"
        "add.u32 x, %1, 0;\n\t"
        "mov.b64 da, {x, %5};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t"
        "setp.eq.u32 p, 0, 0;\n\t"
        "add.u32 y, %2, 2;\n\tmov.b64 db, {y, %5};\n\t"
        "add.u32 x, %1, 2;\n\t"
        "mov.b64 da, {x, %5};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t"
        "add.u32 y, %2, 4;\n\tmov.b64 db, {y, %5};\n\t"
        "add.u32 x, %1, 4;\n\t"
        "mov.b64 da, {x, %5};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t"
        "add.u32 y, %2, 6;\n\tmov.b64 db, {y, %5};\n\t"
        "add.u32 x, %1, 6;\n\t"
        "mov.b64 da, {x, %5};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t"
        "}" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(0), "r"(kDescHigh) : "memory");
}
// (SPREAD: the weights of 32 keys lie in the 16 first of the columns that their scores had)
template <bool SPREAD>
W4A16_DEVICE void pv_block(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
    asm volatile("{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\t.reg .b32 x, y;\n\t"
        "setp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
        "add.u32 y, %2, 0;\n\tmov.b64 db, {y, %5};\n\t"
        "add.u32 x, %1, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], db, %3, p;\n\t"
        "setp.eq.u32 p, 0, 0;\n\t"
        "add.u32 y, %2, 128;\n\tmov.b64 db, {y, %5};\n\t"
        "add.u32 x, %1, %6;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], db, %3, p;\n\t"
        "add.u32 y, %2, 256;\n\tmov.b64 db, {y, %5};\n\t"
        "add.u32 x, %1, %7;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], db, %3, p;\n\t"
        "add.u32 y, %2, 384;\n\tmov.b64 db, {y, %5};\n\t"
        "add.u32 x, %1, %8;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], db, %3, p;\n\t"
        "add.u32 y, %2, 512;\n\tmov.b64 db, {y, %5};\n\t"
        "add.u32 x, %1, %9;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], db, %3, p;\n\t"
        "add.u32 y, %2, 640;\n\tmov.b64 db, {y, %5};\n\t"
        "add.u32 x, %1, %10;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], db, %3, p;\n\t"
        "add.u32 y, %2, 768;\n\tmov.b64 db, {y, %5};\n\t"
        "add.u32 x, %1, %11;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], db, %3, p;\n\t"
        "add.u32 y, %2, 896;\n\tmov.b64 db, {y, %5};\n\t"
        "add.u32 x, %1, %12;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], db, %3, p;\n\t"
        "}" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(kDescHigh), "n"(8), "n"(SPREAD ? 32 : 16),
        "n"(SPREAD ? 40 : 24), "n"(SPREAD ? 64 : 32), "n"(SPREAD ? 72 : 40), "n"(SPREAD ? 96 : 48), "n"(SPREAD ? 104 : 56)
        : "memory");
}
template <typename Ty>
__device__ constexpr uint32_t idesc_ch(int N, bool v) {
    return (1u << 4) | (Ty::idesc_type << 7) | (Ty::idesc_type << 10) | ((v ? 1u : 0u) << 16) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
#define W4A16_R32(v, o)                                                                                            \
    "r"((v)[o]), "r"((v)[o + 1]), "r"((v)[o + 2]), "r"((v)[o + 3]), "r"((v)[o + 4]), "r"((v)[o + 5]),              \
        "r"((v)[o + 6]), "r"((v)[o + 7]), "r"((v)[o + 8]), "r"((v)[o + 9]), "r"((v)[o + 10]), "r"((v)[o + 11]),    \
        "r"((v)[o + 12]), "r"((v)[o + 13]), "r"((v)[o + 14]), "r"((v)[o + 15]), "r"((v)[o + 16]),                  \
        "r"((v)[o + 17]), "r"((v)[o + 18]), "r"((v)[o + 19]), "r"((v)[o + 20]), "r"((v)[o + 21]),                  \
        "r"((v)[o + 22]), "r"((v)[o + 23]), "r"((v)[o + 24]), "r"((v)[o + 25]), "r"((v)[o + 26]),                  \
        "r"((v)[o + 27]), "r"((v)[o + 28]), "r"((v)[o + 29]), "r"((v)[o + 30]), "r"((v)[o + 31])
W4A16_DEVICE void tmem_st32(uint32_t taddr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        W4A16_R32(v, 0)
        : "memory");
}
W4A16_DEVICE void tmem_st16(uint32_t taddr, const uint32_t* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
W4A16_DEVICE void tmem_ld32(uint32_t taddr, uint32_t* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr)
        : "memory");
}

// the two halves of v, 0 in the place of infinities and NaN
template <typename Ty>
W4A16_DEVICE uint32_t finite(uint32_t v) {
    return v & ~(((Ty::all_ones(v) >> 15) & 0x00010001u) * 0xffffu);
}

W4A16_DEVICE float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// two f32 operations in one instruction
W4A16_DEVICE float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
        "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
W4A16_DEVICE float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
W4A16_DEVICE float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// ---- the line of key tiles --------------------------------------------------
struct ChunkItem {
    int i0, tokens;      // first token (of the request) and their number
    int e0, e1;          // last position that all tokens see, and that any does
    int lo0, lo1;        // first position that any token sees, and that all do
    int t0, tiles;       // first key tile and their number
};
template <bool TREE>
W4A16_DEVICE ChunkItem item_of(const PagedAttnParams& p, const Request& r, int q, int span) {
    ChunkItem it;
    it.i0 = q * span;
    it.tokens = min(span, r.n - it.i0);
    const Seen see = seen_by<TREE>(p, r, it.i0, it.i0 + it.tokens - 1);
    it.e0 = see.e_all;
    it.e1 = see.last;
    it.lo0 = see.first;
    it.lo1 = see.lo_all;
    it.t0 = it.lo0 / kChKeys;
    it.tiles = it.e1 < it.lo0 ? 1 : it.e1 / kChKeys + 1 - it.t0;  // nothing seen: one masked tile
    return it;
}
W4A16_DEVICE int items_of(const PagedAttnParams& p, const Request& r, int span) {
    return r.n * p.G <= p.small_rows ? 0 : (r.n + span - 1) / span;
}
struct ChunkPiece {
    Request r;
    ChunkItem it;
    int b, hk, q;
    int off, take;            // key tiles of the item before this piece, and in it
    int64_t first;            // the item's first tile on the line
    bool duo;                 // two row tiles (else both warpgroups share the first)
    bool two;                 // weights in two parts
};
// Ring entries of a piece of n tiles, from its first on.  With items of one row
// tile (ONE) they come in the order in which the MMA warp takes them, the scores
// of two tiles ahead: K0 K1 V0 K2 V1 .. K(n-1) V(n-2) V(n-1); else K0 V0 K1 V1 ..
template <bool ONE>
W4A16_DEVICE uint32_t keys_at(uint32_t t) { return !ONE ? 2 * t : t ? 2 * t - 1 : 0; }
template <bool ONE>
W4A16_DEVICE uint32_t values_at(uint32_t t, uint32_t n) { return !ONE || t + 1 == n ? 2 * t + 1 : 2 * t + 2; }
// Walks a CTA's part of the line; every warp walks it for itself.
struct ChunkWalk {
    int b, hk, q, off, items;
    int64_t at, left;
    Request r;
    template <bool ONE, bool TREE>
    W4A16_DEVICE bool next(const PagedAttnParams& p, int toks, ChunkPiece& c) {
        const int span = ONE ? toks : 2 * toks;
        if (left <= 0) return false;
        c.r = r;
        c.it = item_of<TREE>(p, r, q, span);
        c.b = b;
        c.hk = hk;
        c.q = q;
        c.off = off;
        c.take = (int)(left < c.it.tiles - off ? left : c.it.tiles - off);
        c.first = at - off;
        c.duo = !ONE && c.it.tokens > toks;
        c.two = c.it.e0 - c.it.lo0 + 1 < kChTwo;
        at += c.take;
        left -= c.take;
        if (left > 0) {
            off = 0;
            if (++hk == p.Hkv) {
                hk = 0;
                if (++q == items) {
                    q = 0;
                    do {
                        r = request_of(p, ++b);
                        items = items_of(p, r, span);
                    } while (items == 0);
                }
            }
        }
        return true;
    }
};

// Adds the values that were taken out of an item's value tiles to the columns
// x0 .. x1 of a row that sees the positions lo .. e (and in a tree the nodes that
// its bits say): those that are not finite at positions that not all rows see.
template <typename Ty, bool TREE>
W4A16_DEVICE void add_taken_out(const PagedAttnParams& p, const ChunkPiece& pc, int t, int lo, int e, uint16_t* out, int x0,
                                int x1) {
    const int* table = p.table + (int64_t)pc.b * p.table_stride;
    auto add = [&](int j) {
        const int pg = __ldcg(table + (j >> p.shift));
        if (pg < 0 || pg >= p.pages) return;
        const uint16_t* v = p.v + pg * p.vp + pc.hk * p.vh + (int64_t)(j & ((1 << p.shift) - 1)) * p.vs;
#pragma unroll 1
        for (int x = x0; x < x1; x += 2) {
            const uint32_t y = __ldcg(reinterpret_cast<const uint32_t*>(v + x)), t = Ty::all_ones(y) & 0x80008000u;
            if (t == 0) continue;
            uint32_t* o = reinterpret_cast<uint32_t*>(out + x);
            *o = Ty::pack(Ty::lo(*o) + (t & 0x8000u ? Ty::lo(y) : 0.f), Ty::hi(*o) + (t >> 31 ? Ty::hi(y) : 0.f));
        }
    };
#pragma unroll 1
    for (int j = lo; j <= e; ++j) {
        if (j >= pc.it.lo1 && j <= pc.it.e0) {  // all rows see these
            j = pc.it.e0;
            continue;
        }
        add(j);
    }
    if constexpr (TREE) {
        const int past = pc.r.L - pc.r.n;
#pragma unroll 1
        for (int k = max(0, -past); k < pc.r.n; ++k)
            if ((tree_word(p, t, pc.r.n, k >> 5) >> (k & 31)) & 1u) add(past + k);
    }
}

// ---- keys and values of an 8-bit cache --------------------------------------
// Weights carry their values' scales.  In bf16 these have f32's range.  In fp16 (for
// fp16 queries, whose outputs a weight of 8 bits would spoil) the base that scores
// are taken against goes by the sum of the largest score and the logarithm of the
// largest scale (a power of two, out of 2^-60 .. 2^100) that the row has seen: a
// weight is at most 2^14, what the largest score and the largest scale would make
// at least 2^5, and a weight is rounded by 2^-11 of itself or by 2^-25.  (Two bf16
// parts did it before: the chunk above 408 us.)
// The base lies 66 binades below the row's largest score to 94 above it, so that
// the sum of the weights before their scales is 2^-94 at least and, with the lag of
// 2^8 of a maximum, 2^74 a position at most; scales below 2^-60 make outputs of 0.
// As the scales run, a base may move by more than the 126 binades that an f32 factor
// has, with a sum that lies in range on both sides of the move: such factors are
// taken as their square root, twice.
constexpr float kChShift = 6.f;  // of the base: weights are up to 2^(8 + 6)
W4A16_DEVICE float scale_log(float largest) {  // an exponent that the scale is not above
    return fminf(fmaxf((float)((int)(__float_as_uint(largest) >> 23) - 126), -60.f), 100.f);
}
// 2^x as a factor, and products with it; TWICE: kept as its root
template <bool TWICE>
W4A16_DEVICE float power_of_2(float x) { return exp2_approx(TWICE ? 0.5f * x : x); }
template <bool TWICE>
W4A16_DEVICE float times(float x, float f) { return TWICE ? x * f * f : x * f; }
template <bool TWICE>
W4A16_DEVICE float add_times(float x, float f, float sum) { return fmaf(TWICE ? x * f : x, f, sum); }

// Weights of 32 scores, times their values' scales: hi, and with TWO what hi lacks; the sums l0 and l1 are of the weights
// alone.
template <typename Ty, bool TWO>
W4A16_DEVICE void scaled_weights(const uint32_t (&v)[32], const float* kc, const float* vc, float2 nb, float2& l0, float2& l1,
                                 uint32_t (&hi)[16], uint32_t* lo) {
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
        const float4 c = *reinterpret_cast<const float4*>(kc + 2 * i);
        const float4 d = *reinterpret_cast<const float4*>(vc + 2 * i);
        float2 a = make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
        float2 b = make_float2(__uint_as_float(v[2 * i + 2]), __uint_as_float(v[2 * i + 3]));
        a = fma2(a, make_float2(c.x, c.y), nb);
        b = fma2(b, make_float2(c.z, c.w), nb);
        a.x = exp2_approx(a.x);
        a.y = exp2_approx(a.y);
        b.x = exp2_approx(b.x);
        b.y = exp2_approx(b.y);
        l0 = add2(l0, a);
        l1 = add2(l1, b);
        a = mul2(a, make_float2(d.x, d.y));
        b = mul2(b, make_float2(d.z, d.w));
        hi[i] = Ty::pack(a.x, a.y);
        hi[i + 1] = Ty::pack(b.x, b.y);
        if constexpr (TWO) {
            lo[i] = Ty::pack(a.x - Ty::lo(hi[i]), a.y - Ty::hi(hi[i]));
            lo[i + 1] = Ty::pack(b.x - Ty::lo(hi[i + 1]), b.y - Ty::hi(hi[i + 1]));
        }
    }
}
// Those of a row's 128 scores in two parts, for the rows of few positions: out of line, so that the loop of the long
// ones fits the instruction caches (350 us instead of 379 for the chunk above, before the next steps).
template <typename Ty>
__device__ __noinline__ float2 weights_in_two_parts(uint32_t ts, const float* kc, const float* vc, float base) {
    float2 l0 = make_float2(0.f, 0.f), l1 = l0;
#pragma unroll 1
    for (int x = 0; x < 4; ++x) {
        uint32_t v[32], hi[16], lo[16];
        tmem_ld32(ts + 32 * x, v);
        tmem_wait_ld();
        scaled_weights<Ty, true>(v, kc + 32 * x, vc + 32 * x, make_float2(-base, -base), l0, l1, hi, lo);
        tmem_st16(ts + 32 * x, hi);
        tmem_st16(ts + 32 * x + 16, lo);
    }
    return add2(l0, l1);
}

// The four unpacking warps.  A tile's codes lie in the upper half of its ring slot
// and become 16-bit numbers over the whole slot, in the layout that tensor copies
// of such would give: a thread takes the same 16 columns of 64 of every 32nd row.
// Thread i brings the scales of key i, a tile ahead, and leaves them as the softmax
// takes them.
template <typename Ty, int D, bool ONE, bool TREE, bool E4M3>
W4A16_DEVICE void unpack_codes(const PagedAttnParams& p, ChunkWalk walk, int toks, unsigned char* smem, uint64_t* full,
                               uint64_t* raw, float* scales, volatile int* abort_flag) {
    using L = Ch<D, ONE, true>;
    constexpr int NS = L::kSlots;
    constexpr bool BF = Ty::idesc_type == 1;
    const uint32_t base = code_base<BF>();
    const int tid = threadIdx.x & 127, lane = tid & 31, prow = tid >> 2, pcol = tid & 3;
    const uint32_t ring = smem_u32(smem) + L::kRingOff, from = ring + L::kTile / 2 + prow * D + pcol * 16;
    const uint32_t to = ring + prow * 128 + (((pcol * 2) ^ (prow & 7)) << 4);  // (row & 7 is prow & 7 in every step)
    ChunkPiece pc;
    uint32_t e = 0, tile0 = 0;
    while (walk.next<ONE, TREE>(p, toks, pc)) {
        const uint32_t n = pc.take;
        // of tile t: the page of key tid (-1: not there, or no row sees it), and the key's scales from that
        const int* table = p.table + (int64_t)pc.b * p.table_stride;
        const int first = (pc.it.t0 + pc.off) * kChKeys + tid;
        auto page_of = [&](uint32_t t) {
            const int j = first + (int)t * kChKeys, col = j >> p.shift;
            return t < n && j >= pc.it.lo0 && j <= pc.it.e1 && col < p.columns ? __ldcg(table + col) : -1;
        };
        float ks, vs;
        auto scales_of = [&](uint32_t t, int pg) {
            const int64_t at = (first + (int)t * kChKeys) & ((1 << p.shift) - 1);
            const bool there = pg >= 0 && pg < p.pages;
            ks = there ? __ldcg(p.k_scale + pg * p.ksp + pc.hk * p.ksh + at * p.kss) : 0.f;
            vs = there ? __ldcg(p.v_scale + pg * p.vsp + pc.hk * p.vsh + at * p.vss) : 0.f;
        };
        int pg = page_of(0);
        uint32_t t = ~0u;  // scales of tile t + 1 are on their way, or t + 1 is 0
#pragma unroll 1
        for (uint32_t i = 0; i < 2 * n; ++i, ++e) {
            // entry i is tile t's keys (values_at and keys_at of ChunkWalk's order), or values
            const bool keys = !ONE ? !(i & 1) : i == 0 || ((i & 1) && i + 1 < 2 * n);
            const uint32_t sl = e % NS, off = sl * L::kTile;
            const bool ok = mbar_wait_warp(raw + sl, (e / NS) & 1, abort_flag, &g_chunk_status);
            auto put = [&](uint32_t a, const uint4& v) {
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                uint32_t y[8];
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int h = 0; h < 2; ++h)  // bytes 2 h, 2 h + 1 to where code_pair has them
                        y[2 * c + h] = code_pair<E4M3, BF, E4M3>(
                            __byte_perm(w[c], 0u, E4M3 ? (h ? 0x3424 : 0x1404) : (h ? 0x4342 : 0x4140)), base);
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3])
                             : "memory");
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a ^ 16u), "r"(y[4]), "r"(y[5]), "r"(y[6]), "r"(y[7])
                             : "memory");
            };
            auto unpack = [&] {
                if constexpr (D == 128) {
                    // a row's 128 codes lie where the last 64 of its numbers go: four lanes read and write them
#pragma unroll 1
                    for (int k = 0; k < 4; ++k) {
                        const uint4 x = lds_v4(from + off + k * 32 * 128), y = lds_v4(from + off + k * 32 * 128 + 64);
                        __syncwarp();
                        put(to + off + k * 32 * 128, x);
                        put(to + off + k * 32 * 128 + 16384, y);
                    }
                    return ok;
                } else {
                    // a row of numbers lies over two rows of codes: all are in registers first
                    uint4 v[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[k] = lds_v4(from + off + k * 32 * 64);
                    if (!bar_and(3, 128, ok)) return false;  // all have read theirs (or one gave up, and all do)
#pragma unroll
                    for (int k = 0; k < 4; ++k) put(to + off + k * 32 * 128, v[k]);
                    return true;
                }
            };
            if (keys) {
                if (t == ~0u) {
                    scales_of(0, pg);
                    pg = page_of(1);
                }
                ++t;
                float* sc = scales + ((tile0 + t) & 7) * 384 + tid;
                const float f = finite_or_nan(vs);
                sc[0] = finite_or_nan(ks) * p.scale2;
                sc[128] = f;
                const float g = fabsf(f) < INFINITY ? f : 0.f;
                sc[256] = g;
                if constexpr (!BF) {  // (0 where no row sees the key)
                    const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(g)));
                    if (lane == 0) scales[25 * 128 + ((tile0 + t) & 7) * 4 + (tid >> 5)] = __uint_as_float(most);
                }
                scales_of(t + 1, pg);
                pg = page_of(t + 2);
            }
            if (!unpack()) return;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(full + sl);
        }
        tile0 += n;
    }
}

template <typename Ty, int D, bool ONE, bool TREE, bool Q8>
__global__ void __launch_bounds__(kChThreads<Q8>, 1)
    paged_chunk_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                       const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ PagedAttnParams p) {
    using L = Ch<D, ONE, Q8>;
    constexpr int NS = L::kSlots;
    // The loops over a row's scores are rolled, and weights in two parts lie over their own scores' columns: for an
    // 8-bit cache since the code of the CTA's roles has to fit the instruction caches (a 2048-token chunk: 416 us with
    // the loops written out, 283 so), for trees since their short calls run most lines once (13 nodes: 24.5 us written
    // out, 22.4 so, before the join's present form; 16 trees of 64 nodes alike).
    constexpr bool SPREAD = Q8 || TREE;
    constexpr bool BASED = Q8 && Ty::idesc_type == 0;  // scores against a base that the values' scales are part of
    extern __shared__ __align__(1024) unsigned char smem[];
    if (smem_u32(smem) & 1023u) {  // the swizzled tiles need it
        if (threadIdx.x == 0) atomicExch(&g_chunk_status, (int)W4A16_ECUDA);
        return;
    }
    float2* ml = reinterpret_cast<float2*>(smem + L::kMlOff);  // [2][128] m and l of both warpgroups
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
    uint64_t* empty = full + NS;
    uint64_t* s_full = empty + NS;   // [2]
    uint64_t* p_full = s_full + 2;   // [2]
    uint64_t* o_full = p_full + 2;   // [2]
    uint64_t* o_free = o_full + 2;   // [2]
    uint64_t* q_full = o_free + 2;
    uint64_t* q_free = q_full + 1;
    uint64_t* join = q_free + 1;     // both warpgroups' maxima and sums are in ml
    uint64_t* done = join + 1;       // every MMA of the CTA is done
    uint64_t* raw = done + 1;        // Q8: [NS] a slot's codes are there
    static_assert(((Q8 ? 3 : 2) * NS + 12) * 8 <= 384, "barriers");
    volatile uint32_t* miss = reinterpret_cast<volatile uint32_t*>(smem + L::kMissOff);
    volatile int* misc = reinterpret_cast<volatile int*>(smem + L::kMiscOff);
    volatile int* abort_flag = misc;  // misc: abort, request, head, item, offset, pieces with values taken out (2), -,
                                      // tensor memory
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + L::kMiscOff) + 8;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = (int)blockIdx.x;
    const int toks = 128 / p.G, span = L::kRows * toks;  // tokens of a row tile and of an item

    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(full + i, Q8 ? 4 : 1);  // (Q8: a lane of each unpacking warp arrives)
            if constexpr (Q8) mbar_init(raw + i, 1);
            mbar_init(empty + i, 1);
        }
        for (int g = 0; g < 2; ++g) {
            mbar_init(s_full + g, 1);
            mbar_init(p_full + g, 4);  // a lane of each warp arrives
            mbar_init(o_full + g, 1);
            mbar_init(o_free + g, 8);  // the warps that may read it, or four of them twice
        }
        mbar_init(q_full, 1);
        mbar_init(q_free, 1);
        mbar_init(join, 8);
        mbar_init(done, 1);
        *abort_flag = 0;
        misc[5] = misc[6] = 0;
        fence_mbar_init();
    }
    if (warp == 8) {
        tmem_alloc(tmem_holder, 512);
        tmem_relinquish();
    }
    if (warp == 9 && lane == 0) {
        prefetch_tmap(&tmap_q);
        prefetch_tmap(&tmap_k);
        prefetch_tmap(&tmap_v);
    }
    float* scales = reinterpret_cast<float*>(smem + L::kScaleOff);
    if constexpr (Q8)
        if (threadIdx.x < 128) scales[8 * 3 * 128 + threadIdx.x] = 1.f;
    // Behind the small-row kernel of the same call there is nothing to wait for:
    // that kernel let this one start once everything before it was done, and the
    // two have requests, counters and workspace of their own.  What earlier kernels
    // wrote is in L2, and is read from there (tensor copies, __ldcg).
    if (!p.after_small) pdl_wait();
    pdl_launch_dependents();

    // ---- this CTA's part of the line --------------------------------------
    // The line runs over the requests, their items, the key heads and the key
    // tiles.  Pair j = (request, item): start[b] is request b's first pair (in
    // the ring's memory, not yet in use); a thread takes a pair at a time.
    int* warp_sum = reinterpret_cast<int*>(ml);                        // (not in use before the first item's end)
    int64_t* cut = reinterpret_cast<int64_t*>(warp_sum + 16);
    constexpr int NT = kChThreads<Q8>;
    int* start = reinterpret_cast<int*>(smem);
    auto scan = [&](int x, int& total) {  // exclusive sum over the threads
        int y = x;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int z = __shfl_up_sync(0xffffffffu, y, d);
            if (lane >= d) y += z;
        }
        __syncthreads();
        if (lane == 31) warp_sum[warp] = y;
        __syncthreads();
        const int w = lane < NT / 32 ? warp_sum[lane] : 0;
        total = __reduce_add_sync(0xffffffffu, w);
        return y - x + __reduce_add_sync(0xffffffffu, lane < warp ? w : 0);
    };
    int pairs = 0;
    for (int b = 0; b < p.B; b += NT) {
        int n = 0, total;
        if (b + (int)threadIdx.x < p.B) n = items_of(p, request_of(p, b + threadIdx.x), span);
        const int at = pairs + scan(n, total);
        if (b + (int)threadIdx.x < p.B) start[b + threadIdx.x] = at;
        pairs += total;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    Request pr{0, 0, 0};
    int pb = 0, pq = 0;
    auto tiles_of = [&](int j) {  // key tiles of pair j (0 past the last)
        if (j >= pairs) return 0;
        int lo = 0, hi = p.B;  // the last request whose first pair is j or before it and that has a pair
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (start[mid] <= j) lo = mid; else hi = mid;
        }
        pb = lo;
        pq = j - start[lo];
        pr = request_of(p, lo);
        return item_of<TREE>(p, pr, pq, span).tiles;
    };
    int64_t U = 0;
    int first_tiles = 0, first_at = 0;  // of this thread's first pair
    for (int j = 0; j < pairs; j += NT) {
        int total;
        const int n = tiles_of(j + threadIdx.x), at = scan(n, total);
        if (j == 0) first_tiles = n, first_at = at;
        U += total;
    }
    U *= p.Hkv;
    const int most = [&] {  // key tiles of the longest item
        int m = first_tiles;
        for (int j = NT; j < pairs; j += NT) m = max(m, tiles_of(j + threadIdx.x));
        m = __reduce_max_sync(0xffffffffu, m);
        __syncthreads();
        if (lane == 0) warp_sum[warp] = m;
        __syncthreads();
        return __reduce_max_sync(0xffffffffu, lane < NT / 32 ? warp_sum[lane] : 0);
    }();
    // An item split over CTAs costs about kChJoin tiles' time on each side: the
    // piece written, waited for and joined.  So with no more items than CTAs
    // every CTA takes one, unless the longest would take that much longer than
    // an even share; and a cut less than kChSnap tiles from an item's end moves
    // to the end.
    const int64_t n_items = (int64_t)pairs * p.Hkv;
    const bool single = n_items <= gridDim.x && (int64_t)(most - kChJoin) * gridDim.x <= U;
    int C = single ? (int)n_items : (int)(U < gridDim.x ? U : gridDim.x);
    // A piece more costs the joining CTA about two fifths of a tile's time, so that few items are not cut below
    // sqrt(2 / 5 tiles) tiles a piece: 13 nodes over 2303 positions, 8 items of 19 tiles, 36 us in 152 pieces.  (kChJoin
    // was fitted to an earlier and slower join, and so was the causal form over 16 bits, which has no such least share.)
    if ((TREE || Q8) && !single) {
        int least = 1;
        while (5 * least * least < 2 * most) ++least;
        C = (int)min((int64_t)C, (U + least - 1) / least);
    }
    ChunkWalk walk;
    walk.left = 0;
    if (c < C) {
        int64_t u0 = (int64_t)c * U / C, u1 = (int64_t)(c + 1) * U / C;
        if (single) {
            if (threadIdx.x == 0) {
                const int n = tiles_of(c / p.Hkv);
                misc[1] = pb;
                misc[2] = c % p.Hkv;
                misc[3] = pq;
                misc[4] = 0;
                cut[0] = 0;
                cut[1] = n;
            }
            __syncthreads();
        } else {
            // the items that hold this CTA's first unit and the next CTA's
            int64_t before = 0;
            for (int j = 0; j < pairs; j += NT) {
                int total = 0, n = first_tiles, at = first_at;
                if (pairs > NT) {
                    n = tiles_of(j + threadIdx.x);
                    at = scan(n, total);
                }
                const int64_t a = (before + at) * p.Hkv;
                auto snapped = [&](int64_t u) {
                    const int d = (int)(u - a) % n;
                    return d <= kChSnap && d <= n - d ? u - d : n - d <= kChSnap ? u + n - d : u;
                };
                if (n > 0 && u0 >= a && u0 < a + (int64_t)n * p.Hkv) {
                    cut[0] = snapped(u0);
                    int rest = (int)(cut[0] - a);
                    const bool next = rest == n * p.Hkv;  // at the next pair's first item
                    if (next && j + (int)threadIdx.x + 1 < pairs) {
                        (void)tiles_of(j + threadIdx.x + 1);
                        rest = 0;
                    }
                    misc[1] = pb;
                    misc[2] = rest / n;
                    misc[3] = pq;
                    misc[4] = rest % n;
                }
                if (n > 0 && u1 >= a && u1 < a + (int64_t)n * p.Hkv) cut[1] = snapped(u1);
                if (u1 == U && threadIdx.x == 0) cut[1] = U;
                before += total;
            }
            __syncthreads();
        }
        walk.left = cut[1] - cut[0];
        if (walk.left > 0) {
            walk.b = misc[1];
            walk.hk = misc[2];
            walk.q = misc[3];
            walk.off = misc[4];
            walk.r = request_of(p, walk.b);
            walk.items = items_of(p, walk.r, span);
            walk.at = cut[0];
        }
        fence_proxy_async_smem();  // copies will overwrite `start`
        __syncthreads();
    }
    // the CTAs that share an item of `n` tiles whose first unit is `first`
    auto sharers = [&](int64_t first, int n, int& lo, int& hi) {
        lo = (int)(((first + kChSnap + 1) * C + U - 1) / U) - 1;
        hi = (int)(((first + n - kChSnap) * C + U - 1) / U) - 1;
    };

    ChunkPiece pc;
    if (Q8 && warp >= 12) {
        // ---------------------------------------- codes of an 8-bit cache to numbers
        if constexpr (Q8) {
            fewer_registers<kChUnpackRegs>();
            if (p.e4m3) unpack_codes<Ty, D, ONE, TREE, true>(p, walk, toks, smem, full, raw, scales, abort_flag);
            else unpack_codes<Ty, D, ONE, TREE, false>(p, walk, toks, smem, full, raw, scales, abort_flag);
        }
    } else if (warp >= 8) {
      if constexpr (Q8) fewer_registers<kChMmaRegs>();
      if (warp == 9) {
        // ---------------------------------------------------------- copies
        const int page = 1 << p.shift, rows = page < kChKeys ? page : kChKeys, boxes = kChKeys / rows;
        uint32_t e = 0, tile0 = 0;  // the next ring entry, and the piece's first tile
        bool ok = true;
        while (ok && walk.next<ONE, TREE>(p, toks, pc)) {
            const int* row = p.table + (int64_t)pc.b * p.table_stride;
            auto entry = [&](int t) {  // lane's box of the piece's tile t
                const int j = (pc.it.t0 + pc.off + t) * kChKeys + lane * rows, col = j >> p.shift;
                // boxes that no row sees are not read: -2
                if (t >= pc.take || lane >= boxes || j > pc.it.e1 || j + rows <= pc.it.lo0) return -2;
                return col < p.columns ? __ldcg(row + col) : -1;
            };
            auto load = [&](int t, int kv, int ent) {  // the next ring entry: tile t's keys or values
                const int slot = ((pc.it.t0 + pc.off + t) * kChKeys + lane * rows) & (page - 1), sl = e % NS;
                const bool there = ent >= 0 && ent < p.pages;
                const int pg = there ? ent : p.pages;  // past the tensor: filled with zeros
                const uint32_t no = __ballot_sync(0xffffffffu, !there && ent != -2);
                if (e >= NS) ok = mbar_wait_warp(empty + sl, (e / NS - 1) & 1, abort_flag, &g_chunk_status);
                if (!ok) return;
                if (lane == 0) {
                    if (kv == 0) miss[(tile0 + t) & 7] = no;
                    mbar_arrive_expect_tx((Q8 ? raw : full) + sl, (uint32_t)(Q8 ? L::kTile / 2 : L::kTile));
                }
                __syncwarp();
                if constexpr (Q8) {
                    if (lane < boxes)
                        tma_load_4d(smem + L::kRingOff + sl * L::kTile + L::kTile / 2 + lane * rows * D, kv ? &tmap_v : &tmap_k, 0,
                                    slot, pc.hk, pg, raw + sl);
                } else if (lane < boxes) {
                    unsigned char* dst = smem + L::kRingOff + sl * L::kTile + lane * rows * 128;
#pragma unroll
                    for (int s = 0; s < L::kSlabs; ++s)
                        tma_load_4d(dst + s * 16384, kv ? &tmap_v : &tmap_k, 64 * s, slot, pc.hk, pg, full + sl);
                }
                __syncwarp();
                ++e;
            };
            int ent = entry(0);  // of tile t
            if constexpr (ONE) {
                int next = entry(1);
                load(0, 0, ent);
                for (int t = 0; t < pc.take && ok; ++t) {
                    const int after = entry(t + 2);
                    if (t + 1 < pc.take) load(t + 1, 0, next);
                    if (ok) load(t, 1, ent);
                    ent = next;
                    next = after;
                }
            } else {
                for (int t = 0; t < pc.take && ok; ++t) {
                    const int cur = ent;
                    ent = entry(t + 1);
                    load(t, 0, cur);
                    if (ok) load(t, 1, cur);
                }
            }
            tile0 += pc.take;
        }
        // the copies in flight land before the CTA ends
        for (uint32_t i = e > NS ? e - NS : 0; i < e; ++i)
            (void)mbar_wait_warp((Q8 ? raw : full) + i % NS, (i / NS) & 1, nullptr, &g_chunk_status);
      } else if (warp == 10) {
        // --------------------------------------------------------- queries
        uint32_t items = 0;
        while (walk.next<ONE, TREE>(p, toks, pc)) {
            if (items > 0 && !mbar_wait_warp(q_free, (items - 1) & 1, abort_flag, &g_chunk_status)) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(q_full, (uint32_t)((pc.duo ? 2 : 1) * L::kSlabs * toks * p.G * 128));
                for (int g = 0; g < (pc.duo ? 2 : 1); ++g)
                    for (int s = 0; s < L::kSlabs; ++s)
                        tma_load_3d(smem + g * L::kTile + s * 16384, &tmap_q, 64 * s, pc.hk * p.G,
                                    pc.r.t0 + pc.it.i0 + g * toks, q_full);
            }
            __syncwarp();
            ++items;
        }
        if (items > 0) (void)mbar_wait_warp(q_full, (items - 1) & 1, nullptr, &g_chunk_status);
      } else if (warp == 8) {
        // ------------------------------------------------------------ MMAs
        // The warpgroups in turn: P V of a tile and the scores of the next one
        // go out together.
        // What steers the loop is made uniform, for the descriptors' sake: the chunk
        // above took 206 us with it and 218 without.
        constexpr uint32_t id_s = idesc_ch<Ty>(kChKeys, false), id_o = idesc_ch<Ty>(D, true);
        const uint32_t tm = uniform(tmem), sm = uniform(smem_u32(smem));
        auto tile_at = [&](uint32_t slot, uint32_t kind) {  // a descriptor's low word; tile 0 is Q's first
            return ((sm + slot * (uint32_t)L::kTile) >> 4) | kind;
        };
        uint32_t tile0 = 0, items = 0, np[2] = {0, 0};
        bool ok = true;
        while (ok && walk.next<ONE, TREE>(p, toks, pc)) {
            const int take = (int)uniform((uint32_t)pc.take);
            const bool duo = !ONE && uniform(pc.duo) != 0, two = uniform(pc.two) != 0;
            const int cnt[2] = {duo ? take : (take + 1) / 2, duo ? take : take / 2};
            int scores = cnt[0] + cnt[1];
            auto tile_of = [&](int g, int k) { return (uint32_t)(duo ? k : 2 * k + g); };
            auto keys_of = [&](int g, int k) { return 2 * tile0 + keys_at<ONE>(tile_of(g, k)); };
            auto arrived = [&](uint32_t e) {
                return mbar_wait_warp(full + e % NS, (e / NS) & 1, abort_flag, &g_chunk_status);
            };
            auto score = [&](int g, int k) {  // S_g of the group's k-th tile
                const uint32_t sl = keys_of(g, k) % NS;
                tc_fence_after();
                score_block<D>(tm + L::kTS + 128 * g, tile_at(duo ? g : 0, kDescK), tile_at(L::kRows + sl, kDescK), id_s);
                mma_commit_warp(s_full + g);
                if (!duo || g == 1) mma_commit_warp(empty + sl);
                if (--scores == 0) mma_commit_warp(q_free);
            };
            ok = mbar_wait_warp(q_full, items & 1, abort_flag, &g_chunk_status);
#pragma unroll
            for (int g = 0; g < 2; ++g) {
                if (!ok || cnt[g] == 0) continue;
                if (!duo || g == 0) ok = arrived(keys_of(g, 0));
                if (ok) score(g, 0);
            }
            for (int k = 0; k < cnt[0] && ok; ++k) {
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    if (!ok || k >= cnt[g]) continue;
                    const uint32_t e = 2 * tile0 + values_at<ONE>(tile_of(g, k), (uint32_t)take), sl = e % NS;
                    const bool next = k + 1 < cnt[g];
                    if (k == 0 && items > 0)
                        ok = mbar_wait_warp(o_free + g, (items - 1) & 1, abort_flag, &g_chunk_status);
                    ok = ok && arrived(e);
                    ok = ok && mbar_spin_warp(p_full + g, np[g] & 1, abort_flag, &g_chunk_status);
                    if (!ok) continue;
                    ++np[g];
                    tc_fence_after();
                    const uint32_t va = tile_at(L::kRows + sl, kDescV), pa = tm + L::kTS + 128 * g, od = tm + L::kTO + D * g;
                    if constexpr (SPREAD) {
                        if (two) {
                            pv_block<true>(od, pa, va, id_o, k > 0 ? 1u : 0u);
                            pv_block<true>(od, pa + 16, va, id_o, 1u);
                        } else {
                            pv_block<false>(od, pa, va, id_o, k > 0 ? 1u : 0u);
                        }
                    } else {
                        pv_block<false>(od, pa, va, id_o, k > 0 ? 1u : 0u);
                        if (two) pv_block<false>(od, pa + 64, va, id_o, 1u);
                    }
                    if (!duo || g == 1) mma_commit_warp(empty + sl);
                    if (!next) {
                        mma_commit_warp(o_full + g);
                    } else {
                        ok = arrived(keys_of(g, k + 1));
                        if (ok) score(g, k + 1);
                    }
                }
            }
            if (ok && cnt[1] == 0) {  // a single tile: warpgroup 1 has nothing to wait for but the count
                if (items > 0) ok = mbar_wait_warp(o_free + 1, (items - 1) & 1, abort_flag, &g_chunk_status);
                mma_commit_warp(o_full + 1);
            }
            tile0 += take;
            ++items;
        }
        mma_commit_warp(done);
        (void)mbar_wait_warp(done, 0, nullptr, &g_chunk_status);
      }
    } else {
        // --------------------------------------------------------- softmax
        if constexpr (Q8) more_registers<kChSoftmaxRegs>();
        const int g = warp >> 2, row = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + lanes + L::kTS + 128 * g, to = tmem + lanes + L::kTO + D * g;
        const int tok = row / p.G, hh = row - tok * p.G;
        uint32_t tile0 = 0, items = 0, ns = 0, joins = 0;
        bool ok = true;
        const float scale2 = Q8 ? 1.f : p.scale2;  // of the scores as they are read (Q8: the keys' scales have it)
        while (ok && walk.next<ONE, TREE>(p, toks, pc)) {
            const bool two = pc.two;
            const int base_tok = pc.duo ? g * toks : 0;
            const int mytok = base_tok + tok;  // of the item
            const bool valid = tok < toks && mytok < pc.it.tokens;
            const int my_t = pc.r.t0 + pc.it.i0 + mytok, past = pc.r.L - pc.r.n;
            int e = -1, lo = 0;
            if constexpr (TREE) {
                if (valid) e = past - 1, lo = tree_first(p, pc.r, my_t);
            } else {
                if (valid) e = last_seen(p, pc.r, pc.it.i0 + mytok);
                lo = first_seen(p, e);
            }
            const int cnt = pc.duo ? pc.take : (pc.take + 1 - g) / 2;
            float m = -INFINITY, l = 0.f;
            // a thread that takes a value out says so here first (the warpgroups may be a piece apart)
            volatile int* taken_out = misc + 5 + (items & 1);
            for (int k = 0; k < cnt; ++k) {
                const int t = pc.duo ? k : 2 * k + g;
                const int j0 = (pc.it.t0 + pc.off + t) * kChKeys;
                ok = mbar_spin_warp(s_full + g, ns & 1, abort_flag, &g_chunk_status);
                ++ns;
                if (!ok) break;
                tc_fence_after();
                const uint32_t no = miss[(tile0 + t) & 7];
                // Q8: the tile's scales -- of the scores, and of the weights
                const float* kc = scales + ((tile0 + t) & 7) * 384;
                const float* vc = kc + 128;
                float largest = 0.f;  // of the values' scales that the row sees
                if constexpr (BASED) {
                    const float4 x = *reinterpret_cast<const float4*>(scales + 25 * 128 + ((tile0 + t) & 7) * 4);
                    largest = fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w));
                }
                if (j0 < pc.it.lo1 || j0 + kChKeys - 1 > pc.it.e0 || no) {
                    // an edge: scores outside the row's positions become -inf, 32 at a time
                    const int rl = lo - j0, re = e - j0;
                    bool bad = false;
                    if constexpr (BASED) largest = 0.f;
                    uint32_t nodes[5];  // the words with the nodes at the tile's positions
                    if constexpr (TREE)
#pragma unroll
                        for (int i = 0; i < 5; ++i) nodes[i] = valid ? tree_word(p, my_t, pc.r.n, ((j0 - past) >> 5) + i) : 0u;
#pragma unroll 1
                    for (int x = 0; x < 128; x += 32) {
                        uint32_t seen = re >= x + 31 ? ~0u : re < x ? 0u : (2u << (re - x)) - 1u;
                        seen &= rl <= x ? ~0u : rl > x + 31 ? 0u : ~0u << (rl - x);
                        if constexpr (TREE) {  // node k is position past + k
                            seen |= __funnelshift_r(nodes[0], nodes[1], (j0 - past) & 31);
#pragma unroll
                            for (int i = 0; i < 4; ++i) nodes[i] = nodes[i + 1];
                        }
                        if (no) {  // pages that are not there: 2^sh keys a bit
                            const int sh = p.shift < 7 ? p.shift : 7;
                            for (int i = 0; i < 32; i += 8)
                                if ((no >> ((x + i) >> sh)) & 1u) seen &= ~(0xffu << i);
                        }
                        if constexpr (Q8) {
                            // a row that sees a value without a finite scale takes all scales as they are, and
                            // becomes NaN; the others take 0 for such scales
                            if (__ballot_sync(0xffffffffu, !(fabsf(kc[128 + x + lane]) < INFINITY)) & seen) bad = true;
                        } else if (__all_sync(0xffffffffu, seen == ~0u)) {
                            continue;
                        }
                        uint32_t sv[32];
                        tmem_ld32(ts + x, sv);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            if constexpr (Q8) sv[i] = __float_as_uint(__uint_as_float(sv[i]) * kc[x + i]);
                            if constexpr (BASED)
                                if ((seen >> i) & 1u) largest = fmaxf(largest, fabsf(kc[256 + x + i]));
                            if (!((seen >> i) & 1u)) sv[i] = 0xff800000u;
                        }
                        tmem_st32(ts + x, sv);
                    }
                    tmem_wait_st();
                    if constexpr (Q8) {
                        kc = scales + 8 * 384;  // (scaled by now)
                        if (!bad) vc += 128;
                    } else {
                        // values: a thread looks at one key's
                        const int j = j0 + row;
                        const bool none = j < pc.it.lo0 || j > pc.it.e1;  // seen by no row of the item
                        const bool some = !none && (j < pc.it.lo1 || j > pc.it.e0);
                        const uint32_t en = 2 * tile0 + values_at<ONE>(t, pc.take), sl = en % NS;
                        ok = mbar_wait_warp(full + sl, (en / NS) & 1, abort_flag, &g_chunk_status);
                        if (!ok) break;
                        if (none || some) {
                            const uint32_t va = smem_u32(smem + L::kRingOff + sl * L::kTile) + row * 128;
#pragma unroll 4
                            for (int x = 0; x < 8 * L::kSlabs; ++x) {
                                const uint32_t a = va + (x >> 3) * 16384 + (((x & 7) ^ (row & 7)) << 4);
                                if (none) {
                                    asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(a), "r"(0) : "memory");
                                } else {
                                    // (a half whose exponent is all ones has its top bit set after the addition)
                                    const uint4 v = lds_v4(a);
                                    if ((Ty::all_ones(v.x) | Ty::all_ones(v.y) | Ty::all_ones(v.z) | Ty::all_ones(v.w)) &
                                        0x80008000u) {
                                        *taken_out = (int)items + 1;
                                        __threadfence_block();
                                        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a),
                                                     "r"(finite<Ty>(v.x)), "r"(finite<Ty>(v.y)), "r"(finite<Ty>(v.z)),
                                                     "r"(finite<Ty>(v.w))
                                                     : "memory");
                                    }
                                }
                            }
                        }
                    fence_proxy_async_smem();
                    }
                }
                // the row's maximum, 32 scores at a time and the next 32 on their way
                uint32_t sv[2][32];
                tmem_ld32(ts, sv[0]);
                float mx = BASED ? -INFINITY : m, mo = mx;
#pragma unroll(SPREAD ? 1 : 2)
                for (int x0 = 0; x0 < 4; x0 += 2)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int x = x0 + y;
                    tmem_wait_ld();
                    if (x < 3) tmem_ld32(ts + 32 * (x + 1), sv[1 - y]);
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        float2 a = make_float2(__uint_as_float(sv[y][i]), __uint_as_float(sv[y][i + 1]));
                        float2 b = make_float2(__uint_as_float(sv[y][i + 2]), __uint_as_float(sv[y][i + 3]));
                        if constexpr (Q8) {
                            const float4 c = *reinterpret_cast<const float4*>(kc + 32 * x + i);
                            a = mul2(a, make_float2(c.x, c.y));
                            b = mul2(b, make_float2(c.z, c.w));
                        }
                        mx = max3(mx, a.x, a.y);
                        mo = max3(mo, b.x, b.y);
                    }
                }
                mx = fmaxf(mx, mo);
                if constexpr (BASED) mx = fmaxf(m, mx + (scale_log(largest) - kChShift));
                // (rows behind the item's take what shared memory held for queries: they move no neighbour's maximum)
                const bool grew = valid && (mx - m) * scale2 > 8.f;  // also from -inf
                if (__any_sync(0xffffffffu, grew)) {
                    const float f = mx == -INFINITY ? 1.f : power_of_2<BASED>((m - mx) * scale2);
                    l = times<BASED>(l, f);
                    m = mx;
                    if (k > 0) {
                        // all MMAs before this tile's scores are done: nothing adds to O now
#pragma unroll 1
                        for (int i = 0; i < D; i += 16) {
                            uint32_t ov[16];
                            tmem_ld_x16(to + i, ov);
                            tmem_wait_ld();
#pragma unroll
                            for (int x = 0; x < 16; ++x) ov[x] = __float_as_uint(times<BASED>(__uint_as_float(ov[x]), f));
                            tmem_st_x8(to + i, *reinterpret_cast<const uint32_t(*)[8]>(ov));
                            tmem_st_x8(to + i + 8, *reinterpret_cast<const uint32_t(*)[8]>(ov + 8));
                        }
                    }
                }
                const float base = m == -INFINITY ? 0.f : m * scale2;
                // weights: scores 32 x .. become the 16 columns 16 x .., over scores read before
                float2 l0 = make_float2(0.f, 0.f), l1 = l0;
                const float2 sc = make_float2(scale2, scale2), nb = make_float2(-base, -base);
                auto weights = [&](const uint32_t* v, uint32_t* pk) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float2 a = make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
                        a = fma2(a, sc, nb);
                        a.x = exp2_approx(a.x);
                        a.y = exp2_approx(a.y);
                        if (i & 1) l1 = add2(l1, a);
                        else l0 = add2(l0, a);
                        pk[i] = Ty::pack(a.x, a.y);
                    }
                };
                auto second = [&](const uint32_t* v, const uint32_t* pk, uint32_t* pl) {  // what the first parts lack
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float a = exp2_approx(fmaf(__uint_as_float(v[2 * i]), scale2, -base));
                        const float b = exp2_approx(fmaf(__uint_as_float(v[2 * i + 1]), scale2, -base));
                        pl[i] = Ty::pack(a - Ty::lo(pk[i]), b - Ty::hi(pk[i]));
                    }
                };
                if constexpr (Q8) {
                    if (two) {
                        l0 = weights_in_two_parts<Ty>(ts, kc, vc, base);
                    } else {
#pragma unroll 1
                        for (int x = 0; x < 4; ++x) {  // (the next 32 ahead cost more code than they save time: 301 us, 290 so)
                            uint32_t hi[16];
                            tmem_ld32(ts + 32 * x, sv[0]);
                            tmem_wait_ld();
                            scaled_weights<Ty, false>(sv[0], kc + 32 * x, vc + 32 * x, nb, l0, l1, hi, nullptr);
                            tmem_st16(ts + 16 * x, hi);
                        }
                    }
                } else if constexpr (SPREAD) {
#pragma unroll 1
                    for (int x = 0; x < 4; ++x) {
                        uint32_t pk[16], pl[16];
                        tmem_ld32(ts + 32 * x, sv[0]);
                        tmem_wait_ld();
                        weights(sv[0], pk);
                        if (!two) {
                            tmem_st16(ts + 16 * x, pk);
                        } else {
                            second(sv[0], pk, pl);
                            tmem_st16(ts + 32 * x, pk);
                            tmem_st16(ts + 32 * x + 16, pl);
                        }
                    }
                } else {
                tmem_ld32(ts, sv[0]);
                if (!two) {
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        tmem_wait_ld();
                        if (x < 3) tmem_ld32(ts + 32 * (x + 1), sv[(x + 1) & 1]);
                        uint32_t pk[16];
                        weights(sv[x & 1], pk);
                        tmem_st16(ts + 16 * x, pk);
                    }
                } else {
                    // second parts go to columns 64 + 16 x .., once all scores are read
                    uint32_t pk[4][16], pl[4][16];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        tmem_wait_ld();
                        weights(sv[x & 1], pk[x]);
                        second(sv[x & 1], pk[x], pl[x]);
                        if (x < 3) tmem_ld32(ts + 32 * (x + 1), sv[(x + 1) & 1]);
                    }
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        tmem_st16(ts + 16 * x, pk[x]);
                        tmem_st16(ts + 64 + 16 * x, pl[x]);
                    }
                }
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full + g);
                l += (l0.x + l0.y) + (l1.x + l1.y);
            }
            // ---- the item's (or the piece's) result; the warpgroup goes on or gives up together.
            // Warpgroups with rows of their own write them; where they share the rows, each
            // joins both outputs for half of the columns.
            const int g0 = pc.duo ? g : 0;
            if (!pc.duo) {
                // (the last item's are read)
                if (items > 0) ok = ok && mbar_wait_warp(o_free + g, (items - 1) & 1, abort_flag, &g_chunk_status);
                ml[g * 128 + row] = make_float2(m, l);
                __syncwarp();
                if (lane == 0) mbar_arrive(join);
                ok = ok && mbar_wait_warp(join, joins & 1, abort_flag, &g_chunk_status);
                ++joins;
            }
            ok = ok && mbar_wait_warp(o_full + g, items & 1, abort_flag, &g_chunk_status) &&
                 (pc.duo || mbar_wait_warp(o_full + 1 - g, items & 1, abort_flag, &g_chunk_status));
            ok = bar_and(1 + g, 128, ok);
            if (!ok) break;
            float f0 = 1.f, f1 = 0.f;
            const bool other = !pc.duo && pc.take > 1;
            if (!pc.duo) {
                const float2 a = ml[row], o = ml[128 + row];
                m = a.x;
                l = a.y;
                if (other) {
                    const float M = fmaxf(m, o.x), b = M == -INFINITY ? 0.f : M;
                    f0 = power_of_2<BASED>((m - b) * scale2);
                    f1 = power_of_2<BASED>((o.x - b) * scale2);
                    // a sum that is not a number stays one
                    l = (l == 0.f ? 0.f : times<BASED>(l, m == -INFINITY ? 1.f : f0)) +
                        (o.y == 0.f ? 0.f : times<BASED>(o.y, o.x == -INFINITY ? 1.f : f1));
                    m = M;
                }
            }
            auto both = [&](uint32_t x, uint32_t y) {  // both warpgroups' outputs
                return times<BASED>(__uint_as_float(x), f0) + times<BASED>(__uint_as_float(y), f1);
            };
            // (where the other warpgroup took it out of a tile of both, it said so before this one found it gone)
            const bool odd = !bar_and(1 + g, 128, *taken_out != (int)items + 1);
            const uint32_t toa = tmem + lanes + L::kTO + D * g0, tob = toa + D;
            const int x0 = pc.duo ? 0 : g * (D / 2), x1 = pc.duo ? D : x0 + D / 2;  // columns
            tc_fence_after();
            const bool whole = pc.off == 0 && pc.take == pc.it.tiles;
            const int64_t t = pc.r.t0 + pc.it.i0 + mytok;
            const int h = pc.hk * p.G + hh;
            uint16_t* out = p.out + t * p.o_token + (int64_t)h * p.o_head;
            // the CTAs that share the item, and where CTA i keeps its piece of this row tile
            int c0 = c, c1 = c;
            unsigned* counter = nullptr;
            if (!whole) {
                sharers(pc.first, pc.it.tiles, c0, c1);
                counter = p.counters + kChCounters + 2 * c0 + g;
            }
            auto piece = [&](int i) { return p.part + ((int64_t)(2 * i + (i == c0)) * 2 + g) * L::kPartHalf; };
            // a piece's sums (>= 0, or NaN) carry in their sign whether values were taken out
            const float mine_m = m * scale2, mine_l = __uint_as_float(__float_as_uint(l) | (odd ? 0x80000000u : 0u));
            // Where all other pieces are there already, this one need not be written:
            // it goes into the sum from tensor memory, in its place of the order.
            bool last = whole, kept = true;  // kept: this piece's output is still in tensor memory only
            if (!whole) {
                bool all = true;
                if (row == 0) {
                    unsigned n;
                    asm volatile("ld.acquire.gpu.u32 %0, [%1];" : "=r"(n) : "l"(counter) : "memory");
                    all = n == (unsigned)(c1 - c0);
                    if (all) *counter = 0;
                }
                last = bar_and(1 + g, 128, all);
                if (!last) {
                    kept = false;
                    float* part = piece(c);
#pragma unroll 1
                    for (int i = x0; i < x1; i += 32) {
                        uint32_t ov[32];
                        tmem_ld32(toa + i, ov);
                        tmem_wait_ld();
                        if (other) {
                            uint32_t ow[32];
                            tmem_ld32(tob + i, ow);
                            tmem_wait_ld();
#pragma unroll
                            for (int x = 0; x < 32; ++x)
                                ov[x] = __float_as_uint(both(ov[x], ow[x]));
                        }
                        if (valid)
#pragma unroll
                        for (int x = 0; x < 32; x += 4)  // [column / 4][row]: neighbours write neighbours
                            *reinterpret_cast<uint4*>(part + 256 + (((i + x) >> 2) * 128 + row) * 4) =
                                make_uint4(ov[x], ov[x + 1], ov[x + 2], ov[x + 3]);
                    }
                    reinterpret_cast<float2*>(part)[row] = make_float2(mine_m, mine_l);
                    named_bar(1 + g, 128);
                    bool is_last = true;
                    if (row == 0) {
                        __threadfence();  // the warpgroup's stores, ordered before by the barrier
                        is_last = atomicAdd(counter, 1u) == (unsigned)(c1 - c0);
                        if (is_last) *counter = 0;
                        __threadfence();
                    }
                    last = bar_and(1 + g, 128, is_last);
                }
            }
            bool again = odd;  // values to add
            float S = l;
            if (last) {
                float M = m * scale2;
                auto put = [&](int x, const float* acc) {  // 8 columns
                    const float w = S == 0.f ? 0.f : 1.f / S;
                    *reinterpret_cast<uint4*>(out + x) =
                        S == 0.f ? make_uint4(0u, 0u, 0u, 0u)
                                 : make_uint4(Ty::pack(acc[0] * w, acc[1] * w), Ty::pack(acc[2] * w, acc[3] * w),
                                              Ty::pack(acc[4] * w, acc[5] * w), Ty::pack(acc[6] * w, acc[7] * w));
                };
                if (whole) {
#pragma unroll 1
                    for (int x = x0; x < x1; x += 32) {
                        uint32_t ov[32];
                        float acc[32];
                        tmem_ld32(toa + x, ov);
                        tmem_wait_ld();
                        if (other) {
                            uint32_t ow[32];
                            tmem_ld32(tob + x, ow);
                            tmem_wait_ld();
#pragma unroll
                            for (int y = 0; y < 32; ++y)
                                ov[y] = __float_as_uint(both(ov[y], ow[y]));
                        }
#pragma unroll
                        for (int y = 0; y < 32; ++y) acc[y] = __uint_as_float(ov[y]) + 0.f;  // (-0 becomes 0)
                        if (valid)
#pragma unroll
                            for (int y = 0; y < 32; y += 8) put(x + y, acc + y);
                        __syncwarp();
                    }
                } else {
                    // 16 columns at a time, of four pieces in flight (32 of one piece: 34 us for 13 tokens over 2303
                    // positions, whose 19 pieces come one after the other then), under a running maximum, so that
                    // nothing waits for the maxima of all (a microsecond more with a pass over these before)
                    bool bad = false;
#pragma unroll 1
                    for (int x = x0; x < x1; x += 16) {
                        float acc[16];
#pragma unroll
                        for (int y = 0; y < 16; ++y) acc[y] = 0.f;
                        M = -INFINITY;
                        S = 0.f;
#pragma unroll 1
                        for (int i0 = c0; i0 <= c1; i0 += 4) {
                            float4 v[4][4];
                            float2 mi[4];
                            float fs[4];
#pragma unroll
                            for (int u = 0; u < 4; ++u) {  // (all on their way before any is waited for)
                                const int i = i0 + u;
                                const bool there = i <= c1 && !(i == c && kept) && valid;
                                const float* q = piece(there ? i : c0);
                                mi[u] = there                 ? __ldcg(reinterpret_cast<const float2*>(q) + row)
                                        : i == c && kept ? make_float2(mine_m, mine_l)
                                                         : make_float2(-INFINITY, 0.f);
#pragma unroll
                                for (int y = 0; y < 4; ++y)
                                    v[u][y] = there ? __ldcg(reinterpret_cast<const float4*>(q + 256) + ((x >> 2) + y) * 128 + row)
                                                    : make_float4(0.f, 0.f, 0.f, 0.f);
                            }
                            const float before = M;
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                bad |= __float_as_uint(mi[u].y) >> 31;
                                M = fmaxf(M, mi[u].x);
                            }
                            const float b = M == -INFINITY ? 0.f : M;
                            if (i0 != c0) {
                                const float f = power_of_2<BASED>(before == -INFINITY ? 0.f : before - b);
                                S = times<BASED>(S, f);
#pragma unroll
                                for (int y = 0; y < 16; ++y) acc[y] = times<BASED>(acc[y], f);
                            }
#pragma unroll
                            for (int u = 0; u < 4; ++u) {  // no seen key: zeros
                                fs[u] = mi[u].y == 0.f ? 0.f : power_of_2<BASED>(mi[u].x == -INFINITY ? 0.f : mi[u].x - b);
                                if (mi[u].y != 0.f) S = add_times<BASED>(fabsf(mi[u].y), fs[u], S);
                            }
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                if (i0 + u == c && kept) {  // this piece's, by every lane: tensor-memory loads are the warp's
                                    uint32_t ov[16];
                                    tmem_ld_x16(toa + x, ov);
                                    tmem_wait_ld();
                                    if (other) {
                                        uint32_t ow[16];
                                        tmem_ld_x16(tob + x, ow);
                                        tmem_wait_ld();
#pragma unroll
                                        for (int y = 0; y < 16; ++y)
                                            ov[y] = __float_as_uint(both(ov[y], ow[y]));
                                    }
#pragma unroll
                                    for (int y = 0; y < 16; ++y) acc[y] = add_times<BASED>(__uint_as_float(ov[y]), fs[u], acc[y]);
                                } else {
#pragma unroll
                                    for (int y = 0; y < 4; ++y) {
                                        acc[4 * y] = add_times<BASED>(v[u][y].x, fs[u], acc[4 * y]);
                                        acc[4 * y + 1] = add_times<BASED>(v[u][y].y, fs[u], acc[4 * y + 1]);
                                        acc[4 * y + 2] = add_times<BASED>(v[u][y].z, fs[u], acc[4 * y + 2]);
                                        acc[4 * y + 3] = add_times<BASED>(v[u][y].w, fs[u], acc[4 * y + 3]);
                                    }
                                }
                            }
                        }
                        if (valid) {
                            put(x, acc);
                            put(x + 8, acc + 8);
                        }
                        __syncwarp();
                    }
                    again = !bar_and(1 + g, 128, !bad);
                }
                if (valid && p.lse && x0 == 0) p.lse[t * p.Hq + h] = S == 0.f ? -INFINITY : kLn2 * (M + log2f(S));
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(o_free + g);
                mbar_arrive(o_free + (pc.duo ? g : 1 - g));
            }
            if constexpr (!Q8)
                if (again && last && valid && S != 0.f) add_taken_out<Ty, TREE>(p, pc, my_t, lo, e, out, x0, x1);
            tile0 += pc.take;
            ++items;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (p.after_small) pdl_wait();  // the call is done when both kernels are
}

template <typename Ty, int D, bool ONE, bool TREE, bool Q8>
static cudaError_t launch(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const PagedAttnParams& p,
                          int ctas, cudaStream_t s, bool pdl) {
    static bool set_for[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    auto kernel = paged_chunk_kernel<Ty, D, ONE, TREE, Q8>;
    constexpr int smem = Ch<D, ONE, Q8>::kSmem;
    if (!set_for[dev]) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        set_for[dev] = true;
    }
    return launch_kernel(kernel, dim3(ctas), dim3(kChThreads<Q8>), (size_t)smem, s, pdl, tq, tk, tv, p);
}

template <typename Ty, int D, bool TREE, bool Q8>
static cudaError_t launch(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const PagedAttnParams& p,
                          bool one, int ctas, cudaStream_t s, bool pdl) {
    return one ? launch<Ty, D, true, TREE, Q8>(tq, tk, tv, p, ctas, s, pdl)
               : launch<Ty, D, false, TREE, Q8>(tq, tk, tv, p, ctas, s, pdl);
}

template <bool TREE, bool Q8>
cudaError_t launch_paged_chunk(const PagedAttnParams& p, bool bf16, int d, bool one, int sms, cudaStream_t s, bool pdl) {
    CUtensorMap tq, tk, tv;
    const int box = (1 << p.shift) < kChKeys ? 1 << p.shift : kChKeys;
    if (!paged_tmap(&tk, p, bf16, Q8, d, false, box) || !paged_tmap(&tv, p, bf16, Q8, d, true, box) ||
        !query_tmap(&tq, p, bf16, d, 128 / p.G))
        return cudaErrorInvalidValue;
    if (bf16)
        return d == 128 ? launch<Bf16, 128, TREE, Q8>(tq, tk, tv, p, one, sms, s, pdl)
                        : launch<Bf16, 64, TREE, Q8>(tq, tk, tv, p, one, sms, s, pdl);
    return d == 128 ? launch<F16, 128, TREE, Q8>(tq, tk, tv, p, one, sms, s, pdl)
                    : launch<F16, 64, TREE, Q8>(tq, tk, tv, p, one, sms, s, pdl);
}

template <bool TREE, bool Q8>
int paged_chunk_status() {
    int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_chunk_status, sizeof(int)) != cudaSuccess) return W4A16_ECUDA;
    if (cudaMemcpyToSymbol(g_chunk_status, &zero, sizeof(int)) != cudaSuccess) return W4A16_ECUDA;
    return v;
}

}  // namespace w4a16
