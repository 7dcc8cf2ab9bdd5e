// Block tables, slot map and positions of a serving step, from the requests'
// lengths, in one launch.
//
//     held_b = ceil(past_b / p), need_b = ceil((past_b + new_b) / p)
//     q_start = exclusive sum of new, first = exclusive sum of need - held
//     entry(b, c) = table[b][c] (c < held_b) | free[first_b + c - held_b] | -1
//     slot(t) = entry(b, pos / p) p + pos % p
//
// Both sums run over at most 16384 requests, so every CTA computes them for
// itself in shared memory (8 bytes a request, read from L2) instead of waiting
// for another: one launch, no hand-off between CTAs.  A token's page comes
// from the lengths and the free list, never from an entry that another CTA
// writes in this launch.  Bound: launch and a chain of two dependent loads.
// Measured: 64 decoding requests 4.2 us, 2048 requests, an eighth of them with
// up to 2048 new tokens (5.4 MB in and out), 7.8 us; called one by one from the
// host 6.9 and 9.8 us.
#include "common.cuh"
#include "kernels.h"

namespace w4a16 {

constexpr int kPlanThreads = 512;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPlanRun = 4;  // tokens a lane takes per warp pass, 32 apart

// Lengths come from memory, so no sum of them may wrap into an index: sums of
// numbers >= 0 stop at INT_MAX (in any order of addition), which is past every
// token and free page.
W4A16_DEVICE int add_up(int a, int b) { return (int)min((unsigned)a + (unsigned)b, 0x7fffffffu); }
// a request's tokens in the cache and new ones: >= 0, together INT_MAX at most
struct PlanLengths {
    int past, n;
    W4A16_DEVICE PlanLengths(const w4a16_page_plan_args& p, int b) {
        past = max(p.past_len[b], 0);
        n = min(max(p.new_len[b], 0), 0x7fffffff - past);
    }
};
W4A16_DEVICE int pages_of(int tokens, int shift) { return (tokens >> shift) + ((tokens & ((1 << shift) - 1)) != 0); }

// exclusive sums of two ints >= 0 over the CTA's threads
W4A16_DEVICE void plan_scan(int a, int f, int* sa, int* sf, int& ea, int& ef) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int ia = a, jf = f;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, ia, d), y = __shfl_up_sync(0xffffffffu, jf, d);
        if (lane >= d) {
            ia = add_up(ia, x);
            jf = add_up(jf, y);
        }
    }
    if (lane == 31) {
        sa[warp] = ia;
        sf[warp] = jf;
    }
    __syncthreads();
    const int xa = __shfl_up_sync(0xffffffffu, ia, 1), xf = __shfl_up_sync(0xffffffffu, jf, 1);
    ea = lane ? xa : 0;
    ef = lane ? xf : 0;
    for (int w = 0; w < warp; ++w) {
        ea = add_up(ea, sa[w]);
        ef = add_up(ef, sf[w]);
    }
}

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const w4a16_page_plan_args p, const int shift) {
    extern __shared__ int plan_smem[];
    const int B = p.requests, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int* qs = plan_smem;       // [B + 1] first token of each request
    int* fs = qs + B + 1;      // [B + 1] first free page of each request
    __shared__ int sa[kPlanWarps], sf[kPlanWarps];
    const int page = 1 << shift;
    // In this order: with the next launch let go before the wait, several waiting
    // kernels queue up behind one another; a host that launches about as fast as the
    // kernel runs (2048 requests) then saw 15 us a call instead of 9.5.
    pdl_wait();
    pdl_launch_dependents();

    // the two sums: thread i takes the requests [i * per, i * per + per)
    const int per = (B + kPlanThreads - 1) / kPlanThreads;
    for (int b = threadIdx.x; b < B; b += kPlanThreads) {
        const PlanLengths l(p, b);
        qs[b] = l.n;
        fs[b] = pages_of(l.past + l.n, shift) - pages_of(l.past, shift);
    }
    __syncthreads();
    int a = 0, f = 0;
    const int b0 = min((int)threadIdx.x * per, B), b1 = min(b0 + per, B);
    for (int b = b0; b < b1; ++b) {
        a = add_up(a, qs[b]);
        f = add_up(f, fs[b]);
    }
    int ea, ef;
    plan_scan(a, f, sa, sf, ea, ef);
    for (int b = b0; b < b1; ++b) {
        const int n = qs[b], m = fs[b];
        qs[b] = ea;
        fs[b] = ef;
        ea = add_up(ea, n);
        ef = add_up(ef, m);
    }
    if (threadIdx.x == kPlanThreads - 1) {
        qs[B] = ea;
        fs[B] = ef;
    }
    __syncthreads();
    const int total = qs[B];

    // per request: lengths, and the entries past the pages held (a warp a row)
    const int gw = blockIdx.x * kPlanWarps + warp, nw = gridDim.x * kPlanWarps;
    for (int b = gw; b < B; b += nw) {
        const PlanLengths l(p, b);
        const int held = pages_of(l.past, shift), need = pages_of(l.past + l.n, shift);
        if (lane == 0) {
            p.q_start[b] = qs[b];
            p.kv_len[b] = l.past + l.n;
        }
        int* row = p.block_table + (int64_t)b * p.table_stride;
        for (int64_t c = held + lane; c < p.columns; c += 32) {
            const int64_t at = fs[b] + c - held;
            row[c] = c < need && at < p.num_free ? p.free_pages[at] : -1;
        }
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        p.q_start[B] = total;
        p.pages_used[0] = fs[B];
    }

    // per token: its request by bisection over the first tokens
    for (int64_t t0 = (int64_t)gw * (32 * kPlanRun); t0 < p.tokens; t0 += (int64_t)nw * (32 * kPlanRun)) {
#pragma unroll
        for (int u = 0; u < kPlanRun; ++u) {
            const int64_t t = t0 + 32 * u + lane;
            if (t >= p.tokens) break;
            int pos = -1, slot = -1;
            if (t < total) {
                int lo = 0, hi = B;  // the last request that starts at or before t
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (qs[mid] <= (int)t) lo = mid; else hi = mid;
                }
                const PlanLengths l(p, lo);
                const int held = pages_of(l.past, shift);
                pos = l.past + ((int)t - qs[lo]);  // (t is below the next request's first token: pos < past + n)
                const int c = pos >> shift;
                int entry = -1;
                if (c < p.columns) {
                    if (c < held) {
                        entry = p.block_table[(int64_t)lo * p.table_stride + c];
                    } else {
                        const int64_t at = (int64_t)fs[lo] + c - held;
                        if (at < p.num_free) entry = p.free_pages[at];
                    }
                }
                if (entry >= 0 && entry <= (0x7fffffff >> shift)) slot = (entry << shift) + (pos & (page - 1));
            }
            p.positions[t] = pos;
            p.slot_map[t] = slot;
        }
    }
}

cudaError_t launch_page_plan(const w4a16_page_plan_args& a, int sms, cudaStream_t s) {
    int shift = 0;
    while ((1 << shift) < a.page_size) ++shift;
    const size_t smem = 2 * ((size_t)a.requests + 1) * sizeof(int);
    static bool set_for[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!set_for[dev]) {
        e = cudaFuncSetAttribute(page_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 2 * (kPlanMaxRequests + 1) * (int)sizeof(int));
        if (e != cudaSuccess) return e;
        set_for[dev] = true;
    }
    // a warp per request or per 128 tokens, up to one CTA an SM: every CTA repeats the sums
    const int64_t warps = a.tokens / (32 * kPlanRun) + 1 > a.requests ? a.tokens / (32 * kPlanRun) + 1 : a.requests;
    int64_t ctas = (warps + kPlanWarps - 1) / kPlanWarps;
    if (ctas > sms) ctas = sms;
    return launch_kernel(page_plan_kernel, dim3((unsigned)ctas), dim3(kPlanThreads), smem, s,
                         (a.flags & W4A16_FLAG_PDL) != 0, a, shift);
}

}  // namespace w4a16
