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
// Measured: 64 decoding requests 4.8 us, 2048 requests, an eighth of them with
// up to 2048 new tokens (5.4 MB in and out), 8.2 us; called one by one from the
// host 7.2 and 9.5 us.
#include "common.cuh"
#include "kernels.h"

namespace w4a16 {

constexpr int kPlanThreads = 512;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kPlanRun = 4;  // tokens a lane takes per warp pass, 32 apart

// exclusive sums of two ints over the CTA's threads, and their totals
W4A16_DEVICE void plan_scan(int a, int f, int* sa, int* sf, int& ea, int& ef) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int ia = a, jf = f;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, ia, d), y = __shfl_up_sync(0xffffffffu, jf, d);
        if (lane >= d) {
            ia += x;
            jf += y;
        }
    }
    if (lane == 31) {
        sa[warp] = ia;
        sf[warp] = jf;
    }
    __syncthreads();
    int ba = 0, bf = 0;
    for (int w = 0; w < warp; ++w) {
        ba += sa[w];
        bf += sf[w];
    }
    ea = ba + ia - a;
    ef = bf + jf - f;
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
        const int past = max(p.past_len[b], 0), n = max(p.new_len[b], 0);
        qs[b] = n;
        fs[b] = ((past + n + page - 1) >> shift) - ((past + page - 1) >> shift);
    }
    __syncthreads();
    int a = 0, f = 0;
    const int b0 = min((int)threadIdx.x * per, B), b1 = min(b0 + per, B);
    for (int b = b0; b < b1; ++b) {
        a += qs[b];
        f += fs[b];
    }
    int ea, ef;
    plan_scan(a, f, sa, sf, ea, ef);
    for (int b = b0; b < b1; ++b) {
        const int n = qs[b], m = fs[b];
        qs[b] = ea;
        fs[b] = ef;
        ea += n;
        ef += m;
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
        const int past = max(p.past_len[b], 0), n = qs[b + 1] - qs[b];
        const int held = (past + page - 1) >> shift, need = (past + n + page - 1) >> shift;
        if (lane == 0) {
            p.q_start[b] = qs[b];
            p.kv_len[b] = past + n;
        }
        int* row = p.block_table + (int64_t)b * p.table_stride;
        for (int c = held + lane; c < p.columns; c += 32) {
            const int at = fs[b] + c - held;
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
                const int past = max(p.past_len[lo], 0);
                pos = past + ((int)t - qs[lo]);
                const int held = (past + page - 1) >> shift, c = pos >> shift;
                int entry = -1;
                if (c < p.columns) {
                    if (c < held) {
                        entry = p.block_table[(int64_t)lo * p.table_stride + c];
                    } else {
                        const int at = fs[lo] + c - held;
                        if (at < p.num_free) entry = p.free_pages[at];
                    }
                }
                if (entry >= 0) slot = (entry << shift) + (pos & (page - 1));
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
