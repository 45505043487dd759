// Pages and slots for the new tokens of a batch of requests (definition: q4k.h).
//
// Every step of the definition is a running sum over requests: tokens up to T, pages that come back, pages that are
// lacking against what the list holds, then the granted ones.  One CTA makes them (scan_requests), a thread taking a
// run of consecutive requests, so a sum is one block-wide scan of the threads' totals.  What is left is independent
// per token and per page (fill): a token finds its request by bisection of starts; the j-th page taken is entry
// there - 1 - j of the list as it stands after the returns, which is either an old entry or, found by bisection, one
// that another request has just given back, so nothing waits for the list to be written.
// Bound by latency: some tens of bytes a request, twelve a token.  A small batch runs in one CTA; a larger
// one fills with a second launch over the whole GPU.
#include <cuda_runtime.h>

#include "decode_ops.h"
#include "q4k_ptx.cuh"

namespace q4k {
namespace {

constexpr int kThreads = 1024;
constexpr int kFillThreads = 256;
// What the scanning CTA fills itself, at most: tokens, and table entries that may change hands.
constexpr int64_t kSmallTokens = 8192, kSmallPages = 1 << 17;

// Exclusive prefix of v over the CTA's threads; `total` receives the sum.  Every thread calls it.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t &total, int64_t *scratch) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t sum = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t t = __shfl_up_sync(0xFFFFFFFFu, sum, o);
        if (lane >= o) sum += t;
    }
    if (lane == 31) scratch[warp] = sum;
    __syncthreads();
    int64_t of = lane < kThreads / 32 ? scratch[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t t = __shfl_up_sync(0xFFFFFFFFu, of, o);
        if (lane >= o) of += t;
    }
    total = __shfl_sync(0xFFFFFFFFu, of, 31);
    const int64_t before = __shfl_sync(0xFFFFFFFFu, of, warp > 0 ? warp - 1 : 0);
    __syncthreads();  // scratch is free for the next scan
    return sum - v + (warp > 0 ? before : 0);
}

// ceil(slots / page_size) for 0 <= slots < 2^31
__device__ __forceinline__ int pages_for(const KvView &c, int64_t slots) {
    return slots > 0 ? (int)page_of(c, (uint32_t)(slots - 1)) + 1 : 0;
}

struct Request {
    int64_t len, tokens;  // tokens that would fit into its pages
    int held;
    bool over;
};

__device__ __forceinline__ Request request(const PlanArgs &a, int b, unsigned &bad) {
    Request r;
    const int len = __ldg(a.seq_lens + b), held = __ldg(a.held + b), n = __ldg(a.n_new + b);
    r.len = min(max(len, 0), a.c.capacity);
    r.held = min(max(held, 0), a.c.max_pages);
    r.over = n < 0;
    r.tokens = n > 0 ? n : 0;
    if (r.len != len || r.held != held) bad = 1;
    if (r.len + r.tokens > a.c.capacity) r.tokens = 0, bad = 1;
    return r;
}

// All sums of the definition; writes what a request has, and for fill() the running sums of pages returned and taken.
__device__ __forceinline__ void scan_requests(const PlanArgs &a) {
    __shared__ int64_t scratch[32];
    const int B = a.c.batch, per = (B + kThreads - 1) / kThreads;
    const int first = min((int)threadIdx.x * per, B), last = min(first + per, B);
    unsigned bad = 0;
    const int count0 = __ldg(a.free_count), count = min(max(count0, 0), (int)a.c.n_pages);
    if (count != count0) bad = 1;
    int64_t asked = 0, all;
    for (int b = first; b < last; ++b) asked += request(a, b, bad).tokens;
    asked = block_scan(asked, all, scratch);
    // pages, with the tokens that stay below T
    int64_t run = asked, back = 0, lack = 0;
    auto pages = [&](const Request &r, int64_t &tokens, int &want) {
        run += r.tokens;
        tokens = run <= a.T ? r.tokens : 0;
        want = r.over ? 0 : pages_for(a.c, r.len + tokens);
    };
    for (int b = first; b < last; ++b) {
        const Request r = request(a, b, bad);
        int64_t tokens;
        int want;
        pages(r, tokens, want);
        if (want < r.held) back += r.held - want;
        else lack += want - r.held;
    }
    int64_t all_back, all_lack;
    const int64_t back0 = block_scan(back, all_back, scratch), lack0 = block_scan(lack, all_lack, scratch);
    int64_t there = count + all_back;
    if (there > a.c.n_pages) there = a.c.n_pages, bad = 1;
    // what is granted
    run = asked;
    int64_t lacking = lack0, tokens_in = 0, taken = 0;
    auto grant = [&](const Request &r, int64_t &tokens, int &want, int &take) {
        pages(r, tokens, want);
        take = 0;
        if (want > r.held) {
            lacking += want - r.held;
            if (lacking <= there) take = want - r.held;
            else tokens = 0, want = r.held;
        }
    };
    for (int b = first; b < last; ++b) {
        const Request r = request(a, b, bad);
        int64_t tokens;
        int want, take;
        grant(r, tokens, want, take);
        tokens_in += tokens;
        taken += take;
    }
    int64_t all_tokens, all_taken;
    tokens_in = block_scan(tokens_in, all_tokens, scratch);
    taken = block_scan(taken, all_taken, scratch);
    run = asked, lacking = lack0, back = back0;
    for (int b = first; b < last; ++b) {
        const Request r = request(a, b, bad);
        int64_t tokens;
        int want, take;
        grant(r, tokens, want, take);
        a.starts[b] = (int)tokens_in;
        a.back_at[b] = (int)min(back, (int64_t)INT32_MAX);
        a.take_at[b] = (int)taken;
        if (want < r.held) back += r.held - want;
        tokens_in += tokens;
        taken += take;
        // (last: they may be the arrays that request() reads, each by its own thread)
        a.held_out[b] = want;
        a.after_lens[b] = r.over ? 0 : (int)(r.len + tokens);
    }
    if (threadIdx.x == 0) {
        a.starts[B] = (int)all_tokens;
        a.back_at[B] = (int)min(all_back, (int64_t)INT32_MAX);
        a.take_at[B] = (int)all_taken;
        a.list[0] = count;
        a.list[1] = (int)there;
        *a.count_out = (int)(there - all_taken);
    }
    if (bad) atomicOr(a.c.status, kDevIndex);
}

// The last b in [0, n) with at[b] <= v (at does not decrease, at[0] <= v): the one whose range holds v.
template <typename Load>
__device__ __forceinline__ int find(int n, int v, Load &&at) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (at(mid) <= v) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Thread `id` of `threads`: its tokens and pages.  Plain loads: the scan may have written these in the same kernel.
__device__ __forceinline__ void fill(const PlanArgs &a, int64_t id, int64_t threads) {
    const int B = a.c.batch, tokens = a.starts[B];
    for (int64_t t = id; t < a.T; t += threads) {
        int seq = -1, slot = 0, pos = 0;
        if (t < tokens) {
            seq = find(B, (int)t, [&](int b) { return a.starts[b]; });
            const int begin = a.starts[seq], i = (int)t - begin;
            slot = a.after_lens[seq] - (a.starts[seq + 1] - begin) + i;
            pos = a.first_pos ? __ldg(a.first_pos + seq) + i : slot;
        }
        a.seq[t] = seq, a.slot[t] = slot, a.pos[t] = pos;
    }
    const int count = a.list[0], there = a.list[1], back = a.back_at[B], taken = a.take_at[B];
    bool bad = false;
    // page r of those returned
    auto returned = [&](int r) {
        const int b = find(B, r, [&](int i) { return a.back_at[i]; });
        return a.table[b * a.c.ld_table + a.held_out[b] + (r - a.back_at[b])];
    };
    for (int64_t r = id; r < back; r += threads) {
        if (count + r >= there) continue;  // no room
        const int page = returned((int)r);
        bad |= !page_ok(a.c, page);
        a.free_pages[count + r] = page;
    }
    for (int64_t j = id; j < taken; j += threads) {
        const int from = there - 1 - (int)j;
        const int page = from >= count ? returned(from - count) : a.free_pages[from];
        const int b = find(B, (int)j, [&](int i) { return a.take_at[i]; });
        const int take = a.take_at[b + 1] - a.take_at[b];
        bad |= !page_ok(a.c, page);
        a.table[b * a.c.ld_table + a.held_out[b] - take + ((int)j - a.take_at[b])] = page;
    }
    if (bad) atomicOr(a.c.status, kDevIndex);
}

template <bool FILL>
__global__ void __launch_bounds__(kThreads) plan_kernel(const PlanArgs a) {
    pdl_wait();
    pdl_trigger();
    scan_requests(a);
    if constexpr (FILL) {
        __syncthreads();  // its writes are seen by the CTA
        fill(a, threadIdx.x, kThreads);
    }
}

__global__ void __launch_bounds__(kFillThreads) plan_fill_kernel(const PlanArgs a) {
    pdl_wait();
    pdl_trigger();
    fill(a, (int64_t)blockIdx.x * kFillThreads + threadIdx.x, (int64_t)gridDim.x * kFillThreads);
}

}  // namespace

cudaError_t launch_batch_plan(const DeviceInfo &di, const PlanArgs &a, cudaStream_t s) {
    if (a.T <= kSmallTokens && (int64_t)a.c.batch * a.c.max_pages <= kSmallPages)
        return launch_pdl(plan_kernel<true>, dim3(1), dim3(kThreads), 0, s, dim3(1), a);
    const cudaError_t e = launch_pdl(plan_kernel<false>, dim3(1), dim3(kThreads), 0, s, dim3(1), a);
    if (e != cudaSuccess) return e;
    int64_t ctas = (a.T + 2 * kFillThreads - 1) / (2 * kFillThreads);
    const int64_t most = (int64_t)di.sm_count * 8;
    if (ctas > most) ctas = most;
    return launch_pdl(plan_fill_kernel, dim3((unsigned)ctas), dim3(kFillThreads), 0, s, dim3(1), a);
}

}  // namespace q4k
