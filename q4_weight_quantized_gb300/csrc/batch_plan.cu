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
// Measured: 64 requests with a token each 7.6 us (four scans and three rounds of loads, one after the other); 256 requests
// with 0 to 509 tokens 10.5 us, two launches (13.5 with the sums bisected in global memory, a token a thread).
#include <cuda_runtime.h>

#include "decode_ops.h"
#include "q4k_ptx.cuh"

namespace q4k {
namespace {

constexpr int kThreads = 1024;
constexpr int kFillThreads = 256;
constexpr int kShared = 2048;
// What the scanning CTA fills itself, at most: tokens, and table entries that may change hands.
constexpr int64_t kSmallTokens = 8192, kSmallPages = 1 << 17;

struct Pair {
    int64_t x, y;
    __device__ __forceinline__ Pair operator+(const Pair &o) const { return {x + o.x, y + o.y}; }
};

// Exclusive prefix of v over the CTA's threads; `total` receives the sum.  Every thread calls it; two scratch arrays in turn.
__device__ __forceinline__ Pair block_scan(Pair v, Pair &total, Pair (*scratches)[32], int &turn) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto up = [](Pair p, int o) { return Pair{__shfl_up_sync(0xFFFFFFFFu, p.x, o), __shfl_up_sync(0xFFFFFFFFu, p.y, o)}; };
    Pair *const scratch = scratches[turn];
    turn ^= 1;
    Pair sum = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Pair t = up(sum, o);
        if (lane >= o) sum = sum + t;
    }
    if (lane == 31) scratch[warp] = sum;
    __syncthreads();
    Pair of = lane < (int)blockDim.x / 32 ? scratch[lane] : Pair{0, 0};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Pair t = up(of, o);
        if (lane >= o) of = of + t;
    }
    total = {__shfl_sync(0xFFFFFFFFu, of.x, 31), __shfl_sync(0xFFFFFFFFu, of.y, 31)};
    const int from = warp > 0 ? warp - 1 : 0;
    const Pair before = {__shfl_sync(0xFFFFFFFFu, of.x, from), __shfl_sync(0xFFFFFFFFu, of.y, from)};
    return {sum.x - v.x + (warp > 0 ? before.x : 0), sum.y - v.y + (warp > 0 ? before.y : 0)};
}

// ceil(slots / page_size) for 0 <= slots < 2^31
__device__ __forceinline__ int pages_for(const KvView &c, int64_t slots) {
    return slots > 0 ? (int)page_of(c, (uint32_t)(slots - 1)) + 1 : 0;
}

// The running sums of a batch of few requests.
struct Sums {
    int starts[kShared + 1], back_at[kShared + 1], take_at[kShared + 1], list[2];
};

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
// (sums: the running sums in shared memory, too, or null.)
__device__ __forceinline__ void scan_requests(const PlanArgs &a, Sums *sums) {
    __shared__ Pair scratch[2][32];
    int turn = 0;
    const int B = a.c.batch, per = (B + (int)blockDim.x - 1) / (int)blockDim.x;
    const int first = min((int)threadIdx.x * per, B), last = min(first + per, B);
    unsigned bad = 0;
    const int count0 = __ldg(a.free_count), count = min(max(count0, 0), (int)a.c.n_pages);
    if (count != count0) bad = 1;
    Pair all;
    int64_t asked = 0;
    for (int b = first; b < last; ++b) asked += request(a, b, bad).tokens;
    asked = block_scan({asked, 0}, all, scratch, turn).x;
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
    const Pair before = block_scan({back, lack}, all, scratch, turn);
    const int64_t all_back = all.x, back0 = before.x, lack0 = before.y;
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
    const Pair in = block_scan({tokens_in, taken}, all, scratch, turn);
    const int64_t all_tokens = all.x, all_taken = all.y;
    tokens_in = in.x, taken = in.y;
    run = asked, lacking = lack0, back = back0;
    for (int b = first; b < last; ++b) {
        const Request r = request(a, b, bad);
        int64_t tokens;
        int want, take;
        grant(r, tokens, want, take);
        const int at[3] = {(int)tokens_in, (int)min(back, (int64_t)INT32_MAX), (int)taken};
        a.starts[b] = at[0];
        if (sums) sums->starts[b] = at[0], sums->back_at[b] = at[1], sums->take_at[b] = at[2];
        else a.back_at[b] = at[1], a.take_at[b] = at[2];
        if (want < r.held) back += r.held - want;
        tokens_in += tokens;
        taken += take;
        // (last: they may be the arrays that request() reads, each by its own thread)
        a.held_out[b] = want;
        a.after_lens[b] = r.over ? 0 : (int)(r.len + tokens);
    }
    if (threadIdx.x == 0) {
        const int at[3] = {(int)all_tokens, (int)min(all_back, (int64_t)INT32_MAX), (int)all_taken};
        a.starts[B] = at[0];
        if (sums) {
            sums->starts[B] = at[0], sums->back_at[B] = at[1], sums->take_at[B] = at[2];
            sums->list[0] = count, sums->list[1] = (int)there;
        } else {
            a.back_at[B] = at[1], a.take_at[B] = at[2];
            a.list[0] = count, a.list[1] = (int)there;
        }
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

// Thread `id` of `threads`: its tokens and pages.  Plain loads: the scan may have written these in the same kernel.  The running
// sums of few requests lie in shared memory (bisection over L2 takes ten of its latencies).
__device__ __forceinline__ void fill(const PlanArgs &a, const Sums *sums, int64_t id, int64_t threads) {
    const int B = a.c.batch;
    const int *starts = sums ? sums->starts : a.starts, *back_at = sums ? sums->back_at : a.back_at;
    const int *take_at = sums ? sums->take_at : a.take_at, *list = sums ? sums->list : a.list;
    const int tokens = starts[B];
    // four tokens each
    for (int64_t t0 = 4 * id; t0 < a.T; t0 += 4 * threads) {
        int seq = t0 < tokens ? find(B, (int)t0, [&](int b) { return starts[b]; }) : 0, begin = 0, end = -1, first = 0, from = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t t = t0 + k;
            if (t >= a.T) break;
            if (t < tokens) {
                if (t >= end) {
                    while (t >= starts[seq + 1]) ++seq;
                    begin = starts[seq], end = starts[seq + 1];
                    first = a.after_lens[seq] - (end - begin);
                    from = a.first_pos ? __ldg(a.first_pos + seq) : first;
                }
                const int i = (int)t - begin;
                a.seq[t] = seq, a.slot[t] = first + i, a.pos[t] = from + i;
            } else {
                a.seq[t] = -1, a.slot[t] = 0, a.pos[t] = 0;
            }
        }
    }
    const int count = list[0], there = list[1], back = back_at[B], taken = take_at[B];
    bool bad = false;
    // page r of those returned
    auto returned = [&](int r) {
        const int b = find(B, r, [&](int i) { return back_at[i]; });
        return a.table[b * a.c.ld_table + a.held_out[b] + (r - back_at[b])];
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
        const int b = find(B, (int)j, [&](int i) { return take_at[i]; });
        const int take = take_at[b + 1] - take_at[b];
        bad |= !page_ok(a.c, page);
        a.table[b * a.c.ld_table + a.held_out[b] - take + ((int)j - take_at[b])] = page;
    }
    if (bad) atomicOr(a.c.status, kDevIndex);
}

template <bool FILL>
__global__ void __launch_bounds__(kThreads) plan_kernel(const PlanArgs a) {
    __shared__ Sums sums;
    pdl_wait();
    pdl_trigger();
    Sums *const own = FILL && a.c.batch <= kShared ? &sums : nullptr;
    scan_requests(a, own);
    if constexpr (FILL) {
        __syncthreads();  // its writes are seen by the CTA
        fill(a, own, threadIdx.x, blockDim.x);
    }
}

__global__ void __launch_bounds__(kFillThreads) plan_fill_kernel(const PlanArgs a) {
    __shared__ Sums sums;
    pdl_wait();
    pdl_trigger();
    const int B = a.c.batch;
    Sums *const own = B <= kShared ? &sums : nullptr;
    if (own) {
        for (int i = threadIdx.x; i <= B; i += kFillThreads) sums.starts[i] = a.starts[i], sums.back_at[i] = a.back_at[i], sums.take_at[i] = a.take_at[i];
        if (threadIdx.x < 2) sums.list[threadIdx.x] = a.list[threadIdx.x];
        __syncthreads();
    }
    fill(a, own, (int64_t)blockIdx.x * kFillThreads + threadIdx.x, (int64_t)gridDim.x * kFillThreads);
}

}  // namespace

cudaError_t launch_batch_plan(const DeviceInfo &di, const PlanArgs &a, cudaStream_t s) {
    if (a.T <= kSmallTokens && (int64_t)a.c.batch * a.c.max_pages <= kSmallPages) {
        // few requests and tokens: few warps, whose barriers cost less
        const int threads = a.c.batch <= 128 && a.T <= 512 ? 128 : kThreads;
        return launch_pdl(plan_kernel<true>, dim3(1), dim3(threads), 0, s, dim3(1), a);
    }
    const cudaError_t e = launch_pdl(plan_kernel<false>, dim3(1), dim3(kThreads), 0, s, dim3(1), a);
    if (e != cudaSuccess) return e;
    int64_t ctas = (a.T + 4 * kFillThreads - 1) / (4 * kFillThreads);
    if (ctas < di.sm_count) ctas = di.sm_count;  // (pages may be more than tokens)
    const int64_t most = (int64_t)di.sm_count * 8;
    if (ctas > most) ctas = most;
    return launch_pdl(plan_fill_kernel, dim3((unsigned)ctas), dim3(kFillThreads), 0, s, dim3(1), a);
}

}  // namespace q4k
