// Pages of a step's tokens, handed out on the GPU, and the slots of tokens.
//
//   held' = min(held, keep),  pages [ceil(held' / P), ceil(held / P)) go back,
//   pages [ceil(held' / P), ceil((held' + new) / P)) are taken,
//   token i of the new ones stands at held' + i in slot P table[pos / P] + pos % P
//
// Prefix sums over the sequences give every page and token its place. What is read and
// written is little: launches and chains of dependent loads are what it costs.
#include "paging_launch.hpp"

namespace sffn {

namespace {

// Sums of lanes 0 .. l, in lane l.
__device__ __forceinline__ int64_t wave_prefix(int64_t v) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int64_t q = __shfl_up(v, o, 64);
        if (lane >= o) v += q;
    }
    return v;
}

// Inclusive sums over the workgroup's threads and their total. `lds` is read by nobody
// after the next barrier.
template <int NT>
__device__ __forceinline__ int64_t block_prefix(int64_t v, int64_t* lds, int64_t& total) {
    const int wave = threadIdx.x >> 6;
    v = wave_prefix(v);
    if ((threadIdx.x & 63) == 63) lds[wave] = v;
    __syncthreads();
    int64_t before = 0;
    total = 0;
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) {
        const int64_t q = lds[i];
        if (i < wave) before += q;
        total += q;
    }
    return v + before;
}

// The first of n ascending sums that is more than x (n if none).
__device__ __forceinline__ int first_above(const int64_t* sums, int n, int64_t x) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (sums[mid] > x) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

__device__ __forceinline__ int64_t slot_in(int64_t n_pages, int32_t page, int pos, int shift) {
    return page >= 0 && page < n_pages ? ((int64_t)page << shift) + (pos & ((1 << shift) - 1)) : -1;
}

struct Request {
    int kept, fresh;        // tokens
    int had, from, to;      // pages held before, kept, held then
};

__device__ __forceinline__ Request request_of(const PlanArgs& a, int b) {
    Request r{};
    if (b >= a.B) return r;
    const int held = max(a.lens[b], 0);
    r.kept = a.keep ? min(held, max(a.keep[b], 0)) : held;
    r.fresh = min(max(a.fresh[b], 0), 0x7fffffff - r.kept);
    auto pages = [&](int n) { return min((int)(((int64_t)n + (1 << a.shift) - 1) >> a.shift), a.max_pages); };
    r.had = pages(held);
    r.from = pages(r.kept);
    r.to = pages(r.kept + r.fresh);
    return r;
}

// One workgroup of NT threads, which takes as many sequences at a time, and kIn pages a
// thread, whose loads are in flight together (200 sequences of up to 8000 tokens, of which
// some end and some get prompts: one page a thread 10.8 us, four 8.4, eight 10.0);
// with_tokens: positions and slots too.
constexpr int kIn = 4;
template <int NT>
__global__ __launch_bounds__(NT) void k_page_plan(const PlanArgs a, bool with_tokens) {
    __shared__ int64_t sums[2][NT], scan[2][NT / 64];
    __shared__ int2 places[NT];       // of each sequence: kept tokens, kept pages
    const int tid = threadIdx.x;
    int64_t n_free = min((int64_t)max(a.n_free[0], 0), a.n_pages), total;

    if (a.keep) {
        for (int b0 = 0; b0 < a.B; b0 += NT) {
            const Request r = request_of(a, b0 + tid);
            int64_t back;
            const int64_t s = block_prefix<NT>(max(r.had - r.from, 0), scan[0], back);
            sums[0][tid] = s;
            places[tid].y = r.from;
            __syncthreads();
            for (int64_t k0 = 0; k0 < back; k0 += kIn * NT) {
                const int64_t first = k0 + kIn * tid;
                int at = first < back ? first_above(sums[0], NT, first) : 0, known = 0;
                int32_t page[kIn];
#pragma unroll
                for (int j = 0; j < kIn; ++j) {
                    page[j] = -1;
                    if (first + j < back) {
                        while (sums[0][at] <= first + j) ++at;
                        const int64_t i = first + j - (at > 0 ? sums[0][at - 1] : 0) + places[at].y;
                        page[j] = a.table[(int64_t)(b0 + at) * a.table_stride + i];
                    }
                }
#pragma unroll
                for (int j = 0; j < kIn; ++j) known += page[j] >= 0 && page[j] < a.n_pages;
                int64_t nth = n_free + block_prefix<NT>(known, scan[1], total) - known;
#pragma unroll
                for (int j = 0; j < kIn; ++j)
                    if (page[j] >= 0 && page[j] < a.n_pages) {
                        if (nth < a.n_pages) a.free_pages[nth] = page[j];
                        ++nth;
                    }
                n_free = min(n_free + total, a.n_pages);
                __syncthreads();
            }
        }
        // what went onto the stack is read again below, by other threads
        __syncthreads();
    }

    int64_t tokens = 0, taken = 0;          // before the sequences at hand
    for (int b0 = 0; b0 < a.B; b0 += NT) {
        const int b = b0 + tid;
        const Request r = request_of(a, b);
        int64_t new_tokens, new_pages;
        const int64_t s = block_prefix<NT>(r.fresh, scan[0], new_tokens);
        const int64_t p = block_prefix<NT>(max(r.to - r.from, 0), scan[1], new_pages);
        sums[0][tid] = s;
        sums[1][tid] = p;
        places[tid] = make_int2(r.kept, r.from);
        if (b < a.B) {
            a.lens_out[b] = r.kept + r.fresh;
            a.cu[b + 1] = (int32_t)min(tokens + s, (int64_t)0x7fffffff);
        }
        if (b == 0) a.cu[0] = 0;
        __syncthreads();
        auto page_of = [&](int64_t k) {     // the k-th page that is taken
            return k < n_free ? a.free_pages[n_free - 1 - k] : -1;
        };
        for (int64_t k0 = tid; k0 < new_pages; k0 += kIn * NT) {
            int32_t page[kIn];
#pragma unroll
            for (int j = 0; j < kIn; ++j) page[j] = k0 + j * NT < new_pages ? page_of(taken + k0 + j * NT) : -1;
#pragma unroll
            for (int j = 0; j < kIn; ++j) {
                const int64_t k = k0 + j * NT;
                if (k >= new_pages) break;
                const int at = first_above(sums[1], NT, k);
                const int64_t i = k - (at > 0 ? sums[1][at - 1] : 0) + places[at].y;
                a.table[(int64_t)(b0 + at) * a.table_stride + i] = page[j];
            }
        }
        if (with_tokens) {
            const int64_t left = a.T - tokens, n = left < new_tokens ? left : new_tokens;
            for (int64_t t = tid; t < n; t += NT) {
                const int at = first_above(sums[0], NT, t);
                const int2 place = places[at];
                const int pos = place.x + (int)(t - (at > 0 ? sums[0][at - 1] : 0)), i = pos >> a.shift;
                int32_t page = -1;
                if (i < place.y) page = a.table[(int64_t)(b0 + at) * a.table_stride + i];
                else if (i < a.max_pages) page = page_of(taken + (at > 0 ? sums[1][at - 1] : 0) + i - place.y);
                a.positions[tokens + t] = pos;
                // a sequence that leaves the call has no slots, as in k_slots
                a.slots[tokens + t] = tokens + sums[0][at] <= a.T ? slot_in(a.n_pages, page, pos, a.shift) : -1;
            }
        }
        tokens += new_tokens;
        taken += new_pages;
        __syncthreads();
    }
    if (with_tokens)
        for (int64_t t = tokens + tid; t < a.T; t += NT) {
            a.positions[t] = 0;
            a.slots[t] = -1;
        }
    if (tid == 0) {
        a.n_free_out[0] = (int32_t)(taken < n_free ? n_free - taken : 0);
        a.n_free_out[1] = (int32_t)min(taken < n_free ? 0 : taken - n_free, (int64_t)0x7fffffff);
    }
    if (a.B == 0 && tid == 0) a.cu[0] = 0;      // no sequence above wrote it
}

// A thread for each token. The sequence by halving: over every step-th offset in LDS,
// then over those between.
constexpr int kCoarse = 1024;
__global__ __launch_bounds__(256) void k_slots(const SlotArgs a, int64_t first) {
    __shared__ int32_t coarse[kCoarse];
    const int64_t t = first + (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int step = a.B / kCoarse + 1, n = (a.B + step - 1) / step;
    if (a.cu) {
        for (int i = threadIdx.x; i < n; i += 256) coarse[i] = a.cu[i * step];
        __syncthreads();
    }
    if (t >= a.T) return;
    int b = (int)t, from = (int)t, to = (int)t + 1;
    if (a.cu) {
        auto last_at_most = [&](int lo, int hi, auto at) {      // at(lo) <= t is taken for granted
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (at(mid) <= t) lo = mid;
                else hi = mid;
            }
            return lo;
        };
        b = 0;
        if (a.B > 0) {
            b = step * last_at_most(0, n, [&](int i) { return coarse[i]; });
            if (step > 1) b = last_at_most(b, min(b + step, a.B), [&](int i) { return a.cu[i]; });
            from = a.cu[b];
            to = a.cu[b + 1];
        }
    }
    int pos = 0;
    int64_t slot = -1;
    if (a.B > 0 && t >= from && t < to) {
        const int i = (int)t - from;
        const int64_t at = (int64_t)a.lens[b] - (to - from) + i;
        pos = (int)at;
        if (from >= 0 && to <= a.T && i < a.max_new && at >= 0 && (at >> a.shift) < a.max_pages)
            slot = slot_in(a.n_pages, a.table[(int64_t)b * a.table_stride + (at >> a.shift)], pos, a.shift);
    }
    a.positions[t] = pos;
    a.slots[t] = slot;
}

}  // namespace

hipError_t launch_slots(const SlotArgs& a, hipStream_t s) {
    constexpr int64_t most = (int64_t)1 << 22;      // workgroups: below 2^32 threads in a grid
    const int64_t blocks = (a.T + 255) / 256;
    for (int64_t b = 0; b < blocks; b += most) {
        k_slots<<<dim3((unsigned)(blocks - b < most ? blocks - b : most)), 256, 0, s>>>(a, b * 256);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// One workgroup: of 256 threads for as many sequences and few pages (32 single tokens 4.4 us,
// by 1024 threads 6.6; 8 prompts of 8192 tokens, 1024 pages, 9.05 and 9.35), else of 1024 (as
// many single tokens 7.6, by 256 threads 12.4). How many pages go back the device alone
// knows: where 50 of 200 sequences of 8000 tokens end at once 256 threads take 19.9 us, 1024
// 14.0; one of them 6.5 and 9.5. It writes the positions and slots of up to
// two tokens a thread itself (by 256: 256 tokens 4.6 us, with a second launch 6.0, 1024
// tokens 7.6 and 6.9; by 1024: 2048 tokens 8.4 and 9.1, 4096 10.2 and 9.2).
hipError_t launch_page_plan(const PlanArgs& a, hipStream_t s) {
    const bool few = a.B <= 256 && a.T >> a.shift <= 1024;
    const bool with_tokens = a.T <= (few ? 512 : 2048);
    if (few) k_page_plan<256><<<dim3(1), 256, 0, s>>>(a, with_tokens);
    else k_page_plan<1024><<<dim3(1), 1024, 0, s>>>(a, with_tokens);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || with_tokens) return e;
    SlotArgs q{};
    q.table = a.table;
    q.table_stride = a.table_stride;
    q.lens = a.lens_out;
    q.cu = a.cu;
    q.B = a.B;
    q.max_pages = a.max_pages;
    q.max_new = 0x7fffffff;
    q.shift = a.shift;
    q.n_pages = a.n_pages;
    q.T = a.T;
    q.positions = a.positions;
    q.slots = a.slots;
    return launch_slots(q, s);
}

}  // namespace sffn
