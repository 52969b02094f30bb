// pages.cu -- the pages and rows of a paged cache that move between decode
// steps: accepted drafted tokens, resized and forked sequences.
//
// accept_kernel. One CTA per (sequence, cache); each thread owns 16 bytes of
// a token row and moves them for the accepted tokens in ascending order. The
// indices ascend strictly, so a destination never lies past its source: four
// rows are read before the first of them is written, and no later source can
// have been overwritten. Bound by its chain of dependent loads (length, list,
// table, rows): in a captured graph 64 sequences in 64 caches of 8 heads (41 MB
// moved, in L2) take 7.5 us and one sequence in 56 caches 2.7; otherwise the
// host's call is longer (12 us with the caches' descriptors made once, 190
// with them made at every call).
//
// take_kernel (resize, and the first half of a fork). Page counts only, no
// free list: a page is free when its count is 0, and free pages are handed
// out lowest first, in order of (sequence, entry). One cluster of CTAs: the
// demands' prefix sums in shared memory (each CTA computes them all), returns
// dealt out by element, a cluster barrier, then every warp counts the zeros
// of a contiguous stretch of page_refs, the CTAs exchange their counts through
// distributed shared memory, and each zero of rank r < demand goes to the
// entry that the prefix sums give r. Every result follows from the inputs
// alone: atomics only add and subtract counts. Bound by latency: five round
// trips to memory and as many barriers of the CTA (256 rows, 16384 pages: 6.6 us
// a call), then, when very many pages are given out, by the instructions of 16
// SMs (4096 rows of up to 100 pages, 524288 pages: 19 us a call on average).
//
// share_kernel (the second half of a fork). CTAs of (fork, cache, 16 KB) copy
// the partial last page; CTAs of (fork, stretch of the table) copy the shared
// entries and raise their pages' counts. Bound by memory: 96 forks in 64 caches
// of 16 KB pages (195 MB) take 20 us of the call's 26.
#include <algorithm>
#include <atomic>

#include "pkv_internal.h"
#include "pkv_ptx.cuh"

namespace pkv {
namespace {

template <typename V>
__device__ __forceinline__ V ld_as(const uint8_t* p) {
    return *reinterpret_cast<const V*>(p);
}
template <typename V>
__device__ __forceinline__ void st_as(uint8_t* p, V v) {
    *reinterpret_cast<V*>(p) = v;
}

// ---- accepted drafted tokens --------------------------------------------------
constexpr int kAcceptThreads = 128;
constexpr int kBatch = 4;  // rows in flight per thread

template <typename V>
__device__ __forceinline__ void move_rows(const PoolPart& c, const int64_t* src, const int64_t* dst, int n) {
    const int per_row = c.row / static_cast<int>(sizeof(V));
    const int units = c.n1 * per_row;
    for (int u = threadIdx.x; u < units; u += kAcceptThreads) {
        const int h = u / per_row;
        const int64_t off = h * c.s1 + static_cast<int64_t>(u - h * per_row) * sizeof(V);
        for (int j = 0; j < n; j += kBatch) {
            V v[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                if (j + k < n && src[j + k] >= 0) v[k] = ld_as<V>(c.p + src[j + k] + off);
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                if (j + k < n && src[j + k] >= 0) st_as<V>(c.p + dst[j + k] + off, v[k]);
        }
    }
}

__global__ void __launch_bounds__(kAcceptThreads) accept_kernel(const __grid_constant__ AcceptArgs a) {
    __shared__ int64_t src[kMaxAccepted], dst[kMaxAccepted];
    __shared__ int bad, n_moves;
    // seq_lens and the tables may be written by the preceding grid, and
    // seq_lens_out is an index input of the next: no early trigger.
    grid_dep_wait();
    const int b = blockIdx.x;
    const bool first = blockIdx.y == 0 && a.write_lens;
    const int L = a.seq_lens[b];
    const int64_t N64 = static_cast<int64_t>(a.q_start[b + 1]) - a.q_start[b];
    const int n = a.n_accepted[b];
    const int64_t cap = static_cast<int64_t>(a.max_pages) * a.page_size;
    int flags = 0;
    if (L < 0 || L > cap) flags |= PKV_FLAG_SEQ_LEN_RANGE;
    else if (N64 < 0 || N64 > L || n < 0 || n > N64 || n > a.A) flags |= PKV_FLAG_DRAFT_RANGE;
    if (flags) {
        if (threadIdx.x == 0 && first) {
            flag_error(a.err, flags);
            a.seq_lens_out[b] = L;
        }
        return;
    }
    const int N = static_cast<int>(N64), base = L - N;
    if (threadIdx.x == 0) bad = 0, n_moves = 0;
    __syncthreads();
    for (int j = threadIdx.x; j < n; j += kAcceptThreads) {
        const int32_t* row = a.accepted + b * a.ac_s0;
        const int x = row[j], prev = j ? row[j - 1] : -1;
        if (x <= prev || x >= N) bad = 1;
    }
    __syncthreads();
    if (bad) {
        if (threadIdx.x == 0 && first) {
            flag_error(a.err, PKV_FLAG_DRAFT_RANGE);
            a.seq_lens_out[b] = L;
        }
        return;
    }
    if (threadIdx.x == 0 && first) a.seq_lens_out[b] = base + n;
    if (a.n_caches == 0) return;
    const PoolPart& c = a.c[blockIdx.y];
    for (int j = threadIdx.x; j < n; j += kAcceptThreads) {
        const int sp = base + a.accepted[b * a.ac_s0 + j], dp = base + j;
        int64_t s = -1, d = -1;
        if (sp != dp) {  // accepted from j on: everything before it is in place already
            const int ps = a.block_tables[b * a.bt_s0 + sp / a.page_size];
            const int pd = a.block_tables[b * a.bt_s0 + dp / a.page_size];
            if (ps < 0 || ps >= a.num_pages || pd < 0 || pd >= a.num_pages) {
                if (first) flag_error(a.err, PKV_FLAG_PAGE_RANGE);
            } else {
                s = ps * c.s_page + (sp % a.page_size) * c.s0;
                d = pd * c.s_page + (dp % a.page_size) * c.s0;
            }
        }
        src[j] = s;
        dst[j] = d;
        if (s >= 0) n_moves = 1;
    }
    __syncthreads();
    if (!n_moves) return;
    switch (c.vec) {
        case 16: move_rows<uint4>(c, src, dst, n); break;
        case 8: move_rows<uint2>(c, src, dst, n); break;
        case 4: move_rows<uint32_t>(c, src, dst, n); break;
        default: move_rows<uint8_t>(c, src, dst, n); break;
    }
}

// ---- pages taken from and returned to the pool ----------------------------------
constexpr int kTakeThreads = 1024;
constexpr int kTakeWarps = kTakeThreads / 32;
static_assert(kTakeWarps == 32, "a warp reads the warps' sums, one per lane");
constexpr int kMaxCluster = 16;
// Pools that one CTA looks through; larger ones take a cluster of 16. A trim and a
// growth, captured, us by one CTA and by 16: 256 rows that change by a page, 8192
// pages 12.1 and 13.5, 32,768 14.1 and 13.3, 131,072 19.3 and 15.2; 1024 rows given
// up and taken again, 16,384 pages 27.8 and 15.5. (Four CTAs: 2% better than 16 at
// most, 30% worse.)
constexpr int64_t kSoloPages = 8192;
constexpr int kKeptPages = 1024;           // pages of a warp whose free masks stay in a register
constexpr uint32_t kDemandCap = 1u << 30;  // sums saturate here, above any pool

__device__ __forceinline__ uint32_t sat_add(uint32_t x, uint32_t y) { return min(x + y, kDemandCap); }
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// All threads of the cluster; what they wrote before (shared memory of any
// CTA, device memory) is visible to all of them after it. (SOLO: one CTA, whose
// own barrier does: sixteen forks in 28 layers 21 us and not 23.)
template <bool SOLO>
__device__ __forceinline__ void cluster_barrier() {
    if constexpr (SOLO) __syncthreads();
    else asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t local_addr, uint32_t rank, uint32_t v) {
    asm volatile(
        "{\n\t.reg .u32 ra;\n\tmapa.shared::cluster.u32 ra, %0, %1;\n\tst.shared::cluster.u32 [ra], %2;\n\t}" ::"r"(
            local_addr),
        "r"(rank), "r"(v)
        : "memory");
}

// Exclusive saturating prefix sums of each of the arrays x[k][0, n) in place,
// x[k][n] = the total. All threads of the CTA; thread t owns a contiguous stretch.
template <int K>
__device__ void block_prefix(uint32_t* const (&x)[K], int n, uint32_t (*warp_sum)[kTakeWarps]) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int seg = (n + kTakeThreads - 1) / kTakeThreads;
    const int i0 = min(tid * seg, n), i1 = min(i0 + seg, n);
    __syncthreads();
    uint32_t excl[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        uint32_t sum = 0;
        for (int i = i0; i < i1; ++i) sum = sat_add(sum, x[k][i]);
        uint32_t inc = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc = sat_add(inc, y);
        }
        if (lane == 31) warp_sum[k][warp] = inc;
        excl[k] = __shfl_up_sync(0xffffffffu, inc, 1);
        if (lane == 0) excl[k] = 0;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
        uint32_t sums = warp_sum[k][lane];             // (as many warps as lanes)
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, sums, d);
            if (lane >= d) sums = sat_add(sums, y);
        }
        const uint32_t total = __shfl_sync(0xffffffffu, sums, 31);
        const uint32_t base = __shfl_sync(0xffffffffu, sums, (warp + 31) & 31);
        uint32_t run = warp ? sat_add(base, excl[k]) : excl[k];
        for (int i = i0; i < i1; ++i) {
            const uint32_t d = x[k][i];
            x[k][i] = run;
            run = sat_add(run, d);
        }
        if (tid == 0) x[k][n] = total;
    }
    __syncthreads();
}

// Largest i with x[i] <= r, for x[0] = 0 <= r < x[n].
__device__ __forceinline__ int owner_of(const uint32_t* x, int n, uint32_t r) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (x[mid] <= r) lo = mid;
        else hi = mid;
    }
    return lo;
}

// The pages that a row of `have` pages is to have for `len` tokens; flags set when it stays as it is.
__device__ __forceinline__ int pages_wanted(const TakeArgs& a, int have, int len, int& flags) {
    if (have < 0 || have > a.max_pages) {
        flags |= PKV_FLAG_PAGE_STATE;
        return have;
    }
    if (len < 0) return have;
    const int need = len / a.page_size + (len % a.page_size != 0);
    if (need <= a.max_pages) return need;
    flags |= PKV_FLAG_SEQ_LEN_RANGE;
    return have;
}

// Returns of a large batch, by all SMs: a warp takes 256 entries of a row at a
// time, every gridDim.x-th such stretch. The counts of entries stay as they are
// for the take behind it.
constexpr int kReturnSpan = 256;
__global__ void __launch_bounds__(256) return_kernel(const __grid_constant__ TakeArgs a) {
    grid_dep_wait();  // (the table is an index input: no early trigger, but for the take, which waits)
    grid_dep_launch();
    const int b = blockIdx.y * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (b >= a.n) return;
    int flags = 0;
    const int have = a.page_counts[b], want = pages_wanted(a, have, a.new_lens[b], flags);
    flags = 0;  // the take reports them
    for (int64_t j0 = want + static_cast<int64_t>(blockIdx.x) * kReturnSpan; j0 < have; j0 += static_cast<int64_t>(gridDim.x) * kReturnSpan) {
        int32_t* entry = a.block_tables + b * a.bt_s0 + j0;
        const int m = static_cast<int>(min(static_cast<int64_t>(kReturnSpan), have - j0));
        int page[kReturnSpan / 32], old[kReturnSpan / 32];
#pragma unroll
        for (int k = 0; k < kReturnSpan / 32; ++k) {
            const int j = lane + 32 * k;
            page[k] = -2;
            if (j < m) {
                page[k] = entry[j];
                entry[j] = -1;
                if (page[k] < 0 || page[k] >= a.num_pages) {
                    flags |= PKV_FLAG_PAGE_RANGE;
                    page[k] = -2;
                }
            }
        }
#pragma unroll
        for (int k = 0; k < kReturnSpan / 32; ++k) old[k] = page[k] >= 0 ? atomicSub(a.page_refs + page[k], 1) : 1;
#pragma unroll
        for (int k = 0; k < kReturnSpan / 32; ++k)
            if (old[k] <= 0) {
                atomicAdd(a.page_refs + page[k], 1);
                flags |= PKV_FLAG_PAGE_STATE;
            }
    }
    if (flags) flag_error(a.err, flags);
}

// The four counts from page p on as a mask of the free ones (p a multiple of 4).
__device__ __forceinline__ uint32_t free_mask(const int32_t* refs, int64_t p, int64_t end, bool vec) {
    if (p + 4 <= end && vec) {
        const int4 v = __ldcg(reinterpret_cast<const int4*>(refs + p));
        return (v.x == 0) | (v.y == 0) << 1 | (v.z == 0) << 2 | (v.w == 0) << 3;
    }
    uint32_t m = 0;
    for (int k = 0; k < 4; ++k)
        if (p + k < end && __ldcg(refs + p + k) == 0) m |= 1u << k;
    return m;
}

// Dynamic shared memory: words for n rows or forks, then a page list per warp.
__host__ __device__ constexpr size_t take_words(int n) { return 3 * static_cast<size_t>(n) + 2; }

template <bool FORK, bool SOLO>
__global__ void __launch_bounds__(kTakeThreads) take_kernel(const __grid_constant__ TakeArgs a) {
    extern __shared__ uint32_t dyn[];
    __shared__ uint32_t warp_sum[2][kTakeWarps], warp_free[kTakeWarps], cta_free[kMaxCluster];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = SOLO ? 0 : cluster_rank(), C = SOLO ? 1 : cluster_size();
    const int n = a.n;
    uint32_t* need = dyn;                              // [n + 1]: demands, then their prefix sums
    int32_t* held = reinterpret_cast<int32_t*>(dyn + (n + 1));  // resize: [n] entries in use; fork: parent's length, -1 = not made
    uint32_t* give = dyn + (2 * n + 1);                // resize: [n + 1] returns, then their prefix sums; entries wanted where they are made already
    int32_t* tail = reinterpret_cast<int32_t*>(give);  // fork: [n] page to copy, -1 = none
    uint32_t* list = dyn + take_words(n) + warp * 128; // this warp's free pages, in order

    // Counts, tables and lengths may be written by the preceding grid. What
    // this grid writes are index inputs: a resize lets nothing start early, a
    // fork only its own second half (which waits before it reads).
    grid_dep_wait();
    if (FORK) grid_dep_launch();

    int flags = 0;
    if constexpr (!FORK) {
        for (int b0 = tid; b0 < n; b0 += 4 * kTakeThreads) {
            int have[4], len[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int b = b0 + k * kTakeThreads;
                have[k] = b < n ? a.page_counts[b] : 0;
                len[k] = b < n ? a.new_lens[b] : -1;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int b = b0 + k * kTakeThreads;
                if (b >= n) break;
                const int want = pages_wanted(a, have[k], len[k], flags);
                held[b] = have[k];
                need[b] = want > have[k] ? want - have[k] : 0;
                give[b] = a.returned ? want : want < have[k] ? have[k] - want : 0;
            }
        }
        // Returns (unless a kernel of their own made them), dealt out by entry
        // over the cluster, four per thread on their way.
        if (a.returned) block_prefix<1>({need}, n, warp_sum);
        else block_prefix<2>({need, give}, n, warp_sum);
        const uint32_t total = a.returned ? 0 : give[n], span = C * kTakeThreads;
        for (uint32_t e0 = rank * kTakeThreads + tid; e0 < total; e0 += 4 * span) {
            int page[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t e = e0 + k * span;
                page[k] = -2;
                if (e < total) {
                    const int b = owner_of(give, n, e);
                    // the row keeps held - returns entries
                    int32_t* entry = a.block_tables + b * a.bt_s0 + held[b] - static_cast<int>(give[b + 1] - e);
                    page[k] = *entry;
                    *entry = -1;
                    if (page[k] < 0 || page[k] >= a.num_pages) {
                        flags |= PKV_FLAG_PAGE_RANGE;
                        page[k] = -2;
                    }
                }
            }
            int old[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) old[k] = page[k] >= 0 ? atomicSub(a.page_refs + page[k], 1) : 1;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (old[k] <= 0) {
                    atomicAdd(a.page_refs + page[k], 1);
                    flags |= PKV_FLAG_PAGE_STATE;
                }
        }
    } else {
        // A child's count of 0 becomes a claim: kClaim + i of its first fork i (the
        // lowest value stays). Every CTA makes the same claims, and none takes
        // another's for a count: those start where the claims end.
        constexpr int kClaim = INT32_MIN;
        auto no_child = [&](int count) { return count > 0 || (count < 0 && count >= kClaim + n); };
        for (int i = tid; i < n; i += kTakeThreads) {
            const int p = a.forks[2 * i], c = a.forks[2 * i + 1];
            int L = -1, src = -1;
            if (p >= 0) {
                if (p >= a.rows || c < 0 || c >= a.rows || no_child(a.page_counts[c])) {
                    flags |= PKV_FLAG_PAGE_STATE;
                } else {
                    const int x = a.seq_lens[p];
                    const int full = x / a.page_size, part = x % a.page_size != 0;
                    if (x < 0 || full + part > min(max(a.page_counts[p], 0), a.max_pages)) {
                        flags |= PKV_FLAG_SEQ_LEN_RANGE;
                    } else {
                        if (part) src = a.block_tables[p * a.bt_s0 + full];
                        if (part && (src < 0 || src >= a.num_pages)) {
                            flags |= PKV_FLAG_PAGE_RANGE;
                        } else {
                            L = x;
                            atomicMin(a.page_counts + c, kClaim + i);
                        }
                    }
                }
            }
            held[i] = L;
            tail[i] = L < 0 ? -1 : src;
        }
        cluster_barrier<SOLO>();
        for (int i = tid; i < n; i += kTakeThreads) {
            if (held[i] >= 0 && __ldcg(a.page_counts + a.forks[2 * i + 1]) != kClaim + i) {
                flags |= PKV_FLAG_PAGE_STATE;  // an earlier fork has this child
                held[i] = -1;
                tail[i] = -1;
            }
            need[i] = tail[i] >= 0 ? 1 : 0;
        }
        block_prefix<1>({need}, n, warp_sum);
    }
    cluster_barrier<SOLO>();  // every return is counted

    // ---- free pages: each warp a contiguous stretch ------------------------------
    const int64_t cta_span = ((a.num_pages + C - 1) / C + 127) / 128 * 128;
    const int64_t warp_span = ((cta_span + kTakeWarps - 1) / kTakeWarps + 127) / 128 * 128;
    const int64_t cta0 = rank * cta_span, cta1 = min(cta0 + cta_span, a.num_pages);
    const int64_t p0 = min(cta0 + warp * warp_span, cta1), p1 = min(p0 + warp_span, cta1);
    const bool vec = (reinterpret_cast<uintptr_t>(a.page_refs) & 15) == 0;
    const bool kept = warp_span <= kKeptPages;
    const uint32_t wanted = need[n];
    uint32_t cnt = 0, masks = 0;                       // masks: 4 bits per group of 128 pages, when kept
    if (wanted) {
        if (kept) {
#pragma unroll
            for (int g = 0; g < kKeptPages / 128; ++g) {
                const int64_t p = p0 + 128 * g + 4 * lane;
                if (p < p1) masks |= free_mask(a.page_refs, p, p1, vec) << (4 * g);
            }
            cnt = __popc(masks);
        } else {
#pragma unroll 8
            for (int64_t p = p0 + 4 * lane; p < p1; p += 128) cnt += __popc(free_mask(a.page_refs, p, p1, vec));
        }
    }
    cnt = __reduce_add_sync(0xffffffffu, cnt);
    if (lane == 0) warp_free[warp] = cnt;
    __syncthreads();
    if (warp == 0) {
        const uint32_t t = __reduce_add_sync(0xffffffffu, warp_free[lane]);
        if (SOLO) cta_free[0] = t;
        else if (lane < static_cast<int>(C)) st_cluster(smem_u32(&cta_free[rank]), lane, t);
    }
    cluster_barrier<SOLO>();
    const uint32_t of_cta = lane < static_cast<int>(C) ? cta_free[lane] : 0;
    const uint32_t total_free = __reduce_add_sync(0xffffffffu, of_cta);
    uint32_t at = __reduce_add_sync(0xffffffffu, (lane < static_cast<int>(rank) ? of_cta : 0) + (lane < warp ? warp_free[lane] : 0));
    const uint32_t last = min(wanted, total_free);  // ranks past it go to nobody
    int group = 0, owner = -1;                      // the row of the last rank seen
    for (int64_t g = p0; g < p1 && at < last; g += 128, ++group) {
        const int64_t p = g + 4 * lane;
        uint32_t m = kept ? masks >> (4 * group) & 15u : p < p1 ? free_mask(a.page_refs, p, p1, vec) : 0u;
        uint32_t inc = __popc(m);
        const uint32_t own_n = inc;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += y;
        }
        const uint32_t found = __shfl_sync(0xffffffffu, inc, 31);
        // the group's free pages side by side, so that neighbouring lanes write
        // neighbouring entries
        uint32_t o = inc - own_n;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (m >> k & 1) list[o++] = static_cast<uint32_t>(p + k);
        __syncwarp();
        for (uint32_t k0 = 0; k0 < found && at + k0 < last; k0 += 32) {
            const uint32_t end = min(at + found, last);
            const uint32_t r = min(at + k0 + lane, end - 1);
            // 32 neighbouring ranks mostly have few owners: that of the rank before
            // them (at first, a search by the warp's lanes alike) and the rows behind it
            const int i0 = owner < 0 ? owner_of(need, n, at + k0) : owner;
            const uint32_t ends = i0 + 1 + lane <= n ? need[i0 + 1 + lane] : ~0u;
            int i = 0;
#pragma unroll
            for (int d = 16; d; d >>= 1)
                if (__shfl_sync(0xffffffffu, ends, i + d - 1) <= r) i += d;
            i += i0 + (__shfl_sync(0xffffffffu, ends, i) <= r);
            if (need[i + 1] <= r) i = owner_of(need, n, r);  // more than 31 rows on (rows without a demand among them)
            __syncwarp();
            owner = __shfl_sync(0xffffffffu, i, 31);
            if (at + k0 + lane >= end) continue;
            const int page = static_cast<int>(list[k0 + lane]);
            if (need[i + 1] > total_free) continue;    // i, and everyone after it, gets nothing
            if constexpr (!FORK) {
                a.block_tables[i * a.bt_s0 + held[i] + (r - need[i])] = page;
            } else {
                a.block_tables[a.forks[2 * i + 1] * a.bt_s0 + held[i] / a.page_size] = page;
                a.copies[2 * i] = tail[i];
                a.copies[2 * i + 1] = page;
            }
            a.page_refs[page] = 1;
        }
        at += found;
        __syncwarp();
    }
    if (flags) flag_error(a.err, flags);
    cluster_barrier<SOLO>();  // every CTA has read the counts and lengths
    if (rank != 0) return;
    for (int i = tid; i < n; i += kTakeThreads) {
        if constexpr (!FORK) {
            // (tables of returns made here are small: their sums do not saturate)
            const int want = static_cast<int>(a.returned ? give[i] : held[i] + (need[i + 1] - need[i]) - (give[i + 1] - give[i]));
            const bool fails = want > held[i] && need[i + 1] > total_free;
            if (fails) flag_error(a.err, PKV_FLAG_POOL_EMPTY);
            else if (want != held[i]) a.page_counts[i] = want;
        } else {
            const bool fails = tail[i] >= 0 && need[i + 1] > total_free;
            if (fails) flag_error(a.err, PKV_FLAG_POOL_EMPTY);
            if (held[i] >= 0) {
                const int c = a.forks[2 * i + 1], pages = held[i] / a.page_size + (tail[i] >= 0);
                a.page_counts[c] = fails ? 0 : pages;
                if (!fails) a.seq_lens[c] = held[i];
            }
            if (held[i] < 0 || fails) a.copies[2 * i] = a.copies[2 * i + 1] = -2;
            else if (tail[i] < 0) a.copies[2 * i] = a.copies[2 * i + 1] = -1;
        }
    }
}

// ---- shared entries and copied pages of a fork --------------------------------------
constexpr int kShareThreads = 256;
constexpr int kShareSpan = 2048;  // table entries per CTA

template <typename V>
__device__ __forceinline__ void copy_page(const PoolPart& c, int64_t src, int64_t dst) {
    const int per_row = c.row / static_cast<int>(sizeof(V));
    const int units = c.n0 * c.n1 * per_row;
    auto at = [&](int u) -> int64_t {
        const int row = u / per_row, i0 = row / c.n1;
        return i0 * c.s0 + (row - i0 * c.n1) * c.s1 + static_cast<int64_t>(u - row * per_row) * sizeof(V);
    };
    for (int u0 = threadIdx.x; u0 < units; u0 += 8 * kShareThreads) {
        V v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (u0 + k * kShareThreads < units) v[k] = ld_as<V>(c.p + src + at(u0 + k * kShareThreads));
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (u0 + k * kShareThreads < units) st_as<V>(c.p + dst + at(u0 + k * kShareThreads), v[k]);
    }
}

// A page in one piece, 16-byte aligned: kBulkBytes of it through shared memory
// by two bulk copies of one thread (96 forks in 64 caches of 16 KB pages: 66 us a
// step with loads and stores by 256 threads, 44 with bulk copies).
constexpr int kBulkBytes = 16384;
__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(reinterpret_cast<uint64_t>(dst)), "r"(src),
                 "r"(bytes)
                 : "memory");
}
__device__ void copy_bulk(uint8_t* dst, const uint8_t* src, uint32_t bytes, uint32_t buf, uint32_t bar, int32_t* err) {
    mbar_init(bar, 1);
    fence_mbar_init();
    mbar_arrive_expect_tx(bar, bytes);
    bulk_load(buf, src, bytes, bar, l2_policy_evict_first());
    if (!mbar_wait_bounded(bar, 0, 1000000000ull)) {
        flag_error(err, PKV_FLAG_WAIT_TIMEOUT);
        // the copy under way lands, if it still does, before the CTA gives its shared memory back
        (void)mbar_wait_bounded(bar, 0, 1000000000ull);
        return;
    }
    bulk_store(dst, buf, bytes);
    asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group 0;" ::: "memory");
}

__global__ void __launch_bounds__(kShareThreads) share_kernel(const __grid_constant__ ShareArgs a) {
    __shared__ __align__(128) uint8_t buf[kBulkBytes];
    __shared__ uint64_t bar;
    grid_dep_wait();  // the first half's results; the table is an index input: no early trigger
    const int i = blockIdx.x;
    const int src = a.copies[2 * i], dst = a.copies[2 * i + 1];
    if (src == -2) return;  // not made
    const int y = static_cast<int>(blockIdx.y) - a.table_ctas;
    if (y >= 0) {
        if (src < 0) return;
        const PoolPart& c = a.c[y];
        const int64_t s = src * c.s_page, d = dst * c.s_page;
        if (c.vec == 16 && c.n0 * c.n1 == 1) {
            const int64_t o = static_cast<int64_t>(blockIdx.z) * kBulkBytes;
            if (threadIdx.x == 0 && o < c.row && src != dst)
                copy_bulk(c.p + d + o, c.p + s + o, static_cast<uint32_t>(min(static_cast<int64_t>(kBulkBytes), c.row - o)),
                          smem_u32(buf), smem_u32(&bar), a.err);
            return;
        }
        if (blockIdx.z > 0) return;
        switch (c.vec) {
            case 16: copy_page<uint4>(c, s, d); break;
            case 8: copy_page<uint2>(c, s, d); break;
            case 4: copy_page<uint32_t>(c, s, d); break;
            default: copy_page<uint8_t>(c, s, d); break;
        }
        return;
    }
    if (blockIdx.z > 0) return;
    const int p = a.forks[2 * i], c = a.forks[2 * i + 1];
    const int full = a.seq_lens[c] / a.page_size;
    const int j1 = min(full, (static_cast<int>(blockIdx.y) + 1) * kShareSpan);
    const int32_t* from = a.block_tables + p * a.bt_s0;
    int32_t* to = a.block_tables + c * a.bt_s0;
    int bad = 0;
#pragma unroll 4
    for (int j = blockIdx.y * kShareSpan + threadIdx.x; j < j1; j += kShareThreads) {
        const int page = from[j];
        to[j] = page;
        if (page < 0 || page >= a.num_pages) bad = 1;
        else atomicAdd(a.page_refs + page, 1);
    }
    if (bad) flag_error(a.err, PKV_FLAG_PAGE_RANGE);
}

// The CTAs of a take over a pool of so many pages, its kernel's attributes set:
// before anything of the call is queued, so that a call that cannot be made leaves
// the state as it is. The attributes are of the kernel, not of the call, and
// another host thread may be about to launch it: always the same values.
constexpr size_t kTakeSmemMax = (take_words(kMaxRows) + kTakeWarps * 128) * 4;

template <bool FORK>
cudaError_t plan_take(int64_t num_pages, unsigned* ctas) {
    static std::atomic<unsigned> largest[64];              // per device: the largest cluster that fits, at most 16
    *ctas = num_pages <= kSoloPages ? 1 : kMaxCluster;
    auto kern = *ctas == 1 ? take_kernel<FORK, true> : take_kernel<FORK, false>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kTakeSmemMax));
    if (e != cudaSuccess || *ctas == 1) return e;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    int dev = 0;
    e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    unsigned C = dev < 64 ? largest[dev].load(std::memory_order_relaxed) : 0;
    if (C == 0) {
        // 16 CTAs are past the portable 8 and need not fit (part of a GPU, say)
        cudaLaunchConfig_t cfg{};
        cudaLaunchAttribute attr[1];
        cfg.gridDim = dim3(kMaxCluster);
        cfg.blockDim = dim3(kTakeThreads);
        cfg.dynamicSmemBytes = kTakeSmemMax;
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = kMaxCluster;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        C = cudaOccupancyMaxActiveClusters(&n, kern, &cfg) == cudaSuccess && n > 0 ? kMaxCluster : 8;
        if (C == 8) (void)cudaGetLastError();
        if (dev < 64) largest[dev].store(C, std::memory_order_relaxed);
    }
    *ctas = C;
    return cudaSuccess;
}

template <bool FORK>
cudaError_t launch_take(const TakeArgs& a, unsigned C, cudaStream_t s) {
    auto kern = C == 1 ? take_kernel<FORK, true> : take_kernel<FORK, false>;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(C);
    cfg.blockDim = dim3(kTakeThreads);
    cfg.dynamicSmemBytes = (take_words(a.n) + kTakeWarps * 128) * 4;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = C;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace

cudaError_t launch_accept(const AcceptArgs& a, cudaStream_t s) {
    if (a.B == 0) return cudaSuccess;
    return launch_dependent(accept_kernel, dim3(a.B, std::max(a.n_caches, 1)), dim3(kAcceptThreads), 0, s, a);
}

cudaError_t launch_resize(const TakeArgs& a0, cudaStream_t s) {
    if (a0.n == 0) return cudaSuccess;
    TakeArgs a = a0;
    unsigned C = 0;
    cudaError_t e = plan_take<false>(a.num_pages, &C);
    if (e != cudaSuccess) return e;
    // With room for 64 Ki entries in the tables and more, the returns may be more
    // than the take's one cluster does quickly, and are worth a launch of their
    // own: their number is known on the device alone. A trim and a growth, captured,
    // us a pair in one kernel and in two: 256 rows of 2048 entries that change by a
    // page 12.4 and 13.6, by 500 pages 27 and 21; 4096 rows of 100 entries, by a
    // page 35.4 and 34.6, by 50 57 and 41.
    a.returned = static_cast<int64_t>(a.n) * a.max_pages >= 65536;
    if (a.returned) {
        // One warp per row, and as many more as four CTAs per SM leave room for:
        // a grid for the tables' width was 131,072 CTAs for 4096 rows of 65,536
        // entries, whatever is returned.
        int sms = 0;
        e = device_sm_count(&sms);
        if (e != cudaSuccess) return e;
        const int rows = (a.n + 7) / 8, spans = (a.max_pages + kReturnSpan - 1) / kReturnSpan;
        e = launch_dependent(return_kernel, dim3(std::min(spans, std::max(1, 4 * sms / rows)), rows), dim3(256), 0, s, a);
        if (e != cudaSuccess) return e;
    }
    return launch_take<false>(a, C, s);
}

cudaError_t launch_fork_take(const TakeArgs& a, cudaStream_t s) {
    if (a.n == 0) return cudaSuccess;
    unsigned C = 0;
    const cudaError_t e = plan_take<true>(a.num_pages, &C);
    return e != cudaSuccess ? e : launch_take<true>(a, C, s);
}

cudaError_t launch_fork_share(const ShareArgs& a0, int32_t n, int32_t max_pages, bool tables, cudaStream_t s) {
    if (n == 0) return cudaSuccess;
    ShareArgs a = a0;
    a.table_ctas = tables ? (max_pages + kShareSpan - 1) / kShareSpan : 0;
    int chunks = 1;
    for (int i = 0; i < a.n_caches; ++i)
        if (a.c[i].vec == 16 && a.c[i].n0 * a.c[i].n1 == 1)
            chunks = std::max(chunks, (a.c[i].row + kBulkBytes - 1) / kBulkBytes);
    return launch_dependent(share_kernel, dim3(n, a.table_ctas + a.n_caches, chunks), dim3(kShareThreads), 0, s, a);
}

}  // namespace pkv
