// tree_decode.cu -- attention of drafted tokens over a paged cache on the
// fifth-generation tensor cores: the context in full, the drafted tokens under
// a tree mask or as a chain.
//
// Rows. The N drafted tokens of a sequence and the G query heads of a kv head
// share the same K and V: row r = i G + g of (sequence, kv head) is head g of
// token i. With rows on the M side of the MMA (128 tensor-memory lanes), one
// pass over K and V serves up to 256 rows, a softmax thread owns one row, and
// its maximum and sum need no exchange.
//
// Work. An item is (sequence, kv head, group of 256 rows); a unit is one tile
// of 128 positions of one item. All units of the batch, in order, are cut into
// equal stretches, one per CTA (one CTA per SM): every CTA streams the same
// number of tiles whatever the lengths are, with no plan from the host. Each
// CTA finds its stretch from prefix sums over the batch. An item that is cut
// leaves partial sums in the workspace (at most two per CTA: the end of one
// item, the start of another), which a second kernel joins.
//
// A CTA's roles, per tile:
//   warp 0        TMA tile loads of K and V (16 rows x 128 bytes a copy) into a
//                 ring; pages that do not exist are read out of range, which
//                 fills zeros
//   warp 1        S = Q . K^T and O += P . V (M = 128; P from tensor memory, V
//                 as an MN-major operand: nothing is transposed)
//   warps 4 - 7,
//   warps 8 - 11  two softmax groups, each with S, P and O of its own in tensor
//                 memory. Up to 128 rows: both have the same rows and take the
//                 tiles in turn, and their sums are joined at the end (either
//                 group reads the other's O directly). Past 128: each has its
//                 own 128 rows of every tile. While one group is in its softmax
//                 the tensor cores work for the other.
//   warps 12 - 15 FP8 caches: E4M3 bytes to f16 operand tiles (exact)
//
// The online softmax keeps a reference maximum per row that moves only when a
// tile's maximum passes it by more than 8 (log2), so P <= 2^8 and O is scaled
// rarely. P is rounded to bf16 (f16 for FP8 caches): half a step of 2^-8
// (2^-11) of each weight, which the bf16 output's own 2^-8 covers; the sums of
// the weights are taken before the rounding, in fp32. For FP8 caches q is
// scaled by a power of two per row into f16's range, which is exact for
// every value within 2^29 of the row's largest.
//
// Weights of zero do not cover values that are not finite: rows of V behind
// the sequence's end are zeroed in the tile, and a drafted token whose V is
// not finite is zeroed there too and added to the rows that see it by hand.
//
// Waits are bounded (about one second): a role that gives up sets
// PKV_FLAG_WAIT_TIMEOUT and a CTA-wide flag that ends the others' waits.
#include <algorithm>

#include "pkv_internal.h"
#include "pkv_ptx.cuh"

namespace pkv {
namespace {

constexpr int kTile = 128;    // positions per tile
constexpr int kRows = 256;    // rows per item
constexpr int kTilePages = kTile / kPageSize;
constexpr int kSnap = 2;      // no piece of a cut item is shorter than this many tiles
constexpr int kMinUnits = 2;  // units per CTA before another CTA is used
constexpr uint64_t kWaitLimitNs = 1000000000ull;
constexpr float kRescaleLog2 = 8.f;
constexpr int kMetaBytes = 4096 * 16;  // workspace: one int4 per CTA, then the partial sums

template <int D, bool FP8>
struct Cfg {
    static constexpr int NB = D / 64;                      // 128-byte column blocks of an operand row
    static constexpr int TILE = kTile * D * 2;             // operand tile (bf16 or f16)
    static constexpr int BLOCK = kTile * 128;              // one column block of it
    static constexpr int RAW = kTile * D;                  // FP8 tile as it lands
    static constexpr int RBOX = D >= 128 ? 128 : D;        // its row (and swizzle span)
    static constexpr int ST = FP8 ? (D == 128 ? 3 : 6) : (D == 128 ? 5 : 8);  // operand ring
    static constexpr int RST = FP8 ? (D == 128 ? 3 : 6) : 0;                  // raw ring
    static constexpr int THREADS = FP8 ? 512 : 384;
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_T = OFF_Q + 2 * TILE;
    static constexpr int OFF_R = OFF_T + ST * TILE;
    static constexpr int OFF_SC = OFF_R + RST * RAW;       // FP8: [256] floats, 2^-k of each row
    static constexpr int OFF_BAR = OFF_SC + (FP8 ? kRows * 4 : 0);
    static constexpr int NBAR = 2 * ST + 2 * RST + 7;
    static constexpr int OFF_MISC = OFF_BAR + 8 * NBAR;
    static constexpr int SMEM = OFF_MISC + 256 + 1024;     // + alignment slack
    static_assert(SMEM <= 232448, "shared memory of one CTA");
    // tensor-memory columns of a softmax group: S (P over it, or beside it where O leaves room), then O
    static constexpr uint32_t P_COL = D == 64 ? 192 : 0;
    static constexpr uint32_t O_COL = 128;
};

struct Seq {
    int q0, N, L, ctx, R, RG;
};
// Sequence b, its values clamped; `flags` collects what was out of range.
__device__ __forceinline__ Seq seq_of(const TreeArgs& a, int b, int& flags) {
    Seq s;
    const int q0 = __ldg(a.q_start + b), q1 = __ldg(a.q_start + b + 1);
    s.q0 = min(max(q0, 0), a.T);
    const int e = min(max(q1, s.q0), a.T);
    if (s.q0 != q0 || e != q1) flags |= PKV_FLAG_DRAFT_RANGE;
    s.N = e - s.q0;
    const int cap = a.max_pages * kPageSize;
    const int L = __ldg(a.seq_lens + b);
    s.L = min(max(L, 0), cap);
    if (s.N > 0) {
        if (s.L != L) flags |= PKV_FLAG_SEQ_LEN_RANGE;
        if (s.N > s.L || (a.mask != nullptr && s.N > 32 * a.W)) flags |= PKV_FLAG_DRAFT_RANGE;
    }
    s.ctx = s.L - s.N;
    s.R = s.N * a.G;
    s.RG = (s.R + kRows - 1) / kRows;
    return s;
}
// Positions that row group rg can see (a chain's earlier rows see less), and its tiles (at least one: a row
// that sees nothing has an output).
__device__ __forceinline__ int kv_end(const TreeArgs& a, const Seq& s, int rg) {
    if (a.mask != nullptr) return s.L;
    return min(s.L, s.ctx + (min(s.R, (rg + 1) * kRows) - 1) / a.G + 1);
}
__device__ __forceinline__ int tiles_of(const TreeArgs& a, const Seq& s, int rg) {
    return max((kv_end(a, s, rg) + kTile - 1) / kTile, 1);
}
__device__ __forceinline__ int64_t units_per_head(const TreeArgs& a, const Seq& s) {
    if (s.RG <= 1 || a.mask != nullptr) return s.RG ? static_cast<int64_t>(s.RG) * tiles_of(a, s, 0) : 0;
    int64_t n = 0;
    for (int rg = 0; rg < s.RG; ++rg) n += tiles_of(a, s, rg);
    return n;
}

// A place in the order of units: tile t of item k = kvh RG + rg of sequence b.
struct Place {
    int b, k, t;
};
// Unit `off` of sequence b; a cut closer than kSnap to an end of its item moves there.
__device__ __forceinline__ Place place_of(const TreeArgs& a, const Seq& s, int b, int64_t off) {
    const int64_t per = units_per_head(a, s);
    const int kvh = static_cast<int>(off / per);
    int64_t rem = off - kvh * per;
    int rg = 0, nt = tiles_of(a, s, 0);
    while (rem >= nt) {
        rem -= nt;
        nt = tiles_of(a, s, ++rg);
    }
    Place p{b, kvh * s.RG + rg, static_cast<int>(rem)};
    if (p.t < kSnap) {
        p.t = 0;
    } else if (nt - p.t < kSnap) {
        p.t = 0;
        if (++p.k == a.Hkv * s.RG) {
            p.k = 0;
            ++p.b;
        }
    }
    return p;
}

// The pieces of items between two places, in order. Every role walks them by itself.
struct Walk {
    int b, k, t0, t1, nt, kvh, rg, rows;
    Seq s;
    Place end;
    bool first;
    __device__ __forceinline__ Walk(const Place& from, const Place& to) : b(from.b), k(from.k), t0(from.t), end(to), first(true) {}
    // Next piece [t0, t1) of item (b, k); false at the end.
    __device__ __forceinline__ bool next(const TreeArgs& a) {
        int ignored = 0;
        if (first) {
            if (!in_range()) return false;
            first = false;
            s = seq_of(a, b, ignored);
        } else {
            t0 = 0;
            ++k;
        }
        while (k >= a.Hkv * s.RG) {
            k = 0;
            t0 = 0;
            ++b;
            if (!in_range() || b >= a.B) return false;
            s = seq_of(a, b, ignored);
        }
        if (!in_range()) return false;
        kvh = k / s.RG;
        rg = k - kvh * s.RG;
        rows = min(s.R - rg * kRows, kRows);
        nt = tiles_of(a, s, rg);
        t1 = b == end.b && k == end.k ? end.t : nt;
        return true;
    }
    __device__ __forceinline__ bool in_range() const {
        return b < end.b || (b == end.b && (k < end.k || (k == end.k && end.t > t0)));
    }
};

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,"
        "%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
// D (tensor memory) = A (tensor memory) . B^T (+ D): 16-bit A, two values per 32-bit column.
__device__ __forceinline__ void umma_f16_ts_warp(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                                 uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }

// Workspace of partial sums: [2 per CTA][256 rows] of {m, l}, then of D floats.
__device__ __forceinline__ float* part_ml(void* ws, int slot, int row) {
    return reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kMetaBytes) +
           (static_cast<int64_t>(slot) * kRows + row) * 2;
}
template <int D>
__device__ __forceinline__ float* part_o(void* ws, int ctas, int slot, int row) {
    return reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kMetaBytes) + static_cast<int64_t>(ctas) * 2 * kRows * 2 +
           (static_cast<int64_t>(slot) * kRows + row) * D;
}

template <int D, bool FP8>
__global__ void __launch_bounds__(Cfg<D, FP8>::THREADS, 1)
    tree_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv, const TreeArgs a) {
    using C = Cfg<D, FP8>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t s0 = smem_u32(smem);
    enum : int { bFull = 0, bFree = C::ST, bRawFull = 2 * C::ST, bRawFree = bRawFull + C::RST, bS = bRawFree + C::RST,
                 bP = bS + 2, bO = bP + 2, bQ = bO + 2 };
    auto bar = [&](int i) -> uint32_t { return s0 + C::OFF_BAR + 8 * i; };
    uint32_t* misc = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
    uint32_t* bad_tok = misc + 4;                         // [2 jobs][2 groups][4 words]: drafted tokens, V not finite
    Place* place = reinterpret_cast<Place*>(misc + 20);   // [2]: this CTA's first unit and the one past its last
    int64_t* warp_units = reinterpret_cast<int64_t*>(misc + 26);  // [16]

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t num_pages = a.num_pages;

    if (tid == 0) {
        for (int i = 0; i < C::ST; ++i) {
            mbar_init(bar(bFull + i), FP8 ? 4 : 1);
            mbar_init(bar(bFree + i), 1);
        }
        for (int i = 0; i < C::RST; ++i) {
            mbar_init(bar(bRawFull + i), 1);
            mbar_init(bar(bRawFree + i), 4);
        }
        for (int w = 0; w < 2; ++w) {
            mbar_init(bar(bS + w), 1);
            mbar_init(bar(bP + w), 4);
            mbar_init(bar(bO + w), 1);
        }
        mbar_init(bar(bQ), 8);
        *abort_flag = 0;
        place[0] = place[1] = Place{a.B, 0, 0};
        fence_mbar_init();
        tma_prefetch_desc(&tmk);
        tma_prefetch_desc(&tmv);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(misc), 512);
        tmem_relinquish();
    }

    // ---- this CTA's stretch of the units (index inputs only) ------------------
    int64_t total;
    int n_ctas;
    {
        const int seg = (a.B + C::THREADS - 1) / C::THREADS;
        const int b0 = min(tid * seg, a.B), b1 = min(b0 + seg, a.B);
        int64_t sum = 0;
        int flags = 0;
        for (int b = b0; b < b1; ++b) sum += a.Hkv * units_per_head(a, seq_of(a, b, flags));
        if (flags && blockIdx.x == 0) flag_error(a.err, flags);
        int64_t inc = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += y;
        }
        if (lane == 31) warp_units[warp] = inc;
        __syncthreads();
        int64_t base = 0;
        total = 0;
        for (int w = 0; w < C::THREADS / 32; ++w) {
            if (w == warp) base = total;
            total += warp_units[w];
        }
        n_ctas = static_cast<int>(min(static_cast<int64_t>(gridDim.x), (total + kMinUnits - 1) / kMinUnits));
        const int c = blockIdx.x;
        if (c < n_ctas) {
            int64_t at = base + inc - sum;
            const int64_t x[2] = {c * total / n_ctas, (c + 1) * total / n_ctas};
            if (x[1] >= at && x[0] < at + sum) {
                for (int b = b0; b < b1; ++b) {
                    int ignored = 0;
                    const Seq s = seq_of(a, b, ignored);
                    const int64_t n = a.Hkv * units_per_head(a, s);
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (x[e] >= at && x[e] < at + n) place[e] = place_of(a, s, b, x[e] - at);
                    at += n;
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];
    const Place from = place[0], to = place[1];

    // q and the cache may still be being written by the preceding grid.
    grid_dep_wait();
    grid_dep_launch();

    auto give_up = [&]() {
        *abort_flag = 1;
        flag_error(a.err, PKV_FLAG_WAIT_TIMEOUT);
    };
    auto warp_wait = [&](uint32_t bb, uint32_t par) -> bool {
        const bool r = __all_sync(0xffffffffu, mbar_wait_or_abort(bb, par, abort_flag, kWaitLimitNs));
        if (!r && lane == 0) give_up();
        return r;
    };
    // Slot n of the operand ring (K of tile i is 2 i, V is 2 i + 1; tiles are
    // numbered through the CTA's stretch).
    auto stage = [](int n) { return n % C::ST; };
    auto phase = [](int n) -> uint32_t { return (n / C::ST) & 1; };

    if (warp == 0) {
        // ======================= copies ===========================================
        constexpr int RING = FP8 ? C::RST : C::ST;
        constexpr int FULL = FP8 ? bRawFull : bFull, FREE = FP8 ? bRawFree : bFree;
        constexpr int COPIES = FP8 ? kTilePages : kTilePages * C::NB;  // per tile of K or V
        const int pg = lane % kTilePages, blk = lane / kTilePages;     // this lane's copy
        int n = 0;
        bool ok = true;
        Walk w(from, to);
        while (ok && w.next(a)) {
            // evict-first: one read of the cache serves all rows, unless the item has several row groups
            const uint64_t policy = l2_policy_evict_first();
            const int npages = (w.s.L + kPageSize - 1) / kPageSize;
            auto page_at = [&](int t) -> int {
                const int p = t * kTilePages + pg;
                return p < npages && t < w.t1 ? __ldg(a.block_tables + w.b * a.bt_s0 + p) : -1;
            };
            int nxt = page_at(w.t0);
            bool bad = false;
            for (int t = w.t0; ok && t < w.t1; ++t) {
                int id = nxt;
                nxt = page_at(t + 1);
                if (id < 0 || id >= num_pages) {
                    bad |= t * kTilePages + pg < npages;
                    id = static_cast<int>(num_pages);  // out of range: the copy fills zeros
                }
                for (int v = 0; v < 2; ++v, ++n) {
                    const int st = n % RING;
                    if (n >= RING && !warp_wait(bar(FREE + st), (n / RING - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    const uint32_t fb = bar(FULL + st);
                    if (lane == 0) mbar_arrive_expect_tx(fb, FP8 ? C::RAW : C::TILE);
                    __syncwarp();
                    if (lane < COPIES) {
                        const uint32_t dst = FP8 ? s0 + C::OFF_R + st * C::RAW + pg * kPageSize * C::RBOX
                                                 : s0 + C::OFF_T + st * C::TILE + blk * C::BLOCK + pg * kPageSize * 128;
                        const bool hnd = a.layout == PKV_HND;
                        tma_load_4d(dst, v ? &tmv : &tmk, fb, FP8 ? 0 : blk * 64, hnd ? 0 : w.kvh, hnd ? w.kvh : 0, id,
                                    policy);
                    }
                    __syncwarp();
                }
            }
            if (bad && blk == 0) flag_error(a.err, PKV_FLAG_PAGE_RANGE);
        }
        // Copies under way land before the CTA may exit.
        if (lane == 0)
            for (int i = max(n - RING, 0); i < n; ++i) (void)mbar_wait_bounded(bar(FULL + i % RING), (i / RING) & 1, kWaitLimitNs);
        __syncwarp();
    } else if (warp == 1) {
        // ======================= tensor-core issue ================================
        constexpr int FMT = FP8 ? 0 : 1;  // f16 or bf16 operands
        constexpr uint32_t kIdescQk = umma_idesc(128, kTile, FMT, FMT, false, false);
        constexpr uint32_t kIdescPv = umma_idesc(128, D, FMT, FMT, false, true);
        int tile0 = 0, seg = 0;  // tiles before this piece, pieces
        int jobs[2] = {0, 0}, scores[2] = {0, 0};  // P . V and Q . K^T issued per group
        bool ok = true;
        Walk w(from, to);
        while (ok && w.next(a)) {
            const bool two = w.rows > 128;  // each group its own rows of every tile
            const int nt = w.t1 - w.t0, nj = two ? 2 * nt : nt;
            auto tile_of = [&](int j) { return tile0 + (two ? j >> 1 : j); };
            auto qk = [&](int j) -> bool {
                const int g = j & 1, n = 2 * tile_of(j);
                if (!warp_wait(bar(bFull + stage(n)), phase(n))) return false;
                tc_fence_after();
                const uint32_t q = s0 + C::OFF_Q + (two ? g * C::TILE : 0), kt = s0 + C::OFF_T + stage(n) * C::TILE;
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    umma_f16_warp(tmem + 256 * g, umma_desc_sw128(q + (k >> 2) * C::BLOCK + (k & 3) * 32, 16, 1024),
                                  umma_desc_sw128(kt + (k >> 2) * C::BLOCK + (k & 3) * 32, 16, 1024), kIdescQk, k > 0);
                umma_commit_warp(bar(bS + g));
                if (!two || g == 1) umma_commit_warp(bar(bFree + stage(n)));
                ++scores[g];
                return true;
            };
            auto pv = [&](int j) -> bool {
                const int g = j & 1, n = 2 * tile_of(j) + 1;
                if (!warp_wait(bar(bP + g), jobs[g] & 1)) return false;
                if (!warp_wait(bar(bFull + stage(n)), phase(n))) return false;
                tc_fence_after();
                const uint32_t vt = s0 + C::OFF_T + stage(n) * C::TILE;
#pragma unroll
                for (int k = 0; k < kTile / 16; ++k)
                    umma_f16_ts_warp(tmem + 256 * g + C::O_COL, tmem + 256 * g + C::P_COL + 8 * k,
                                     umma_desc_sw128(vt + k * 2048, C::BLOCK, 1024), kIdescPv, j > 1 || k > 0);
                umma_commit_warp(bar(bO + g));
                if (!two || g == 1) umma_commit_warp(bar(bFree + stage(n)));
                ++jobs[g];
                return true;
            };
            ok = warp_wait(bar(bQ), seg & 1);
            ++seg;
            ok = ok && qk(0) && (nj < 2 || qk(1));
            for (int j = 0; ok && j < nj; ++j) ok = pv(j) && (j + 2 >= nj || qk(j + 2));
            tile0 += nt;
        }
        // Every operation issued is done before the tensor memory is freed:
        // the softmax groups wait for their last O, and give-ups for both here.
        if (!ok) {
            for (int g = 0; g < 2; ++g) {
                if (scores[g] > 0) (void)mbar_wait_bounded(bar(bS + g), (scores[g] - 1) & 1, kWaitLimitNs);
                if (jobs[g] > 0) (void)mbar_wait_bounded(bar(bO + g), (jobs[g] - 1) & 1, kWaitLimitNs);
            }
        }
    } else if (warp >= 4 && warp < 12) {
        // ======================= softmax ==========================================
        const int grp = (warp - 4) >> 2, wq = warp & 3;
        const int row_l = 32 * wq + lane;              // this thread's lane of tensor memory
        const uint32_t tl = tmem + (static_cast<uint32_t>(wq) << 21);  // lanes 32 wq .. (bits 16 and up)
        const uint32_t tS = tl + 256 * grp, tP = tS + C::P_COL, tO = tS + C::O_COL;
        float* q_scale = reinterpret_cast<float*>(smem + C::OFF_SC);
        int tile0 = 0, job = 0;  // tiles before this piece, this group's jobs
        bool ok = true;
        Walk w(from, to);
        while (w.next(a)) {
            const bool two = w.rows > 128;
            const int r0 = w.rg * kRows;               // the item's first row
            // ---- Q rows into the operand tiles (128-byte swizzle) ------------------
            {
                const int stid = tid - 128;            // 0 .. 255
                constexpr int CH = D / 8;              // 16-byte chunks per row
                const int n_rows = two ? kRows : 128;
                const int ch = stid % CH;
                const bool neg = a.scale_log2 < 0.f;   // the sign of the scale goes into q
                for (int r = stid / CH; r < n_rows; r += 256 / CH) {
                    uint4 x = make_uint4(0u, 0u, 0u, 0u);
                    if (r < w.rows) {
                        const int i = (r0 + r) / a.G, g = (r0 + r) - i * a.G;
                        x = *reinterpret_cast<const uint4*>(a.q + (w.s.q0 + i) * a.q_s0 + (w.kvh * a.G + g) * a.q_s1 + 8 * ch);
                    }
                    if (neg) {
                        x.x ^= 0x80008000u;
                        x.y ^= 0x80008000u;
                        x.z ^= 0x80008000u;
                        x.w ^= 0x80008000u;
                    }
                    if constexpr (FP8) {
                        // 2^k with 2^k max|q| in [2^14, 2^15): exponent arithmetic on the row's largest value
                        const uint32_t v[4] = {x.x, x.y, x.z, x.w};
                        uint32_t mx = 0;
#pragma unroll
                        for (int e = 0; e < 4; ++e) mx = max(mx, max(v[e] & 0x7F80u, (v[e] >> 16) & 0x7F80u));
#pragma unroll
                        for (int d = 1; d < CH; d <<= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                        int ex = static_cast<int>(mx >> 7);                    // biased exponent
                        ex = ex == 255 ? 127 : max(ex, 20);                    // not finite: as it is; tiny rows: 2^121
                        const float up = __uint_as_float(static_cast<uint32_t>(127 + 141 - ex) << 23);
                        if (ch == 0) q_scale[r] = __uint_as_float(static_cast<uint32_t>(127 + ex - 141) << 23);
                        x.x = pack_f16(bf16_lo(v[0]) * up, bf16_hi(v[0]) * up);
                        x.y = pack_f16(bf16_lo(v[1]) * up, bf16_hi(v[1]) * up);
                        x.z = pack_f16(bf16_lo(v[2]) * up, bf16_hi(v[2]) * up);
                        x.w = pack_f16(bf16_lo(v[3]) * up, bf16_hi(v[3]) * up);
                    }
                    sts128u(s0 + C::OFF_Q + (r >> 7) * C::TILE + (ch >> 3) * C::BLOCK + (r & 127) * 128 + ((ch ^ r) & 7) * 16, x.x, x.y,
                            x.z, x.w);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(bQ));
                // the other warps wrote parts of the row scales
                if (FP8) ok = named_bar_and(1, 256, ok);
            }
            const int row = two ? 128 * grp + row_l : row_l;
            const bool live = row < w.rows;
            const bool warp_live = (two ? 128 * grp : 0) + 32 * wq < w.rows;
            const int tok = live ? (r0 + row) / a.G : 0;         // this row's drafted token
            const uint32_t* mrow = a.mask != nullptr && live ? a.mask + (w.s.q0 + tok) * a.mask_s0 : nullptr;
            float sl = fabsf(a.scale_log2);
            float vs = 1.f;
            if constexpr (FP8) {
                sl *= __ldg(a.k_scale + (a.n_scale == 1 ? 0 : w.kvh)) * q_scale[row];
                vs = __ldg(a.v_scale + (a.n_scale == 1 ? 0 : w.kvh));
            }
            const int L = w.s.L, ctx = w.s.ctx;
            const int npages = (L + kPageSize - 1) / kPageSize;
            const int job0 = job;
            float m = -INFINITY, l = 0.f;
            const int step = two ? 1 : 2;
            auto page_ok = [&](int t) -> uint32_t {
                bool good = true;
                if (t < w.t1 && lane < kTilePages && t * kTilePages + lane < npages) {
                    const int id = __ldg(a.block_tables + w.b * a.bt_s0 + t * kTilePages + lane);
                    good = id >= 0 && id < num_pages;
                }
                return __ballot_sync(0xffffffffu, good);
            };
            const int tb = w.t0 + (two ? 0 : grp);
            uint32_t pages = page_ok(tb);
            for (int t = tb; t < w.t1; t += step, ++job) {
                const int p0 = t * kTile;
                const int n = 2 * (tile0 + t - w.t0) + 1;        // ring slot of the tile's V
                const uint32_t pages_now = pages;
                pages = page_ok(t + step);
                const bool inner = p0 + kTile <= ctx && pages_now == ~0u;
                uint32_t vis[4] = {~0u, ~0u, ~0u, ~0u};
                if (!inner) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int q0 = p0 + 32 * k, j0 = q0 - ctx;
                        uint32_t v = live ? low_bits(L - q0) : 0u;
                        if (j0 > -32) {
                            if (a.mask == nullptr) {
                                v &= low_bits(tok - j0 + 1);
                            } else if (live) {
                                const int wd = j0 >> 5;
                                const uint32_t lo = wd < 0 ? ~0u : wd < a.W ? __ldg(mrow + wd) : 0u;
                                const uint32_t hi = wd + 1 < a.W ? __ldg(mrow + wd + 1) : 0u;
                                v &= __funnelshift_r(lo, hi, j0 & 31);
                            }
                        }
                        if (!(pages_now >> (2 * k) & 1)) v &= 0xFFFF0000u;
                        if (!(pages_now >> (2 * k + 1) & 1)) v &= 0x0000FFFFu;
                        vis[k] = v;
                    }
                }
                // The scores first: they tell that every slot up to this tile's K
                // has landed, so the wait for V below is at most one phase ahead.
                if (ok) ok = warp_wait(bar(bS + grp), job & 1);
                tc_fence_after();
                // ---- V rows that a weight of zero would not silence --------------------
                uint32_t bad[4] = {0u, 0u, 0u, 0u};
                if (p0 + kTile > ctx) {
                    const bool landed = ok && warp_wait(bar(bFull + stage(n)), phase(n));
                    const int pos = p0 + row_l;                  // thread = row of the tile here
                    const uint32_t vrow = s0 + C::OFF_T + stage(n) * C::TILE + row_l * 128;
                    bool odd = false;
                    if (landed && pos >= ctx && pos < L) {
                        constexpr uint32_t EX = FP8 ? 0x7C00u : 0x7F80u;
#pragma unroll
                        for (int c = 0; c < D / 8; ++c) {
                            const uint4 x = lds128(vrow + (c >> 3) * C::BLOCK + ((c ^ row_l) & 7) * 16);
                            const uint32_t v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) odd |= (v[e] & EX) == EX || (v[e] >> 16 & EX) == EX;
                        }
                    }
                    const uint32_t word = __ballot_sync(0xffffffffu, odd);
                    uint32_t* words = bad_tok + 8 * (job & 1) + 4 * grp;
                    if (lane == 0) words[wq] = word;
                    // all who share the tile have looked at it before a row is zeroed
                    ok = two ? named_bar_and(1, 256, landed) : named_bar_and(2 + grp, 128, landed);
#pragma unroll
                    for (int k = 0; k < 4; ++k) bad[k] = words[k];
                    if (ok && (odd || pos >= L)) {
#pragma unroll
                        for (int c = 0; c < D / 8; ++c) sts128u(vrow + (c >> 3) * C::BLOCK + c % 8 * 16, 0u, 0u, 0u, 0u);
                    }
                    fence_proxy_async_smem();
                }
                if (ok && warp_live) {
                    // ---- tile maximum ----------------------------------------------------
                    float mx = -INFINITY;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t x[32];
                        tmem_ld32(tS + 32 * c, x);
                        tmem_wait_ld();
                        if (inner) {
#pragma unroll
                            for (int e = 0; e < 32; ++e) mx = fmaxf(mx, __uint_as_float(x[e]));
                        } else {
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                mx = fmaxf(mx, (vis[c] >> e & 1) ? __uint_as_float(x[e]) : -INFINITY);
                        }
                    }
                    mx *= sl;
                    if (!(mx == mx)) mx = -INFINITY;             // 0 x -inf: a scale of zero and nothing seen
                    const bool move = mx > m + kRescaleLog2 || (m == -INFINITY && mx > m);
                    if (__any_sync(0xffffffffu, move)) {
                        const float nm = move ? mx : m;
                        const float al = move ? fast_exp2(m - nm) : 1.f;
                        if (job > job0) {
                            ok = warp_wait(bar(bO + grp), (job - 1) & 1);
                            tc_fence_after();
#pragma unroll
                            for (int c = 0; c < D / 16; ++c) {
                                uint32_t o[16];
                                tmem_ld16(tO + 16 * c, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * al);
                                tmem_st16(tO + 16 * c, o);
                            }
                        }
                        l *= al;
                        m = nm;
                    }
                    // ---- weights ------------------------------------------------------------
                    const float mm = m == -INFINITY ? 0.f : m;
                    float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t x[32], p[16];
                        tmem_ld32(tS + 32 * c, x);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float p0f = fast_exp2(fmaf(__uint_as_float(x[2 * e]), sl, -mm));
                            float p1f = fast_exp2(fmaf(__uint_as_float(x[2 * e + 1]), sl, -mm));
                            if (!inner) {
                                if (!(vis[c] >> (2 * e) & 1)) p0f = 0.f;
                                if (!(vis[c] >> (2 * e + 1) & 1)) p1f = 0.f;
                            }
                            s4[(2 * e) & 3] += p0f;
                            s4[(2 * e + 1) & 3] += p1f;
                            if (!inner) {
                                if (bad[c] >> (2 * e) & 1) p0f = 0.f;
                                if (bad[c] >> (2 * e + 1) & 1) p1f = 0.f;
                            }
                            p[e] = FP8 ? pack_f16(p0f, p1f) : pack_bf16(p0f, p1f);
                        }
                        tmem_st16(tP + 16 * c, p);
                    }
                    l += (s4[0] + s4[1]) + (s4[2] + s4[3]);
                    tmem_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0 && ok) mbar_arrive(bar(bP + grp));
                // ---- drafted tokens whose V is not finite, for the rows that see them ----
                if ((bad[0] | bad[1] | bad[2] | bad[3]) != 0u) {
                    if (ok) ok = warp_wait(bar(bO + grp), job & 1);
                    tc_fence_after();
                    for (int j = 0; ok && j < kTile; ++j) {
                        if (!(bad[j >> 5] >> (j & 31) & 1)) continue;
                        const int id = __ldg(a.block_tables + w.b * a.bt_s0 + (p0 + j) / kPageSize);
                        if (id < 0 || id >= num_pages) continue;
                        const int off = (p0 + j) % kPageSize;
                        const int64_t kb = id * a.kc_s0 + off * a.kc_st + w.kvh * a.kc_sh;
                        const int64_t vb = id * a.vc_s0 + off * a.vc_st + w.kvh * a.vc_sh;
                        auto at = [&](const void* base, int64_t i) -> float {
                            if constexpr (FP8)
                                return __half2float(__ushort_as_half(static_cast<unsigned short>(
                                    e4m3x2_to_f16x2(static_cast<const uint8_t*>(base)[i]) & 0xFFFFu)));
                            return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(base)[i]) << 16);
                        };
                        const bool sees = live && (vis[j >> 5] >> (j & 31) & 1);
                        float x = 0.f;
                        if (sees) {
                            const int g = (r0 + row) - tok * a.G;
                            const uint16_t* qr = a.q + (w.s.q0 + tok) * a.q_s0 + (w.kvh * a.G + g) * a.q_s1;
                            for (int d = 0; d < D; ++d)
                                x += __uint_as_float(static_cast<uint32_t>(qr[d]) << 16) * at(a.k_cache, kb + d);
                            x *= a.scale_log2 * (FP8 ? __ldg(a.k_scale + (a.n_scale == 1 ? 0 : w.kvh)) : 1.f);
                            x = fast_exp2(x - (m == -INFINITY ? 0.f : m));
                        }
                        for (int c = 0; c < D / 16; ++c) {
                            uint32_t o[16];
                            tmem_ld16(tO + 16 * c, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                if (sees) o[e] = __float_as_uint(fmaf(x, at(a.v_cache, vb + 16 * c + e), __uint_as_float(o[e])));
                            tmem_st16(tO + 16 * c, o);
                            tmem_wait_st();
                        }
                    }
                    tc_fence_before();
                }
            }
            // ---- the piece's sums ---------------------------------------------------
            const bool mine = job > job0;
            if (ok && mine) ok = warp_wait(bar(bO + grp), (job - 1) & 1);
            tc_fence_after();
            float mo = -INFINITY, lo = 0.f;  // the other group's
            const bool theirs = !two && w.t1 - w.t0 > 1 - grp;
            if (!two) {
                uint32_t x[8] = {__float_as_uint(m), __float_as_uint(l), 0u, 0u, 0u, 0u, 0u, 0u};
                tmem_st8(tS, x);
                tmem_wait_st();
            }
            tc_fence_before();
            ok = named_bar_and(1, 256, ok);  // (also: every S of this piece is read, so Q may be overwritten)
            tc_fence_after();
            if (!ok) break;
            if (!two) {
                uint32_t x[8];
                tmem_ld8(tl + 256 * (1 - grp), x);
                tmem_wait_ld();
                mo = __uint_as_float(x[0]);
                lo = __uint_as_float(x[1]);
            }
            if (warp_live) {
                const float M = fmaxf(m, mo);
                const float f0 = m == -INFINITY ? 0.f : fast_exp2(m - M), f1 = mo == -INFINITY ? 0.f : fast_exp2(mo - M);
                const float sum = (mine ? l * f0 : 0.f) + (theirs ? lo * f1 : 0.f);
                const bool whole = w.t0 == 0 && w.t1 == w.nt;
                const bool none = sum == 0.f;
                const float k0 = whole ? (none ? 0.f : f0 * vs / sum) : f0 * vs, k1 = whole ? (none ? 0.f : f1 * vs / sum) : f1 * vs;
                const int g = (r0 + row) - tok * a.G, h = w.kvh * a.G + g;
                const int slot = 2 * static_cast<int>(blockIdx.x) + (w.t0 == 0 ? 1 : 0);
                uint16_t* out = a.out + (w.s.q0 + tok) * a.o_s0 + h * a.o_s1;
                float* part = part_o<D>(a.workspace, gridDim.x, slot, row);
                if (live && (two || grp == 0)) {
                    if (!whole) {
                        float* ml = part_ml(a.workspace, slot, row);
                        ml[0] = M;
                        ml[1] = sum;
                    } else if (a.lse) {
                        a.lse[(w.s.q0 + tok) * a.l_s0 + h * a.l_s1] =
                            none ? -INFINITY : (M + __log2f(sum)) * 0.69314718055994530942f;
                    }
                }
                // two row groups: all of this row's columns; else each group half of them
                const int c0 = two ? 0 : grp * (D / 32), c1 = two ? D / 16 : c0 + D / 32;
#pragma unroll 1
                for (int c = c0; c < c1; ++c) {
                    uint32_t x[16], y[16];
                    if (mine) tmem_ld16(tO + 16 * c, x);
                    if (theirs) tmem_ld16(tl + 256 * (1 - grp) + C::O_COL + 16 * c, y);
                    tmem_wait_ld();
                    float o[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        o[e] = mine ? __uint_as_float(x[e]) * k0 : 0.f;
                        if (theirs) o[e] = fmaf(__uint_as_float(y[e]), k1, o[e]);
                    }
                    if (!live) continue;
                    if (whole) {
                        uint32_t p[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) p[e] = pack_bf16(o[2 * e], o[2 * e + 1]);
                        uint4* dst = reinterpret_cast<uint4*>(out + 16 * c);
                        dst[0] = make_uint4(p[0], p[1], p[2], p[3]);
                        dst[1] = make_uint4(p[4], p[5], p[6], p[7]);
                    } else {
                        float4* dst = reinterpret_cast<float4*>(part + 16 * c);
#pragma unroll
                        for (int e = 0; e < 4; ++e) dst[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    }
                }
            }
            tc_fence_before();
            named_bar_and(1, 256, true);  // O, m and l are read
            tile0 += w.t1 - w.t0;
        }
    } else if (FP8 && warp >= 12) {
        // ======================= E4M3 bytes to f16 tiles ==========================
        const int ct = tid - 384;
        constexpr int CH = D / 16;  // 16-byte chunks of a raw row
        int n = 0;
        bool ok = true;
        Walk w(from, to);
        while (ok && w.next(a)) {
            for (int t = w.t0; ok && t < w.t1; ++t) {
                for (int v = 0; v < 2; ++v, ++n) {
                    const int rs = n % C::RST;
                    ok = warp_wait(bar(bRawFull + rs), (n / C::RST) & 1);
                    if (ok && n >= C::ST) ok = warp_wait(bar(bFree + stage(n)), (n / C::ST - 1) & 1);
                    if (!ok) break;
                    const uint32_t src = s0 + C::OFF_R + rs * C::RAW, dst = s0 + C::OFF_T + stage(n) * C::TILE;
                    const int ch = ct % CH;
#pragma unroll 4
                    for (int r = ct / CH; r < kTile; r += 128 / CH) {
                        const int sw = C::RBOX == 128 ? (ch ^ r) & 7 : (ch ^ (r >> 1)) & 3;
                        const uint4 x = lds128(src + r * C::RBOX + sw * 16);
                        const uint32_t d0 = dst + (ch >> 2) * C::BLOCK + r * 128;
                        const int c0 = (2 * ch) & 7;
                        const uint32_t e0 = d0 + ((c0 ^ r) & 7) * 16, e1 = d0 + (((c0 + 1) ^ r) & 7) * 16;
                        uint32_t h[8];
                        h[0] = e4m3x2_to_f16x2(static_cast<uint16_t>(x.x)), h[1] = e4m3x2_to_f16x2(static_cast<uint16_t>(x.x >> 16));
                        h[2] = e4m3x2_to_f16x2(static_cast<uint16_t>(x.y)), h[3] = e4m3x2_to_f16x2(static_cast<uint16_t>(x.y >> 16));
                        h[4] = e4m3x2_to_f16x2(static_cast<uint16_t>(x.z)), h[5] = e4m3x2_to_f16x2(static_cast<uint16_t>(x.z >> 16));
                        h[6] = e4m3x2_to_f16x2(static_cast<uint16_t>(x.w)), h[7] = e4m3x2_to_f16x2(static_cast<uint16_t>(x.w >> 16));
                        sts128u(e0, h[0], h[1], h[2], h[3]);
                        sts128u(e1, h[4], h[5], h[6], h[7]);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(bar(bFull + stage(n)));
                        mbar_arrive(bar(bRawFree + rs));
                    }
                }
            }
        }
    }

    // ---- what the joining kernel is to do with this CTA's cut item --------------
    if (warp == 2 && lane == 0) {
        int4 meta = make_int4(0, 0, 0, 0);
        Walk w(from, to);
        while (w.next(a)) {
            if (w.t0 != 0 || w.t1 == w.nt) continue;
            const int64_t i0 = (static_cast<int64_t>(blockIdx.x) + 1) * total / n_ctas - w.t1;
            const int64_t last = i0 + w.nt - kSnap + 1;  // cuts before this unit are inside the item
            const int c1 = min(static_cast<int>((last * n_ctas + total - 1) / total) - 1, n_ctas - 1);
            meta = make_int4(w.s.q0, w.rg * kRows, w.rows | (c1 - static_cast<int>(blockIdx.x) + 1) << 12, w.kvh);
        }
        reinterpret_cast<int4*>(a.workspace)[blockIdx.x] = meta;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

// ---- joining the pieces of cut items ------------------------------------------------
constexpr int kJoinRows = 8;  // rows (warps) per CTA

template <int D>
__global__ void __launch_bounds__(kJoinRows * 32) tree_join_kernel(const TreeArgs a, int ctas) {
    grid_dep_wait();
    const int c = blockIdx.x, lane = threadIdx.x & 31;
    const int row = blockIdx.y * kJoinRows + (threadIdx.x >> 5);
    const int4 meta = reinterpret_cast<const int4*>(a.workspace)[c];
    if (row >= (meta.z & 0xFFF)) return;
    const int n = meta.z >> 12;  // pieces: slot 1 of CTA c, slot 0 of the next ones
    auto slot = [&](int i) { return 2 * (c + i) + (i == 0 ? 1 : 0); };
    float M = -INFINITY;
    for (int i = lane; i < n; i += 32) M = fmaxf(M, part_ml(a.workspace, slot(i), row)[0]);
    M = warp_max(M);
    float sum = 0.f;
    constexpr int V = D / 32;
    float o[V];
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] = 0.f;
#pragma unroll 8
    for (int i = 0; i < n; ++i) {
        const float* ml = part_ml(a.workspace, slot(i), row);
        const float f = ml[0] == -INFINITY ? 0.f : fast_exp2(ml[0] - M);
        const float* p = part_o<D>(a.workspace, ctas, slot(i), row) + V * lane;
        sum += f * ml[1];
        if constexpr (V == 4) {
            const float4 x = *reinterpret_cast<const float4*>(p);
            o[0] += f * x.x, o[1] += f * x.y, o[2] += f * x.z, o[3] += f * x.w;
        } else {
            const float2 x = *reinterpret_cast<const float2*>(p);
            o[0] += f * x.x, o[1] += f * x.y;
        }
    }
    const bool none = sum == 0.f;
    const float inv = none ? 0.f : 1.f / sum;
    const int tok = (meta.y + row) / a.G, h = meta.w * a.G + (meta.y + row) - tok * a.G;
    uint32_t* out = reinterpret_cast<uint32_t*>(a.out + (meta.x + tok) * a.o_s0 + h * a.o_s1 + V * lane);
#pragma unroll
    for (int e = 0; e < V; e += 2) out[e / 2] = pack_bf16(none ? 0.f : o[e] * inv, none ? 0.f : o[e + 1] * inv);
    if (lane == 0 && a.lse)
        a.lse[(meta.x + tok) * a.l_s0 + h * a.l_s1] = none ? -INFINITY : (M + __log2f(sum)) * 0.69314718055994530942f;
}

template <int D, bool FP8>
cudaError_t launch_t(const TreeArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s) {
    using C = Cfg<D, FP8>;
    int sms = 0;
    cudaError_t e = device_sm_count(&sms);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(tree_kernel<D, FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    e = launch_dependent(tree_kernel<D, FP8>, dim3(sms), dim3(C::THREADS), C::SMEM, s, tk, tv, a);
    if (e != cudaSuccess) return e;
    const int rows = static_cast<int>(std::min<int64_t>(kRows, static_cast<int64_t>(a.T) * a.G));
    return launch_dependent(tree_join_kernel<D>, dim3(sms, (rows + kJoinRows - 1) / kJoinRows), dim3(kJoinRows * 32), 0, s, a, sms);
}

}  // namespace

int64_t tree_decode_workspace(int64_t T, int32_t Hq, int32_t D, int32_t sm_count) {
    (void)T, (void)Hq;
    return kMetaBytes + static_cast<int64_t>(sm_count) * 2 * kRows * (D + 2) * 4;
}

cudaError_t launch_tree_decode(const TreeArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s) {
    const bool fp8 = a.kind == kFp8;
    if (a.D == 128) return fp8 ? launch_t<128, true>(a, tk, tv, s) : launch_t<128, false>(a, tk, tv, s);
    return fp8 ? launch_t<64, true>(a, tk, tv, s) : launch_t<64, false>(a, tk, tv, s);
}

}  // namespace pkv
