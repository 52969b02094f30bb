// prompt_attention.cu -- causal attention over packed prompts on the
// fifth-generation tensor cores.
//
// Rows. The tokens of a sequence and the G query heads of a kv head share the
// same K and V. A row tile is 128 / G tokens (rounded down) times G heads on the
// M side of the MMA (128 tensor-memory lanes): q lands in operand layout by
// TMA, and a softmax thread owns one row. One pass over K and V serves two row
// tiles.
//
// Work. An item is (sequence, kv head, pair of row tiles). Its cost is counted
// in keys: those that its last row sees, and kItemKeys for its start and
// output. All items of the call, in order, are cut into equal stretches, one per
// CTA (one CTA per SM), so every CTA does the same amount of work whatever the
// lengths are, with no plan from the host; sums over a sequence's items are
// closed forms. An item that is cut leaves partial sums in the workspace (at
// most two per CTA), which a second kernel joins. Where no item of the whole call is
// longer than what partial sums and joining cost (kSnapKeys), the cuts are moved to
// the next item's start instead.
//
// A CTA's roles:
//   warp 0        TMA loads of K and V, 128 positions at a time
//   warp 1        one thread issues S = Q . K^T and O += P . V (M = 128; P from
//                 tensor memory, V as an MN-major operand: nothing is transposed)
//   warp 2        V of the tiles that some row sees in part: zeroes rows behind
//                 the sequence's end and rows that are not finite, which a
//                 weight of zero would not silence, and notes the latter
//   warp 3        walks the CTA's items, hands the pieces to the other roles, and
//                 loads q by TMA
//   warps 4 - 11,
//   warps 12 - 19 two softmax groups, each with a row tile, S, P and O of its own
//                 in tensor memory. While one group is in its softmax the tensor
//                 cores work for the other: P . V and the next scores of one
//                 group (1024 cycles, D = 128) hide the other's softmax. An
//                 item's first scores are computed while the item before writes
//                 its output. Two threads share a row, 64 positions of a tile
//                 each: 4 warps a group, a thread for a whole row, leave the
//                 exponential unit waiting for the warps' other instructions
//                 (8,192 tokens, 28 heads: 418 us and not 390 at that step; D = 64, 32
//                 heads, 408 and not 343).
//
// Softmax. The weights are exp2(score - m) with a reference m per row: the
// maximum of the tile where it last moved. It moves where the sum of a half's 64
// weights passes 2^12, by 2^6 at least; the row's two threads agree on
// that at a barrier of their two warps, which they need anyway before P goes over
// S. So one pass over S does, with no maximum in it, and O is scaled rarely (a
// maximum in every tile: 1949 us and not 1566 for 16,384 tokens, with the MMAs from one
// thread). fp32 holds what is between: nothing that counts underflows, and a tile adds at
// most 2^13 times its largest value to O. Sums and O are fp32. The tensor cores cut a
// product off below about 2^-25 of the sum it goes to, so a sum over n keys of one
// sign falls short by about n 2^-27 of itself (v = 1 with a tenth of noise, 2^20 keys: 0.4
// to 0.65%; 2^27 ones: a half). After kFold tiles, 2^16 keys, O therefore goes to the
// workspace and starts anew: a piece of its own, added to what is there at its output.
// P meets V as bf16, rounded once (by at most 2^-8 of a weight): that rounding
// and the output's are of one size, and independent (the output is off by 2.0 to 2.3e-3
// relative to its norm, 1.5e-3 of it the output's own rounding). The weight of the
// maximum itself is one and exact, so rows of a few keys lose less (2 prompts of 45
// and 54 tokens 1.8e-3; with a reference rounded up to a whole number 2.1 to 2.5e-3, and
// 32 of 1 to 2048 tokens 2.3e-3 and not 2.0), and a row that sees one key gives its
// value. A second term, as in the attention of drafted tokens, is half as much tensor
// work again.
//
// Bound: the tensor cores' turns with the softmax. 16,384 tokens of 28 heads, D = 128:
// 1264 us, 1.52 PFLOP/s, 79% of the rate of a large library product; a group's softmax
// of a tile (1400 cycles) and the hand-overs are a little longer than the other
// group's MMAs. D = 64, 8,192 tokens of 32 heads: 323 us, 0.85 PFLOP/s; the same softmax
// beside half the tensor work. Short prompts: an item's start, the tile on the diagonal
// and the output (32 prompts of 1 to 2048 tokens, 32 heads: 187 us, 0.81 PFLOP/s of
// visible pairs).
//
// Waits. The thread that copies K and V is the one that keeps time: what it waits
// for comes within a tile's turn of the others, whatever the length of an item, and
// with its last copy done it waits for the other roles' end. After a second
// without that it sets a CTA-wide flag, which ends the others' waits and the call
// with PKV_FLAG_WAIT_TIMEOUT. The others keep no time, as some of their waits last as
// long as an item. From the flag on, copies, MMAs and V's warp leave their
// tiles; the softmax warps go through the pieces in the ring, no longer waiting.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "pkv_internal.h"
#include "pkv_ptx.cuh"
#include "umma_row.cuh"

namespace pkv {
namespace {

constexpr int kTile = 128;      // positions per tile
// What an item costs beyond its tiles, in keys. (256, 512 and 768: 8,192 tokens, 28 heads 348, 331, 335 us; 32 prompts of 1
// to 2048 tokens, 32 heads 193, 199, 218, D = 64 156, 165, 183; 2 prompts of 1,000 tokens 36.7, 39.2, 39.2.)
constexpr int kItemKeys = 512;
// Longest item (keys and kItemKeys) up to which a call's items are not cut. (0, 1024, 1536 and 2560, 32 heads of 128: a prompt of
// 600 tokens 22.5, 22.4, 16.9, 16.8 us; of 1,000 31.8, 31.7, 22.1, 22.0; 2 of 1,000 39.7, 39.7, 39.2, 33.2; 4 of 500 31.5,
// 29.6, 29.7, 24.5; the ragged prompts above, D = 64, 166, 166, 165, 171.)
constexpr int kSnapKeys = 1536;
constexpr int kPieces = 4;      // ring of pieces
constexpr int kFold = 512;      // most tiles of a piece
constexpr float kRaise = 4096.f; // sum of 64 weights past which their row's reference moves
constexpr uint64_t kWaitLimitNs = 1000000000ull;
constexpr int kFix = 4;         // ring of the fixed tiles' notes: no fewer than there are stages of V

template <int D>
struct Cfg {
    static constexpr int NB = D / 64;            // 128-byte column blocks of an operand row
    static constexpr int TILE = kTile * D * 2;
    static constexpr int BLOCK = kTile * 128;    // one column block of it
    static constexpr int SK = D == 128 ? 2 : 4, SV = D == 128 ? 3 : 4;  // stages of K, of V
    static constexpr int THREADS = 640;
    // (96 registers a thread, the same for all roles: handing them over from the copies' and the MMAs' warps made
    // those spill, which took 10% more)
    static constexpr int OFF_Q = 0;              // two row tiles of q
    static constexpr int OFF_K = OFF_Q + 2 * TILE;
    static constexpr int OFF_V = OFF_K + SK * TILE;
    static constexpr int OFF_BAR = OFF_V + SV * TILE;
    static constexpr int NBAR = 2 * SK + 2 * SV + kFix + 2 * 6 + 1 + 2 * kPieces + 8 + 1;
    static constexpr int OFF_MISC = OFF_BAR + 8 * NBAR;
    static constexpr int OFF_PIECE = (OFF_MISC + 128 + 2048 + 128 + 15) / 16 * 16;  // [kPieces] Piece
    static constexpr int SMEM = OFF_PIECE + kPieces * 80;
    static_assert(SMEM <= 232448, "shared memory of one CTA");
    // tensor-memory columns of a softmax group: S (P over it), then O
    static constexpr uint32_t O_COL = 128;
};

struct Seq {
    int q0, N, k0, L, ctx, RG, W;  // W: tokens of a pair of row tiles
    // Keys that pair rg may see (where there are fewer keys than tokens: that many, the rest masked).
    __device__ __forceinline__ int end(int rg) const { return max(ctx, 0) + min(N, (rg + 1) * W); }
    __device__ __forceinline__ int tiles(int rg) const { return (end(rg) + kTile - 1) / kTile; }
    // Cost of the pairs before rg < RG, and of all of them.
    __device__ __forceinline__ int64_t before(int64_t rg) const {
        return rg * (kItemKeys + max(ctx, 0)) + rg * (rg + 1) / 2 * W;
    }
    __device__ __forceinline__ int64_t all() const { return RG ? before(RG - 1) + kItemKeys + end(RG - 1) : 0; }
};
// Sequence b, its values clamped; `flags` collects what was out of range.
__device__ __forceinline__ Seq seq_of(const PromptArgs& a, int b, int& flags) {
    Seq s;
    const int q0 = __ldg(a.q_start + b), q1 = __ldg(a.q_start + b + 1);
    s.q0 = min(max(q0, 0), a.T);
    const int e = min(max(q1, s.q0), a.T);
    s.N = e - s.q0;
    s.k0 = s.q0;
    s.L = s.N;
    bool bad = s.q0 != q0 || e != q1;
    if (a.k_start != nullptr) {
        const int k0 = __ldg(a.k_start + b), k1 = __ldg(a.k_start + b + 1);
        s.k0 = min(max(k0, 0), a.Tk);
        s.L = min(max(k1, s.k0), a.Tk) - s.k0;
        bad |= s.k0 != k0 || s.k0 + s.L != k1 || s.N > s.L;
    }
    if (bad) flags |= PKV_FLAG_ROW_RANGE;
    s.ctx = s.L - s.N;
    s.W = 2 * a.tile_toks;
    s.RG = s.N <= s.W ? (s.N > 0) : (s.N + s.W - 1) / s.W;
    return s;
}

// CTA c of n starts at unit cut(c); the first total % n stretches are one unit longer.
struct Cuts {
    int n;
    int64_t per, rem;
    __device__ __forceinline__ Cuts(int64_t total, int ctas) : n(0), per(0), rem(0) {
        // (stretches of a tile and more: cuts of one item are a tile apart)
        n = static_cast<int>(min(static_cast<int64_t>(ctas), (total + kTile - 1) / kTile));
        if (n > 1 && total / n < kTile) --n;
        if (n > 0) {
            per = total / n;
            rem = total - per * n;
        }
    }
    __device__ __forceinline__ int64_t cut(int c) const { return c * per + min(static_cast<int64_t>(c), rem); }
    // the last CTA that starts at or before unit x
    __device__ __forceinline__ int at_or_before(int64_t x) const {
        const int64_t c = x < rem * (per + 1) ? x / (per + 1) : rem + (x - rem * (per + 1)) / per;
        return static_cast<int>(min(c, static_cast<int64_t>(n - 1)));
    }
};

// A place in the order of items: tile t of item k = kvh RG + rg of sequence b; the item's first unit.
struct Place {
    int b, k, t, pad;
    int64_t item;
};
// Unit `off` of sequence b, whose first unit is `base`.
__device__ __forceinline__ Place place_of(const Seq& s, int64_t per_head, int b, int64_t base, int64_t off, bool snap) {
    const int kvh = static_cast<int>(off / per_head);
    const int64_t rem = off - kvh * per_head;
    // the last rg with before(rg) <= rem
    const double w = s.W, h = kItemKeys + max(s.ctx, 0) + 0.5 * w;
    int rg = static_cast<int>((sqrt(h * h + 2.0 * w * static_cast<double>(rem)) - h) / w);
    rg = min(max(rg, 0), s.RG - 1);
    while (rg > 0 && s.before(rg) > rem) --rg;
    while (rg + 1 < s.RG && s.before(rg + 1) <= rem) ++rg;
    const int64_t in = rem - s.before(rg);
    Place p{b, kvh * s.RG + rg, 0, 0, base + kvh * per_head + s.before(rg)};
    if (snap) {
        if (in > 0) ++p.k;  // (which may be one past the sequence's last)
    } else {
        p.t = static_cast<int>(max(in - kItemKeys, static_cast<int64_t>(0)) / kTile);
    }
    return p;
}

// The pieces of items between two places, in order.
struct Walk {
    int b, k, t0, t1, nt, kvh, rg;
    Seq s;
    Place end;
    bool first;
    __device__ __forceinline__ Walk(const Place& from, const Place& to)
        : b(from.b), k(from.k), t0(from.t), end(to), first(true) {}
    // Next piece [t0, t1) of item (b, k); false at the end.
    __device__ __forceinline__ bool next(const PromptArgs& a) {
        int ignored = 0;
        bool load = first;
        if (!first) {
            t0 = 0;
            load = ++k >= a.Hkv * s.RG;
            if (load) {
                k = 0;
                ++b;
            }
        }
        first = false;
        for (;; ++b, k = 0, load = true) {  // past the sequences without tokens
            if (b >= a.B || !in_range()) return false;
            if (load) s = seq_of(a, b, ignored);
            if (k < a.Hkv * s.RG) break;
        }
        kvh = s.RG == 1 ? k : k / s.RG;
        rg = k - kvh * s.RG;
        nt = s.tiles(rg);
        t1 = b == end.b && k == end.k ? end.t : nt;
        return true;
    }
    __device__ __forceinline__ bool in_range() const {
        return b < end.b || (b == end.b && (k < end.k || (k == end.k && end.t > t0)));
    }
};

// A piece: tiles [t0, t1) of an item, all of the CTA's or kFold of them (the tokens [tok0, tok0 + toks) of sequence b).
struct Piece {
    int b, kvh, q0, k0;      // b < 0: there are no more
    int L, ctx, tok0, toks;
    int t0, t1, whole, two;  // whole: with it, all of the item; two: two row tiles
    int tf;                  // tiles before this one are seen in full by every row
    int end[2];              // keys that either row tile may see
    int cont;                // the item goes on: its O so far is in the workspace
    int slot;                // where there: 1 if the CTA has the item's first tile
    int pad[3];
};
static_assert(sizeof(Piece) == 80, "as laid out");

template <int D>
__global__ void __launch_bounds__(Cfg<D>::THREADS, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                  const __grid_constant__ CUtensorMap tmv, const PromptArgs a) {
    using C = Cfg<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t s0 = smem_u32(smem);
    enum : int { bKFull = 0, bKFree = C::SK, bVFull = 2 * C::SK, bVFree = bVFull + C::SV, bFix = bVFree + C::SV,
                 bS = bFix + kFix, bP = bS + 2, bO = bP + 2, bOFree = bO + 2, bQ = bOFree + 2, bQFree = bQ + 2,
                 bPiece = bQFree + 2, bPieceFree = bPiece + kPieces, bEnd = bPieceFree + kPieces,
                 bPair = bEnd + 1, bDone = bPair + 8 };
    static_assert(bDone + 1 == C::NBAR, "barriers");
    auto bar = [&](int i) -> uint32_t { return s0 + C::OFF_BAR + 8 * i; };
    uint32_t* misc = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
    volatile uint32_t* go_on = misc + 2;                       // [2 groups]: O has been started by hand
    volatile uint32_t* bad_rows = misc + 4;                    // [kFix][4 words]: rows of V that are not finite
    Place* place = reinterpret_cast<Place*>(misc + 20);                 // [2]: from, to
    int64_t* warp_units = reinterpret_cast<int64_t*>(misc + 32);        // [THREADS / 32]
    int* warp_longest = reinterpret_cast<int*>(misc + 72);              // [THREADS / 32]
    float* theirs = reinterpret_cast<float*>(misc + 32);                // (later) [2 groups][2 halves][128 rows]: what the halves tell each other
    volatile int* handed_out = reinterpret_cast<volatile int*>(misc + 544);  // pieces, where a give-up ended them (else -1)
    volatile uint32_t* pair_uses = misc + 545;                 // [2 groups][4 pairs][2 halves]
    static_assert(sizeof(Place) == 24, "as laid out");
    Piece* pieces = reinterpret_cast<Piece*>(smem + C::OFF_PIECE);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    if (tid == C::THREADS - 32) {  // (the first threads have sequences to look at)
        for (int i = 0; i < C::SK; ++i) {
            mbar_init(bar(bKFull + i), 1);
            mbar_init(bar(bKFree + i), 1);
        }
        for (int i = 0; i < C::SV; ++i) {
            mbar_init(bar(bVFull + i), 1);
            mbar_init(bar(bVFree + i), 2);  // the last P . V, and warp 2
        }
        static_assert(kFix >= C::SV, "a note lasts as long as its tile");
        for (int i = 0; i < kFix; ++i) mbar_init(bar(bFix + i), 1);
        for (int w = 0; w < 2; ++w) {
            mbar_init(bar(bS + w), 1);
            mbar_init(bar(bP + w), 8);
            mbar_init(bar(bO + w), 1);
            mbar_init(bar(bOFree + w), 8);
            mbar_init(bar(bQ + w), 1);
            mbar_init(bar(bQFree + w), 1);
        }
        for (int i = 0; i < kPieces; ++i) {
            mbar_init(bar(bPiece + i), 1);
            mbar_init(bar(bPieceFree + i), 19);  // copies, MMA, V, softmax
        }
        mbar_init(bar(bEnd), 1);
        for (int i = 0; i < 8; ++i) mbar_init(bar(bPair + i), 2);
        mbar_init(bar(bDone), C::THREADS / 32 - 1);  // all warps but the copies'
        for (int i = 0; i < 16; ++i) pair_uses[i] = 0u;
        *handed_out = -1;
        *abort_flag = 0;
        place[0] = place[1] = Place{a.B, 0, 0, 0, 0};
        fence_mbar_init();
        tma_prefetch_desc(&tmq);
        tma_prefetch_desc(&tmk);
        tma_prefetch_desc(&tmv);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(misc), 512);
        tmem_relinquish();
    }

    // ---- this CTA's stretch (index inputs only) --------------------------------
    int64_t total = 0;
    bool snap = false;
    {
        const int seg = (a.B + C::THREADS - 1) / C::THREADS;
        const int b0 = min(tid * seg, a.B), b1 = min(b0 + seg, a.B);
        int64_t sum = 0, per = 0;
        int flags = 0, longest = 0;
        Seq s{};
        for (int b = b0; b < b1; ++b) {
            s = seq_of(a, b, flags);
            per = s.all();
            sum += a.Hkv * per;
            if (s.RG) longest = max(longest, kItemKeys + s.end(s.RG - 1));
        }
        if (flags && blockIdx.x == 0) flag_error(a.err, flags);
        int64_t inc = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += y;
        }
        longest = __reduce_max_sync(0xffffffffu, longest);
        if (lane == 31) {
            warp_units[warp] = inc;
            warp_longest[warp] = longest;
        }
        __syncthreads();
        int64_t base = 0;
        for (int w = 0; w < C::THREADS / 32; ++w) {
            if (w == warp) base = total;
            total += warp_units[w];
            longest = max(longest, warp_longest[w]);
        }
        snap = longest <= kSnapKeys;
        const Cuts cuts(total, gridDim.x);
        const int c = blockIdx.x;
        int64_t at = base + inc - sum;
        if (c < cuts.n && sum > 0) {
            const int64_t x0 = cuts.cut(c), x1 = cuts.cut(c + 1);
            if (x1 >= at && x0 < at + sum) {
                for (int b = b0; b < b1; ++b) {
                    if (seg > 1) {
                        int ignored = 0;
                        s = seq_of(a, b, ignored);
                        per = s.all();
                    }
                    const int64_t n = a.Hkv * per;
                    if (x0 >= at && x0 < at + n) place[0] = place_of(s, per, b, at, x0 - at, snap);
                    if (x1 >= at && x1 < at + n) place[1] = place_of(s, per, b, at, x1 - at, snap);
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

    // q, k and v may still be being written by the preceding grid: every role waits for it.
    //
    // Waits that the copying thread watches over. One that is given up on returns like any other: what follows works
    // on what is there, in bounds, until the role leaves. (try_wait holds the warp until the phase is over, for about
    // 1 us; polling with test_wait takes the issue slots of the others: 347 us and not 333.)
    auto lane_wait = [&](uint32_t bb, uint32_t par) -> bool { return mbar_wait_watched(bb, par, abort_flag); };
    auto warp_wait = [&](uint32_t bb, uint32_t par) -> bool { return mbar_warp_wait_watched(bb, par, abort_flag); };
    auto piece_bar = [&](int i) { return bar(bPiece + i % kPieces); };
    auto piece_par = [](int i) -> uint32_t { return (i / kPieces) & 1; };

    if (warp < 4) {
        if (warp == 0 && lane == 0) {
            // ======================= copies of K and V ================================
            grid_dep_wait();
            int nk = 0, nv = 0;  // tiles of K, of V
            auto timed_wait = [&](uint32_t bb, uint32_t par) -> bool {
                if (mbar_wait_or_abort(bb, par, abort_flag, kWaitLimitNs)) return true;
                *abort_flag = 1;
                return false;
            };
            for (int i = 0; timed_wait(piece_bar(i), piece_par(i)); ++i) {
                const Piece w = pieces[i % kPieces];
                mbar_arrive(bar(bPieceFree + i % kPieces));
                if (w.b < 0) break;
                bool ok = true;
                for (int t = w.t0; t < w.t1; ++t) {
                    const int row = w.k0 + t * kTile;
                    const int sk = nk % C::SK, sv = nv % C::SV;
                    ok = nk < C::SK || timed_wait(bar(bKFree + sk), (nk / C::SK - 1) & 1);
                    if (!ok) break;
                    mbar_arrive_expect_tx(bar(bKFull + sk), C::TILE);
                    for (int c = 0; c < C::NB; ++c)
                        tma_load_3d(s0 + C::OFF_K + sk * C::TILE + c * C::BLOCK, &tmk, bar(bKFull + sk), 64 * c, w.kvh,
                                    row);
                    ++nk;
                    ok = nv < C::SV || timed_wait(bar(bVFree + sv), (nv / C::SV - 1) & 1);
                    if (!ok) break;
                    mbar_arrive_expect_tx(bar(bVFull + sv), C::TILE);
                    for (int c = 0; c < C::NB; ++c)
                        tma_load_3d(s0 + C::OFF_V + sv * C::TILE + c * C::BLOCK, &tmv, bar(bVFull + sv), 64 * c, w.kvh,
                                    row);
                    ++nv;
                }
                if (!ok) break;
            }
            // Copies under way land before the CTA may exit.
            bool landed = true;
            for (int i = max(nk - C::SK, 0); landed && i < nk; ++i)
                landed = mbar_wait_bounded(bar(bKFull + i % C::SK), (i / C::SK) & 1, kWaitLimitNs);
            for (int i = max(nv - C::SV, 0); landed && i < nv; ++i)
                landed = mbar_wait_bounded(bar(bVFull + i % C::SV), (i / C::SV) & 1, kWaitLimitNs);
            if (!landed) *abort_flag = 1;
            timed_wait(bar(bDone), 0);
        } else if (warp == 3 && lane == 0) {
            // ======================= the CTA's pieces, and q ==========================
            int4 meta = make_int4(0, 0, 0, 0);  // what the joining kernel is to do with the cut item
            const Cuts cuts(total, gridDim.x);
            const uint64_t policy = l2_policy_evict_first();
            int uses[2] = {0, 0};
            Walk walk(from, to);
            int at = 0, upto = 0;               // the item's tiles yet to be handed out
            for (int i = 0;; ++i) {
                Piece w{};
                bool there = at < upto;
                w.cont = there;
                if (!there && walk.next(a)) {
                    at = walk.t0, upto = walk.t1;
                    there = true;
                }
                w.b = there ? walk.b : -1;
                if (there) {
                    w.kvh = walk.kvh, w.q0 = walk.s.q0, w.k0 = walk.s.k0, w.L = walk.s.L, w.ctx = walk.s.ctx;
                    w.tok0 = walk.rg * 2 * a.tile_toks;
                    w.toks = min(walk.s.N - w.tok0, 2 * a.tile_toks);
                    w.t0 = at, w.t1 = at = min(at + kFold, upto);
                    w.slot = walk.t0 == 0;
                    w.whole = walk.t0 == 0 && at == walk.nt;
                    w.two = w.toks > a.tile_toks;
                    w.tf = max(min(w.ctx + w.tok0 + 1, w.L), 0) / kTile;
                    w.end[0] = w.ctx + w.tok0 + min(w.toks, a.tile_toks);
                    w.end[1] = w.ctx + w.tok0 + w.toks;
                }
                if (i >= kPieces) lane_wait(bar(bPieceFree + i % kPieces), (i / kPieces - 1) & 1);
                if (*abort_flag) {  // (what is in the ring stays as it is)
                    *handed_out = i;
                    break;
                }
                pieces[i % kPieces] = w;
                mbar_arrive(piece_bar(i));
                if (w.b < 0) break;
                if (walk.t0 == 0 && upto < walk.nt) {
                    // the CTA that has the item's last unit
                    const int c1 = cuts.at_or_before(to.item + kItemKeys + walk.s.end(walk.rg) - 1);
                    meta = make_int4(w.q0 + w.tok0, w.toks, c1 - static_cast<int>(blockIdx.x) + 1, w.kvh);
                }
                if (i == 0) grid_dep_wait();
                // tile_toks tokens x G heads are consecutive operand rows
                for (int g = 0; g <= w.two; ++g) {
                    if (uses[g] > 0 && !lane_wait(bar(bQFree + g), (uses[g] - 1) & 1)) break;
                    mbar_arrive_expect_tx(bar(bQ + g), a.tile_toks * a.G * D * 2);
                    for (int c = 0; c < C::NB; ++c)
                        tma_load_3d(s0 + C::OFF_Q + g * C::TILE + c * C::BLOCK, &tmq, bar(bQ + g), 64 * c, w.kvh * a.G,
                                    w.q0 + w.tok0 + g * a.tile_toks, policy);
                    ++uses[g];
                }
            }
            grid_dep_wait();
            reinterpret_cast<int4*>(a.workspace)[blockIdx.x] = meta;
            for (int g = 0; g < 2; ++g)
                if (uses[g]) (void)mbar_wait_bounded(bar(bQ + g), (uses[g] - 1) & 1, kWaitLimitNs);
        } else if (warp == 1) {
            // ======================= tensor-core issue (one thread) ===================
            grid_dep_wait();
            if (elect_one()) {
                // the sign of softmax_scale goes into q (bit 13 negates A); N in bits 17 and up
                const uint32_t idesc_qk = umma_idesc(128, 0, 1, 1, false, false) | (a.scale_log2 < 0.f ? 1u << 13 : 0u);
                constexpr uint32_t kIdescPv = umma_idesc(128, D, 1, 1, false, true);
                // 128-byte-swizzled operands, 1024 bytes between groups of 8 rows
                constexpr uint64_t kDescHi = static_cast<uint64_t>((1024 >> 4) | (1u << 14) | (2u << 29)) << 32;
                auto desc = [](uint32_t addr, uint32_t lead) -> uint64_t { return kDescHi | ((addr >> 4) & 0x3FFFu) | (lead >> 4) << 16; };
                // Stages and phases of the next tile of K, of V. Per group: the phase of the P that is next (bit g), and
                // in two bits at 2 g the items whose scores were begun, 2 or 3 for all of that parity from there on.
                int sk = 0, sv = 0, n_fix = 0;
                bool on = true;  // no wait was given up on
                auto wait = [&](uint32_t bb, uint32_t par) { on = lane_wait(bb, par) && on; };
                uint32_t pk = 0, pv = 0, n_p = 0, items = 0, issued = 0;
                auto next_k = [&]() {
                    if (++sk == C::SK) sk = 0, pk ^= 1;
                };
                auto next_v = [&]() {
                    if (++sv == C::SV) sv = 0, pv ^= 1;
                };
                struct Job {  // of a piece
                    int there, t0, t1, two, tf, end0, end1;
                };
                auto job_of = [&](int i) {
                    const Piece& w = pieces[i % kPieces];
                    Job j{w.b >= 0 && !*abort_flag, w.t0, w.t1, w.two, w.tf, w.end[0], w.end[1]};
                    if (!j.there) j.two = 0;
                    return j;
                };
                auto cols_of = [](const Job& w, int g, int t) {
                    return min(max(((g ? w.end1 : w.end0) - t * kTile + 15) & ~15, 16), kTile);
                };
                // Scores for row tile g of the tile of K that is next.
                auto scores = [&](int g, int cols) {
                    const uint64_t q = desc(s0 + C::OFF_Q + g * C::TILE, 16), kt = desc(s0 + C::OFF_K + sk * C::TILE, 16);
                    const uint32_t idesc = idesc_qk | static_cast<uint32_t>(cols >> 3) << 17;
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t at = ((k >> 2) * C::BLOCK + (k & 3) * 32) >> 4;
                        umma_ss(tmem + 256 * g, q + at, kt + at, idesc, k > 0);
                    }
                    umma_commit(bar(bS + g));
                };
                // The first scores of a piece for row tile g.
                auto begin = [&](const Job& w, int g) {
                    if (g == 0) wait(bar(bKFull + sk), pk);
                    wait(bar(bQ + g), items >> (2 * g) & 1);
                    items = (items >> (2 * g) & 3u) == 3u ? items ^ 1u << (2 * g) : items + (1u << (2 * g));
                    scores(g, cols_of(w, g, w.t0));
                    issued = 1;
                    if (g == w.two) next_k();
                };
                wait(piece_bar(0), piece_par(0));
                Job w = job_of(0), next;
#pragma unroll 1
                for (int g = 0; w.there && g <= w.two; ++g) begin(w, g);
#pragma unroll 1
                for (int i = 0; on && w.there; ++i) {
                    next.there = next.two = 0;
                    const int fix = min(w.tf, w.t1);
#pragma unroll 1
                    for (int t = w.t0; on && t < w.t1;) {
                        // Tiles that both row tiles see in full, as the next one: the loop to be fast.
                        if (t > w.t0 && w.two && t + 1 < fix) {
#pragma unroll 1
                            for (; on && t + 1 < fix; ++t) {
                                wait(bar(bVFull + sv), pv);
                                const uint64_t vt = desc(s0 + C::OFF_V + sv * C::TILE, C::BLOCK);
#pragma unroll
                                for (int g = 0; g < 2; ++g) {
                                    wait(bar(bP + g), n_p >> g & 1);
                                    tc_fence_after();
#pragma unroll
                                    for (int k = 0; k < kTile / 16; ++k)
                                        umma_ts(tmem + 256 * g + C::O_COL, tmem + 256 * g + 8 * k, vt + k * (2048 >> 4), kIdescPv, 1u);
                                    if (g == 0) wait(bar(bKFull + sk), pk);
                                    scores(g, kTile);
                                }
                                n_p ^= 3u;
                                next_v();
                                next_k();
                            }
                            continue;
                        }
                        const bool last = t + 1 == w.t1;
                        if (t >= w.tf) {
                            wait(bar(bFix + n_fix % kFix), (n_fix / kFix) & 1);
                            ++n_fix;
                        } else {
                            wait(bar(bVFull + sv), pv);
                        }
                        const uint64_t vt = desc(s0 + C::OFF_V + sv * C::TILE, C::BLOCK);
#pragma unroll 1
                        for (int g = 0; g <= w.two; ++g) {
                            // the item before has been read out of O
                            if (t == w.t0 && (items >> (2 * g) & 2u)) wait(bar(bOFree + g), items >> (2 * g) & 1);
                            const int steps = cols_of(w, g, t) >> 4;
                            wait(bar(bP + g), n_p >> g & 1);
                            n_p ^= 1u << g;
                            tc_fence_after();
                            const uint32_t more_o = t > w.t0 ? 1u : go_on[g];  // O goes on, or starts
#pragma unroll 1
                            for (int k = 0; k < steps; ++k)
                                umma_ts(tmem + 256 * g + C::O_COL, tmem + 256 * g + 8 * k, vt + k * (2048 >> 4), kIdescPv, k > 0 ? 1u : more_o);
                            if (last) {
                                umma_commit(bar(bO + g));
                            } else {
                                if (g == 0) wait(bar(bKFull + sk), pk);
                                scores(g, cols_of(w, g, t + 1));
                                if (g == w.two) next_k();
                            }
                        }
                        if (last) {
                            // (q of the next piece may be on its way yet: nothing waits behind it but its scores)
                            wait(piece_bar(i + 1), piece_par(i + 1));
                            next = job_of(i + 1);
#pragma unroll 1
                            for (int g = 0; next.there && g <= next.two; ++g) begin(next, g);
                        }
                        next_v();
                        ++t;
                    }
                    mbar_arrive(bar(bPieceFree + i % kPieces));
                    w = next;
                }
                // Every operation issued is done before the tensor memory is freed: the
                // softmax groups wait for their last O, and a give-up for all of them here.
                if (*abort_flag && issued) {
                    umma_commit(bar(bEnd));
                    (void)mbar_wait_bounded(bar(bEnd), 0, kWaitLimitNs);
                }
            }
            __syncwarp();
        } else if (warp == 2) {
            // ======================= V of partly visible tiles ========================
            grid_dep_wait();
            int n = 0, n_fix = 0;
            bool on = true;
            for (int i = 0; on; ++i) {
                if (!warp_wait(piece_bar(i), piece_par(i))) break;
                const Piece w = pieces[i % kPieces];
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(bPieceFree + i % kPieces));
                if (__any_sync(0xffffffffu, w.b < 0)) break;
                const int lim = max(min(w.ctx + w.tok0 + 1, w.L), 0);  // keys that every row sees
                for (int t = w.t0; t < w.t1; ++t, ++n) {
                    on = warp_wait(bar(bVFull + n % C::SV), (n / C::SV) & 1);
                    if (!on) break;
                    if (t < w.tf) {
                        if (lane == 0) mbar_arrive(bar(bVFree + n % C::SV));
                        continue;
                    }
                    const uint32_t tile = s0 + C::OFF_V + (n % C::SV) * C::TILE;
                    uint32_t words[4];
                    for (int k = 0; k < 4; ++k) {
                        const int r = 32 * k + lane, pos = t * kTile + r;
                        const uint32_t row = tile + r * 128;
                        uint32_t acc = 0u;  // sums of 0 v: zero unless some v is not finite
                        if (pos >= lim && pos < w.L) {
#pragma unroll
                            for (int c = 0; c < D / 8; ++c) {
                                const uint4 x = lds128(row + (c >> 3) * C::BLOCK + ((c ^ r) & 7) * 16);
                                acc = fma_bf16x2(x.x, 0u, acc);
                                acc = fma_bf16x2(x.y, 0u, acc);
                                acc = fma_bf16x2(x.z, 0u, acc);
                                acc = fma_bf16x2(x.w, 0u, acc);
                            }
                        }
                        const bool odd = (acc & 0x7FFF7FFFu) != 0u;
                        words[k] = __ballot_sync(0xffffffffu, odd);
                        if (odd || pos >= w.L) {
#pragma unroll
                            for (int c = 0; c < D / 8; ++c)
                                sts128u(row + (c >> 3) * C::BLOCK + c % 8 * 16, 0u, 0u, 0u, 0u);
                        }
                    }
                    if (lane < 4)
                        bad_rows[4 * (n_fix % kFix) + lane] = lane == 0 ? words[0] : lane == 1 ? words[1] : lane == 2 ? words[2] : words[3];
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(bar(bFix + n_fix % kFix));
                        mbar_arrive(bar(bVFree + n % C::SV));
                    }
                    ++n_fix;
                }
            }
        }
        __syncwarp();
    } else {
        // ======================= softmax ==========================================
        grid_dep_wait();
        grid_dep_launch();
        const int grp = (warp - 4) >> 3, half = (warp - 4) >> 2 & 1, wq = warp & 3;
        const int row_l = 32 * wq + lane;              // this thread's lane of tensor memory
        const uint32_t tl = tmem + (static_cast<uint32_t>(wq) << 21);  // lanes 32 wq .. (bits 16 and up)
        // its columns of S, of P, of O (the row's other half is warp + 4's or warp - 4's)
        const uint32_t tS = tl + 256 * grp + 64 * half, tP = tl + 256 * grp + 32 * half;
        const uint32_t tO = tl + 256 * grp + C::O_COL + D / 2 * half;
        const int tok_l = row_l / a.G, g_l = row_l - tok_l * a.G;      // its token in the row tile, its head
        const bool speaker = wq == 0 && half == 0 && lane == 0;        // for its group
        const int pair = 1 + 4 * grp + wq;             // barrier of the two warps that share rows
        float* mine = theirs + (2 * grp + half) * 128 + row_l;         // what this half tells the other, and hears
        const float* other = theirs + (2 * grp + 1 - half) * 128 + row_l;
        const float sl = fmaxf(fabsf(a.scale_log2), 1.2e-38f);         // -inf times it stays -inf
        const float2 sl2 = make_float2(sl, sl);
        int n = 0, job = 0, n_o = 0, n_fix = 0;        // the CTA's tiles, this group's jobs and pieces, fixed tiles
        float m = -INFINITY, l = 0.f;                  // of the item (l: of this half's columns)
        for (int i = 0;; ++i) {
            // A group's warps meet at barriers, which know no limit: they take up the same pieces, and a wait that was
            // given up on changes nothing of what they do with one. A warp that gives up waiting for a piece learns
            // from warp 3, whose waits end too, whether there is one.
            bool more = true;
            if (!warp_wait(piece_bar(i), piece_par(i))) {
                const uint64_t t0 = global_ns();
                while (*handed_out < 0 && !mbar_try_wait(piece_bar(i), piece_par(i)) && global_ns() - t0 < 4 * kWaitLimitNs) {}
                more = mbar_try_wait(piece_bar(i), piece_par(i));
            }
            const Piece& w = pieces[i % kPieces];
            if (__any_sync(0xffffffffu, !more || w.b < 0)) break;
            const int t0 = w.t0, t1 = w.t1, tf = w.tf;
            if (grp > w.two) {
                n += t1 - t0;
                n_fix += max(t1 - max(t0, tf), 0);
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(bPieceFree + i % kPieces));
                continue;
            }
            const bool frees = speaker && grp == w.two;                // the tile's last use is this group's
            const int tok_t = tok_l + grp * a.tile_toks;               // token in the pair of row tiles
            const bool live = tok_l < a.tile_toks && tok_t < w.toks;
            const int tok = w.tok0 + tok_t;
            const int lim = live ? min(w.ctx + tok + 1, w.L) : 0;      // positions that this row sees
            // tiles that every row of this group sees in full
            const int inner_end = max(min(w.ctx + w.tok0 + grp * a.tile_toks + 1, w.L), 0) / kTile;
            const bool cont = w.cont != 0;
            if (!cont) m = -INFINITY, l = 0.f;
            for (int t = t0; t < t1; ++t, ++n, ++job) {
                const bool first = t == t0;
                const int vis = lim - t * kTile - 64 * half;   // of this half's columns, those that the row sees
                const bool inner = t < inner_end;
                warp_wait(bar(bS + grp), job & 1);
                tc_fence_after();
                if (speaker) {
                    if (frees) {
                        mbar_arrive(bar(bKFree + n % C::SK));
                        if (!first) mbar_arrive(bar(bVFree + (n - 1) % C::SV));
                    }
                    if (t == t1 - 1) mbar_arrive(bar(bQFree + grp));
                    if (first) go_on[grp] = 0u;
                }
                uint32_t bad[4] = {0u, 0u, 0u, 0u};
                if (t >= tf) {
                    warp_wait(bar(bFix + n_fix % kFix), (n_fix / kFix) & 1);
#pragma unroll
                    for (int k = 0; k < 4; ++k) bad[k] = bad_rows[4 * (n_fix % kFix) + k];
                    ++n_fix;
                }
                {
                    // The half's weights; where their sum asks for another reference, twice.
                    bool start = first && !cont;       // there is no reference yet
                    uint32_t p[32];
                    float sum;
                    bool raised = false;
#pragma unroll 1
                    for (;;) {
                        sum = 0.f;
                        if (!start) {
                            const float mm = m == -INFINITY ? 0.f : -m;
                            const float2 mm2 = make_float2(mm, mm);
                            float2 s2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                uint32_t x[32];
                                tmem_ld32(tS + 32 * c, x);
                                tmem_wait_ld();
                                pin(x);
                                if (!inner) {
#pragma unroll
                                    for (int e = 0; e < 32; ++e)
                                        if (32 * c + e >= vis) x[e] = 0xFF800000u;
                                }
#pragma unroll
                                for (int e = 0; e < 16; ++e) {
                                    float2 y = fma2(make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), sl2, mm2);
                                    y.x = fast_exp2(y.x);
                                    y.y = fast_exp2(y.y);
                                    s2[e & 1] = add2(s2[e & 1], y);
                                    p[16 * c + e] = pack_bf16(y.x, y.y);
                                }
                            }
                            sum = (s2[0].x + s2[1].x) + (s2[0].y + s2[1].y);
                            // (also: both have read S, and P may go over it)
                            const bool move = !raised && live && (sum > kRaise || (m == -INFINITY && vis > 0));
                            if (named_bar_and(pair, 64, !move)) break;
                        }
                        // The reference goes up to the tile's maximum, where that is 2^6 above it (as it is
                        // where a sum is too large) or there was none.
                        float mx = -INFINITY;
#pragma unroll 1
                        for (int c = 0; c < 2; ++c) {
                            uint32_t x[32];
                            tmem_ld32(tS + 32 * c, x);
                            tmem_wait_ld();
                            pin(x);
                            if (!inner) {
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    if (32 * c + e >= vis) x[e] = 0xFF800000u;
                            }
                            float mx4[4] = {mx, mx, mx, mx};
#pragma unroll
                            for (int e = 0; e < 32; e += 2)
                                mx4[e >> 1 & 3] = fmaxf(fmaxf(mx4[e >> 1 & 3], __uint_as_float(x[e])), __uint_as_float(x[e + 1]));
                            mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
                        }
                        *mine = mx;
                        (void)named_bar_and(pair, 64, true);
                        mx = fmaxf(mx, *other);
                        const float top = mx * sl, nm = top > m + 6.f ? top : m;
                        const float al = m == -INFINITY ? 0.f : fast_exp2(m - nm);
                        l *= al;
                        m = nm;
                        if (!first) {
#pragma unroll 1
                            for (int c = 0; c < D / 32; ++c) {
                                uint32_t o[16];
                                tmem_ld16(tO + 16 * c, o);
                                tmem_wait_ld();
                                pin(o);
#pragma unroll
                                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * al);
                                tmem_st16(tO + 16 * c, o);
                            }
                        }
                        start = false;
                        raised = true;
                    }
                    tmem_st32(tP, p);
                    l += sum;
                    tmem_wait_st();
                    // ---- rows of V that are not finite, for the rows that see them ---------
                    if ((bad[0] | bad[1] | bad[2] | bad[3]) != 0u) {  // (uniform)
                        if (first) {  // there is no O yet: it starts here, and P . V goes on from it
                            uint32_t zero[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) zero[e] = 0u;
#pragma unroll 1
                            for (int c = 0; c < D / 32; ++c) tmem_st16(tO + 16 * c, zero);
                            tmem_wait_st();
                            if (speaker) go_on[grp] = 1u;
                        }
                        tc_fence_before();
                        {   // (a barrier with a limit: where the wait above was given up on, the other half may not be here)
                            const uint32_t uses = pair_uses[8 * grp + 2 * wq + half];
                            __syncwarp();
                            if (lane == 0) {
                                pair_uses[8 * grp + 2 * wq + half] = uses + 1;
                                mbar_arrive(bar(bPair + 4 * grp + wq));
                            }
                            warp_wait(bar(bPair + 4 * grp + wq), uses & 1);
                        }
                        tc_fence_after();
                        const int sees = live ? vis + 64 * half : 0;
#pragma unroll 1
                        for (int j = 0; j < kTile; ++j) {
                            if (!(word_of(bad, j >> 5) >> (j & 31) & 1)) continue;
                            const float pj = tmem_ld_half(tl + 256 * grp + (j >> 1), j & 1);
                            const uint16_t* vr = a.v + static_cast<int64_t>(w.k0 + t * kTile + j) * a.v_s0 +
                                                 static_cast<int64_t>(w.kvh) * a.v_s1 + D / 2 * half;
#pragma unroll 1
                            for (int c = 0; c < D / 32; ++c) {
                                uint32_t o[16];
                                tmem_ld16(tO + 16 * c, o);
                                tmem_wait_ld();
                                pin(o);
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    if (j < sees)
                                        o[e] = __float_as_uint(fmaf(
                                            pj, __uint_as_float(static_cast<uint32_t>(vr[16 * c + e]) << 16), __uint_as_float(o[e])));
                                tmem_st16(tO + 16 * c, o);
                                tmem_wait_st();
                            }
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(bP + grp));
            }
            // ---- the piece's output, or its partial sums -----------------------------
            warp_wait(bar(bO + grp), n_o & 1);
            ++n_o;
            tc_fence_after();
            if (frees) mbar_arrive(bar(bVFree + (n - 1) % C::SV));
            {
                const int row = 128 * grp + row_l;             // its place in partial sums
                const int slot = 2 * static_cast<int>(blockIdx.x) + w.slot;
                // What is there of the item was taken against an earlier reference.
                float older = 0.f;
                if (cont && live) {
                    const float m0 = *part_ml(a.workspace, slot, row);
                    older = m0 == m ? 1.f : exp2f(m0 - m);
                }
                *mine = l;
                (void)named_bar_and(pair, 64, true);
                const float sum = l + *other;
                (void)named_bar_and(pair, 64, true);
                const bool none = sum == 0.f, whole = w.whole;
                const int h = w.kvh * a.G + g_l;
                const int64_t q_row = w.q0 + tok;
                const float inv = whole ? (none ? 0.f : 1.f / sum) : 1.f;
                if (live && half == 0) {
                    if (!whole) {
                        *reinterpret_cast<float2*>(part_ml(a.workspace, slot, row)) = make_float2(m, sum);
                    } else if (a.lse) {
                        a.lse[q_row * a.l_s0 + h * a.l_s1] = none ? -INFINITY : (m + __log2f(sum)) * 0.69314718055994530942f;
                    }
                }
                float* part = part_o<D>(a.workspace, gridDim.x, slot, row) + static_cast<int64_t>(D / 8 * half) * kJoinRows * 4;
                uint16_t* out = a.out + q_row * a.o_s0 + h * a.o_s1 + D / 2 * half;
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[16];
                    tmem_ld16(tO + 16 * c, o);
                    tmem_wait_ld();
                    pin(o);
                    if (c == D / 32 - 1) {  // O is read
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(bOFree + grp));
                    }
                    if (!live) continue;
                    if (cont) {  // (this thread's own, of the piece before)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float4 x = *reinterpret_cast<const float4*>(part + static_cast<int64_t>(4 * c + e) * kJoinRows * 4);
                            o[4 * e] = __float_as_uint(fmaf(x.x, older, __uint_as_float(o[4 * e])));
                            o[4 * e + 1] = __float_as_uint(fmaf(x.y, older, __uint_as_float(o[4 * e + 1])));
                            o[4 * e + 2] = __float_as_uint(fmaf(x.z, older, __uint_as_float(o[4 * e + 2])));
                            o[4 * e + 3] = __float_as_uint(fmaf(x.w, older, __uint_as_float(o[4 * e + 3])));
                        }
                    }
                    if (whole) {
                        uint32_t q[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            q[e] = none ? 0u : pack_bf16(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
                        // (32 rows a store: the load-store unit takes a row at a time, whatever its bytes)
                        if (a.wide) {
                            stg256(out + 16 * c, q);
                        } else {
                            reinterpret_cast<uint4*>(out)[2 * c] = make_uint4(q[0], q[1], q[2], q[3]);
                            reinterpret_cast<uint4*>(out)[2 * c + 1] = make_uint4(q[4], q[5], q[6], q[7]);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            *reinterpret_cast<uint4*>(part + static_cast<int64_t>(4 * c + e) * kJoinRows * 4) =
                                make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(bPieceFree + i % kPieces));
        }
    }

    if (warp != 0) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(bDone));
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0 && *abort_flag) flag_error(a.err, PKV_FLAG_WAIT_TIMEOUT);
    if (warp == 1) tmem_dealloc(tmem, 512);
}

template <int D>
cudaError_t launch_t(const PromptArgs& a, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s) {
    using C = Cfg<D>;
    int sms = 0;
    cudaError_t e = device_sm_count(&sms);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(prompt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    e = launch_dependent(prompt_kernel<D>, dim3(sms), dim3(C::THREADS), C::SMEM, s, tq, tk, tv, a);
    if (e != cudaSuccess) return e;
    // No item is longer than all keys, or all tokens where a sequence has more of them than keys: nothing is cut.
    if (std::max(a.T, a.Tk) + kItemKeys <= kSnapKeys) return cudaSuccess;
    TreeArgs j{};
    j.T = a.T, j.Hq = a.Hq, j.G = a.G, j.tile_toks = a.tile_toks, j.D = D;
    j.out = a.out, j.o_s0 = a.o_s0, j.o_s1 = a.o_s1;
    j.lse = a.lse, j.l_s0 = a.l_s0, j.l_s1 = a.l_s1;
    j.workspace = a.workspace;
    return launch_row_join(j, sms, s);
}

}  // namespace

int64_t prompt_attention_workspace(int32_t D, int32_t sm_count) {
    return kJoinMetaBytes + static_cast<int64_t>(sm_count) * 2 * kJoinRows * (D + 2) * 4;
}

cudaError_t launch_prompt_attention(const PromptArgs& a, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                    cudaStream_t s) {
    return a.D == 128 ? launch_t<128>(a, tq, tk, tv, s) : launch_t<64>(a, tq, tk, tv, s);
}

}  // namespace pkv
