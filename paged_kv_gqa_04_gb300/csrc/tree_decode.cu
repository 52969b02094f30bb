// tree_decode.cu -- attention of drafted tokens over a paged cache on the
// fifth-generation tensor cores: the context in full, the drafted tokens under
// a tree mask or as a chain.
//
// Rows. The drafted tokens of a sequence and the G query heads of a kv head
// share the same K and V. A row tile is 128 / G tokens (rounded down) times G
// heads on the M side of the MMA (128 tensor-memory lanes), so q lands in
// operand layout by TMA, a softmax thread owns one row, and its maximum and
// sum need no exchange. One pass over K and V serves two row tiles.
//
// Work. An item is (sequence, kv head, pair of row tiles); a unit is one tile
// of 128 positions of one item, and an item counts four units more for its
// start and output (measured: counting two, 64 contexts of 1 to 8192 with 32
// query heads took 105 us and not 91, counting five or three 93 and 96; FP8, 16
// contexts of 2 to 16 Ki, 73 and not 68). All units of the batch, in order, are cut
// into equal stretches, one per CTA (one CTA per SM): every CTA does the same
// amount of work whatever the lengths are, with no plan from the host. Each
// CTA finds its stretch from prefix sums over the batch. An item that is cut
// leaves partial sums in the workspace (at most two per CTA: the end of one
// item, the start of another), which a second kernel joins.
//
// A CTA's roles, per tile:
//   warps 0, 2    TMA tile loads of K and of V (a warp starts a 16-row x 128-byte
//                 copy in about 85 cycles: one for both would be the limit).
//                 Pages that do not exist are read out of range, which fills
//                 zeros
//   warp 3        walks the CTA's items, hands the pieces to the other roles, and
//                 loads q by TMA
//   warp 1        one thread issues S = Q . K^T and O += P . V (M = 128; P from
//                 tensor memory, V as an MN-major operand: nothing is
//                 transposed). A tcgen05.commit holds the products behind it
//                 up for about 105 cycles (16 MMAs: 1054 cycles, 1481 with four
//                 commits), so a tile has one, for S: that S is there also says
//                 that its K, and the V and the P before it, are done with, and
//                 the softmax warps release them
//   warps 4 - 7,
//   warps 8 - 11  two softmax groups, each with S, P and O of its own in tensor
//                 memory. One row tile: both have the same rows and take the
//                 tiles in turn, and their sums are joined at the end (either
//                 group reads the other's O directly). Two: each has its own
//                 row tile, and every tile. While one group is in its softmax
//                 the tensor cores work for the other; the next item's first
//                 scores are computed while the item before writes its output.
//   warps 12 - 15 FP8 caches: E4M3 bytes to f16 operand tiles (exact), q too
//
// The online softmax keeps a reference maximum per row that moves only when a
// tile's maximum passes it by more than 8 (log2), so P <= 2^8 and O is scaled
// rarely. bf16 alone is too few bits for P where the weighted values cancel, so
// P is its bf16 rounding (2^-8 of it) and the rest, rounded again (2^-16 in all),
// and V meets both, as in the one-token decode; the scores' columns hold both.
// One term: 64 contexts of 1 to 8192 82 us and not 91, 16 of 8 Ki with 64 drafted
// tokens 141 and not 176, but outputs of weights near one another up to 11 times
// their bound off. FP8 caches: one f16 term of 2^7 P (<= 2^15), 2^-11 of it down to
// weights of 2^-21 of the reference, 2^-32 of the reference below (P itself would
// lose all weights below 2^-25 beside one dominant position: 0.03 of V after 2^20
// others). The sums of the weights are taken before the rounding, in fp32. For
// FP8 caches q is scaled by a power of two per row into f16's range, which is
// exact for every value within 2^29 of the row's largest.
//
// Weights of zero do not cover values that are not finite: rows of V behind
// the sequence's end are zeroed in the tile, and a drafted token whose V is
// not finite is zeroed there too and added to the rows that see it by hand.
//
// Bound. With one row tile a tile of K and V (64 KB, bf16, D = 128) takes an SM
// 1.43 us, HBM's rate (7.0 TB/s); 64 contexts of 1 to 8192 (413 MB) take 91 us in
// all, 4.5 TB/s, the rest being the start (6 us to the first scores), the ends of
// items and the joining kernel. With two row tiles it takes 2.7 us: scores,
// softmax, P and P . V of a group follow one another, and tensor memory has room
// for two groups (S and O of each, 512 columns); the products are 1536 cycles
// of either group. 16 contexts of 8 Ki with 64 drafted tokens (519 MB, 129 GFLOP)
// take 176 us, 2.9 TB/s and 0.73 PFLOP/s, P . V counted once. FP8 (32 KB): 1.74 and
// 2.3 us, the conversion, which shares a pipe with the exponentials. Measured and not kept
// (that case, by one term of P, 141 us at the end): scores and P in two halves of
// 64 positions each with its own barriers (199 us: products of 64 columns take as
// long as those of 128, and the issuing thread becomes the limit), sixteen softmax
// warps (169 and not 150), all eight warps on every set of scores (160 and not
// 144), two issuing threads, P handed over in halves (147 and not 144). By two
// terms: the rest of the truncated weight (180), the split by fused
// multiply-adds (185), the terms by two stores (183).
//
// Waits are bounded (about one second): a role that gives up sets
// PKV_FLAG_WAIT_TIMEOUT and a CTA-wide flag that ends the others' waits.
#include <algorithm>
#include <atomic>

#include "pkv_internal.h"
#include "pkv_ptx.cuh"

namespace pkv {
namespace {

constexpr int kTile = 128;    // positions per tile
constexpr int kRows = 256;    // rows (lanes of two row tiles) per item
constexpr int kTilePages = kTile / kPageSize;
constexpr int kItemUnits = 4; // what an item costs beyond its tiles (start, output, joining), in tiles
constexpr int kPieces = 4;    // ring of pieces
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
    // Operand tiles: K and V have rings of their own (so either copy warp's waits
    // for a free stage are never two phases behind). FP8: one ring of K and V in
    // turn, filled in order by the conversion, and one of tiles of bytes.
    static constexpr int SK = D == 128 ? 3 : 4, SV = D == 128 ? 2 : 4;
    static constexpr int ST = FP8 ? (D == 128 ? 3 : 6) : SK + SV;
    // Slot n: K of tile n / 2 or, n odd, its V (tiles numbered through the CTA's stretch).
    static __device__ __forceinline__ int stage(int n) {
        return FP8 ? n % ST : n & 1 ? SK + (n >> 1) % SV : (n >> 1) % SK;
    }
    static __device__ __forceinline__ int round(int n) { return FP8 ? n / ST : n & 1 ? (n >> 1) / SV : (n >> 1) / SK; }
    // The same for the ring that the copies fill.
    static __device__ __forceinline__ int copy_stage(int n) { return FP8 ? n % RST : stage(n); }
    static __device__ __forceinline__ int copy_round(int n) { return FP8 ? n / RST : round(n); }
    static constexpr int RST = FP8 ? (D == 128 ? 3 : 6) : 0;
    static constexpr int THREADS = FP8 ? 512 : 384;
    // Registers a thread: launched with 168 (128), dealt out again by role.
    static constexpr int REG_IO = 88, REG_SM = FP8 ? 168 : 208, REG_CV = 88;
    static constexpr int OFF_Q = 0;                        // two row tiles of q
    static constexpr int OFF_T = OFF_Q + 2 * TILE;
    static constexpr int OFF_R = OFF_T + ST * TILE;
    static constexpr int OFF_SC = OFF_R + RST * RAW;       // FP8: [2][128] floats, 2^-k of each row
    static constexpr int OFF_BAR = OFF_SC + (FP8 ? kRows * 4 : 0);
    static constexpr int NBAR = 2 * ST + 2 * RST + 13 + 3 * kPieces;
    static constexpr int OFF_MISC = OFF_BAR + 8 * NBAR;
    static constexpr int OFF_PIECE = OFF_MISC + 192;       // [kPieces] Piece
    static constexpr int SMEM = OFF_PIECE + kPieces * 64 + 1024;  // + alignment slack
    static_assert(SMEM <= 232448, "shared memory of one CTA");
    static constexpr int REGS = 128 * (REG_IO + 2 * REG_SM + (FP8 ? REG_CV : 0));
    static_assert(REGS <= (FP8 ? 128 : 168) * THREADS, "registers as launched");
    // Tensor-memory columns of a softmax group: S (P over it, or behind O, where that leaves room), then O.
    // 32 positions of P are 16 columns; bf16: those of the rounded rest beside those of the rounded term, the
    // columns of S that they were.
    static constexpr int TERMS = FP8 ? 1 : 2;
    static constexpr float P_LOG2 = FP8 ? 7.f : 0.f;       // P and its sums are held times 2^this (P <= 2^15)
    static constexpr uint32_t P_COL = FP8 && D == 64 ? 192 : 0;
    static constexpr uint32_t O_COL = 128;
    static __device__ __forceinline__ constexpr uint32_t p_col(int k, int term) {  // of positions 16 k ..
        return P_COL + 16 * TERMS * (k >> 1) + 8 * (k & 1) + 16 * term;
    }
};

struct Seq {
    int q0, N, L, ctx, RG;
};
// Sequence b, its values clamped; `flags` collects what was out of range.
__device__ __forceinline__ Seq seq_of(const TreeArgs& a, int b, int& flags) {
    Seq s;
    const int q0 = __ldg(a.q_start + b), q1 = __ldg(a.q_start + b + 1);
    const int L = __ldg(a.seq_lens + b);
    s.q0 = min(max(q0, 0), a.T);
    const int e = min(max(q1, s.q0), a.T);
    if (s.q0 != q0 || e != q1) flags |= PKV_FLAG_DRAFT_RANGE;
    s.N = e - s.q0;
    s.L = min(max(L, 0), a.max_pages * kPageSize);
    if (s.N > 0) {
        if (s.L != L) flags |= PKV_FLAG_SEQ_LEN_RANGE;
        if (s.N > s.L || (a.mask != nullptr && s.N > 32 * a.W)) flags |= PKV_FLAG_DRAFT_RANGE;
    }
    s.ctx = s.L - s.N;
    s.RG = s.N <= 2 * a.tile_toks ? (s.N > 0) : (s.N + 2 * a.tile_toks - 1) / (2 * a.tile_toks);
    return s;
}
// Positions that pair rg of row tiles can see (a chain's earlier rows see less), and its tiles (at least one: a
// row that sees nothing has an output).
__device__ __forceinline__ int kv_end(const TreeArgs& a, const Seq& s, int rg) {
    return a.mask != nullptr ? s.L : min(s.L, s.ctx + min(s.N, (rg + 1) * 2 * a.tile_toks));
}
__device__ __forceinline__ int tiles_of(const TreeArgs& a, const Seq& s, int rg) {
    return max((kv_end(a, s, rg) + kTile - 1) / kTile, 1);
}
// Units of one kv head.
__device__ __forceinline__ int units_per_head(const TreeArgs& a, const Seq& s) {
    if (s.RG <= 1 || a.mask != nullptr) return s.RG ? s.RG * (tiles_of(a, s, 0) + kItemUnits) : 0;
    int n = 0;
    for (int rg = 0; rg < s.RG; ++rg) n += tiles_of(a, s, rg) + kItemUnits;
    return n;
}

// Sums of units. The host has checked that the drafted tokens' come to less than
// kMaxUnits; those of ranges that overlap may not, and stay there.
constexpr int kMaxUnits = 0x7FFFFFFF;
__device__ __forceinline__ int add_units(int x, int y) {
    return static_cast<int>(min(static_cast<uint32_t>(x) + static_cast<uint32_t>(y), static_cast<uint32_t>(kMaxUnits)));
}

// CTA c of n starts at unit cut(c); the first total % n stretches are one unit longer.
struct Cuts {
    int n, per, rem;
    __device__ __forceinline__ Cuts(int total, int ctas) : n(min(ctas, total)), per(0), rem(0) {
        if (n > 0) {
            per = total / n;
            rem = total - per * n;
        }
    }
    __device__ __forceinline__ int cut(int c) const { return c * per + min(c, rem); }
    // the last CTA that starts at or before unit x
    __device__ __forceinline__ int at_or_before(int x) const {
        const int c = x < rem * (per + 1) ? x / (per + 1) : rem + (x - rem * (per + 1)) / per;
        return min(c, n - 1);
    }
};

// A place in the order of units: tile t of item k = kvh RG + rg of sequence b.
struct Place {
    int b, k, t;
};
// Unit `off` of sequence b, of `per` units a kv head.
__device__ __forceinline__ Place place_of(const TreeArgs& a, const Seq& s, int per, int b, int off) {
    const int kvh = off / per;
    int rem = off - kvh * per;
    int rg = 0, nt = tiles_of(a, s, 0);
    while (rem >= nt + kItemUnits) {
        rem -= nt + kItemUnits;
        nt = tiles_of(a, s, ++rg);
    }
    return Place{b, kvh * s.RG + rg, max(rem - kItemUnits, 0)};
}

// The pieces of items between two places, in order.
struct Walk {
    int b, k, t0, t1, nt, kvh, rg;
    Seq s;
    Place end;
    bool first;
    __device__ __forceinline__ Walk(const Place& from, const Place& to) : b(from.b), k(from.k), t0(from.t), end(to), first(true) {}
    // Next piece [t0, t1) of item (b, k); false at the end.
    __device__ __forceinline__ bool next(const TreeArgs& a) {
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
        for (;; ++b, k = 0, load = true) {  // past the sequences without drafted tokens
            if (b >= a.B || !in_range()) return false;
            if (load) s = seq_of(a, b, ignored);
            if (k < a.Hkv * s.RG) break;
        }
        kvh = s.RG == 1 ? k : k / s.RG;
        rg = k - kvh * s.RG;
        nt = tiles_of(a, s, rg);
        t1 = b == end.b && k == end.k ? end.t : nt;
        return true;
    }
    __device__ __forceinline__ bool in_range() const {
        return b < end.b || (b == end.b && (k < end.k || (k == end.k && end.t > t0)));
    }
};

// A piece: tiles [t0, t1) of an item (its drafted tokens [tok0, tok0 + toks)).
struct Piece {
    int b, kvh, q0, L, ctx, tok0, toks;  // b < 0: there are no more
    int t0, t1, whole;                   // whole: all of the item
    int two, buf;                        // two row tiles, or one, whose q is in this buffer
    int uses0, uses1;                    // earlier pieces in either buffer of q
    // q's buffers of this piece: fn(buffer, uses of it before)
    template <typename F>
    __device__ __forceinline__ void buffers(F fn) const {
        if (two || buf == 0) fn(0, uses0);
        if (two || buf == 1) fn(1, uses1);
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
// 32 columns: the 16 of r, then the 16 of q; complete after tmem_wait_st().
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[16], const uint32_t (&q)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,"
        "%31,%32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(q[0]), "r"(q[1]), "r"(q[2]),
        "r"(q[3]), "r"(q[4]), "r"(q[5]), "r"(q[6]), "r"(q[7]), "r"(q[8]), "r"(q[9]), "r"(q[10]), "r"(q[11]), "r"(q[12]),
        "r"(q[13]), "r"(q[14]), "r"(q[15])
        : "memory");
}
// The values of a tensor-memory load are used only past this point (which follows its wait).
template <int N>
__device__ __forceinline__ void pin(uint32_t (&r)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}
// One thread's MMA and commit (the warp forms elect a lane at each call).
// Descriptors as a start address (>> 4, low word with the leading offset) and
// a constant high word: a step along K is one 32-bit add.
// D (tensor memory) = A . B^T (+ D unless FIRST), both operands in shared memory.
template <bool FIRST>
__device__ __forceinline__ void umma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tmov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\tsetp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "n"(FIRST ? 0 : 1)
        : "memory");
}
// A in tensor memory: 16-bit values, two per 32-bit column.
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t hi, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tmov.b64 b, {%2, %3};\n\tsetp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void umma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
template <int N>
__device__ __forceinline__ void reg_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// Lane-wise fma and add of two floats.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 w, x, y;\n\t"
        "mov.b64 {%0, %1}, w;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ uint16_t lo16(uint32_t w) { return static_cast<uint16_t>(w & 0xFFFFu); }
__device__ __forceinline__ uint16_t hi16(uint32_t w) { return static_cast<uint16_t>(w >> 16); }
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; }
// v[k] without an array in local memory
__device__ __forceinline__ uint32_t word_of(const uint32_t (&v)[4], int k) {
    return k == 0 ? v[0] : k == 1 ? v[1] : k == 2 ? v[2] : v[3];
}

// Workspace of partial sums: [2 per CTA][256 rows] of {m, l}, then [2 per
// CTA][D / 4][256 rows] of 4 floats (a warp's rows are neighbours).
__device__ __forceinline__ float* part_ml(void* ws, int slot, int row) {
    return reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kMetaBytes) +
           (static_cast<int64_t>(slot) * kRows + row) * 2;
}
template <int D>
__device__ __forceinline__ float* part_o(void* ws, int ctas, int slot, int row) {
    return reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kMetaBytes) + static_cast<int64_t>(ctas) * 2 * kRows * 2 +
           static_cast<int64_t>(slot) * kRows * D + row * 4;
}

template <int D, bool FP8>
__global__ void __launch_bounds__(Cfg<D, FP8>::THREADS, 1)
    tree_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                const __grid_constant__ CUtensorMap tmv, const TreeArgs a) {
    using C = Cfg<D, FP8>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t s0 = smem_u32(smem);
    enum : int { bFull = 0, bFree = C::ST, bRawFull = 2 * C::ST, bRawFree = bRawFull + C::RST, bS = bRawFree + C::RST,
                 bP = bS + 2, bO = bP + 2, bQ = bO + 2, bQFree = bQ + 2, bQRaw = bQFree + 2, bX = bQRaw + 2,
                 bPiece = bX + kPieces, bPieceFree = bPiece + kPieces, bEnd = bPieceFree + kPieces };
    static_assert(bEnd + 1 == C::NBAR, "barriers");
    auto bar = [&](int i) -> uint32_t { return s0 + C::OFF_BAR + 8 * i; };
    uint32_t* misc = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
    uint32_t* bad_tok = misc + 4;                         // [2 jobs][2 groups][4 words]: drafted tokens, V not finite
    Place* place = reinterpret_cast<Place*>(misc + 20);   // [2]: this CTA's first unit and the one past its last
    int* warp_units = reinterpret_cast<int*>(misc + 26);  // [16]
    Piece* pieces = reinterpret_cast<Piece*>(smem + C::OFF_PIECE);
    uint32_t* go_on = misc + 2;                           // [2 groups]: O has been started by hand
    float* q_scale = reinterpret_cast<float*>(smem + C::OFF_SC);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t num_pages = a.num_pages;

    if (tid == C::THREADS - 32) {  // (the first threads have sequences to look at)
        for (int i = 0; i < C::ST; ++i) {
            mbar_init(bar(bFull + i), FP8 ? 4 : 1);
            mbar_init(bar(bFree + i), 2);  // either group's use (two arrivals where one group has the tile)
        }
        for (int i = 0; i < C::RST; ++i) {
            mbar_init(bar(bRawFull + i), 1);
            mbar_init(bar(bRawFree + i), 4);
        }
        for (int w = 0; w < 2; ++w) {
            mbar_init(bar(bS + w), 1);
            mbar_init(bar(bP + w), 4);
            mbar_init(bar(bO + w), 1);
            mbar_init(bar(bQ + w), FP8 ? 4 : 1);
            mbar_init(bar(bQFree + w), 8);  // the softmax warps (the last S, and the staged output)
            mbar_init(bar(bQRaw + w), 1);
        }
        mbar_init(bar(bEnd), 1);
        for (int i = 0; i < kPieces; ++i) {
            mbar_init(bar(bX + i), 8);
            mbar_init(bar(bPiece + i), 1);
            mbar_init(bar(bPieceFree + i), FP8 ? 15 : 11);  // copies, MMA, softmax, conversion
        }
        *abort_flag = 0;
        place[0] = place[1] = Place{a.B, 0, 0};
        fence_mbar_init();
        tma_prefetch_desc(&tmq);
        tma_prefetch_desc(&tmk);
        tma_prefetch_desc(&tmv);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(misc), 512);
        tmem_relinquish();
    }

    // ---- this CTA's stretch of the units (index inputs only) ------------------
    int total = 0;
    {
        const int seg = (a.B + C::THREADS - 1) / C::THREADS;
        const int b0 = min(tid * seg, a.B), b1 = min(b0 + seg, a.B);
        int sum = 0, flags = 0, per = 0;
        Seq s{};
        for (int b = b0; b < b1; ++b) {
            s = seq_of(a, b, flags);
            per = units_per_head(a, s);
            sum = add_units(sum, a.Hkv * per);
        }
        if (flags && blockIdx.x == 0) flag_error(a.err, flags);
        int inc = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc = add_units(inc, y);
        }
        if (lane == 31) warp_units[warp] = inc;
        __syncthreads();
        int base = 0;
        for (int w = 0; w < C::THREADS / 32; ++w) {
            if (w == warp) base = total;
            total = add_units(total, warp_units[w]);
        }
        if (total == kMaxUnits) total = 0;             // (ranges that overlap; flagged)
        const Cuts cuts(total, gridDim.x);
        const int c = blockIdx.x;
        int at = base + inc - sum;
        const int x0 = cuts.cut(c), x1 = cuts.cut(c + 1);
        if (c < cuts.n && x1 >= at && x0 < at + sum) {
            for (int b = b0; b < b1; ++b) {
                if (seg > 1) {
                    int ignored = 0;
                    s = seq_of(a, b, ignored);
                    per = units_per_head(a, s);
                }
                const int n = a.Hkv * per;
                if (x0 >= at && x0 < at + n) place[0] = place_of(a, s, per, b, x0 - at);
                if (x1 >= at && x1 < at + n) place[1] = place_of(a, s, per, b, x1 - at);
                at += n;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];
    const Place from = place[0], to = place[1];

    // q, the mask, the scales and the cache may still be being written by the
    // preceding grid: every role waits for it, the walker and the copies once
    // they have the first piece and its pages, which are index inputs too (1 us
    // a call, back to back).
    auto give_up = [&]() {
        *abort_flag = 1;
        flag_error(a.err, PKV_FLAG_WAIT_TIMEOUT);
    };
    auto lane_wait = [&](uint32_t bb, uint32_t par) -> bool {
        if (mbar_test_wait(bb, par)) return true;  // (cheaper than try_wait when the phase is over)
        uint64_t t0 = 0;
        while (!mbar_try_wait(bb, par)) {
            const uint64_t now = global_ns();
            if (t0 == 0) t0 = now;
            if (*abort_flag || now - t0 > kWaitLimitNs) {
                give_up();
                return false;
            }
        }
        return true;
    };
    auto warp_wait = [&](uint32_t bb, uint32_t par) -> bool { return __all_sync(0xffffffffu, lane_wait(bb, par)); };
    // Piece i of this CTA, handed over in a ring
    auto piece_bar = [&](int i) { return bar(bPiece + i % kPieces); };
    auto piece_par = [](int i) -> uint32_t { return (i / kPieces) & 1; };
    auto stage = [](int n) { return C::stage(n); };
    auto phase = [](int n) -> uint32_t { return C::round(n) & 1; };

    if (warp < 4) {
        reg_dec<C::REG_IO>();
        if (warp == 0 || warp == 2) {
            // ======================= copies of K, of V ================================
            const int v = warp >> 1;
            constexpr int FULL = FP8 ? bRawFull : bFull, FREE = FP8 ? bRawFree : bFree;
            constexpr int COPIES = FP8 ? kTilePages : kTilePages * C::NB;  // per tile
            const int pg = lane % kTilePages, blk = lane / kTilePages;     // this lane's copy
            const bool hnd = a.layout == PKV_HND;
            // (Items of one (sequence, kv head) read the same tiles, so the hint might hurt where there are many;
            // it does not: chunks of 128 to 2048 tokens behind 8 to 256 Ki take the same time without, the
            // drafted tokens' widest case 184 us and not 182.)
            const uint64_t policy = l2_policy_evict_first();
            int n = v;
            bool ok = true, bad = false;
            for (int i = 0; ok; ++i) {
                if (!warp_wait(piece_bar(i), piece_par(i))) break;
                const Piece w = pieces[i % kPieces];
                __syncwarp();
                if (w.b < 0) break;
                if (lane == 0) mbar_arrive(bar(bPieceFree + i % kPieces));
                const int npages = (w.L + kPageSize - 1) / kPageSize;
                auto page_at = [&](int t) -> int {
                    const int p = t * kTilePages + pg;
                    return p < npages && t < w.t1 ? __ldg(a.block_tables + w.b * a.bt_s0 + p) : -1;
                };
                int nxt = page_at(w.t0);
                if (i == 0) grid_dep_wait();
                for (int t = w.t0; t < w.t1; ++t, n += 2) {
                    int id = nxt;
                    nxt = page_at(t + 1);
                    if (id < 0 || id >= num_pages) {
                        bad |= t * kTilePages + pg < npages;
                        id = static_cast<int>(num_pages);  // out of range: the copy fills zeros
                    }
                    const int st = C::copy_stage(n), rd = C::copy_round(n);
                    if (rd > 0) ok = warp_wait(bar(FREE + st), (rd - 1) & 1);
                    if (!ok) break;
                    const uint32_t fb = bar(FULL + st);
                    if (lane == 0) mbar_arrive_expect_tx(fb, FP8 ? C::RAW : C::TILE);
                    __syncwarp();
                    if (lane < COPIES) {
                        const uint32_t dst = FP8 ? s0 + C::OFF_R + st * C::RAW + pg * kPageSize * C::RBOX
                                                 : s0 + C::OFF_T + st * C::TILE + blk * C::BLOCK + pg * kPageSize * 128;
                        tma_load_4d(dst, v ? &tmv : &tmk, fb, FP8 ? 0 : blk * 64, hnd ? 0 : w.kvh, hnd ? w.kvh : 0, id,
                                    policy);
                    }
                    __syncwarp();
                }
            }
            if (bad && blk == 0 && v == 0) flag_error(a.err, PKV_FLAG_PAGE_RANGE);
            if (lane == 0) {
                // Copies under way land before the CTA may exit: the last ones of every
                // stage that neither copy warp has taken again.
                constexpr int BACK = FP8 ? C::RST : 2 * (C::SK > C::SV ? C::SK : C::SV);
                for (int i = n - 2; i >= 0 && i > n - 1 - v - BACK; i -= 2)
                    if (FP8 || i + 2 * (v ? C::SV : C::SK) >= n)
                        (void)mbar_wait_bounded(bar(FULL + C::copy_stage(i)), C::copy_round(i) & 1, kWaitLimitNs);
            }
        } else if (warp == 3 && lane == 0) {
            // ======================= the CTA's pieces, and q ==========================
            int4 meta = make_int4(0, 0, 0, 0);     // what the joining kernel is to do with the cut item
            const Cuts cuts(total, gridDim.x);
            const uint64_t policy = l2_policy_evict_first();
            int uses0 = 0, uses1 = 0, buf = 1;
            bool ok = true;
            Walk walk(from, to);
            for (int i = 0; ok; ++i) {
                Piece w;
                w.b = walk.next(a) ? walk.b : -1;
                if (w.b >= 0) {
                    w.kvh = walk.kvh, w.q0 = walk.s.q0, w.L = walk.s.L, w.ctx = walk.s.ctx;
                    w.tok0 = walk.rg * 2 * a.tile_toks;
                    w.toks = min(walk.s.N - w.tok0, 2 * a.tile_toks);
                    w.t0 = walk.t0, w.t1 = walk.t1;
                    w.whole = w.t0 == 0 && w.t1 == walk.nt;
                    w.two = w.toks > a.tile_toks;
                    if (!w.two) buf ^= 1;
                    w.buf = buf;
                    w.uses0 = uses0, w.uses1 = uses1;
                }
                if (i >= kPieces && !lane_wait(bar(bPieceFree + i % kPieces), (i / kPieces - 1) & 1)) break;
                pieces[i % kPieces] = w;
                mbar_arrive(piece_bar(i));
                if (w.b < 0) break;
                if (w.t0 == 0 && w.t1 < walk.nt) {
                    // the CTA that has the item's last unit
                    const int c1 = cuts.at_or_before(cuts.cut(static_cast<int>(blockIdx.x) + 1) - w.t1 + walk.nt - 1);
                    meta = make_int4(w.q0 + w.tok0, w.toks, c1 - static_cast<int>(blockIdx.x) + 1, w.kvh);
                }
                if (i == 0) grid_dep_wait();
                // q, once the buffer is free: tile_toks tokens x G heads are consecutive operand rows
                w.buffers([&](int bf, int uses) {
                    if (ok && uses > 0) ok = lane_wait(bar(bQFree + bf), (uses - 1) & 1);
                    if (!ok) return;
                    const uint32_t fb = bar((FP8 ? bQRaw : bQ) + bf);
                    mbar_arrive_expect_tx(fb, a.tile_toks * a.G * D * 2);
                    for (int c = 0; c < C::NB; ++c)
                        tma_load_3d(s0 + C::OFF_Q + bf * C::TILE + c * C::BLOCK, &tmq, fb, 64 * c, w.kvh * a.G,
                                    w.q0 + w.tok0 + (w.two ? bf * a.tile_toks : 0), policy);
                    ++(bf ? uses1 : uses0);
                });
            }
            grid_dep_wait();
            reinterpret_cast<int4*>(a.workspace)[blockIdx.x] = meta;
            if (uses0) (void)mbar_wait_bounded(bar(FP8 ? bQRaw : bQ), (uses0 - 1) & 1, kWaitLimitNs);
            if (uses1) (void)mbar_wait_bounded(bar((FP8 ? bQRaw : bQ) + 1), (uses1 - 1) & 1, kWaitLimitNs);
        } else if (warp == 1 && lane == 0) {
            // ======================= tensor-core issue (one thread) ===================
            grid_dep_wait();  // (so that its bounded waits begin behind the preceding grid)
            constexpr int FMT = FP8 ? 0 : 1;  // f16 or bf16 operands
            // the sign of softmax_scale goes into q (bit 13 negates A)
            const uint32_t idesc_qk = umma_idesc(128, kTile, FMT, FMT, false, false) | (a.scale_log2 < 0.f ? 1u << 13 : 0u);
            constexpr uint32_t kIdescPv = umma_idesc(128, D, FMT, FMT, false, true);
            // 128-byte-swizzled operands, 1024 bytes between groups of 8 rows
            constexpr uint32_t kDescHi = (1024 >> 4) | (1u << 14) | (2u << 29);
            auto desc_lo = [](uint32_t addr, uint32_t lead) { return ((addr >> 4) & 0x3FFFu) | (lead >> 4) << 16; };
            int tile0 = 0;                             // tiles before this piece
            int p0 = 0, p1 = 0, n_qk = 0, n_o = 0;     // P taken of either group, scores and items issued
            bool ok = true;
            for (int i = 0; ok; ++i) {
                ok = lane_wait(piece_bar(i), piece_par(i));
                const Piece w = pieces[i % kPieces];
                if (!ok || w.b < 0) break;
                const int nt = w.t1 - w.t0, nj = w.two ? 2 * nt : nt;
                // the item before has no more use for S
                if (i > 0) ok = lane_wait(bar(bX + (i - 1) % kPieces), ((i - 1) / kPieces) & 1);
                w.buffers([&](int bf, int uses) { ok = ok && lane_wait(bar(bQ + bf), uses & 1); });
                auto landed = [&](int n) -> bool { return lane_wait(bar(bFull + stage(n)), phase(n)); };
                // Job j is tile j / 2 for group j % 2 (two row tiles), or tile j for group
                // j % 2. P . V of a job, then the scores of that group's next one, which
                // take S from under P: the tensor cores execute in order of issue.
                for (int j = -2; ok && j < nj; ++j) {
                    const int g = j & 1, t = w.two ? j >> 1 : j, tn = w.two ? t + 1 : t + 2;
                    const int n = 2 * (tile0 + t) + 1, n2 = 2 * (tile0 + tn);  // V here, the next K
                    const uint32_t tS = tmem + 256 * g;
                    const bool more = j + 2 < nj;
                    bool here = false;
                    if (j >= 0) {
                        // (what has landed is looked up before P is waited for)
                        ok = landed(n);
                        here = ok && more && mbar_test_wait(bar(bFull + stage(n2)), phase(n2));
                        ok = ok && lane_wait(bar(bP + g), (g ? p1 : p0) & 1);
                        if (!ok) break;
                        ++(g ? p1 : p0);
                        tc_fence_after();
                        const uint32_t vt = desc_lo(s0 + C::OFF_T + stage(n) * C::TILE, C::BLOCK);
                        const uint32_t more_o = j > 1 || *reinterpret_cast<volatile uint32_t*>(go_on + g) != 0u;  // O goes on, or starts
#pragma unroll
                        for (int k = 0; k < kTile / 16; ++k)
#pragma unroll
                            for (int e = 0; e < C::TERMS; ++e)
                                umma_ts(tS + C::O_COL, tS + C::p_col(k, e), vt + k * (2048 >> 4), kDescHi, kIdescPv,
                                        k + e > 0 ? 1u : more_o);
                        if (!w.two) {
                            // (one row tile is bound by memory: V's stage is wanted back at once)
                            mbar_arrive(bar(bFree + stage(n)));
                            umma_commit(bar(bFree + stage(n)));
                        }
                    }
                    if (more) {
                        ok = here || landed(n2);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t q = desc_lo(s0 + C::OFF_Q + (w.two ? g : w.buf) * C::TILE, 16);
                        const uint32_t kt = desc_lo(s0 + C::OFF_T + stage(n2) * C::TILE, 16);
#pragma unroll
                        for (int k = 0; k < D / 16; ++k) {
                            const uint32_t at = ((k >> 2) * C::BLOCK + (k & 3) * 32) >> 4;
                            if (k == 0) umma_ss<true>(tS, q, kt, kDescHi, idesc_qk);
                            else umma_ss<false>(tS, q + at, kt + at, kDescHi, idesc_qk);
                        }
                        umma_commit(bar(bS + g));
                        ++n_qk;
                    } else if (j >= 0) {
                        umma_commit(bar(bO + g));      // the item's O
                        ++n_o;
                    }
                }
                mbar_arrive(bar(bPieceFree + i % kPieces));
                tile0 += nt;
            }
            // Every operation issued is done before the tensor memory is freed: the
            // softmax groups wait for their last O, and a give-up for all of them here.
            if (!ok && n_qk + n_o > 0) {
                umma_commit(bar(bEnd));
                (void)mbar_wait_bounded(bar(bEnd), 0, kWaitLimitNs);
            }
        }
        __syncwarp();
    } else if (warp < 12) {
        // ======================= softmax ==========================================
        reg_inc<C::REG_SM>();
        grid_dep_wait();
        grid_dep_launch();
        const int grp = (warp - 4) >> 2, wq = warp & 3;
        const int row_l = 32 * wq + lane;              // this thread's lane of tensor memory
        const uint32_t tl = tmem + (static_cast<uint32_t>(wq) << 21);  // lanes 32 wq .. (bits 16 and up)
        const uint32_t tS = tl + 256 * grp, tO = tS + C::O_COL;
        const int tok_l = row_l / a.G, g_l = row_l - tok_l * a.G;      // its token in the row tile, its head
        int tile0 = 0, job = 0;                        // tiles before this piece, this group's jobs
        int n_o = 0, n_oo = 0;                         // items that this and the other group had a part in
        const bool speaker = wq == 0 && lane == 0;     // for its group
        bool ok = true;
        for (int i = 0;; ++i) {
            ok = named_bar_and(1, 256, warp_wait(piece_bar(i), piece_par(i)));
            const Piece& w = pieces[i % kPieces];
            if (!ok || w.b < 0) break;
            const bool two = w.two;
            const int tok_t = tok_l + (two ? grp * a.tile_toks : 0);   // token in the pair of row tiles
            const bool live = tok_l < a.tile_toks && tok_t < w.toks;
            const bool warp_live = __any_sync(0xffffffffu, live);
            const int tok = live ? w.tok0 + tok_t : 0;                 // this row's drafted token
            const int row = (two ? 128 * grp : 0) + row_l;             // its place in partial sums
            const uint32_t* mrow = a.mask != nullptr && live ? a.mask + (w.q0 + tok) * a.mask_s0 : nullptr;
            float sl = fabsf(a.scale_log2), vs = 1.f;
            if constexpr (FP8) {
                w.buffers([&](int bf, int uses) { ok = ok && warp_wait(bar(bQ + bf), uses & 1); });
                sl *= fabsf(__ldg(a.k_scale + (a.n_scale == 1 ? 0 : w.kvh))) * q_scale[128 * (two ? grp : w.buf) + row_l];
                vs = __ldg(a.v_scale + (a.n_scale == 1 ? 0 : w.kvh));
            }
            sl = fmaxf(sl, 1.2e-38f);                  // -inf times it stays -inf (a scale that is no number: see q)
            const int L = w.L, ctx = w.ctx, t1 = w.t1, w_t0 = w.t0;
            const int32_t* table = a.block_tables + w.b * a.bt_s0;
            const int npages = (L + kPageSize - 1) / kPageSize;
            const int job0 = job;
            float m = -INFINITY, l = 0.f;
            const int step = two ? 1 : 2;
            // lanes 0-7: the tile's pages, read one tile ahead
            auto page_id = [&](int t) -> int {
                const int p = t * kTilePages + lane;
                return t < t1 && lane < kTilePages && p < npages ? __ldg(table + p) : 0;
            };
            const int tb = w_t0 + (two ? 0 : grp);
            int id_next = page_id(tb);
            for (int t = tb; t < t1; t += step, ++job) {
                const int p0 = t * kTile;
                const int n = 2 * (tile0 + t - w_t0) + 1;        // ring slot of the tile's V
                const int id = id_next;
                id_next = page_id(t + step);
                const uint32_t pages_now = __ballot_sync(0xffffffffu, id >= 0 && id < num_pages);
                const bool inner = p0 + kTile <= ctx && pages_now == ~0u;
                uint32_t vis[4] = {~0u, ~0u, ~0u, ~0u}, bad[4] = {0u, 0u, 0u, 0u};
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
                // P . V of the job before is done with, too.
                if (ok) ok = warp_wait(bar(bS + grp), job & 1);
                tc_fence_after();
                if (speaker && ok) {
                    mbar_arrive(bar(bFree + stage(n - 1)));                            // K
                    if (!two) mbar_arrive(bar(bFree + stage(n - 1)));
                    if (two && job > job0) mbar_arrive(bar(bFree + stage(n - 2)));     // the V before
                    if (job == job0) *reinterpret_cast<volatile uint32_t*>(go_on + grp) = 0u;
                }
                // ---- V rows that a weight of zero would not silence --------------------
                if (p0 + kTile > ctx) {
                    const bool landed = ok && warp_wait(bar(bFull + stage(n)), phase(n));
                    const int pos = p0 + row_l;                  // thread = row of the tile here
                    const uint32_t vrow = s0 + C::OFF_T + stage(n) * C::TILE + row_l * 128;
                    bool odd = false;
                    if (landed && pos >= ctx && pos < L) {
                        constexpr uint32_t EX = FP8 ? 0x7C00u : 0x7F80u;
#pragma unroll 4
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
                const bool any_bad = (bad[0] | bad[1] | bad[2] | bad[3]) != 0u;  // (uniform)
                // ---- the tile's softmax, 32 columns at a time: short loops stay in the
                // ---- instruction cache (64 at a time, and 128 held so that S is read only
                // ---- once, were slower by 2% and 8%)
                auto columns = [&](int c, uint32_t (&x)[32]) {
                    tmem_ld32(tS + 32 * c, x);
                    tmem_wait_ld();
                    pin(x);
                    if (!inner) {
                        const uint32_t v0 = word_of(vis, c);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!(v0 & (1u << e))) x[e] = 0xFF800000u;
                    }
                };
                const bool work = ok && warp_live;
                if (work) {
                    float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        uint32_t x[32];
                        columns(c, x);
#pragma unroll
                        for (int e = 0; e < 32; e += 2)
                            mx4[e >> 1 & 3] = fmaxf(fmaxf(mx4[e >> 1 & 3], __uint_as_float(x[e])), __uint_as_float(x[e + 1]));
                    }
                    const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * sl;
                    const bool move = mx > m + kRescaleLog2 || (m == -INFINITY && mx > m);
                    if (__any_sync(0xffffffffu, move)) {
                        const float nm = move ? mx : m;
                        const float al = move ? fast_exp2(m - nm) : 1.f;
                        if (job > job0) {
#pragma unroll 1
                            for (int c = 0; c < D / 32; ++c) {
                                uint32_t o[32];
                                tmem_ld32(tO + 32 * c, o);
                                tmem_wait_ld();
                                pin(o);
                                uint32_t h0[16], h1[16];
#pragma unroll
                                for (int e = 0; e < 16; ++e) {
                                    h0[e] = __float_as_uint(__uint_as_float(o[e]) * al);
                                    h1[e] = __float_as_uint(__uint_as_float(o[16 + e]) * al);
                                }
                                tmem_st16(tO + 32 * c, h0);
                                tmem_st16(tO + 32 * c + 16, h1);
                            }
                        }
                        l *= al;
                        m = nm;
                    }
                }
                const float mm = m == -INFINITY ? 0.f : C::P_LOG2 - m;
                const float2 sl2 = make_float2(sl, sl), mm2 = make_float2(mm, mm);
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    if (work) {
                        uint32_t x[32];
                        columns(c, x);
                        uint32_t p[16], rest[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float2 y = fma2(make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), sl2, mm2);
                            y.x = fast_exp2(y.x);
                            y.y = fast_exp2(y.y);
                            sum[e & 1] = add2(sum[e & 1], y);
                            if constexpr (FP8) {
                                p[e] = pack_f16(y.x, y.y);
                            } else {
                                p[e] = pack_bf16(y.x, y.y);
                                y = fma2(make_float2(bf16_lo(p[e]), bf16_hi(p[e])), make_float2(-1.f, -1.f), y);  // (exact)
                                rest[e] = pack_bf16(y.x, y.y);
                            }
                        }
                        if (any_bad) {
                            const uint32_t b = word_of(bad, c);
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const uint32_t keep = (b & (1u << (2 * e)) ? 0u : 0x0000FFFFu) | (b & (2u << (2 * e)) ? 0u : 0xFFFF0000u);
                                p[e] &= keep;
                                if constexpr (!FP8) rest[e] &= keep;
                            }
                        }
                        if constexpr (FP8) {
                            tmem_st16(tS + C::p_col(2 * c, 0), p);
                        } else {
                            tmem_st32(tS + C::p_col(2 * c, 0), p, rest);
                        }
                    }
                }
                tmem_wait_st();
                l += (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
                // ---- drafted tokens whose V is not finite, for the rows that see them ----
                if (any_bad) {
                    if (job == job0) {  // there is no O yet: it starts here, and P . V goes on from it
                        const uint32_t zero[16] = {};
#pragma unroll 1
                        for (int c = 0; c < D / 16; ++c) tmem_st16(tO + 16 * c, zero);
                        tmem_wait_st();
                        if (speaker) *reinterpret_cast<volatile uint32_t*>(go_on + grp) = 1u;
                    }
                    for (int j = 0; ok && j < kTile; ++j) {
                        if (!(word_of(bad, j >> 5) >> (j & 31) & 1)) continue;
                        const int id = __ldg(table + (p0 + j) / kPageSize);
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
                        const bool sees = live && (word_of(vis, j >> 5) >> (j & 31) & 1);
                        float x = 0.f;
                        if (sees) {
                            const uint16_t* qr = a.q + (w.q0 + tok) * a.q_s0 + (w.kvh * a.G + g_l) * a.q_s1;
                            for (int d = 0; d < D; ++d)
                                x += __uint_as_float(static_cast<uint32_t>(qr[d]) << 16) * at(a.k_cache, kb + d);
                            x *= a.scale_log2 * (FP8 ? __ldg(a.k_scale + (a.n_scale == 1 ? 0 : w.kvh)) : 1.f);
                            x = fast_exp2(x + mm);
                        }
#pragma unroll 1
                        for (int c = 0; c < D / 16; ++c) {
                            uint32_t o[16];
                            tmem_ld16(tO + 16 * c, o);
                            tmem_wait_ld();
                            pin(o);
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                if (sees) o[e] = __float_as_uint(fmaf(x, at(a.v_cache, vb + 16 * c + e), __uint_as_float(o[e])));
                            tmem_st16(tO + 16 * c, o);
                            tmem_wait_st();
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0 && ok) mbar_arrive(bar(bP + grp));
            }
            // ---- the piece's sums ---------------------------------------------------
            const int nt = t1 - w_t0;
            const bool mine = job > job0;
            const bool theirs = !two && nt > 1 - grp;
            float mo = -INFINITY, lo = 0.f;            // the other group's
            tc_fence_before();
            ok = named_bar_and(1, 256, ok);            // every S of this piece is read, and q done with
            tc_fence_after();
            if (!ok) break;
            tc_fence_before();
            if (lane == 0) mbar_arrive(bar(bX + i % kPieces));  // S may be written for the next item
            // q's buffer is free for m and l, and then the output
            const uint32_t stage_row = s0 + C::OFF_Q + (two ? grp : w.buf) * C::TILE + row_l * 128;
            if (!two) {
                // where the thread that reads them writes its first 16 bytes of output
                auto ml_at = [&](int reader) -> uint32_t {
                    const int ch = reader * (D / 16);
                    return stage_row + (ch >> 3) * C::BLOCK + ((ch ^ row_l) & 7) * 16;
                };
                sts128u(ml_at(1 - grp), __float_as_uint(m), __float_as_uint(l), 0u, 0u);
                (void)named_bar_and(1, 256, true);
                const uint4 x = lds128(ml_at(grp));
                mo = __uint_as_float(x.x);
                lo = __uint_as_float(x.y);
            }
            if (mine) ok = warp_wait(bar(bO + grp), n_o & 1);
            if (theirs) ok = ok && warp_wait(bar(bO + 1 - grp), n_oo & 1);
            tc_fence_after();
            n_o += mine;
            n_oo += two || nt > 1 - grp;
            if (speaker && ok && two) mbar_arrive(bar(bFree + stage(2 * (tile0 + nt) - 1)));  // the last V
            if (ok && warp_live) {
                const float M = fmaxf(m, mo), M0 = M - C::P_LOG2;  // (M0: what P and its sums are relative to)
                const float f0 = m == -INFINITY ? 0.f : fast_exp2(m - M), f1 = mo == -INFINITY ? 0.f : fast_exp2(mo - M);
                const float sum = (mine ? l * f0 : 0.f) + (theirs ? lo * f1 : 0.f);
                const bool whole = w.whole;
                const bool none = sum == 0.f;
                const float inv = whole ? (none ? 0.f : vs / sum) : vs, k0 = f0 * inv, k1 = f1 * inv;
                const int h = w.kvh * a.G + g_l;
                const int slot = 2 * static_cast<int>(blockIdx.x) + (w_t0 == 0 ? 1 : 0);
                float* part = part_o<D>(a.workspace, gridDim.x, slot, row);
                if (live && (two || grp == 0)) {
                    if (!whole) {
                        *reinterpret_cast<float2*>(part_ml(a.workspace, slot, row)) = make_float2(M0, sum);
                    } else if (a.lse) {
                        a.lse[(w.q0 + tok) * a.l_s0 + h * a.l_s1] =
                            none ? -INFINITY : (M0 + __log2f(sum)) * 0.69314718055994530942f;
                    }
                }
                // Two row tiles: all of this row's columns; else each group half of them.
                // A whole item's output goes through q's buffer (the warp's own 32
                // rows), so that the warp writes rows and not columns.
                const int c0 = two ? 0 : grp * (D / 32), c1 = two ? D / 16 : c0 + D / 32;  // 16 columns each
#pragma unroll 1
                for (int c = c0; c < c1; ++c) {
                    uint32_t x[16], y[16];
                    if (mine) tmem_ld16(tO + 16 * c, x);
                    if (theirs) tmem_ld16(tl + 256 * (1 - grp) + C::O_COL + 16 * c, y);
                    tmem_wait_ld();
                    pin(x);
                    pin(y);
                    float o[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        o[e] = mine ? __uint_as_float(x[e]) * k0 : 0.f;
                        if (theirs) o[e] = fmaf(__uint_as_float(y[e]), k1, o[e]);
                    }
                    if (whole) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int ch = 2 * c + e;
                            sts128u(stage_row + (ch >> 3) * C::BLOCK + ((ch ^ row_l) & 7) * 16, pack_bf16(o[8 * e], o[8 * e + 1]),
                                    pack_bf16(o[8 * e + 2], o[8 * e + 3]), pack_bf16(o[8 * e + 4], o[8 * e + 5]),
                                    pack_bf16(o[8 * e + 6], o[8 * e + 7]));
                        }
                    } else if (live) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            *reinterpret_cast<float4*>(part + static_cast<int64_t>(4 * c + e) * kRows * 4) =
                                make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                    }
                }
                if (whole) {
                    __syncwarp();
                    const int64_t off = live ? (w.q0 + tok) * a.o_s0 + h * a.o_s1 : -1;  // this lane's row
                    const int per_row = 2 * (c1 - c0);                                      // 16-byte chunks: 16, 8 or 4
                    const int sub = lane / per_row, ch = 2 * c0 + lane - sub * per_row;
#pragma unroll 4
                    for (int i = 0; i < per_row; ++i) {
                        const int r = i * (32 / per_row) + sub;
                        const int64_t o = __shfl_sync(0xffffffffu, off, r);
                        const uint4 v = lds128(stage_row + (r - lane) * 128 + (ch >> 3) * C::BLOCK + ((ch ^ r) & 7) * 16);
                        if (o >= 0) *reinterpret_cast<uint4*>(a.out + o + 8 * ch) = v;
                    }
                }
            }
            fence_proxy_async_smem();                  // q's next copy comes after the staged rows
            __syncwarp();
            if (lane == 0) {
                w.buffers([&](int bf, int) { mbar_arrive(bar(bQFree + bf)); });
                mbar_arrive(bar(bPieceFree + i % kPieces));
            }
            tc_fence_before();
            if (!two) ok = named_bar_and(1, 256, ok);  // either group's O is read by both
            tile0 += nt;
        }
    } else {
        // ======================= E4M3 bytes and bf16 q to f16 tiles ===============
        reg_dec<C::REG_CV>();
        grid_dep_wait();
        const int ct = tid - 384;
        constexpr int CH = D / 16;  // 16-byte chunks of a raw row
        int n = 0;
        bool ok = true;
        for (int i = 0; ok; ++i) {
            ok = warp_wait(piece_bar(i), piece_par(i));
            const Piece w = pieces[i % kPieces];
            if (!ok || w.b < 0) break;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(bPieceFree + i % kPieces));
            // q takes the sign of k_scale, or its being no number, which then reaches the scores of the positions
            // that a row sees (as a factor of the masked ones' -inf it would not leave them out)
            const float ks = __ldg(a.k_scale + (a.n_scale == 1 ? 0 : w.kvh));
            const float sign = ks != ks ? ks : copysignf(1.f, ks);
            w.buffers([&](int bf, int uses) {
                ok = ok && warp_wait(bar(bQRaw + bf), uses & 1);
                if (!ok) return;
                constexpr int QC = D / 8;              // 16-byte chunks of a row of q
                const int ch = ct % QC;
#pragma unroll 2
                for (int r = ct / QC; r < 128; r += 128 / QC) {
                    const uint32_t at = s0 + C::OFF_Q + bf * C::TILE + (ch >> 3) * C::BLOCK + r * 128 + ((ch ^ r) & 7) * 16;
                    const uint4 x = lds128(at);
                    const uint32_t v[4] = {x.x, x.y, x.z, x.w};
                    // 2^k with 2^k max|q| in [2^14, 2^15), from the exponent of the row's largest value
                    uint32_t mx = 0;
#pragma unroll
                    for (int e = 0; e < 4; ++e) mx = max(mx, max(v[e] & 0x7F80u, (v[e] >> 16) & 0x7F80u));
#pragma unroll
                    for (int d = 1; d < QC; d <<= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, d));
                    int ex = static_cast<int>(mx >> 7);    // biased exponent
                    ex = ex == 255 ? 127 : max(ex, 20);    // not finite: stays so; tiny rows: 2^121
                    const float up = sign * __uint_as_float(static_cast<uint32_t>(127 + 141 - ex) << 23);
                    if (ch == 0) q_scale[128 * bf + r] = __uint_as_float(static_cast<uint32_t>(127 + ex - 141) << 23);
                    sts128u(at, pack_f16(bf16_lo(v[0]) * up, bf16_hi(v[0]) * up), pack_f16(bf16_lo(v[1]) * up, bf16_hi(v[1]) * up),
                            pack_f16(bf16_lo(v[2]) * up, bf16_hi(v[2]) * up), pack_f16(bf16_lo(v[3]) * up, bf16_hi(v[3]) * up));
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(bQ + bf));
            });
            for (int t = w.t0; ok && t < w.t1; ++t) {
                for (int v = 0; v < 2; ++v, ++n) {
                    const int rs = C::RST ? n % C::RST : 0;
                    ok = warp_wait(bar(bRawFull + rs), (n / (C::RST ? C::RST : 1)) & 1);
                    if (ok && n >= C::ST) ok = warp_wait(bar(bFree + stage(n)), (C::round(n) - 1) & 1);
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
                        h[0] = e4m3x2_to_f16x2(lo16(x.x)), h[1] = e4m3x2_to_f16x2(hi16(x.x));
                        h[2] = e4m3x2_to_f16x2(lo16(x.y)), h[3] = e4m3x2_to_f16x2(hi16(x.y));
                        h[4] = e4m3x2_to_f16x2(lo16(x.z)), h[5] = e4m3x2_to_f16x2(hi16(x.z));
                        h[6] = e4m3x2_to_f16x2(lo16(x.w)), h[7] = e4m3x2_to_f16x2(hi16(x.w));
                        // either half first, by column block: eight lanes meet all banks once
                        const bool swap = ch & 4;
                        sts128u(swap ? e1 : e0, swap ? h[4] : h[0], swap ? h[5] : h[1], swap ? h[6] : h[2], swap ? h[7] : h[3]);
                        sts128u(swap ? e0 : e1, swap ? h[0] : h[4], swap ? h[1] : h[5], swap ? h[2] : h[6], swap ? h[3] : h[7]);
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

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

// ---- joining the pieces of cut items ------------------------------------------------
// The work is blocks of rows of the cut items (entry c of the CTAs' notes: the
// item whose first piece CTA c had), numbered through and dealt to a grid that is
// resident at once. A warp reads 8 rows x 4 quads of columns at a time (128-byte
// runs of the partial sums), eight reads of 16 bytes per thread on their way: of
// four row blocks of two pieces (items cut once), or of eight pieces.
template <int D, int R, int U>
__device__ __forceinline__ void join_rows(const TreeArgs& a, int ctas, int c, const int4 meta, int r0) {
    const int lane = threadIdx.x & 31, quad = (threadIdx.x >> 5) * 4 + (lane >> 3);
    const int n = meta.z;                                // pieces: slot 1 of CTA c, slot 0 of the next ones
    int row[R];                                          // places in the partial sums; rows past the item: the last one
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const int r = min(r0 + 8 * k + (lane & 7), meta.y * a.G - 1);  // row: token r / G, head r % G
        row[k] = r < a.tile_toks * a.G ? r : 128 + r - a.tile_toks * a.G;
    }
    float M[R], sum[R];
    float4 o[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
        M[k] = -INFINITY;
        sum[k] = 0.f;
        o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int i0 = 0; i0 < n; i0 += U) {                  // online over the pieces
        float2 ml[U][R];
        float4 x[U][R];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u, slot = 2 * (c + i) + (i == 0 ? 1 : 0);
#pragma unroll
            for (int k = 0; k < R; ++k) {
                ml[u][k] = make_float2(-INFINITY, 0.f);
                x[u][k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i < n) {
                    ml[u][k] = *reinterpret_cast<const float2*>(part_ml(a.workspace, slot, row[k]));
                    x[u][k] = *reinterpret_cast<const float4*>(part_o<D>(a.workspace, ctas, slot, row[k]) + quad * (kRows * 4));
                }
            }
        }
#pragma unroll
        for (int k = 0; k < R; ++k) {
            float m = M[k];
#pragma unroll
            for (int u = 0; u < U; ++u) m = fmaxf(m, ml[u][k].x);
            const float al = M[k] == -INFINITY ? 0.f : fast_exp2(M[k] - m);
            M[k] = m;
            sum[k] *= al;
            o[k].x *= al, o[k].y *= al, o[k].z *= al, o[k].w *= al;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (i0 + u >= n) break;
                const float f = ml[u][k].x == -INFINITY ? 0.f : fast_exp2(ml[u][k].x - m);
                sum[k] += f * ml[u][k].y;
                o[k].x += f * x[u][k].x, o[k].y += f * x[u][k].y, o[k].z += f * x[u][k].z, o[k].w += f * x[u][k].w;
            }
        }
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
        const int r = r0 + 8 * k + (lane & 7), tok = r / a.G, g = r - tok * a.G;
        if (tok >= meta.y) continue;
        const bool none = sum[k] == 0.f;
        const float inv = none ? 0.f : 1.f / sum[k];
        const int h = meta.w * a.G + g;
        uint2* out = reinterpret_cast<uint2*>(a.out + (meta.x + tok) * a.o_s0 + h * a.o_s1 + quad * 4);
        *out = none ? make_uint2(0u, 0u) : make_uint2(pack_bf16(o[k].x * inv, o[k].y * inv), pack_bf16(o[k].z * inv, o[k].w * inv));
        if (quad == 0 && a.lse)
            a.lse[(meta.x + tok) * a.l_s0 + h * a.l_s1] =
                none ? -INFINITY : (M[k] + __log2f(sum[k])) * 0.69314718055994530942f;
    }
}

template <int D>
__global__ void __launch_bounds__(2 * D) tree_join_kernel(const TreeArgs a, int ctas) {
    extern __shared__ int4 note[];                       // [ctas]
    int* first = reinterpret_cast<int*>(note + ctas);    // [ctas + 1]: the first block of entry c's item
    const int4* notes = reinterpret_cast<const int4*>(a.workspace);  // first token, tokens, pieces, kv head
    auto rows_per_block = [](int4 m) { return m.z <= 2 ? 32 : 8; };
    // The next grid may start: everything before the tree kernel is done (it began
    // this one behind its own wait), and neither of the two writes index inputs.
    grid_dep_launch();
    grid_dep_wait();
    for (int c = threadIdx.x; c < ctas; c += 2 * D) {
        const int4 m = notes[c];
        note[c] = m;
        first[c + 1] = (m.y * a.G + rows_per_block(m) - 1) / rows_per_block(m);
    }
    if (threadIdx.x == 0) first[0] = 0;
    __syncthreads();
    if (threadIdx.x < 32) {
        int base = 0;
        for (int c0 = 0; c0 < ctas; c0 += 32) {
            const int c = c0 + threadIdx.x;
            int v = c < ctas ? first[c + 1] : 0;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, v, d);
                if (static_cast<int>(threadIdx.x) >= d) v += y;
            }
            if (c < ctas) first[c + 1] = base + v;
            base += __shfl_sync(0xffffffffu, v, 31);
        }
    }
    __syncthreads();
    const int blocks = first[ctas];
    for (int b = blockIdx.x; b < blocks; b += gridDim.x) {
        int lo = 0, hi = ctas;                           // the entry with first[c] <= b < first[c + 1]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (first[mid] <= b) lo = mid;
            else hi = mid;
        }
        const int4 m = note[lo];
        const int r0 = (b - first[lo]) * rows_per_block(m);
        if (m.z <= 2) join_rows<D, 4, 2>(a, ctas, lo, m, r0);
        else join_rows<D, 1, 8>(a, ctas, lo, m, r0);
    }
}

template <int D, bool FP8>
cudaError_t launch_t(const TreeArgs& a, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s) {
    using C = Cfg<D, FP8>;
    int sms = 0;
    cudaError_t e = device_sm_count(&sms);
    if (e != cudaSuccess) return e;
    // The roles deal out the registers that the kernel is launched with: as many
    // as assumed, or it would wait for more that never come.
    static std::atomic<bool> as_assumed{false};
    if (!as_assumed.load(std::memory_order_relaxed)) {
        cudaFuncAttributes at{};
        e = cudaFuncGetAttributes(&at, tree_kernel<D, FP8>);
        if (e != cudaSuccess) return e;
        if (at.numRegs * C::THREADS < C::REGS) return cudaErrorInvalidConfiguration;
        as_assumed.store(true, std::memory_order_relaxed);
    }
    e = cudaFuncSetAttribute(tree_kernel<D, FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    e = launch_dependent(tree_kernel<D, FP8>, dim3(sms), dim3(C::THREADS), C::SMEM, s, tq, tk, tv, a);
    if (e != cudaSuccess) return e;
    // An item of one tile is not cut (two short chats: 9.5 us with a joining kernel, 7.6 without).
    if (a.max_pages * kPageSize <= kTile) return cudaSuccess;
    // An SM holds three of these at once (D = 128; 64 registers a thread, for four, spill: 43 us and not
    // 38 for two long contexts); no more than there are blocks of 8 rows.
    const int grid = static_cast<int>(std::min<int64_t>(3 * sms, (static_cast<int64_t>(a.T) * a.Hq + 7) / 8));
    return launch_dependent(tree_join_kernel<D>, dim3(grid), dim3(2 * D), sms * sizeof(int4) + (sms + 1) * sizeof(int), s, a, sms);
}

}  // namespace

int64_t tree_decode_workspace(int64_t T, int32_t Hq, int32_t D, int32_t sm_count) {
    (void)T, (void)Hq;  // (at most two cut items per CTA, whatever the rows)
    return kMetaBytes + static_cast<int64_t>(sm_count) * 2 * kRows * (D + 2) * 4;
}

cudaError_t launch_tree_decode(const TreeArgs& a, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s) {
    const bool fp8 = a.kind == kFp8;
    if (a.D == 128) return fp8 ? launch_t<128, true>(a, tq, tk, tv, s) : launch_t<128, false>(a, tq, tk, tv, s);
    return fp8 ? launch_t<64, true>(a, tq, tk, tv, s) : launch_t<64, false>(a, tq, tk, tv, s);
}

}  // namespace pkv
