// qk_norm_write.cu -- RMS norm of every q and k head, RoPE and the paged-KV
// cache write in one pass.
//
// Mapping: as rope_kv_write_kernel, thread c of a row's D/16 owns the 8-value
// chunks at 8c and at D/2 + 8c, partners of one another's rotation pairs. A
// thread takes U heads of one token: its position, its cos / sin and its weights
// are loaded once for them, and all of their rows before any is used. A CTA's
// rows are of one kind (the grid is the CTAs of q, then of k, then of v), in the
// order of tokens and groups of heads; a row's threads are consecutive lanes of
// one warp, and the sum of its squares is a butterfly over them.
//
// Arithmetic: r = rsqrtf(mean(x^2) + eps), the mean in float32 (its sum in a fixed
// order); y = (x r) w, each product rounded; then the rotation and the cache
// formats of rope_kv_write.cu, bit for bit.
//
// Bound: HBM for fills (39,750 tokens of 32 + 2 x 8 heads, D = 128, bf16, keys kept:
// 1,060 MB in 162 us, 6.5 TB/s, 96% of a copy's rate; a thread's four heads of loads
// are what is in flight); the quantisers' instructions for FP8 and NVFP4 caches
// (22,197 tokens of 12 + 2 x 2 heads, FP8: 187 MB in 34.8 us, 79%); latency for a step's
// tokens (61 of 32 + 2 x 8 heads: 2.3 us within a graph, 7.1 us by itself).
#include <type_traits>

#include "pkv_internal.h"
#include "pkv_ptx.cuh"
#include "rope_row.cuh"

namespace pkv {
namespace {

// The thread's 16 weights: chunks 8c and D/2 + 8c of [D] float32 or bf16.
template <int D>
__device__ __forceinline__ void load_weights(const void* w, int is_bf16, int c, Chunk8& lo, Chunk8& hi) {
    if (is_bf16) {
        const uint16_t* p = static_cast<const uint16_t*>(w);
        lo = unpack_bf16x8(*reinterpret_cast<const uint4*>(p + 8 * c));
        hi = unpack_bf16x8(*reinterpret_cast<const uint4*>(p + D / 2 + 8 * c));
    } else {
        const float* p = static_cast<const float*>(w);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float4 x = *reinterpret_cast<const float4*>(p + 8 * c + 4 * k);
            const float4 y = *reinterpret_cast<const float4*>(p + D / 2 + 8 * c + 4 * k);
            lo.v[4 * k] = x.x, lo.v[4 * k + 1] = x.y, lo.v[4 * k + 2] = x.z, lo.v[4 * k + 3] = x.w;
            hi.v[4 * k] = y.x, hi.v[4 * k + 1] = y.y, hi.v[4 * k + 2] = y.z, hi.v[4 * k + 3] = y.w;
        }
    }
}

// Sum of a key's squares, the same in all of its row's lanes, in one order whatever the launch: columns 32 apart first,
// ascending, then neighbours in pairs, pairs of pairs and so on. One unit in the last place of a norm can move an NVFP4
// value by a third of its block's largest, so the order is stated (pkv.h) and tested to the last bit; this one is what a
// plain float32 mean over the rows gave as well where it was tried (PyTorch 2.9.1 on this GPU, 1 to 318,000 rows). (The
// D = 128 lanes that share columns 32 apart, c and c ^ 4, take four of the eight sums each.)
template <int D>
__device__ __forceinline__ float sum_of_squares(const Chunk8& lo, const Chunk8& hi, int c, unsigned row_lanes) {
    float a[8], b[8];
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        mul_rn_x2(lo.v[e], lo.v[e + 1], lo.v[e], lo.v[e + 1], a[e], a[e + 1]);
        mul_rn_x2(hi.v[e], hi.v[e + 1], hi.v[e], hi.v[e + 1], b[e], b[e + 1]);
    }
    float ss;
    if constexpr (D == 128) {
        const bool up = (c & 4) != 0;
        float t[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float ga = __shfl_xor_sync(row_lanes, up ? a[e] : a[4 + e], 4);
            const float gb = __shfl_xor_sync(row_lanes, up ? b[e] : b[4 + e], 4);
            const float oa = up ? a[4 + e] : a[e], ob = up ? b[4 + e] : b[e];
            t[e] = ((oa + ga) + (up ? gb : ob)) + (up ? ob : gb);
        }
        ss = (t[0] + t[1]) + (t[2] + t[3]);
        ss += __shfl_xor_sync(row_lanes, ss, 4);
    } else {
        ss = (((a[0] + b[0]) + (a[1] + b[1])) + ((a[2] + b[2]) + (a[3] + b[3]))) +
             (((a[4] + b[4]) + (a[5] + b[5])) + ((a[6] + b[6]) + (a[7] + b[7])));
    }
    ss += __shfl_xor_sync(row_lanes, ss, 1);
    ss += __shfl_xor_sync(row_lanes, ss, 2);
    return ss;
}

// The same of a query's, in the fewest instructions (the order above takes 8 more shuffles).
template <int D>
__device__ __forceinline__ float quick_sum_of_squares(const Chunk8& lo, const Chunk8& hi, unsigned row_lanes) {
    float2 s2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        s2[0] = fma2(make_float2(lo.v[e], lo.v[e + 1]), make_float2(lo.v[e], lo.v[e + 1]), s2[0]);
        s2[1] = fma2(make_float2(hi.v[e], hi.v[e + 1]), make_float2(hi.v[e], hi.v[e + 1]), s2[1]);
    }
    float ss = (s2[0].x + s2[0].y) + (s2[1].x + s2[1].y);
#pragma unroll
    for (int d = 1; d < D / 16; d <<= 1) ss += __shfl_xor_sync(row_lanes, ss, d);
    return ss;
}

// Small CTAs: one that waits for its loads holds up fewer of the others (32 prompts of 300 to 2000 tokens, bf16,
// keys kept, four heads a thread: 190 us with 2 CTAs of 256 threads an SM, 172 with 5 of 128, 171 with 10 of 64, 251 with 11
// of 64). At ten a thread has 96 registers, and the four-heads forms spill: bytes stored and loaded, D = 128, bf16 52 and
// 92, FP8 32 and 144, NVFP4 68 and 176; D = 64, 0, 4 and 32, 36 and 88.
constexpr int kThreads = 64;
constexpr int kCtas = 10;  // an SM's, that registers are budgeted for

template <int D, bool INTER, int KIND, int U>
__global__ void __launch_bounds__(kThreads, kCtas) qk_norm_write_kernel(const NormArgs n) {
    constexpr int TPR = D / 16;  // threads per row
    const RopeArgs& a = n.rope;
    // As rope_kv_write_kernel: a programmatic dependent, whose successor waits for it.
    grid_dep_wait();
    grid_dep_launch();
    const bool is_q = blockIdx.x < n.ctas_q, is_k = !is_q && blockIdx.x < n.ctas_q + n.ctas_kv;
    const uint32_t cta = blockIdx.x - (is_q ? 0u : n.ctas_q + (is_k ? 0u : n.ctas_kv));
    const int heads = is_q ? a.Hq : a.Hkv;
    const uint32_t groups = (heads + U - 1) / U;   // of heads, of a token
    const uint32_t item = cta * (kThreads / TPR) + threadIdx.x / TPR;
    const int64_t t = item / groups;
    const int h0 = static_cast<int>(item - static_cast<uint32_t>(t) * groups) * U;
    const int c = threadIdx.x % TPR;
    if (t >= a.T) return;

    // Reading the rows of a skipped token stays inside the [T, heads, D] input.
    const int64_t s1 = is_q ? a.q_s1 : (is_k ? a.k_s1 : a.v_s1);
    const uint16_t* src = is_q ? a.q + t * a.q_s0 : (is_k ? a.k + t * a.k_s0 : a.v + t * a.v_s0);
    const int32_t slot = __ldg(a.slots + t), pos = __ldg(a.positions + t);
    uint4 wlo[U], whi[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (h0 + u >= heads) break;
        const uint16_t* p = src + (h0 + u) * s1;
        wlo[u] = *reinterpret_cast<const uint4*>(p + 8 * c);
        whi[u] = *reinterpret_cast<const uint4*>(p + D / 2 + 8 * c);
    }
    if (slot < 0) return;
    const bool lead = h0 == 0 && c == 0;  // flags a bad token once per kind
    if (slot >= a.num_pages * a.page_size) {
        if (lead) flag_error(a.err, PKV_FLAG_SLOT_RANGE);
        return;
    }
    if (pos < 0 || pos >= a.max_pos) {
        if (lead) flag_error(a.err, PKV_FLAG_POSITION_RANGE);
        return;
    }
    float cv[8], sv[8];
    Chunk8 glo, ghi;
    if (is_q || is_k) {
        load_cos_sin<D, INTER>(a.cos_sin + pos * a.cs_s0, c, cv, sv);
        load_weights<D>(is_q ? n.q_weight : n.k_weight, n.weight_bf16, c, glo, ghi);
    }
    int64_t page;
    int off;
    if (a.page_size == 16) {
        page = slot >> 4;
        off = slot & 15;
    } else {
        page = slot / a.page_size;
        off = static_cast<int>(slot - page * a.page_size);
    }
    const int64_t* st = is_k ? a.kc_s : a.vc_s;
    const int64_t cache_row = page * st[0] + off * (a.layout == PKV_HND ? st[2] : st[1]);
    const int64_t cache_head = a.layout == PKV_HND ? st[1] : st[2];
    // (the lanes of this row and of the rows beside it in a half, quarter or eighth of the warp are all here)
    const unsigned row_lanes = ((1u << TPR) - 1u) << (lane_id() & ~(TPR - 1u));
    // A CTA's kind as a constant: its loop over the heads has no branches on it, and keys' sums cost the queries nothing
    // (one loop for all: 171 us and not 162 for the fill above; with the keys' sums in it FP8 40.6 and not 34.8).
    auto heads_of = [&](auto kind) {
        constexpr bool kQ = decltype(kind)::value == 0, kK = decltype(kind)::value == 1;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = h0 + u;
            if (h >= heads) break;
            Chunk8 lo = unpack_bf16x8(wlo[u]), hi = unpack_bf16x8(whi[u]);
            if constexpr (kQ || kK) {
                const float ss = kK ? sum_of_squares<D>(lo, hi, c, row_lanes) : quick_sum_of_squares<D>(lo, hi, row_lanes);
                const float r = rsqrtf(__fadd_rn(ss * (1.f / D), n.eps));
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    mul_rn_x2(lo.v[e], lo.v[e + 1], r, r, lo.v[e], lo.v[e + 1]);
                    mul_rn_x2(hi.v[e], hi.v[e + 1], r, r, hi.v[e], hi.v[e + 1]);
                    mul_rn_x2(lo.v[e], lo.v[e + 1], glo.v[e], glo.v[e + 1], lo.v[e], lo.v[e + 1]);
                    mul_rn_x2(hi.v[e], hi.v[e + 1], ghi.v[e], ghi.v[e + 1], hi.v[e], hi.v[e + 1]);
                }
                rotate_row<INTER>(lo, hi, cv, sv);
            }
            if (kQ || (kK && n.k_out != nullptr)) {
                uint16_t* p = kQ ? a.q + t * a.q_s0 + h * a.q_s1 : n.k_out + t * n.ko_s0 + h * n.ko_s1;
                *reinterpret_cast<uint4*>(p + 8 * c) = pack_bf16x8(lo);
                *reinterpret_cast<uint4*>(p + D / 2 + 8 * c) = pack_bf16x8(hi);
            }
            if (kQ) continue;
            const int64_t e = cache_row + h * cache_head;
            if constexpr (KIND == kBf16) {
                uint16_t* dst = static_cast<uint16_t*>(kK ? a.k_cache : a.v_cache) + e;
                *reinterpret_cast<uint4*>(dst + 8 * c) = kK ? pack_bf16x8(lo) : wlo[u];
                *reinterpret_cast<uint4*>(dst + D / 2 + 8 * c) = kK ? pack_bf16x8(hi) : whi[u];
            } else {
                const float scale = __ldg((kK ? a.k_scale : a.v_scale) + (a.n_scale == 1 ? 0 : h));
                uint8_t* dst = static_cast<uint8_t*>(kK ? a.k_cache : a.v_cache) + e;
                if constexpr (KIND == kFp8) {
                    const E4m3Rcp r8 = e4m3_rcp(scale);
                    *reinterpret_cast<uint2*>(dst + 8 * c) = pack_e4m3x8(lo, scale, r8);
                    *reinterpret_cast<uint2*>(dst + D / 2 + 8 * c) = pack_e4m3x8(hi, scale, r8);
                } else {
                    // both lanes of a pair (chunks c, c^1 of this row) hold a block's halves
                    const float six_g = __fmul_rn(6.f, scale);
                    const E4m3Rcp r6 = bracket_rcp(six_g);
                    const unsigned pair = 3u << (lane_id() & 30u);
                    float am_lo = amax8(lo), am_hi = amax8(hi);
                    am_lo = fmaxf(am_lo, __shfl_xor_sync(pair, am_lo, 1));
                    am_hi = fmaxf(am_hi, __shfl_xor_sync(pair, am_hi, 1));
                    uint32_t s_lo, s_hi;
                    const uint32_t w_lo = nvfp4_half(lo, am_lo, scale, six_g, r6, s_lo);
                    const uint32_t w_hi = nvfp4_half(hi, am_hi, scale, six_g, r6, s_hi);
                    *reinterpret_cast<uint32_t*>(dst + 4 * c) = w_lo;
                    *reinterpret_cast<uint32_t*>(dst + D / 4 + 4 * c) = w_hi;
                    const int64_t* bs = kK ? a.kbs_s : a.vbs_s;
                    uint8_t* bdst = (kK ? a.k_bs : a.v_bs) + page * bs[0] +
                                    (a.layout == PKV_HND ? h * bs[1] + off * bs[2] : off * bs[1] + h * bs[2]);
                    if (c & 1)
                        bdst[D / 32 + c / 2] = static_cast<uint8_t>(s_hi);
                    else
                        bdst[c / 2] = static_cast<uint8_t>(s_lo);
                }
            }
        }
    };
    if (is_q) heads_of(std::integral_constant<int, 0>{});
    else if (is_k) heads_of(std::integral_constant<int, 1>{});
    else heads_of(std::integral_constant<int, 2>{});
}

template <int D, bool INTER, int KIND, int U>
cudaError_t launch_u(const NormArgs& n, cudaStream_t s) {
    const RopeArgs& a = n.rope;
    constexpr int kItems = kThreads / (D / 16);
    auto ctas = [&](int heads) { return (a.T * ((heads + U - 1) / U) + kItems - 1) / kItems; };
    const int64_t q = ctas(a.Hq), kv = ctas(a.Hkv);
    if ((q + 2 * kv) * kItems > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    NormArgs b = n;
    b.ctas_q = static_cast<uint32_t>(q);
    b.ctas_kv = static_cast<uint32_t>(kv);
    return launch_dependent(qk_norm_write_kernel<D, INTER, KIND, U>, dim3(static_cast<unsigned>(q + 2 * kv)), dim3(kThreads), 0,
                            s, b);
}

// Heads a thread: one where there are few rows, four where there are many (32 + 2 x 8 heads, bf16, keys kept, back to
// back: 256 tokens 3.0 us and not 3.7, 1024 tokens 5.3 and not 7.5, 16,384 tokens 80 and not 114; 12 + 2 x 2, FP8: 1024
// tokens 3.4 and 3.6, 2048 tokens 4.8 and not 5.4. Two: between them, but 2.8 us at 256 tokens.)
constexpr int64_t kManyRows = 20480;
template <int D, bool INTER, int KIND>
cudaError_t launch_t(const NormArgs& n, cudaStream_t s) {
    const RopeArgs& a = n.rope;
    if (a.T == 0) return cudaSuccess;
    if (a.T * (a.Hq + 2 * a.Hkv) >= kManyRows) return launch_u<D, INTER, KIND, 4>(n, s);
    return launch_u<D, INTER, KIND, 1>(n, s);
}

template <int D, bool INTER>
cudaError_t launch_k(const NormArgs& n, cudaStream_t s) {
    switch (n.rope.kind) {
        case kBf16: return launch_t<D, INTER, kBf16>(n, s);
        case kFp8: return launch_t<D, INTER, kFp8>(n, s);
        case kFp4: return launch_t<D, INTER, kFp4>(n, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_qk_norm_write(const NormArgs& n, cudaStream_t s) {
    if (n.rope.D == 128) return n.rope.interleaved ? launch_k<128, true>(n, s) : launch_k<128, false>(n, s);
    return n.rope.interleaved ? launch_k<64, true>(n, s) : launch_k<64, false>(n, s);
}

}  // namespace pkv
