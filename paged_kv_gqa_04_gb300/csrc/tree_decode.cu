// tree_decode.cu -- attention of drafted tokens over a paged cache: the
// context in full, the drafted tokens under a tree mask or as a chain.
//
// One CTA per (drafted token, kv head), four warps over the tokens, a lane
// D/32 head-dim values: scores by a warp sum, online softmax per head of the
// group, the warps' states combined at the end. Scores, weights and sums are
// fp32; the output is rounded once.
#include "pkv_internal.h"
#include "pkv_ptx.cuh"

namespace pkv {
namespace {

constexpr int kWarps = 4;
constexpr int kMaxG = 16;

template <int D, bool FP8>
__device__ __forceinline__ void load_vals(const void* base, int64_t off, float (&x)[D / 32]) {
    constexpr int V = D / 32;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int64_t at = off + V * lane + i;
        if constexpr (FP8) {
            const uint32_t h = e4m3x2_to_f16x2(static_cast<const uint8_t*>(base)[at]);
            x[i] = __half2float(__ushort_as_half(static_cast<unsigned short>(h & 0xFFFFu)));
        } else {
            x[i] = __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(base)[at]) << 16);
        }
    }
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kWarps * 32) tree_kernel(const TreeArgs a) {
    constexpr int V = D / 32;
    __shared__ float qs[kMaxG][D], part[kWarps][kMaxG][D], pm[kWarps][kMaxG], pl[kWarps][kMaxG];
    grid_dep_wait();
    const int r = blockIdx.x, kvh = blockIdx.y, G = a.G;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // the sequence of row r (ranges clamped to [0, T] and to ascend)
    int b = -1, s = 0, e = 0;
    for (int k = 0; k < a.B; ++k) {
        const int s0 = a.q_start[k], e0 = a.q_start[k + 1];
        const int sk = min(max(s0, 0), a.T), ek = min(max(e0, sk), a.T);
        if ((sk != s0 || ek != e0) && r == 0 && kvh == 0 && threadIdx.x == 0) flag_error(a.err, PKV_FLAG_DRAFT_RANGE);
        if (b < 0 && r >= sk && r < ek) b = k, s = sk, e = ek;
    }
    if (b < 0) return;
    const int N = e - s, i = r - s, cap = a.max_pages * kPageSize;
    int L = a.seq_lens[b], flags = 0;
    if (L < 0 || L > cap) {
        flags |= PKV_FLAG_SEQ_LEN_RANGE;
        L = L < 0 ? 0 : cap;
    }
    if (N > L || (a.mask && N > 32 * a.W)) flags |= PKV_FLAG_DRAFT_RANGE;
    const int ctx = L - N;
    for (int x = threadIdx.x; x < G * D; x += kWarps * 32)
        qs[x / D][x % D] = __uint_as_float(static_cast<uint32_t>(a.q[r * a.q_s0 + (kvh * G + x / D) * a.q_s1 + x % D]) << 16);
    __syncthreads();
    const float ks = FP8 ? a.k_scale[a.n_scale == 1 ? 0 : kvh] : 1.f, vs = FP8 ? a.v_scale[a.n_scale == 1 ? 0 : kvh] : 1.f;
    float m[kMaxG], l[kMaxG], acc[kMaxG][V];
#pragma unroll
    for (int g = 0; g < kMaxG; ++g) {
        m[g] = -INFINITY;
        l[g] = 0.f;
#pragma unroll
        for (int d = 0; d < V; ++d) acc[g][d] = 0.f;
    }
    for (int t = warp; t < L; t += kWarps) {
        const int j = t - ctx;
        if (j >= 0) {
            const bool seen = a.mask ? j < 32 * a.W && (a.mask[r * a.mask_s0 + (j >> 5)] >> (j & 31) & 1) : j <= i;
            if (!seen) continue;
        }
        const int page = a.block_tables[b * a.bt_s0 + t / kPageSize];
        if (page < 0 || page >= a.num_pages) {
            flags |= PKV_FLAG_PAGE_RANGE;
            continue;
        }
        float kx[V], vx[V];
        load_vals<D, FP8>(a.k_cache, page * a.kc_s0 + (t % kPageSize) * a.kc_st + kvh * a.kc_sh, kx);
        load_vals<D, FP8>(a.v_cache, page * a.vc_s0 + (t % kPageSize) * a.vc_st + kvh * a.vc_sh, vx);
#pragma unroll
        for (int g = 0; g < kMaxG; ++g) {
            if (g >= G) break;
            float x = 0.f;
#pragma unroll
            for (int d = 0; d < V; ++d) x += qs[g][V * lane + d] * kx[d];
#pragma unroll
            for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
            x *= a.scale_log2 * ks;
            const float nm = fmaxf(m[g], x);
            const float al = exp2f(m[g] - nm), p = exp2f(x - nm);
            m[g] = nm;
            l[g] = l[g] * al + p;
#pragma unroll
            for (int d = 0; d < V; ++d) acc[g][d] = acc[g][d] * al + p * vx[d];
        }
    }
    if (flags && lane == 0) flag_error(a.err, flags);
#pragma unroll
    for (int g = 0; g < kMaxG; ++g) {
        if (g >= G) break;
#pragma unroll
        for (int d = 0; d < V; ++d) part[warp][g][V * lane + d] = acc[g][d];
        if (lane == 0) pm[warp][g] = m[g], pl[warp][g] = l[g];
    }
    __syncthreads();
    for (int x = threadIdx.x; x < G * D; x += kWarps * 32) {
        const int g = x / D, d = x % D;
        float M = -INFINITY, sum = 0.f, o = 0.f;
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, pm[w][g]);
        for (int w = 0; w < kWarps; ++w) {
            if (pl[w][g] == 0.f) continue;
            const float f = exp2f(pm[w][g] - M);
            sum += f * pl[w][g];
            o += f * part[w][g][d];
        }
        const int h = kvh * G + g;
        a.out[r * a.o_s0 + h * a.o_s1 + d] =
            static_cast<uint16_t>(pack_bf16(sum == 0.f ? 0.f : o * (vs / sum), 0.f) & 0xFFFFu);
        if (d == 0 && a.lse)
            a.lse[r * a.l_s0 + h * a.l_s1] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * 0.69314718055994530942f;
    }
}

}  // namespace

int64_t tree_decode_workspace(int64_t T, int32_t Hq, int32_t D, int32_t sm_count) {
    (void)T, (void)Hq;
    // two partial tiles of 128 rows per CTA: D sums, a maximum and a total each
    return static_cast<int64_t>(sm_count) * 2 * 128 * (D + 2) * 4;
}

cudaError_t launch_tree_decode(const TreeArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s) {
    (void)tk, (void)tv;
    const dim3 grid(a.T, a.Hkv);
    const bool fp8 = a.kind == kFp8;
    auto kern = a.D == 128 ? (fp8 ? tree_kernel<128, true> : tree_kernel<128, false>)
                           : (fp8 ? tree_kernel<64, true> : tree_kernel<64, false>);
    return launch_dependent(kern, grid, dim3(kWarps * 32), 0, s, a);
}

}  // namespace pkv
