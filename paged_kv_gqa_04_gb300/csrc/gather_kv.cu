// gather_kv.cu -- cached keys and values read back from their pages into packed
// bf16 rows.
//
// Mapping: a CTA takes `rows` consecutive rows of the output. Its first threads
// look up where each lies -- the sequence by bisection of the starts, the page
// in its block table -- once for both caches; then thread (x, y) copies 8 values
// (16 bytes of output) of one head at a time, x over a row's heads and chunks, y
// over the rows, kUnroll rows of K and V on their way at once.
//
// Arithmetic: E4M3 and E2M1 values and their product with a block's E4M3 scale
// are exact in f16; the product with the static scale is float32, rounded once
// more to bf16.
//
// Bound: HBM, where there are rows enough (153,123 rows of 8 heads, D = 128: bf16
// 1,254 MB in 185 us, a copy's rate; 126,341 of FP8 in 120 us, 95%; 64,760 rows of 4
// heads, NVFP4: 170 MB in 31 us, 80%, the start and the end of the grid being the
// rest). 16 values a thread take more registers, so fewer loads in flight (FP8 138 us
// and not 123, NVFP4 41 and not 32).
#include <algorithm>
#include <type_traits>

#include "pkv_internal.h"
#include "pkv_ptx.cuh"

namespace pkv {
namespace {

constexpr int kRows = 32;    // most rows of a CTA (64 take 2% more, 16 as long or 4% more for NVFP4)
constexpr int kThreads = 256;
constexpr int kUnroll = 8;   // (4: NVFP4 2% more)
constexpr int32_t kNobody = -1, kZeros = -2;  // rows of no sequence; rows that no page holds

// 8 values of a cache row as they are stored, with their block's scale byte.
template <int KIND>
struct Raw;
template <>
struct Raw<kBf16> {
    uint4 w;
};
template <>
struct Raw<kFp8> {
    uint2 w;
};
template <>
struct Raw<kFp4> {
    uint32_t w, s;
};

__device__ __forceinline__ uint32_t scaled(uint32_t h, float g) {  // two f16 values times g, as bf16
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    return pack_bf16(__fmul_rn(f.x, g), __fmul_rn(f.y, g));
}

template <int KIND>
__device__ __forceinline__ uint4 values(const Raw<KIND>& r, float g) {
    if constexpr (KIND == kBf16) {
        return r.w;
    } else if constexpr (KIND == kFp8) {
        return make_uint4(scaled(e4m3x2_to_f16x2(static_cast<uint16_t>(r.w.x)), g),
                          scaled(e4m3x2_to_f16x2(static_cast<uint16_t>(r.w.x >> 16)), g),
                          scaled(e4m3x2_to_f16x2(static_cast<uint16_t>(r.w.y)), g),
                          scaled(e4m3x2_to_f16x2(static_cast<uint16_t>(r.w.y >> 16)), g));
    } else {
        uint32_t h[4];
        e2m1x8_to_f16x2(r.w, h);
        const uint32_t s = e4m3x2_to_f16x2(static_cast<uint16_t>(r.s | r.s << 8));
        return make_uint4(scaled(hmul2(h[0], s), g), scaled(hmul2(h[1], s), g), scaled(hmul2(h[2], s), g),
                          scaled(hmul2(h[3], s), g));
    }
}

template <int D, int KIND>
__global__ void __launch_bounds__(kThreads) gather_kernel(const GatherArgs a) {
    constexpr int CPR = D / 8;  // chunks of a row
    __shared__ int32_t page_of[kRows];
    __shared__ int32_t off_of[kRows];
    const int tid = threadIdx.y * blockDim.x + threadIdx.x;
    grid_dep_wait();
    grid_dep_launch();
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.rows;
    const int n = static_cast<int>(min(static_cast<int64_t>(a.rows), a.T - t0));
    bool zeros = false;  // a row here that no page holds
    if (tid < n) {
        const int t = static_cast<int>(t0) + tid;
        // the last sequence that starts at or before row t
        int lo = 0, hi = a.B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (__ldg(a.start + mid) <= t) lo = mid;
            else hi = mid;
        }
        const int first_row = __ldg(a.start + lo);
        int page = kNobody, off = 0, flags = 0;
        if (first_row <= t && t < __ldg(a.start + lo + 1)) {
            const int64_t pos = static_cast<int64_t>(t) - first_row + (a.first ? __ldg(a.first + lo) : 0);
            page = kZeros;
            if (pos < 0 || pos >= static_cast<int64_t>(a.max_pages) * a.page_size) {
                flags = PKV_FLAG_SEQ_LEN_RANGE;
            } else {
                const int entry = static_cast<int>(a.page_shift >= 0 ? pos >> a.page_shift : pos / a.page_size);
                const int id = __ldg(a.block_tables + lo * a.bt_s0 + entry);
                if (id < 0 || id >= a.num_pages) {
                    flags = PKV_FLAG_PAGE_RANGE;
                } else {
                    page = id;
                    off = static_cast<int>(pos - static_cast<int64_t>(entry) * a.page_size);
                }
            }
        }
        if (flags) flag_error(a.err, flags);
        zeros = page == kZeros;
        page_of[tid] = page;
        off_of[tid] = off;
    }
    // (starts that do not ascend within the rows)
    if (blockIdx.x == 0) {
        bool bad = false;
        for (int b = tid; b <= a.B; b += blockDim.x * blockDim.y) {
            const int x = __ldg(a.start + b);
            bad |= x < (b ? __ldg(a.start + b - 1) : 0) || x > a.T;
        }
        if (bad) flag_error(a.err, PKV_FLAG_ROW_RANGE);
    }
    zeros = __syncthreads_or(zeros);

    const int items = a.Hkv * CPR, X = blockDim.x, Y = blockDim.y;
    for (int it = threadIdx.x; it < items; it += X) {
        const int h = it / CPR, c = it % CPR;
        float gk = 1.f, gv = 1.f;
        if constexpr (KIND != kBf16) {
            gk = __ldg(a.k_scale + (a.n_scale == 1 ? 0 : h));
            gv = __ldg(a.v_scale + (a.n_scale == 1 ? 0 : h));
        }
        // (whether there are such rows as a constant: a choice of the factor for each took NVFP4 34 us and not 31)
        auto copy_rows = [&](auto with_zeros) {
            for (int r0 = threadIdx.y; r0 < n; r0 += kUnroll * Y) {
                Raw<KIND> k[kUnroll] = {}, v[kUnroll] = {};
                int page[kUnroll];
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    const int r = r0 + u * Y;
                    page[u] = r < n ? page_of[r] : kNobody;
                    if (page[u] < 0) continue;
                    const int64_t p = page[u];
                    const int off = off_of[r];
                    const int64_t ek = p * a.kc_s0 + off * a.kc_st + h * a.kc_sh, ev = p * a.vc_s0 + off * a.vc_st + h * a.vc_sh;
                    if constexpr (KIND == kBf16) {
                        k[u].w = ldg_nc128(static_cast<const uint16_t*>(a.k_cache) + ek + 8 * c);
                        v[u].w = ldg_nc128(static_cast<const uint16_t*>(a.v_cache) + ev + 8 * c);
                    } else if constexpr (KIND == kFp8) {
                        k[u].w = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.k_cache) + ek + 8 * c));
                        v[u].w = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.v_cache) + ev + 8 * c));
                    } else {
                        k[u].w = __ldg(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.k_cache) + ek + 4 * c));
                        v[u].w = __ldg(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.v_cache) + ev + 4 * c));
                        k[u].s = __ldg(a.k_bs + p * a.kbs_s0 + off * a.kbs_st + h * a.kbs_sh + (c >> 1));
                        v[u].s = __ldg(a.v_bs + p * a.vbs_s0 + off * a.vbs_st + h * a.vbs_sh + (c >> 1));
                    }
                }
#pragma unroll
                for (int u = 0; u < kUnroll; ++u) {
                    if (page[u] == kNobody) continue;
                    const int64_t t = t0 + r0 + u * Y;
                    const bool none = decltype(with_zeros)::value && page[u] == kZeros;
                    *reinterpret_cast<uint4*>(a.k_out + t * a.ko_s0 + h * a.ko_s1 + 8 * c) = values<KIND>(k[u], none ? 0.f : gk);
                    *reinterpret_cast<uint4*>(a.v_out + t * a.vo_s0 + h * a.vo_s1 + 8 * c) = values<KIND>(v[u], none ? 0.f : gv);
                }
            }
        };
        if (zeros) copy_rows(std::true_type{});
        else copy_rows(std::false_type{});
    }
}

template <int D, int KIND>
cudaError_t launch_t(const GatherArgs& a, cudaStream_t s) {
    int sms = 0;
    cudaError_t e = device_sm_count(&sms);
    if (e != cudaSuccess) return e;
    GatherArgs b = a;
    // As many rows a CTA as leave every SM several of them.
    b.rows = kRows;
    while (b.rows > 2 && (a.T + b.rows - 1) / b.rows < 4 * sms) b.rows >>= 1;
    const int items = a.Hkv * (D / 8);
    const int X = std::min(items, kThreads), Y = kThreads / X;
    return launch_dependent(gather_kernel<D, KIND>, dim3(static_cast<unsigned>((a.T + b.rows - 1) / b.rows)), dim3(X, Y), 0, s, b);
}

template <int D>
cudaError_t launch_d(const GatherArgs& a, cudaStream_t s) {
    switch (a.kind) {
        case kBf16: return launch_t<D, kBf16>(a, s);
        case kFp8: return launch_t<D, kFp8>(a, s);
        case kFp4: return launch_t<D, kFp4>(a, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_gather_kv(const GatherArgs& a, cudaStream_t s) {
    return a.D == 128 ? launch_d<128>(a, s) : launch_d<64>(a, s);
}

}  // namespace pkv
