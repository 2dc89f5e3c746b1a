// lq_attn_prefill.cu -- attention of runs of new tokens over the paged
// key-value cache (lq_attn_prefill), causal from each token's own position.
//
// attn_prefill_simt: 64 query rows of one head per block, key tiles staged in
// shared memory as FP32, 4 x 4 register tiles of FP32 FMAs, running maximum
// and sum per row.
#include "lq_attn_common.cuh"

namespace lq {
namespace {

template <int D>
struct Simt {
    static constexpr int kRows = 64, kThreads = 256;
    static constexpr int kKeys = D == 256 ? 32 : 64;
    static constexpr int kCols = kKeys / 16;     // key columns of a thread
    static constexpr int kLd = D + 4;            // row stride of Q and K: rows on distinct banks
    static constexpr int kSmem = (kRows * kLd + kKeys * kLd + kKeys * D + kRows * (kKeys + 4)) * 4;
};

// Four consecutive io elements.
template <bool BF16>
__device__ __forceinline__ float4 load4(const void *p, size_t i) {
    if constexpr (BF16) {
        const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(p) + i);
        return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u),
                           __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u));
    } else {
        return *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
    }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(256) attn_prefill_simt(const AttnArgs a) {
    using S = Simt<D>;
    constexpr int LD = S::kLd, KT = S::kKeys, NC = S::kCols, PL = KT + 4;
    extern __shared__ __align__(16) float sm[];
    float *qs = sm, *ks = qs + S::kRows * LD, *vs = ks + KT * LD, *ps = vs + KT * D;
    __shared__ int find[S::kThreads / 32 + 6];
    // the last tiles see the most keys: they go first
    const QueryTile qt = find_query_tile<S::kRows, S::kThreads>(a, gridDim.x - 1 - (long long)blockIdx.x, find);
    if (qt.rows <= 0) return;
    const int tid = threadIdx.x, rg = tid >> 4, cg = tid & 15;
    const int h = blockIdx.y, kv = h / (a.Hq / a.Hkv);
    for (int i = tid; i < S::kRows * (D / 4); i += S::kThreads) {
        const int r = i / (D / 4), c = 4 * (i % (D / 4));
        float4 x = make_float4(0, 0, 0, 0);
        if (r < qt.rows) x = load4<BF16>(a.q, ((size_t)(qt.base + qt.first + r) * a.Hq + h) * D + c);
        *reinterpret_cast<float4 *>(qs + r * LD + c) = x;
    }
    const int p0 = qt.start + qt.first;               // position of row 0
    const int len = p0 + qt.rows;                     // keys any row sees: [lo, len)
    const int lo = a.window > 0 && p0 + 1 > a.window ? p0 + 1 - a.window : 0;
    float o[4][D / 16], m[4], l[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        m[r] = -INFINITY, l[r] = 0.0f;
#pragma unroll
        for (int e = 0; e < D / 16; ++e) o[r][e] = 0.0f;
    }
    for (int k0 = lo / KT * KT; k0 < len; k0 += KT) {
        __syncthreads();
        for (int i = tid; i < KT * (D / 4); i += S::kThreads) {
            const int r = i / (D / 4), c = 4 * (i % (D / 4)), tok = k0 + r;
            float4 kx = make_float4(0, 0, 0, 0), vx = kx;
            if (tok >= lo && tok < len) {
                const int page = __ldg(a.block_table + (size_t)qt.b * a.max_pages + (tok >> a.page_shift));
                if (page >= 0 && page < a.num_pages) {
                    const size_t at = (((size_t)page * a.Hkv + kv) * a.page_size + (tok & (a.page_size - 1))) * D + c;
                    kx = load4<BF16>(a.k_pages, at);
                    vx = load4<BF16>(a.v_pages, at);
                } else if (c == 0) {
                    atomicOr(&g_dev_error, kErrBadPage);
                }
            }
            *reinterpret_cast<float4 *>(ks + r * LD + c) = kx;
            *reinterpret_cast<float4 *>(vs + r * D + c) = vx;
        }
        __syncthreads();
        float s[4][NC];
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int j = 0; j < NC; ++j) s[r][j] = 0.0f;
#pragma unroll 4
        for (int c = 0; c < D; c += 4) {
            float4 qv[4], kx[NC];
#pragma unroll
            for (int r = 0; r < 4; ++r) qv[r] = *reinterpret_cast<const float4 *>(qs + (4 * rg + r) * LD + c);
#pragma unroll
            for (int j = 0; j < NC; ++j) kx[j] = *reinterpret_cast<const float4 *>(ks + (cg + 16 * j) * LD + c);
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int j = 0; j < NC; ++j) {
                    s[r][j] = fmaf(qv[r].x, kx[j].x, s[r][j]);
                    s[r][j] = fmaf(qv[r].y, kx[j].y, s[r][j]);
                    s[r][j] = fmaf(qv[r].z, kx[j].z, s[r][j]);
                    s[r][j] = fmaf(qv[r].w, kx[j].w, s[r][j]);
                }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int p = p0 + 4 * rg + r;
            float mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < NC; ++j) {
                const int tok = k0 + cg + 16 * j;
                const bool seen = tok <= p && (a.window == 0 || tok > p - a.window);
                float x = a.softcap > 0.0f ? capped_log2<BF16>(s[r][j], a.scale, a.softcap) : s[r][j] * (a.scale * kLog2e);
                s[r][j] = seen ? x : -INFINITY;
                mx = fmaxf(mx, s[r][j]);
            }
            mx = group_max<16>(mx);
            const float n = fmaxf(m[r], mx);
            const float base = n == -INFINITY ? 0.0f : n;
            const float f = ex2(m[r] - base);
            m[r] = n;
            l[r] *= f;
#pragma unroll
            for (int e = 0; e < D / 16; ++e) o[r][e] *= f;
#pragma unroll
            for (int j = 0; j < NC; ++j) {
                const float w = ex2(s[r][j] - base);
                l[r] += w;
                ps[(4 * rg + r) * PL + cg + 16 * j] = w;
            }
        }
        __syncwarp();  // the rows of P are read by the half-warp that wrote them
#pragma unroll 2
        for (int k = 0; k < KT; k += 4) {
            float4 pv[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) pv[r] = *reinterpret_cast<const float4 *>(ps + (4 * rg + r) * PL + k);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                for (int e = 0; e < D / 64; ++e) {
                    const float4 v = *reinterpret_cast<const float4 *>(vs + (k + kk) * D + 64 * e + 4 * cg);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float w = kk == 0 ? pv[r].x : kk == 1 ? pv[r].y : kk == 2 ? pv[r].z : pv[r].w;
                        o[r][4 * e] = fmaf(w, v.x, o[r][4 * e]);
                        o[r][4 * e + 1] = fmaf(w, v.y, o[r][4 * e + 1]);
                        o[r][4 * e + 2] = fmaf(w, v.z, o[r][4 * e + 2]);
                        o[r][4 * e + 3] = fmaf(w, v.w, o[r][4 * e + 3]);
                    }
                }
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const float f = 1.0f / group_sum<16>(l[r]);
        const int row = 4 * rg + r;
        if (row >= qt.rows) continue;
#pragma unroll
        for (int e = 0; e < D / 64; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                store_io<BF16>(a.o, ((size_t)(qt.base + qt.first + row) * a.Hq + h) * D + 64 * e + 4 * cg + i, o[r][4 * e + i] * f);
    }
}

template <int D, bool BF16>
cudaError_t launch_simt(const AttnArgs &a, cudaStream_t stream) {
    using S = Simt<D>;
    static std::atomic<uint64_t> ready{0};
    auto kern = attn_prefill_simt<D, BF16>;
    const cudaError_t e = allow_smem(kern, ready, S::kSmem);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)query_tiles(a, S::kRows), (unsigned)a.Hq);
    kern<<<grid, S::kThreads, S::kSmem, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_prefill(const AttnArgs &a, int D, bool bf16, cudaStream_t stream) {
    switch (D) {
        case 64: return bf16 ? launch_simt<64, true>(a, stream) : launch_simt<64, false>(a, stream);
        case 128: return bf16 ? launch_simt<128, true>(a, stream) : launch_simt<128, false>(a, stream);
        case 256: return bf16 ? launch_simt<256, true>(a, stream) : launch_simt<256, false>(a, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace lq
