// lq_rows.cu -- per-head norm and position rotation of q and k, to dense
// outputs (lq_qk_norm_rotate) or into a paged key-value cache (lq_kv_append).
//
// Per head row x of D channels (FP32 throughout, one rounding at the end):
//   r = 1 / sqrt(sum x^2 + eps)  or  1 / sqrt(sum x^2 / D + eps),  y = x r w,
//   (y0, y1) <- (y0 cos - y1 sin, y1 cos + y0 sin) for each rotated pair.
// Every row is read once and written once, so DRAM bandwidth bounds long
// calls and launch latency short ones.  A row belongs to D / 8 lanes (8
// channels each: one 16-byte load of BF16, two of FP32), so the sum of
// squares is a butterfly of 3 to 5 shuffles and the partner channels of a
// rotation by halves are one shuffle away.  A block takes one token: its
// table row is loaded once per lane and used for all of the block's rows,
// and the row loads (up to four per lane in flight) do not wait for the
// chain cu_tokens -> pos -> block_table / table.
#include "lq_attn.h"
#include "lq_common.cuh"

namespace lq {
namespace {

template <bool BF16>
struct Raw {
    uint4 w[BF16 ? 1 : 2];
};

template <bool BF16>
__device__ __forceinline__ Raw<BF16> load_raw(const void *p, size_t i) {
    Raw<BF16> r;
    const uint4 *s = reinterpret_cast<const uint4 *>(static_cast<const char *>(p) + i * (BF16 ? 2 : 4));
    r.w[0] = s[0];
    if constexpr (!BF16) r.w[1] = s[1];
    return r;
}

template <bool BF16>
__device__ __forceinline__ void store_raw(void *p, size_t i, const Raw<BF16> &r) {
    uint4 *d = reinterpret_cast<uint4 *>(static_cast<char *>(p) + i * (BF16 ? 2 : 4));
    d[0] = r.w[0];
    if constexpr (!BF16) d[1] = r.w[1];
}

template <bool BF16>
__device__ __forceinline__ void unpack(const Raw<BF16> &r, float (&x)[8]) {
#pragma unroll
    for (int j = 0; j < (BF16 ? 1 : 2); ++j) {
        const uint32_t w[4] = {r.w[j].x, r.w[j].y, r.w[j].z, r.w[j].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (BF16) {
                x[2 * e] = __uint_as_float(w[e] << 16);
                x[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
            } else {
                x[4 * j + e] = __uint_as_float(w[e]);
            }
        }
    }
}

template <bool BF16>
__device__ __forceinline__ Raw<BF16> pack(const float (&x)[8]) {
    Raw<BF16> r;
    if constexpr (BF16) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
            w[e] = *reinterpret_cast<const uint32_t *>(&p);
        }
        r.w[0] = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        r.w[0] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
        r.w[1] = make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7]));
    }
    return r;
}

template <int N>
__device__ __forceinline__ void load_f32(float *v, const float *p) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const float4 x = __ldg(reinterpret_cast<const float4 *>(p + i));
        v[i] = x.x, v[i + 1] = x.y, v[i + 2] = x.z, v[i + 3] = x.w;
    }
}

// One block: NR rows for each of its groups of D / 8 lanes, all of token
// blockIdx.x; rows are the q heads, the k heads and, when appending, the v
// heads (copied).
template <int D, bool BF16, bool ADJ, bool APPEND, int NR>
__global__ void __launch_bounds__(256) rows_kernel(const RowsArgs a) {
    constexpr int L = D / 8;
    const int tid = threadIdx.x, l = tid & (L - 1), c = 8 * l;
    const int groups = blockDim.x / L;
    const long long t = blockIdx.x;
    const int R = a.Hq + a.Hkv * (APPEND ? 2 : 1);
    const int r0 = blockIdx.y * groups * NR + tid / L;

    Raw<BF16> raw[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int r = r0 + i * groups;
        if (r >= R) raw[i] = Raw<BF16>{};
        else if (r < a.Hq) raw[i] = load_raw<BF16>(a.q, t * a.q_stride + r * D + c);
        else if (!APPEND || r < a.Hq + a.Hkv) raw[i] = load_raw<BF16>(a.k, t * a.k_stride + (r - a.Hq) * D + c);
        else raw[i] = load_raw<BF16>(a.v, t * a.v_stride + (r - a.Hq - a.Hkv) * D + c);
    }

    // the token's position and, when appending, its place in the cache
    // (the same for the whole block)
    long long p = 0;
    size_t page_row = 0;  // row of the token in head 0 of its page
    if constexpr (APPEND) {
        int b;
        long long i;
        if (a.cu) {
            // sequences whose first row is at or before t
            int n = 0;
            for (int j0 = 0; j0 <= a.B; j0 += blockDim.x) {
                const int j = j0 + tid;
                n += __syncthreads_count(j <= a.B && __ldg(a.cu + j) <= t);
            }
            b = n - 1;
            if (b < 0 || b >= a.B) return;  // padding behind the last sequence
            i = t - __ldg(a.cu + b);
        } else {
            const int per = a.tokens / a.B;
            b = (int)(t / per);
            i = t - (long long)b * per;
        }
        const int first = __ldg(a.pos + b);
        if (first < 0) return;  // idle slot
        p = first + i;
        bool bad_pos = i < 0 || p >= (long long)a.max_pages * a.page_size || (a.rot > 0 && p >= a.table_len);
        int page = 0;
        if (!bad_pos) page = __ldg(a.block_table + (size_t)b * a.max_pages + (int)(p / a.page_size));
        const bool bad_page = page < 0 || page >= a.num_pages;
        if (bad_pos || bad_page) {
            if (tid == 0 && blockIdx.y == 0) atomicOr(&g_dev_error, bad_pos ? kErrBadPosition : kErrBadPage);
            return;
        }
        page_row = (size_t)page * a.Hkv * a.page_size + (size_t)(p % a.page_size);
    } else if (a.positions) {
        p = __ldg(a.positions + t);
        if (p < 0) return;  // padding
        if (a.rot > 0 && p >= a.table_len) {
            if (tid == 0 && blockIdx.y == 0) atomicOr(&g_dev_error, kErrBadPosition);
            return;
        }
    }

    const int half = a.rot / 2;
    const bool turned = c < a.rot;
    // rot is a multiple of 16, so a lane's 8 channels lie on one side of
    // rot / 2 and the partner channels belong to one other lane
    const bool low = c < half;
    const int partner = turned ? (low ? l + half / 8 : l - half / 8) : l;
    constexpr int NT = ADJ ? 4 : 8;
    float cs[NT], sn[NT];
    if (turned) {
        const float *row = a.cos_sin + (size_t)p * a.rot + (ADJ ? c / 2 : (low ? c : c - half));
        load_f32<NT>(cs, row);
        load_f32<NT>(sn, row + half);
    }

#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int r = r0 + i * groups;
        const bool is_v = APPEND && r >= a.Hq + a.Hkv;
        float x[8];
        unpack<BF16>(raw[i], x);
        if (a.norm) {
            float ss = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
            ss = group_sum<L>(ss);
            const float f = 1.0f / sqrtf(a.norm == 2 ? ss * (1.0f / D) + a.eps : ss + a.eps);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= f;
            const float *w = r < a.Hq ? a.q_weight : a.k_weight;
            if (w && !is_v) {
                float wv[8];
                load_f32<8>(wv, w + c);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] *= wv[e];
            }
        }
        if (a.rot > 0) {
            if constexpr (ADJ) {
                if (turned) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float x0 = x[2 * e], x1 = x[2 * e + 1];
                        x[2 * e] = x0 * cs[e] - x1 * sn[e];
                        x[2 * e + 1] = x1 * cs[e] + x0 * sn[e];
                    }
                }
            } else {
                float y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = __shfl_sync(0xffffffffu, x[e], partner, L);
                if (turned) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = low ? x[e] * cs[e] - y[e] * sn[e] : x[e] * cs[e] + y[e] * sn[e];
                }
            }
        }
        if (r >= R) continue;
        const Raw<BF16> out = is_v ? raw[i] : pack<BF16>(x);
        if (r < a.Hq) store_raw<BF16>(a.q_out, ((size_t)t * a.Hq + r) * D + c, out);
        else if constexpr (APPEND) {
            const int h = is_v ? r - a.Hq - a.Hkv : r - a.Hq;
            store_raw<BF16>(is_v ? a.v_pages : a.k_pages, (page_row + (size_t)h * a.page_size) * D + c, out);
        } else store_raw<BF16>(a.k_out, ((size_t)t * a.Hkv + (r - a.Hq)) * D + c, out);
    }
}

template <int D, bool BF16, bool ADJ, bool APPEND>
cudaError_t launch_rows_d(const RowsArgs &a, cudaStream_t stream) {
    constexpr int L = D / 8;
    const int R = a.Hq + a.Hkv * (APPEND ? 2 : 1);
    // one row per group while all of them fit on the GPU at once, else four
    const bool wide = (long long)a.tokens * R * L > 148LL * 2048;
    const int nr = wide ? 4 : 1;
    int threads = (R + nr - 1) / nr * L;
    threads = threads >= 256 ? 256 : (threads + 31) / 32 * 32;
    const int rows = threads / L * nr;
    const dim3 grid((unsigned)a.tokens, (unsigned)((R + rows - 1) / rows));
    if (wide) rows_kernel<D, BF16, ADJ, APPEND, 4><<<grid, threads, 0, stream>>>(a);
    else rows_kernel<D, BF16, ADJ, APPEND, 1><<<grid, threads, 0, stream>>>(a);
    return cudaGetLastError();
}

template <int D, bool BF16>
cudaError_t launch_rows_t(const RowsArgs &a, bool adjacent, bool append, cudaStream_t stream) {
    if (adjacent)
        return append ? launch_rows_d<D, BF16, true, true>(a, stream) : launch_rows_d<D, BF16, true, false>(a, stream);
    return append ? launch_rows_d<D, BF16, false, true>(a, stream) : launch_rows_d<D, BF16, false, false>(a, stream);
}

}  // namespace

cudaError_t launch_rows(const RowsArgs &a, int D, bool bf16, bool adjacent, bool append, cudaStream_t stream) {
    switch (D) {
        case 64: return bf16 ? launch_rows_t<64, true>(a, adjacent, append, stream) : launch_rows_t<64, false>(a, adjacent, append, stream);
        case 128: return bf16 ? launch_rows_t<128, true>(a, adjacent, append, stream) : launch_rows_t<128, false>(a, adjacent, append, stream);
        case 256: return bf16 ? launch_rows_t<256, true>(a, adjacent, append, stream) : launch_rows_t<256, false>(a, adjacent, append, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace lq
