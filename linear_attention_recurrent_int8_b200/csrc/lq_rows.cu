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
//
// Measured on B200 (6.55 TB/s copy): 16,384 tokens of 32 + 32 heads, head size
// 128, BF16, L2 norm: 80 us, 6.6 TB/s of algorithmic traffic.  9,458 ragged
// tokens of 16 + 2 + 2 heads at head size 256, RMS norm, rotation, appended:
// 45 us, 4.3 TB/s; issue takes 65 % of the slots there (conversions, norm and
// rotation of 8 channels are about 40 instructions) and the L1 data pipe 59 %
// (a row's weights are loaded with it).
// Two tokens: 2.1 us.  Lanes of 16 channels (52 us appended), several tokens
// to a block (46 to 72) and a shared-memory ring filled by bulk copies (57)
// were slower.
#include "lq_attn.h"
#include "lq_common.cuh"

namespace lq {
namespace {

// A lane's 8 channels of a row as stored, in two groups of four: channels
// off0 .. off0 + 3 and off1 .. off1 + 3 (off1 = off0 + 4 unless SPLIT).
template <bool BF16>
struct Raw {
    uint32_t w[BF16 ? 4 : 8];
};

template <bool BF16, bool SPLIT>
__device__ __forceinline__ Raw<BF16> load_raw(const void *row, int off0, int off1) {
    Raw<BF16> r;
    if constexpr (BF16) {
        const __nv_bfloat16 *p = static_cast<const __nv_bfloat16 *>(row);
        if constexpr (SPLIT) {
            const uint2 a = *reinterpret_cast<const uint2 *>(p + off0), b = *reinterpret_cast<const uint2 *>(p + off1);
            r.w[0] = a.x, r.w[1] = a.y, r.w[2] = b.x, r.w[3] = b.y;
        } else {
            const uint4 a = *reinterpret_cast<const uint4 *>(p + off0);
            r.w[0] = a.x, r.w[1] = a.y, r.w[2] = a.z, r.w[3] = a.w;
        }
    } else {
        const float *p = static_cast<const float *>(row);
        const uint4 a = *reinterpret_cast<const uint4 *>(p + off0), b = *reinterpret_cast<const uint4 *>(p + off1);
        r.w[0] = a.x, r.w[1] = a.y, r.w[2] = a.z, r.w[3] = a.w;
        r.w[4] = b.x, r.w[5] = b.y, r.w[6] = b.z, r.w[7] = b.w;
    }
    return r;
}

template <bool BF16, bool SPLIT>
__device__ __forceinline__ void store_raw(void *row, int off0, int off1, const Raw<BF16> &r) {
    if constexpr (BF16) {
        __nv_bfloat16 *p = static_cast<__nv_bfloat16 *>(row);
        if constexpr (SPLIT) {
            *reinterpret_cast<uint2 *>(p + off0) = make_uint2(r.w[0], r.w[1]);
            *reinterpret_cast<uint2 *>(p + off1) = make_uint2(r.w[2], r.w[3]);
        } else {
            *reinterpret_cast<uint4 *>(p + off0) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
        }
    } else {
        float *p = static_cast<float *>(row);
        *reinterpret_cast<uint4 *>(p + off0) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
        *reinterpret_cast<uint4 *>(p + off1) = make_uint4(r.w[4], r.w[5], r.w[6], r.w[7]);
    }
}

template <bool BF16>
__device__ __forceinline__ void unpack(const Raw<BF16> &r, float (&x)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if constexpr (BF16) x[e] = __uint_as_float((e & 1) ? (r.w[e / 2] & 0xFFFF0000u) : (r.w[e / 2] << 16));
        else x[e] = __uint_as_float(r.w[e]);
    }
}

template <bool BF16>
__device__ __forceinline__ Raw<BF16> pack(const float (&x)[8]) {
    Raw<BF16> r;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if constexpr (BF16) {
            if ((e & 1) == 0) {
                const __nv_bfloat162 p = __floats2bfloat162_rn(x[e], x[e + 1]);
                r.w[e / 2] = *reinterpret_cast<const uint32_t *>(&p);
            }
        } else r.w[e] = __float_as_uint(x[e]);
    }
    return r;
}

__device__ __forceinline__ void load4(float *v, const float *p) {
    const float4 x = __ldg(reinterpret_cast<const float4 *>(p));
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
}

// 1 / sqrt(x) of a normal x, to 2^-22.9.
__device__ __forceinline__ float rsqrt_normal(float x) {
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// One block: NR rows for each of its groups of D / 8 lanes, all of token
// blockIdx.x; rows are the q heads, the k heads and, when appending, the v
// heads (copied).  SPLIT (rotation by halves): the lanes of the rotated
// channels hold 4 of the first half and their 4 partners of the second, so
// that a pair needs no exchange and its cosine and sine are loaded once.
// (Five blocks of 256 threads on an SM instead of four are worth 4 % to BF16
// rows with a rotation, 42 -> 40 us for 9,458 tokens of 32 + 8 heads at head
// size 128; FP32 and appended rows would spill, 76 against 86 us.)
template <int D, bool BF16, bool SPLIT, bool APPEND, int NR>
__global__ void __launch_bounds__(256, NR == 4 ? (BF16 && !APPEND ? 5 : 4) : 6) rows_kernel(const RowsArgs a) {
    constexpr int L = D / 8;
    const int tid = threadIdx.x, l = tid & (L - 1);
    const int half = a.rot / 2;
    const bool turned = 8 * l < a.rot;
    const int off0 = SPLIT && turned ? 4 * l : 8 * l;
    const int off1 = SPLIT && turned ? half + 4 * l : 8 * l + 4;
    const int groups = blockDim.x / L;
    const long long t = blockIdx.x;
    const int R = a.Hq + a.Hkv * (APPEND ? 2 : 1);
    const int r0 = blockIdx.y * groups * NR + tid / L;
    constexpr int es = BF16 ? 2 : 4;

    const char *qrow = static_cast<const char *>(a.q) + t * a.q_stride * es;
    const char *krow = static_cast<const char *>(a.k) + t * a.k_stride * es;
    const char *vrow = APPEND ? static_cast<const char *>(a.v) + t * a.v_stride * es : nullptr;
    Raw<BF16> raw[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int r = r0 + i * groups;
        const char *row = r < a.Hq ? qrow + r * (D * es) : krow + (r - a.Hq) * (D * es);
        if (APPEND && r >= a.Hq + a.Hkv) row = vrow + (r - a.Hq - a.Hkv) * (D * es);
        raw[i] = Raw<BF16>{};
        if (r < R) raw[i] = load_raw<BF16, SPLIT>(row, off0, off1);
    }

    // the token's position and, when appending, its place in the cache
    // (the same for the whole block)
    long long p = 0;
    size_t page_row = 0;  // row of the token in head 0 of its page
    if constexpr (APPEND) {
        int b, first;
        long long i;
        if (a.cu) {
            // the sequence that holds row t: its thread has read all that is
            // needed of it
            __shared__ int found[3];
            bool here = false;
            for (int j = tid; j < a.B; j += blockDim.x) {
                const int c0 = __ldg(a.cu + j), c1 = __ldg(a.cu + j + 1), f = __ldg(a.pos + j);
                if (c0 <= t && t < c1) {
                    here = true;
                    found[0] = j, found[1] = (int)t - c0, found[2] = f;
                }
            }
            if (__syncthreads_count(here) == 0) return;  // padding behind the last sequence
            b = found[0], i = found[1], first = found[2];
        } else {
            const int per = a.tokens / a.B;
            b = (int)(t / per);
            i = t - (long long)b * per;
            first = __ldg(a.pos + b);
        }
        if (first < 0) return;  // idle slot
        p = first + i;
        const bool bad_pos = p < 0 || p >= (long long)a.max_pages * a.page_size || (a.rot > 0 && p >= a.table_len);
        int page = 0;
        if (!bad_pos) page = __ldg(a.block_table + (size_t)b * a.max_pages + (int)(p >> a.page_shift));
        const bool bad_page = page < 0 || page >= a.num_pages;
        if (bad_pos || bad_page) {
            if (tid == 0 && blockIdx.y == 0) atomicOr(&g_dev_error, bad_pos ? kErrBadPosition : kErrBadPage);
            return;
        }
        page_row = (size_t)page * a.Hkv * a.page_size + (size_t)(p & (a.page_size - 1));
    } else if (a.positions) {
        p = __ldg(a.positions + t);
        if (p < 0) return;  // padding
        if (a.rot > 0 && p >= a.table_len) {
            if (tid == 0 && blockIdx.y == 0) atomicOr(&g_dev_error, kErrBadPosition);
            return;
        }
    }

    // the lane's four pairs: (x[e], x[4 + e]) when split, else (x[2 e], x[2 e + 1])
    float cs[4], sn[4];
    if (turned) {
        const float *row = a.cos_sin + (size_t)p * a.rot + 4 * l;
        load4(cs, row);
        load4(sn, row + half);
    }

    // where the heads of the token go
    char *const qdst = static_cast<char *>(a.q_out) + (size_t)t * a.Hq * (D * es);
    char *const kdst = APPEND ? static_cast<char *>(a.k_pages) + page_row * (D * es)
                              : static_cast<char *>(a.k_out) + (size_t)t * a.Hkv * (D * es);
    char *const vdst = APPEND ? static_cast<char *>(a.v_pages) + page_row * (D * es) : nullptr;
    const unsigned next = (APPEND ? a.page_size : 1) * (D * es);  // from a head to the next

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
            const float f = rsqrt_normal(a.norm == 2 ? fmaf(ss, 1.0f / D, a.eps) : ss + a.eps);
            const float *w = r < a.Hq ? a.q_weight : a.k_weight;
            if (w) {
                float wv[8];
                load4(wv, w + off0);
                load4(wv + 4, w + off1);
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = x[e] * f * wv[e];
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] *= f;
            }
        }
        if (turned) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float &x0 = x[SPLIT ? e : 2 * e], &x1 = x[SPLIT ? e + 4 : 2 * e + 1];
                const float y0 = x0 * cs[e] - x1 * sn[e];
                x1 = x1 * cs[e] + x0 * sn[e];
                x0 = y0;
            }
        }
        if (r >= R) continue;
        const Raw<BF16> out = is_v ? raw[i] : pack<BF16>(x);
        char *dst = r < a.Hq ? qdst + r * (D * es) : kdst + (unsigned)(r - a.Hq) * next;
        if (APPEND && is_v) dst = vdst + (unsigned)(r - a.Hq - a.Hkv) * next;
        store_raw<BF16, SPLIT>(dst, off0, off1, out);
    }
}

template <int D, bool BF16, bool SPLIT, bool APPEND>
cudaError_t launch_rows_d(const RowsArgs &a, cudaStream_t stream) {
    constexpr int L = D / 8;
    const int R = a.Hq + a.Hkv * (APPEND ? 2 : 1);
    // one row per group while all of them fit on the GPU at once, else four
    const bool wide = (long long)a.tokens * R * L > 148LL * 2048;
    const int nr = wide ? 4 : 1;
    // as few blocks of up to 256 threads as hold the token's rows, in equal
    // shares (48 rows of head size 256 as 24 + 24 and not 32 + 16: 120 -> 99 us)
    const int most = 256 / L * nr, blocks = (R + most - 1) / most;
    const int threads = (((R + blocks - 1) / blocks + nr - 1) / nr * L + 31) / 32 * 32;
    const int rows = threads / L * nr;
    const dim3 grid((unsigned)a.tokens, (unsigned)((R + rows - 1) / rows));
    if (wide) rows_kernel<D, BF16, SPLIT, APPEND, 4><<<grid, threads, 0, stream>>>(a);
    else rows_kernel<D, BF16, SPLIT, APPEND, 1><<<grid, threads, 0, stream>>>(a);
    return cudaGetLastError();
}

template <int D, bool BF16>
cudaError_t launch_rows_t(const RowsArgs &a, bool split, bool append, cudaStream_t stream) {
    if (split)
        return append ? launch_rows_d<D, BF16, true, true>(a, stream) : launch_rows_d<D, BF16, true, false>(a, stream);
    return append ? launch_rows_d<D, BF16, false, true>(a, stream) : launch_rows_d<D, BF16, false, false>(a, stream);
}

}  // namespace

cudaError_t launch_rows(const RowsArgs &a, int D, bool bf16, bool adjacent, bool append, cudaStream_t stream) {
    const bool split = a.rot > 0 && !adjacent;
    switch (D) {
        case 64: return bf16 ? launch_rows_t<64, true>(a, split, append, stream) : launch_rows_t<64, false>(a, split, append, stream);
        case 128: return bf16 ? launch_rows_t<128, true>(a, split, append, stream) : launch_rows_t<128, false>(a, split, append, stream);
        case 256: return bf16 ? launch_rows_t<256, true>(a, split, append, stream) : launch_rows_t<256, false>(a, split, append, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace lq
