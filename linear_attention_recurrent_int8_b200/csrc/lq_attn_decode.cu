// lq_attn_decode.cu -- attention of one new token per sequence over the
// paged key-value cache (lq_attn_decode).
//
//   o_h = sum_j p_j v_j / sum_j p_j,   p_j = 2^(x_j - m),
//   x_j = log2(e) cap(scale q_h . k_j),  m = max_j x_j,
//
// over the visible tokens j of the sequence.  Each key and value row is used
// by the Hq / Hkv query heads of its head only, a few operations per byte:
// DRAM bandwidth bounds all but the shortest calls.
//
// Work split.  The visible tokens of every (sequence, key-value head) are cut
// into tiles of 8 or 16 tokens; the tiles of all pairs form one line, and the
// line is dealt out to the warps of a persistent grid in equal runs, whatever
// the lengths of the sequences.  Each warp is on its own: a ring of
// shared-memory stages that one of its lanes fills by TMA (a tile's rows of a
// page, 128-byte swizzle, one mbarrier per stage), its own running maximum,
// sum and output accumulators, no block barrier after the start.  A pair that
// lies within one run is finished by its warp; the others leave unnormalised
// parts (o, m, sum) in the workspace that a second launch joins in the order
// of the line, so results do not depend on scheduling.
//
// BF16 (attn_tiles_bf16): query heads are the rows of a 16-row warp MMA.  The
// softmax weights enter the product with V as two BF16 parts (p = hi + lo,
// relative error 2^-17), so the output carries one rounding, its own.  With at
// most 8 heads per key-value head the lower 8 rows hold hi, the upper 8 lo,
// of one and the same MMA.  Warp MMAs and not tcgen05: a tile needs 2 MMAs
// per token, a fifth of what the warp path can issue while DRAM delivers the
// token, and accumulators in registers keep the warps independent.
//
// FP32 (attn_tiles_f32): FP32 FMAs, 8 query heads at a time.
#include "lq_attn_common.cuh"

namespace lq {
namespace {

template <int D, bool BF16>
struct Tile {
    static constexpr int kTok = BF16 || D == 64 ? 16 : 8;       // tokens of a tile
    static constexpr int kWarps = D < 256 ? 8 : 4;              // warps of a block
    static constexpr int kRowEl = BF16 ? 64 : 32;               // elements of a 128-byte box row
    static constexpr int kBoxes = D / kRowEl;                   // boxes of a tile of K (or V)
    static constexpr int kBoxBytes = kTok * 128;
    static constexpr int kHalfBytes = kBoxes * kBoxBytes;       // K of a tile, then V
    static constexpr int kStageBytes = 2 * kHalfBytes;
    // per-warp scratch of the FP32 path: 8 query rows, weights, factors
    static constexpr int kScratch = BF16 ? 0 : 8 * D * 4 + kTok * 32 + 64;
};

constexpr int kMaxStages = 8;
constexpr int kSmemLimit = 227 * 1024;

// Shared memory of a block: [pad to 1024][ring][per-warp scratch][barriers][prefix B + 1][lengths B][scan]
template <int D, bool BF16>
__host__ __device__ constexpr int fixed_smem(int B) {
    return 1024 + Tile<D, BF16>::kWarps * (Tile<D, BF16>::kScratch + kMaxStages * 8) + (2 * B + 1) * 4 + 64;
}

// Workspace: [tiles of a sequence's pair, prefix sums: B + 1 ints, tiles per worker: int], then
// per worker two parts of RU rows: o [RU][D], then (m, sum) [RU].
__host__ __device__ inline size_t ws_header(int B) { return ((size_t)(B + 2) * 4 + 255) / 256 * 256; }

template <int D, int RU>
__host__ __device__ constexpr size_t part_floats() { return (size_t)RU * (D + 2); }

struct DecodePlan {
    int units;       // row groups of all key-value heads of a sequence
    int per_kv;      // row groups of a key-value head
    int stages;
    int workers;
    int min_tiles;   // tiles of the shortest run
};

// Visible range of a sequence: lo .. len - 1 (nothing for idle slots).
__device__ __forceinline__ int first_visible(int len, int window) {
    return window > 0 && len > window ? len - window : 0;
}

template <int TOK>
__device__ __forceinline__ int tile_count(int len, int window) {
    return len <= 0 ? 0 : (len - 1) / TOK - first_visible(len, window) / TOK + 1;
}

// A place on the line of tiles.
struct Cursor {
    int b, u, t, n, len, lo, t0;  // sequence, row group, tile, tiles of the pair, visible range, first tile
};

template <int TOK>
__device__ __forceinline__ void enter_sequence(Cursor &c, const int *len, int window) {
    c.len = len[c.b];
    c.lo = first_visible(c.len, window);
    c.t0 = c.lo / TOK;
    c.n = tile_count<TOK>(c.len, window);
}

template <int TOK>
__device__ __forceinline__ Cursor cursor_at(long long x, const int *prefix, const int *len, int B, int units, int window) {
    int lo = 0, hi = B - 1;  // the first sequence whose tiles end past x
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if ((long long)prefix[mid + 1] * units > x) hi = mid;
        else lo = mid + 1;
    }
    Cursor c;
    c.b = lo;
    enter_sequence<TOK>(c, len, window);
    const long long r = x - (long long)prefix[lo] * units;
    c.u = (int)(r / c.n);
    c.t = (int)(r - (long long)c.u * c.n);
    return c;
}

// To the next tile; sequences without tiles are passed over.
template <int TOK>
__device__ __forceinline__ void advance(Cursor &c, const int *len, int B, int units, int window) {
    if (++c.t < c.n) return;
    c.t = 0;
    if (++c.u < units) return;
    c.u = 0;
    do ++c.b;
    while (c.b < B && len[c.b] <= 0);
    if (c.b < B) enter_sequence<TOK>(c, len, window);
}

// One warp's softmax state and output accumulators over tiles of BF16 rows.
template <int D, int RU>
struct Bf16Core {
    static constexpr int NK = D / 16, NO = D / 8, NR = RU / 8;
    uint32_t q[NK][2 * NR];
    float o[NO][4], m[NR], l[NR];

    // query rows of the group: rows g and (RU = 16) g + 8 of the MMA
    __device__ __forceinline__ void begin(const AttnArgs &a, int b, int head0, int rows, int lane, unsigned char *) {
        const int g = lane >> 2, t = lane & 3;
        const __nv_bfloat16 *qp = static_cast<const __nv_bfloat16 *>(a.q) + ((size_t)b * a.Hq + head0) * D;
#pragma unroll
        for (int k = 0; k < NK; ++k)
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                const uint32_t *p = reinterpret_cast<const uint32_t *>(qp + (size_t)(g + 8 * r) * D + 16 * k + 2 * t);
                const bool in = g + 8 * r < rows;
                q[k][r] = in ? __ldg(p) : 0u;
                q[k][NR + r] = in ? __ldg(p + 4) : 0u;
            }
#pragma unroll
        for (int j = 0; j < NO; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[j][e] = 0.0f;
#pragma unroll
        for (int r = 0; r < NR; ++r) m[r] = -INFINITY, l[r] = 0.0f;
    }

    // one tile: tokens tok0 .. tok0 + 15, visible lo .. len - 1
    __device__ __forceinline__ void tile(const AttnArgs &a, unsigned char *st, int tok0, int lo, int len, int lane,
                                         unsigned char *) {
        using T = Tile<D, true>;
        const int mi = lane >> 3, ri = lane & 7, t = lane & 3;
        const uint32_t kb = smem_u32(st), vb = kb + T::kHalfBytes;
        float s[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[j][e] = 0.0f;
        {
            const uint32_t row = kb + ((mi >> 1) * 8 + ri) * 128;
#pragma unroll
            for (int k = 0; k < NK; ++k) {
                const int ch = 2 * k + (mi & 1);
                uint32_t bf[4];
                ldsm_x4(bf, row + (ch >> 3) * T::kBoxBytes + (((ch & 7) ^ ri) << 4));
                if constexpr (NR == 1) {
                    mma_16816(s[0], q[k][0], 0u, q[k][1], 0u, bf[0], bf[1]);
                    mma_16816(s[1], q[k][0], 0u, q[k][1], 0u, bf[2], bf[3]);
                } else {
                    mma_16816(s[0], q[k][0], q[k][1], q[k][2], q[k][3], bf[0], bf[1]);
                    mma_16816(s[1], q[k][0], q[k][1], q[k][2], q[k][3], bf[2], bf[3]);
                }
            }
        }
        const bool part = tok0 + 16 > len || tok0 < lo;
        const SoftCap cap = soft_cap<true>(a.scale, a.softcap);
        float mx[NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            mx[r] = -INFINITY;
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float &x = s[j][2 * r + e];
                    x = a.softcap > 0.0f ? capped_log2<true>(x, cap) : x * (a.scale * kLog2e);
                    const int tok = tok0 + 8 * j + 2 * t + e;
                    if (part && (tok < lo || tok >= len)) x = -INFINITY;
                    mx[r] = fmaxf(mx[r], x);
                }
            mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
            mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
        }
        bool grew = mx[0] > m[0];
        if constexpr (NR == 2) grew = grew || mx[1] > m[1];
        if (__any_sync(0xffffffffu, grew)) {
            float f[NR];
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                const float n = fmaxf(m[r], mx[r]);
                f[r] = n == -INFINITY ? 1.0f : ex2(m[r] - n);
                m[r] = n;
                l[r] *= f[r];
            }
#pragma unroll
            for (int j = 0; j < NO; ++j) {
                o[j][0] *= f[0], o[j][1] *= f[0];
                o[j][2] *= f[NR - 1], o[j][3] *= f[NR - 1];
            }
        }
        uint32_t hi[2][NR], lw[2][NR];  // weights of tokens 2t, 2t + 1 (+ 8 j)
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            // a row whose scores so far are all -inf has m = -inf and weights 0
            const float base = m[r] == -INFINITY ? 0.0f : m[r];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float p0 = ex2(s[j][2 * r] - base), p1 = ex2(s[j][2 * r + 1] - base);
                l[r] += p0 + p1;
                const __nv_bfloat162 h = __floats2bfloat162_rn(p0, p1);
                hi[j][r] = *reinterpret_cast<const uint32_t *>(&h);
                const __nv_bfloat162 w = __floats2bfloat162_rn(p0 - __uint_as_float(hi[j][r] << 16),
                                                               p1 - __uint_as_float(hi[j][r] & 0xFFFF0000u));
                lw[j][r] = *reinterpret_cast<const uint32_t *>(&w);
            }
        }
        if (part) {
            // rows of V that are not visible may hold NaN: weight 0 would not silence them
            for (int r = 0; r < 16; ++r) {
                if (tok0 + r >= lo && tok0 + r < len) continue;
                for (int ch = lane; ch < D / 8; ch += 32)
                    *reinterpret_cast<uint4 *>(st + T::kHalfBytes + (ch >> 3) * T::kBoxBytes + r * 128 + (ch & 7) * 16) =
                        make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();  // before the stage's next TMA write
            __syncwarp();
        }
        const uint32_t row = vb + ((mi & 1) * 8 + ri) * 128;
#pragma unroll
        for (int n = 0; n < NO / 2; ++n) {
            const int ch = 2 * n + (mi >> 1);
            uint32_t bf[4];
            ldsm_x4_t(bf, row + (ch >> 3) * T::kBoxBytes + (((ch & 7) ^ ri) << 4));
            if constexpr (NR == 1) {
                mma_16816(o[2 * n], hi[0][0], lw[0][0], hi[1][0], lw[1][0], bf[0], bf[1]);
                mma_16816(o[2 * n + 1], hi[0][0], lw[0][0], hi[1][0], lw[1][0], bf[2], bf[3]);
            } else {
                mma_16816(o[2 * n], hi[0][0], hi[0][1], hi[1][0], hi[1][1], bf[0], bf[1]);
                mma_16816(o[2 * n + 1], hi[0][0], hi[0][1], hi[1][0], hi[1][1], bf[2], bf[3]);
                mma_16816(o[2 * n], lw[0][0], lw[0][1], lw[1][0], lw[1][1], bf[0], bf[1]);
                mma_16816(o[2 * n + 1], lw[0][0], lw[0][1], lw[1][0], lw[1][1], bf[2], bf[3]);
            }
        }
    }

    // the pair is complete: normalised rows to a.o; else the raw part to `part`
    __device__ __forceinline__ void end(const AttnArgs &a, int b, int head0, int rows, float *part, int lane,
                                        unsigned char *) {
        const int g = lane >> 2, t = lane & 3;
        if constexpr (NR == 1) {
#pragma unroll
            for (int j = 0; j < NO; ++j) o[j][0] += o[j][2], o[j][1] += o[j][3];  // hi and lo rows
        }
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            float sum = l[r];
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            const int row = g + 8 * r;
            if (row >= rows) continue;
            if (part) {
#pragma unroll
                for (int j = 0; j < NO; ++j)
                    *reinterpret_cast<float2 *>(part + row * D + 8 * j + 2 * t) = make_float2(o[j][2 * r], o[j][2 * r + 1]);
                if (t == 0) *reinterpret_cast<float2 *>(part + RU * D + 2 * row) = make_float2(m[r], sum);
            } else {
                const float f = 1.0f / sum;
                __nv_bfloat16 *op = static_cast<__nv_bfloat16 *>(a.o) + ((size_t)b * a.Hq + head0 + row) * D + 2 * t;
#pragma unroll
                for (int j = 0; j < NO; ++j)
                    *reinterpret_cast<__nv_bfloat162 *>(op + 8 * j) = __floats2bfloat162_rn(o[j][2 * r] * f, o[j][2 * r + 1] * f);
            }
        }
    }
};

// The same over tiles of FP32 rows, 8 query rows.
template <int D>
struct F32Core {
    using T = Tile<D, false>;
    static constexpr int TOK = T::kTok;
    static constexpr int NP = 32 / TOK;             // lanes of one token in q . k
    static constexpr int NRL = 8 / NP;              // rows a lane holds after the reduction
    static constexpr int LPR = D / 4 < 32 ? D / 4 : 32;  // lanes across a row of V
    static constexpr int TG = 32 / LPR;             // token groups in p V
    static constexpr int NV = D / (4 * LPR);        // float4 of a row per lane
    float o[8][4 * NV], m[NRL], l[NRL];

    __device__ __forceinline__ static float *q_smem(unsigned char *sc) { return reinterpret_cast<float *>(sc); }
    __device__ __forceinline__ static float *p_smem(unsigned char *sc) { return reinterpret_cast<float *>(sc) + 8 * D; }
    __device__ __forceinline__ static float *f_smem(unsigned char *sc) { return reinterpret_cast<float *>(sc) + 8 * D + 8 * TOK; }

    // the first of the rows a lane holds after the reduction
    __device__ __forceinline__ static int row0(int lane) {
        const int part = lane / TOK;
        return NP == 4 ? 4 * (part >> 1) + 2 * (part & 1) : 4 * part;
    }

    __device__ __forceinline__ void begin(const AttnArgs &a, int b, int head0, int rows, int lane, unsigned char *sc) {
        const float4 *qp = reinterpret_cast<const float4 *>(static_cast<const float *>(a.q) + ((size_t)b * a.Hq + head0) * D);
        __syncwarp();
        for (int i = lane; i < 8 * D / 4; i += 32)
            reinterpret_cast<float4 *>(q_smem(sc))[i] = i < rows * (D / 4) ? __ldg(qp + i) : make_float4(0, 0, 0, 0);
        __syncwarp();
#pragma unroll
        for (int r = 0; r < 8; ++r)
#pragma unroll
            for (int e = 0; e < 4 * NV; ++e) o[r][e] = 0.0f;
#pragma unroll
        for (int r = 0; r < NRL; ++r) m[r] = -INFINITY, l[r] = 0.0f;
    }

    __device__ __forceinline__ void tile(const AttnArgs &a, unsigned char *st, int tok0, int lo, int len, int lane,
                                         unsigned char *sc) {
        const int tok = lane % TOK, part = lane / TOK;
        float s[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) s[r] = 0.0f;
        // a lane takes 1 / NP of its token's channels; the parts start at
        // different 16-byte chunks so that their q reads hit distinct banks
        constexpr int BPP = T::kBoxes / NP;
#pragma unroll
        for (int bx = 0; bx < BPP; ++bx) {
            const int box = part * BPP + bx;
            const unsigned char *kr = st + box * T::kBoxBytes + tok * 128;
            const float *qr = q_smem(sc) + box * 32;
#pragma unroll 2
            for (int c0 = 0; c0 < 8; ++c0) {
                const int c = (c0 + part * (8 / NP)) & 7;
                const float4 k = *reinterpret_cast<const float4 *>(kr + ((c ^ (tok & 7)) << 4));
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    const float4 q = *reinterpret_cast<const float4 *>(qr + r * D + 4 * c);
                    s[r] = fmaf(q.x, k.x, s[r]);
                    s[r] = fmaf(q.y, k.y, s[r]);
                    s[r] = fmaf(q.z, k.z, s[r]);
                    s[r] = fmaf(q.w, k.w, s[r]);
                }
            }
        }
        // sums over the parts: halving exchanges leave rows row0 .. row0 + NRL - 1 here
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const bool up = (lane & 16) != 0;
            const float send = up ? s[r] : s[r + 4];
            s[r] = (up ? s[r + 4] : s[r]) + __shfl_xor_sync(0xffffffffu, send, 16);
        }
        if constexpr (NP == 4) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const bool up = (lane & 8) != 0;
                const float send = up ? s[r] : s[r + 2];
                s[r] = (up ? s[r + 2] : s[r]) + __shfl_xor_sync(0xffffffffu, send, 8);
            }
        }
        const bool seen = tok0 + tok >= lo && tok0 + tok < len;
        const SoftCap cap = soft_cap<false>(a.scale, a.softcap);
        bool grew = false;
        float mx[NRL];
#pragma unroll
        for (int r = 0; r < NRL; ++r) {
            s[r] = a.softcap > 0.0f ? capped_log2<false>(s[r], cap) : s[r] * (a.scale * kLog2e);
            if (!seen) s[r] = -INFINITY;
            mx[r] = group_max<TOK>(s[r]);
            grew = grew || mx[r] > m[r];
        }
        const int r0 = row0(lane);
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
            for (int r = 0; r < NRL; ++r) {
                const float n = fmaxf(m[r], mx[r]);
                const float f = n == -INFINITY ? 1.0f : ex2(m[r] - n);
                m[r] = n;
                l[r] *= f;
                if (tok == 0) f_smem(sc)[r0 + r] = f;
            }
            __syncwarp();
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const float f = f_smem(sc)[r];
#pragma unroll
                for (int e = 0; e < 4 * NV; ++e) o[r][e] *= f;
            }
        }
#pragma unroll
        for (int r = 0; r < NRL; ++r) {
            const float p = ex2(s[r] - (m[r] == -INFINITY ? 0.0f : m[r]));
            l[r] += p;
            p_smem(sc)[8 * tok + r0 + r] = p;
        }
        __syncwarp();
        // only visible tokens: the others' values may be NaN
        const int t_lo = lo > tok0 ? lo - tok0 : 0, t_hi = len - tok0 < TOK ? len - tok0 : TOK;
        const int vl = lane % LPR, tg = lane / LPR;
#pragma unroll 4
        for (int t = t_lo + tg; t < t_hi; t += TG) {
            const float4 pa = *reinterpret_cast<const float4 *>(p_smem(sc) + 8 * t);
            const float4 pb = *reinterpret_cast<const float4 *>(p_smem(sc) + 8 * t + 4);
            const float p[8] = {pa.x, pa.y, pa.z, pa.w, pb.x, pb.y, pb.z, pb.w};
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int ch = vl + 32 * i;  // 16-byte chunk of the row
                const float4 v = *reinterpret_cast<const float4 *>(st + T::kHalfBytes + (ch >> 3) * T::kBoxBytes + t * 128 +
                                                                  (((ch & 7) ^ (t & 7)) << 4));
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    o[r][4 * i] = fmaf(p[r], v.x, o[r][4 * i]);
                    o[r][4 * i + 1] = fmaf(p[r], v.y, o[r][4 * i + 1]);
                    o[r][4 * i + 2] = fmaf(p[r], v.z, o[r][4 * i + 2]);
                    o[r][4 * i + 3] = fmaf(p[r], v.w, o[r][4 * i + 3]);
                }
            }
        }
    }

    __device__ __forceinline__ void end(const AttnArgs &a, int b, int head0, int rows, float *part, int lane,
                                        unsigned char *sc) {
        const int tok = lane % TOK, r0 = row0(lane), vl = lane % LPR;
        __syncwarp();
#pragma unroll
        for (int r = 0; r < NRL; ++r) {
            const float sum = group_sum<TOK>(l[r]);
            if (tok == 0) {
                f_smem(sc)[r0 + r] = sum;
                if (part && r0 + r < rows)
                    *reinterpret_cast<float2 *>(part + 8 * D + 2 * (r0 + r)) = make_float2(m[r], sum);
            }
        }
        __syncwarp();
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            if constexpr (TG == 2) {
#pragma unroll
                for (int e = 0; e < 4 * NV; ++e) o[r][e] += __shfl_xor_sync(0xffffffffu, o[r][e], 16);
            }
            if (r < rows && lane < LPR) {
                const float f = part ? 1.0f : 1.0f / f_smem(sc)[r];
                float *dst = part ? part + r * D : static_cast<float *>(a.o) + ((size_t)b * a.Hq + head0 + r) * D;
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    *reinterpret_cast<float4 *>(dst + 4 * (vl + 32 * i)) =
                        make_float4(o[r][4 * i] * f, o[r][4 * i + 1] * f, o[r][4 * i + 2] * f, o[r][4 * i + 3] * f);
            }
        }
        __syncwarp();
    }
};

template <int D, bool BF16, int RU>
struct CoreOf {
    using type = Bf16Core<D, RU>;
};
template <int D, int RU>
struct CoreOf<D, false, RU> {
    using type = F32Core<D>;
};

template <int D, bool BF16, int RU>
__global__ void __launch_bounds__(Tile<D, BF16>::kWarps * 32, 1)
    attn_decode_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                       const AttnArgs a, const DecodePlan pl) {
    using T = Tile<D, BF16>;
    constexpr int TOK = T::kTok, NW = T::kWarps;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    unsigned char *scratch = ring + NW * pl.stages * T::kStageBytes;
    uint64_t *bars = reinterpret_cast<uint64_t *>(scratch + NW * T::kScratch);
    int *prefix = reinterpret_cast<int *>(bars + NW * kMaxStages);
    int *len = prefix + a.B + 1;
    int *scan = len + a.B;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    pdl_release();
    // lengths and the prefix sums of tiles per pair
    const int cap = a.max_pages << a.page_shift;
    const int chunk = (a.B + NW * 32 - 1) / (NW * 32);
    int mine = 0;
    for (int i = 0; i < chunk; ++i) {
        const int b = tid * chunk + i;
        if (b >= a.B) break;
        const int p = __ldg(a.pos + b);
        const bool bad = p >= cap;
        if (bad && blockIdx.x == 0) atomicOr(&g_dev_error, kErrBadPosition);
        const int n = p < 0 || bad ? 0 : p + 1;
        len[b] = n;
        mine += tile_count<TOK>(n, a.window);
    }
    int incl = mine;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, s);
        if (lane >= s) incl += y;
    }
    if (lane == 31) scan[warp] = incl;
    if (lane < pl.stages) mbar_init(bars + warp * kMaxStages + lane, 1);
    __syncthreads();
    int at = incl - mine;
    for (int w = 0; w < warp; ++w) at += scan[w];
    for (int i = 0; i < chunk; ++i) {
        const int b = tid * chunk + i;
        if (b >= a.B) break;
        prefix[b] = at;
        at += tile_count<TOK>(len[b], a.window);
        if (b == a.B - 1) prefix[a.B] = at;
    }
    __syncthreads();
    const long long total = (long long)prefix[a.B] * pl.units;
    long long per = (total + pl.workers - 1) / pl.workers;
    if (per < pl.min_tiles) per = pl.min_tiles;
    if (blockIdx.x == 0) {
        int *h = reinterpret_cast<int *>(a.ws);
        for (int b = tid; b <= a.B; b += NW * 32) h[b] = prefix[b];
        if (tid == 0) h[a.B + 1] = (int)per;
    }
    // runs go to the SMs in turn, so that a short line spreads over all of them
    const int worker = warp * gridDim.x + blockIdx.x;
    const long long x0 = worker * per;
    if (x0 >= total) return;
    const int run = (int)(total - x0 < per ? total - x0 : per);

    unsigned char *my_ring = ring + warp * pl.stages * T::kStageBytes;
    uint64_t *full = bars + warp * kMaxStages;
    unsigned char *sc = scratch + warp * T::kScratch;
    float *part = reinterpret_cast<float *>(a.ws + ws_header(a.B)) + (size_t)worker * 2 * part_floats<D, RU>();
    const int G = a.Hq / a.Hkv;
    Cursor c = cursor_at<TOK>(x0, prefix, len, a.B, pl.units, a.window), pc = c;

    // page of the producer's tile, fetched one tile ahead of its use
    auto page_of = [&](const Cursor &k) -> int {
        return k.b < a.B ? __ldg(a.block_table + (size_t)k.b * a.max_pages + (((k.t0 + k.t) * TOK) >> a.page_shift)) : 0;
    };
    int page = page_of(pc), fill = 0, filled = 0;
    auto issue = [&]() {
        if (lane == 0) {
            const bool bad = page < 0 || page >= a.num_pages;
            if (bad) atomicOr(&g_dev_error, kErrBadPage);
            const int z = bad ? -1 : page * a.Hkv + pc.u / pl.per_kv;
            const int row = ((pc.t0 + pc.t) * TOK) & (a.page_size - 1);
            unsigned char *dst = my_ring + fill * T::kStageBytes;
            mbar_arrive_expect_tx(full + fill, T::kStageBytes);
#pragma unroll
            for (int x = 0; x < T::kBoxes; ++x) tma_page_load(dst + x * T::kBoxBytes, &kmap, x * T::kRowEl, row, z, full + fill);
#pragma unroll
            for (int x = 0; x < T::kBoxes; ++x)
                tma_page_load(dst + T::kHalfBytes + x * T::kBoxBytes, &vmap, x * T::kRowEl, row, z, full + fill);
        }
        if (++fill == pl.stages) fill = 0;
        if (++filled < run) {
            advance<TOK>(pc, len, a.B, pl.units, a.window);
            page = page_of(pc);
        }
    };
    while (filled < run && filled < pl.stages) issue();

    typename CoreOf<D, BF16, RU>::type core;
    int st = 0, ph = 0;
    bool fresh = true, whole = false;  // whole: the run holds the pair's first tile
    int head0 = 0, rows = 0;
    for (int i = 0; i < run; ++i) {
        if (fresh) {
            const int kv = c.u / pl.per_kv, first = (c.u - kv * pl.per_kv) * RU;
            head0 = kv * G + first;
            rows = min(RU, G - first);
            core.begin(a, c.b, head0, rows, lane, sc);
            whole = c.t == 0;
            fresh = false;
        }
        if (!bar_wait(full + st, ph)) {
            // give the copies still in flight their time before the block's shared memory is freed
            for (int k = i + 1; k < filled; ++k) {
                if (++st == pl.stages) st = 0, ph ^= 1;
                bar_wait(full + st, ph);
            }
            return;
        }
        unsigned char *stage = my_ring + st * T::kStageBytes;
        core.tile(a, stage, (c.t0 + c.t) * TOK, c.lo, c.len, lane, sc);
        __syncwarp();
        if (filled < run) issue();
        if (++st == pl.stages) st = 0, ph ^= 1;
        const bool last = c.t + 1 == c.n;
        if (last || i + 1 == run) {
            // a part that began in an earlier run goes to the worker's first
            // slot, one that goes on in the next run to its second
            core.end(a, c.b, head0, rows, last && whole ? nullptr : part + (whole ? part_floats<D, RU>() : 0), lane, sc);
            fresh = true;
        }
        if (i + 1 < run) advance<TOK>(c, len, a.B, pl.units, a.window);
    }
}

// Joins the parts of one query head: block (sequence, head).  Threads take the
// parts in a fixed pattern and are summed in a fixed order.
template <int D, bool BF16, int RU>
__global__ void __launch_bounds__(256) attn_join_kernel(const AttnArgs a, const DecodePlan pl) {
    constexpr int LR = D / 4, NG = 256 / LR;  // lanes of a row, parts taken at a time
    __shared__ float red[8];
    __shared__ __align__(16) float acc[NG][D];
    __shared__ float sums[NG];
    const int tid = threadIdx.x, b = blockIdx.x / a.Hq, head = blockIdx.x % a.Hq;
    const int G = a.Hq / a.Hkv, in = head % G;
    const int u = head / G * pl.per_kv + in / RU, row = in % RU;
    pdl_wait();
    const int *h = reinterpret_cast<const int *>(a.ws);
    const int p0 = h[b], n = h[b + 1] - p0, per = h[a.B + 1];
    if (n == 0) return;
    const long long s0 = (long long)p0 * pl.units + (long long)u * n;
    const int w0 = (int)(s0 / per), parts = (int)((s0 + n - 1) / per) - w0 + 1;
    if (parts == 1) return;  // written by its worker
    const float *ws = reinterpret_cast<const float *>(a.ws + ws_header(a.B));
    auto part_of = [&](int i) { return ws + ((size_t)(w0 + i) * 2 + (i == 0)) * part_floats<D, RU>(); };
    float m = -INFINITY;
    for (int i = tid; i < parts; i += 256) m = fmaxf(m, part_of(i)[RU * D + 2 * row]);
    m = group_max<32>(m);
    if ((tid & 31) == 0) red[tid >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) m = fmaxf(m, red[w]);
    if (m == -INFINITY) m = 0.0f;
    const int g = tid / LR, c = 4 * (tid % LR);
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float sum = 0.0f;
    for (int i = g; i < parts; i += NG) {
        const float *p = part_of(i);
        const float2 ml = *reinterpret_cast<const float2 *>(p + RU * D + 2 * row);
        const float4 v = *reinterpret_cast<const float4 *>(p + row * D + c);
        const float f = ex2(ml.x - m);
        sum = fmaf(ml.y, f, sum);
        o.x = fmaf(v.x, f, o.x), o.y = fmaf(v.y, f, o.y), o.z = fmaf(v.z, f, o.z), o.w = fmaf(v.w, f, o.w);
    }
    *reinterpret_cast<float4 *>(&acc[g][c]) = o;
    if (c == 0) sums[g] = sum;
    __syncthreads();
    if (tid < D) {
        float x = 0.0f, s = 0.0f;
#pragma unroll
        for (int k = 0; k < NG; ++k) x += acc[k][tid], s += sums[k];
        store_io<BF16>(a.o, ((size_t)b * a.Hq + head) * D + tid, x / s);
    }
}

template <int D, bool BF16, int RU>
cudaError_t launch_decode_ru(const AttnArgs &a, cudaStream_t stream) {
    using T = Tile<D, BF16>;
    static std::atomic<uint64_t> ready{0};
    auto kern = attn_decode_kernel<D, BF16, RU>;
    cudaError_t e = allow_smem(kern, ready, kSmemLimit);
    int sms = 0;
    if (e == cudaSuccess) e = device_sms(&sms);
    if (e != cudaSuccess) return e;
    DecodePlan pl;
    const int G = a.Hq / a.Hkv;
    pl.per_kv = (G + RU - 1) / RU;
    pl.units = a.Hkv * pl.per_kv;
    pl.stages = (kSmemLimit - fixed_smem<D, BF16>(a.B)) / (T::kWarps * T::kStageBytes);
    if (pl.stages > kMaxStages) pl.stages = kMaxStages;
    if (pl.stages < 1) return cudaErrorInvalidConfiguration;
    pl.workers = sms * T::kWarps;
    pl.min_tiles = 2;
    CUtensorMap km, vm;
    if (!page_map(&km, a.k_pages, D, a, BF16, T::kTok) || !page_map(&vm, a.v_pages, D, a, BF16, T::kTok))
        return cudaErrorInvalidValue;
    const int smem = fixed_smem<D, BF16>(a.B) + T::kWarps * pl.stages * T::kStageBytes;
    kern<<<sms, T::kWarps * 32, smem, stream>>>(km, vm, a, pl);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)a.B * a.Hq);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_join_kernel<D, BF16, RU>, a, pl);
}

template <int D, bool BF16>
cudaError_t launch_decode_d(const AttnArgs &a, cudaStream_t stream) {
    if constexpr (BF16) {
        if (a.Hq / a.Hkv > 8) return launch_decode_ru<D, true, 16>(a, stream);
    }
    return launch_decode_ru<D, BF16, 8>(a, stream);
}

template <int D, bool BF16>
size_t ws_bytes(int B, int G, int sms) {
    const size_t part = BF16 && G > 8 ? part_floats<D, 16>() : part_floats<D, 8>();
    return ws_header(B) + (size_t)sms * Tile<D, BF16>::kWarps * 2 * part * 4;
}

}  // namespace

size_t attn_decode_workspace_bytes(int B, int Hq, int Hkv, int D, bool bf16, cudaError_t *err) {
    int sms = 0;
    *err = device_sms(&sms);
    if (*err != cudaSuccess) return 0;
    const int G = Hq / Hkv;
    switch (D) {
        case 64: return bf16 ? ws_bytes<64, true>(B, G, sms) : ws_bytes<64, false>(B, G, sms);
        case 128: return bf16 ? ws_bytes<128, true>(B, G, sms) : ws_bytes<128, false>(B, G, sms);
        default: return bf16 ? ws_bytes<256, true>(B, G, sms) : ws_bytes<256, false>(B, G, sms);
    }
}

cudaError_t launch_attn_decode(const AttnArgs &a, int D, bool bf16, cudaStream_t stream) {
    switch (D) {
        case 64: return bf16 ? launch_decode_d<64, true>(a, stream) : launch_decode_d<64, false>(a, stream);
        case 128: return bf16 ? launch_decode_d<128, true>(a, stream) : launch_decode_d<128, false>(a, stream);
        case 256: return bf16 ? launch_decode_d<256, true>(a, stream) : launch_decode_d<256, false>(a, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace lq
