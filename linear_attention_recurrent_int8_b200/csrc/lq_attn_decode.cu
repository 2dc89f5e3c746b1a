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
// Where a key-value head has more query heads than the rows of a warp (16 or
// 8), a run goes to as many warps of neighbouring SMs, which walk it side by
// side, so that the second reads find part of it in the L2 cache (24 heads,
// BF16, 800 MB: 256 -> 203 us at head size 128 against a line with a run for
// each row group).
//
// BF16 (Bf16Core): query heads are the rows of a 16-row warp MMA.  The
// softmax weights enter the product with V as two BF16 parts (p = hi + lo,
// relative error 2^-17), so the output carries one rounding, its own.  With at
// most 8 heads per key-value head the lower 8 rows hold hi, the upper 8 lo,
// of one and the same MMA.  Warp MMAs and not tcgen05: a token of a
// key-value head needs D / 64 of them, a fifth of what the warp path can issue
// while DRAM delivers the token, and accumulators in registers keep the warps
// independent.
//
// FP32 (F32Core): the same with operands split into two TF32 parts, 8 query
// heads at a time.
//
// Measured on B200 (6.55 TB/s copy): BF16, 256 sequences of 15 to 4,095
// tokens, 32 query and 8 key-value heads, head size 128: 320 us, 6.1 TB/s;
// three sequences of 90,000 to 131,071, 16 and 2 heads, head size 256: 114
// us, 6.0 TB/s; one of 700 tokens: 9.3 us, the latency of the two launches.
// The tensor pipe is busy 20 % of the time, 21 % of the issue slots are used.
#include "lq_attn_common.cuh"

namespace lq {
namespace {

template <int D, bool BF16>
struct Tile {
    static constexpr int kTok = BF16 || D == 64 ? 16 : 8;       // tokens of a tile
    // warps of a block (12 over 8 at BF16, head size 64: 73 -> 62 us for 16
    // query heads per key-value head, 64 -> 62 us for 4)
    static constexpr int kWarps = BF16 && D == 64 ? 12 : 8;
    static constexpr int kRowEl = BF16 ? 64 : 32;               // elements of a 128-byte box row
    static constexpr int kBoxes = D / kRowEl;                   // boxes of a tile of K (or V)
    static constexpr int kBoxBytes = kTok * 128;
    static constexpr int kHalfBytes = kBoxes * kBoxBytes;       // K of a tile, then V
    static constexpr int kStageBytes = 2 * kHalfBytes;
    // per-warp scratch: 8 query rows of FP32 (head size 256)
    static constexpr int kScratch = BF16 || D < 256 ? 0 : 8 * (D + 4) * 4;
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
    int units;       // key-value heads of a sequence
    int per_kv;      // row groups of a key-value head, a warp of the team each
    int stages;
    int teams;       // of per_kv warps; a run of the line each
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

// x / y of numbers that mostly fit into 32 bits.
__device__ __forceinline__ long long divide(long long x, int y) {
    return (x >> 32) == 0 ? (long long)((unsigned)x / (unsigned)y) : x / y;
}

// A place on the line of tiles.
struct Cursor {
    int b, u, t, n, len, lo, t0;  // sequence, key-value head, tile, tiles of the pair, visible range, first tile
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
    c.u = (int)divide(r, c.n);
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
                                         unsigned char *, int, int, int) {
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
        const SoftCap cap = soft_cap(a.scale, a.softcap);
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

// The same over tiles of FP32 rows, 8 query rows.  Every FP32 operand enters
// the TF32 MMAs as two parts, x = hi + lo with hi rounded to 11 bits: the upper
// 8 rows of the A operand hold the hi parts and the lower 8 the lo parts of
// the 8 query rows (or of their weights), and B comes once as hi and once as
// lo, so two MMAs give all four products.  A row of scratch (head size 256) is
// D + 4 floats long, which puts the rows on distinct banks.
template <int D>
struct F32Core {
    using T = Tile<D, false>;
    static constexpr int TOK = T::kTok, NT = TOK / 8, NB = T::kBoxes;
    static constexpr bool kKeepQ = D < 256;  // split query rows in registers, else FP32 rows in scratch
    float q[kKeepQ ? NB : 1][2][8];
    float o[NB][4][2], m, l;

    __device__ __forceinline__ static void mma(float (&d)[4], const float *a, float b0, float b1) {
        mma_1688(d, a[0], a[1], a[2], a[3], b0, b1);
    }

    // Channels of a box are dealt to the MMA's K so that a lane reads 16 bytes
    // at a time: lane t holds chunks 2t and 2t + 1 (of 4 channels) of its row.
    __device__ __forceinline__ void begin(const AttnArgs &a, int b, int head0, int rows, int lane, unsigned char *sc) {
        const int g = lane >> 2, t = lane & 3;
        const float *qp = static_cast<const float *>(a.q) + ((size_t)b * a.Hq + head0) * D;
        const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if constexpr (kKeepQ) {
#pragma unroll
            for (int x = 0; x < NB; ++x)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    split_tf32(g < rows ? __ldg(reinterpret_cast<const float4 *>(qp + g * D + 32 * x + 4 * (2 * t + j))) : zero, q[x][j]);
        } else {
            __syncwarp();
            for (int i = lane; i < 8 * (D / 4); i += 32) {
                const int r = i / (D / 4), c = 4 * (i % (D / 4));
                *reinterpret_cast<float4 *>(reinterpret_cast<float *>(sc) + r * (D + 4) + c) =
                    r < rows ? __ldg(reinterpret_cast<const float4 *>(qp + r * D + c)) : zero;
            }
            __syncwarp();
        }
#pragma unroll
        for (int x = 0; x < NB; ++x)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[x][i][0] = o[x][i][1] = 0.0f;
        m = -INFINITY, l = 0.0f;
    }

    __device__ __forceinline__ void tile(const AttnArgs &a, unsigned char *st, int tok0, int lo, int len, int lane,
                                         unsigned char *sc, int b, int head0, int rows) {
        const int g = lane >> 2, t = lane & 3;
        float s[NT][2];  // scores of tokens 8 n + 2 t, 8 n + 2 t + 1 with row g
        {
            // four chains of MMAs per 8 tokens
            float c[NT][4][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) c[n][i][e] = 0.0f;
#pragma unroll
            for (int x = 0; x < NB; ++x)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float qv[8];
                    if constexpr (kKeepQ) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) qv[e] = q[x][j][e];
                    } else {
                        split_tf32(*reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(sc) + g * (D + 4) + 32 * x + 4 * (2 * t + j)), qv);
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float k[8];
                        split_tf32(*reinterpret_cast<const float4 *>(st + x * T::kBoxBytes + (8 * n + g) * 128 + (((2 * t + j) ^ g) << 4)), k);
                        mma(c[n][0], qv, k[0], k[2]);
                        mma(c[n][1], qv, k[1], k[3]);
                        mma(c[n][2], qv + 4, k[4], k[6]);
                        mma(c[n][3], qv + 4, k[5], k[7]);
                    }
                }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    s[n][e] = (c[n][0][e] + c[n][2][e]) + ((c[n][1][e] + c[n][3][e]) + (c[n][0][e + 2] + c[n][2][e + 2]) +
                                                           (c[n][1][e + 2] + c[n][3][e + 2]));
        }
        const bool part = tok0 + TOK > len || tok0 < lo;
        bool seen[NT][2], odd = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int tok = tok0 + 8 * n + 2 * t + e;
                seen[n][e] = !part || (tok >= lo && tok < len);
                odd = odd || (seen[n][e] && s[n][e] != s[n][e]);
            }
        if (__any_sync(0xffffffffu, odd)) {
            // The split turns an infinity into NaN: such scores (and no
            // others, of whatever heads share the warp) are formed again, in
            // FP32.
            const float *qp = static_cast<const float *>(a.q) + ((size_t)b * a.Hq + head0 + g) * D;
#pragma unroll 1
            for (int i = 0; i < 2 * NT && g < rows; ++i) {
                const int r = 8 * (i >> 1) + 2 * t + (i & 1);
                float x = 0.0f;
#pragma unroll 1
                for (int d = 0; d < D; ++d)
                    x = fmaf(__ldg(qp + d), *reinterpret_cast<const float *>(st + (d >> 5) * T::kBoxBytes + r * 128 +
                                                                             ((((d >> 2) & 7) ^ (r & 7)) << 4) + 4 * (d & 3)), x);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (2 * n + e == i && s[n][e] != s[n][e]) s[n][e] = x;
            }
            __syncwarp();
        }
        const SoftCap cap = soft_cap(a.scale, a.softcap);
        float mx = -INFINITY;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                s[n][e] = a.softcap > 0.0f ? capped_log2<false>(s[n][e], cap) : s[n][e] * (a.scale * kLog2e);
                if (!seen[n][e]) s[n][e] = -INFINITY;
                mx = fmaxf(mx, s[n][e]);
            }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        if (__any_sync(0xffffffffu, mx > m)) {
            const float n = fmaxf(m, mx), f = n == -INFINITY ? 1.0f : ex2(m - n);
            m = n;
            l *= f;
#pragma unroll
            for (int x = 0; x < NB; ++x)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[x][i][0] *= f, o[x][i][1] *= f;
        }
        const float base = m == -INFINITY ? 0.0f : m;
        float p[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float p0 = ex2(s[n][0] - base), p1 = ex2(s[n][1] - base);
            l += p0 + p1;
            split_tf32(p0, p[n][0], p[n][1]);
            split_tf32(p1, p[n][2], p[n][3]);
        }
        if (part) {
            // rows of V that are not visible may hold NaN: weight 0 would not silence them
            for (int r = 0; r < TOK; ++r) {
                if (tok0 + r >= lo && tok0 + r < len) continue;
                for (int ch = lane; ch < D / 4; ch += 32)
                    *reinterpret_cast<uint4 *>(st + T::kHalfBytes + (ch >> 3) * T::kBoxBytes + r * 128 + (ch & 7) * 16) =
                        make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();  // before the stage's next TMA write
            __syncwarp();
        }
        // lane (g, t) reads chunk g of the rows of its two tokens: channel
        // 4 g + i of a box is column g of the box's MMA i
#pragma unroll
        for (int x = 0; x < NB; ++x) {
            float c[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) c[i][e] = 0.0f;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const unsigned char *vp = st + T::kHalfBytes + x * T::kBoxBytes + (8 * n + 2 * t) * 128;
                float v0[8], v1[8];
                split_tf32(*reinterpret_cast<const float4 *>(vp + ((g ^ (2 * t)) << 4)), v0);
                split_tf32(*reinterpret_cast<const float4 *>(vp + 128 + ((g ^ (2 * t + 1)) << 4)), v1);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    mma(c[i], p[n], v0[2 * i], v1[2 * i]);
                    mma(c[i], p[n], v0[2 * i + 1], v1[2 * i + 1]);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) o[x][i][0] += c[i][0] + c[i][2], o[x][i][1] += c[i][1] + c[i][3];
        }
    }

    __device__ __forceinline__ void end(const AttnArgs &a, int b, int head0, int rows, float *part, int lane,
                                        unsigned char *) {
        const int g = lane >> 2, t = lane & 3;
        float sum = l;
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        if (g >= rows) return;
        const float f = part ? 1.0f : 1.0f / sum;
        float *dst = part ? part + g * D : static_cast<float *>(a.o) + ((size_t)b * a.Hq + head0 + g) * D;
#pragma unroll
        for (int x = 0; x < NB; ++x)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                *reinterpret_cast<float4 *>(dst + 32 * x + 8 * t + 4 * e) =
                    make_float4(o[x][0][e] * f, o[x][1][e] * f, o[x][2][e] * f, o[x][3][e] * f);
        if (part && t == 0) *reinterpret_cast<float2 *>(part + 8 * D + 2 * g) = make_float2(m, sum);
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
    if (tid == 0) prefetch_map(&kmap), prefetch_map(&vmap);
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
    long long per = divide(total + pl.teams - 1, pl.teams);
    if (per < pl.min_tiles) per = pl.min_tiles;
    if (blockIdx.x == 0) {
        int *h = reinterpret_cast<int *>(a.ws);
        for (int b = tid; b <= a.B; b += NW * 32) h[b] = prefix[b];
        if (tid == 0) h[a.B + 1] = (int)per;
    }
    // runs go to the SMs in turn, so that a short line spreads over all of them
    const int worker = warp * gridDim.x + blockIdx.x, team = pl.per_kv == 1 ? worker : worker / pl.per_kv;
    const int group = worker - team * pl.per_kv;
    const long long x0 = (long long)team * per;
    if (x0 >= total || team >= pl.teams) return;
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
    // (of the first tiles all at once, lane i of the run's i-th)
    Cursor ahead = pc;
    for (int i = 0; i < lane && i < pl.stages && i < run; ++i) advance<TOK>(ahead, len, a.B, pl.units, a.window);
    const int first_pages = page_of(ahead);
    int page = 0, fill = 0, filled = 0;
    // The whole warp prepares a tile's copies from values that the compiler
    // knows to be uniform (shuffled from lane 0) and one lane issues them;
    // prepared inside that lane's branch they took about 900 cycles a tile.
    const uint32_t ring_addr = __shfl_sync(0xffffffffu, smem_u32(my_ring), 0), full_addr = __shfl_sync(0xffffffffu, smem_u32(full), 0);
    auto issue = [&]() {
        const bool bad = page < 0 || page >= a.num_pages;
        const int z = __shfl_sync(0xffffffffu, bad ? -1 : page * a.Hkv + pc.u, 0);
        const int row = __shfl_sync(0xffffffffu, ((pc.t0 + pc.t) * TOK) & (a.page_size - 1), 0);
        const uint32_t dst = ring_addr + fill * T::kStageBytes, bar = full_addr + fill * 8;
        if (elect_one()) {
            if (z < 0) atomicOr(&g_dev_error, kErrBadPage);
            expect_bytes(bar, T::kStageBytes);
#pragma unroll
            for (int x = 0; x < T::kBoxes; ++x) {
                tma_page_load_at(dst + x * T::kBoxBytes, &kmap, x * T::kRowEl, row, z, bar);
                tma_page_load_at(dst + T::kHalfBytes + x * T::kBoxBytes, &vmap, x * T::kRowEl, row, z, bar);
            }
        }
        __syncwarp();
        if (++fill == pl.stages) fill = 0;
        if (++filled < run) advance<TOK>(pc, len, a.B, pl.units, a.window);
    };

    typename CoreOf<D, BF16, RU>::type core;
    int st = 0, ph = 0;
    bool fresh = false, whole = false;  // whole: the run holds the pair's first tile
    int head0 = 0, rows = 0;
    auto begin = [&]() {
        head0 = c.u * G + group * RU;
        rows = min(RU, G - group * RU);
        core.begin(a, c.b, head0, rows, lane, sc);
        whole = c.t == 0;
        fresh = false;
    };
    while (filled < run && filled < pl.stages) {
        page = __shfl_sync(0xffffffffu, first_pages, filled);
        issue();
    }
    if (filled < run) page = page_of(pc);
    begin();
    for (int i = 0; i < run; ++i) {
        if (fresh) begin();
        if (!warp_wait(full + st, ph)) {
            // give the copies in flight (this one again) their time before the
            // block's shared memory is freed
            for (int k = i; k < filled; ++k) {
                bar_wait(full + st, ph);
                if (++st == pl.stages) st = 0, ph ^= 1;
            }
            return;
        }
        unsigned char *stage = my_ring + st * T::kStageBytes;
        core.tile(a, stage, (c.t0 + c.t) * TOK, c.lo, c.len, lane, sc, c.b, head0, rows);
        __syncwarp();
        if (filled < run) {
            issue();
            if (filled < run) page = page_of(pc);
        }
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

// The parts of one query head's output.
struct JoinJob {
    int b, head, group, row, first, parts;  // sequence, head, its row group and row in it, first team, number of parts
};

template <int RU>
__device__ __forceinline__ JoinJob join_job(const AttnArgs &a, const DecodePlan &pl, long long job) {
    JoinJob j{};
    if (job >= (long long)a.B * a.Hq) return j;
    j.b = (int)(job / a.Hq), j.head = (int)(job - (long long)j.b * a.Hq);
    const int *h = reinterpret_cast<const int *>(a.ws);
    const int p0 = h[j.b], n = h[j.b + 1] - p0, per = h[a.B + 1];
    if (n == 0) return j;
    const int G = a.Hq / a.Hkv, kv = j.head / G, in = j.head - kv * G;
    j.row = in % RU;
    j.group = in / RU;
    const long long s0 = (long long)p0 * pl.units + (long long)kv * n;
    j.first = (int)(s0 / per);
    j.parts = (int)((s0 + n - 1) / per) - j.first + 1;
    return j;
}

template <int D, int RU>
__device__ __forceinline__ const float *join_part(const AttnArgs &a, const DecodePlan &pl, const JoinJob &j, int i) {
    // the first part is in its worker's second slot, the others in their worker's first
    return reinterpret_cast<const float *>(a.ws + ws_header(a.B)) + (((size_t)(j.first + i) * pl.per_kv + j.group) * 2 + (i == 0)) * part_floats<D, RU>();
}

// Joins the parts of the query heads, each sum in a fixed order.  A block takes
// JB heads: with 8, each warp joins the few parts of a head by itself, and the
// block comes together for heads of many; with 1 the block joins 64 channels
// of one head (a few long sequences leave hundreds of parts per head).  A head
// whose pair lay in one run was written by its worker.
template <int D, bool BF16, int RU, int JB>
__global__ void __launch_bounds__(256) attn_join_kernel(const AttnArgs a, const DecodePlan pl) {
    constexpr int NC = JB == 1 ? 64 : D, LR = NC / 4, NG = 256 / LR;  // channels of the block, their lanes, parts taken at a time
    constexpr int kFew = JB == 1 ? 1 : 16;    // parts up to which a warp works alone
    constexpr int NV = D / 32;                // channels of a lane of a lone warp
    __shared__ float red[8];
    __shared__ __align__(16) float acc[NG][NC];
    __shared__ float sums[NG];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_wait();
    const JoinJob mine = join_job<RU>(a, pl, JB == 1 ? blockIdx.x / (D / NC) : (long long)blockIdx.x * JB + warp);
    const int c0 = JB == 1 ? blockIdx.x % (D / NC) * NC : 0;
    if (JB > 1 && mine.parts > 1 && mine.parts <= kFew) {
        const int x = lane < mine.parts ? lane : 0;
        const float2 ml = *reinterpret_cast<const float2 *>(join_part<D, RU>(a, pl, mine, x) + RU * D + 2 * mine.row);
        float m = group_max<32>(ml.x);
        if (m == -INFINITY) m = 0.0f;
        const float f = lane < mine.parts ? ex2(ml.x - m) : 0.0f;
        float sum = 0.0f, o[NV];
#pragma unroll
        for (int e = 0; e < NV; ++e) o[e] = 0.0f;
#pragma unroll 4
        for (int i = 0; i < mine.parts; ++i) {
            const float w = __shfl_sync(0xffffffffu, f, i), l = __shfl_sync(0xffffffffu, ml.y, i);
            const float *p = join_part<D, RU>(a, pl, mine, i) + mine.row * D + NV * lane;
            sum = fmaf(l, w, sum);
#pragma unroll
            for (int e = 0; e < NV; e += 2) {
                const float2 v = *reinterpret_cast<const float2 *>(p + e);
                o[e] = fmaf(v.x, w, o[e]), o[e + 1] = fmaf(v.y, w, o[e + 1]);
            }
        }
        const size_t at = ((size_t)mine.b * a.Hq + mine.head) * D + NV * lane;
#pragma unroll
        for (int e = 0; e < NV; ++e) store_io<BF16>(a.o, at + e, o[e] / sum);
    }
    unsigned many = 1;
    if (JB > 1) {
        // which heads the block joins together
        if (lane == 0) red[warp] = mine.parts > kFew ? 1.0f : 0.0f;
        if (!__syncthreads_or(mine.parts > kFew)) return;
        many = 0;
        for (int w = 0; w < 8; ++w) many |= (red[w] != 0.0f ? 1u : 0u) << w;
        __syncthreads();
    } else if (mine.parts <= 1) {
        return;
    }
    for (; many; many &= many - 1) {
        const JoinJob j = JB == 1 ? mine : join_job<RU>(a, pl, (long long)blockIdx.x * JB + __ffs(many) - 1);
        float m = -INFINITY;
        for (int i = tid; i < j.parts; i += 256) m = fmaxf(m, join_part<D, RU>(a, pl, j, i)[RU * D + 2 * j.row]);
        m = group_max<32>(m);
        if (lane == 0) red[warp] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < 8; ++w) m = fmaxf(m, red[w]);
        if (m == -INFINITY) m = 0.0f;
        const int g = tid / LR, c = 4 * (tid % LR);
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float sum = 0.0f;
#pragma unroll 4
        for (int i = g; i < j.parts; i += NG) {
            const float *p = join_part<D, RU>(a, pl, j, i);
            const float2 ml = *reinterpret_cast<const float2 *>(p + RU * D + 2 * j.row);
            const float4 v = *reinterpret_cast<const float4 *>(p + j.row * D + c0 + c);
            const float f = ex2(ml.x - m);
            sum = fmaf(ml.y, f, sum);
            o.x = fmaf(v.x, f, o.x), o.y = fmaf(v.y, f, o.y), o.z = fmaf(v.z, f, o.z), o.w = fmaf(v.w, f, o.w);
        }
        *reinterpret_cast<float4 *>(&acc[g][c]) = o;
        if (c == 0) sums[g] = sum;
        __syncthreads();
        if (tid < NC) {
            float x = 0.0f, s = 0.0f;
#pragma unroll
            for (int k = 0; k < NG; ++k) x += acc[k][tid], s += sums[k];
            store_io<BF16>(a.o, ((size_t)j.b * a.Hq + j.head) * D + c0 + tid, x / s);
        }
        __syncthreads();
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
    pl.units = a.Hkv;
    pl.stages = (kSmemLimit - fixed_smem<D, BF16>(a.B)) / (T::kWarps * T::kStageBytes);
    if (pl.stages > kMaxStages) pl.stages = kMaxStages;
    if (pl.stages < 1) return cudaErrorInvalidConfiguration;
    pl.teams = sms * T::kWarps / pl.per_kv;
    if (pl.teams < 1) return cudaErrorInvalidConfiguration;
    pl.min_tiles = 2;
    CUtensorMap km, vm;
    if (!page_map(&km, a.k_pages, D, a, BF16, T::kTok) || !page_map(&vm, a.v_pages, D, a, BF16, T::kTok))
        return cudaErrorInvalidValue;
    const int smem = fixed_smem<D, BF16>(a.B) + T::kWarps * pl.stages * T::kStageBytes;
    kern<<<sms, T::kWarps * 32, smem, stream>>>(km, vm, a, pl);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    // a block per head while they fill the GPU about once, else one for 8
    const int jobs = a.B * a.Hq;
    const bool few = jobs <= sms * T::kWarps;
    cfg.gridDim = dim3((unsigned)(few ? jobs * (D / 64) : (jobs + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (few) return cudaLaunchKernelEx(&cfg, attn_join_kernel<D, BF16, RU, 1>, a, pl);
    return cudaLaunchKernelEx(&cfg, attn_join_kernel<D, BF16, RU, 8>, a, pl);
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
