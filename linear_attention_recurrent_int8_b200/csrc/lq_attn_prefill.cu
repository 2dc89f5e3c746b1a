// lq_attn_prefill.cu -- attention of runs of new tokens over the paged
// key-value cache (lq_attn_prefill), causal from each token's own position.
//
//   o_t = sum_j p_j v_j / sum_j p_j,   p_j = 2^(x_j - m),
//   x_j = log2(e) cap(scale q_t . k_j),  max(0, P_t + 1 - window) <= j <= P_t,
//
// 4 D operations per query head and visible key; a tile of 256 rows uses each
// key and value 256 times, so the products and the exponentials bound it.
//
// attn_prefill_tc (BF16) runs on tcgen05 with scores, weights and outputs in
// TMEM; attn_prefill_f32 on warp MMAs with TF32 operands in two parts.  Both
// pack the query heads that share a key-value head into the rows of a tile
// (head fastest), so that a tile spans few tokens: its causal edge is short
// and its keys are read once for all of its heads.
//
// Measured on B200 (cuBLAS BF16 burst 1,645 TFLOP/s): 2 x 4,096 tokens behind
// 4,096, 32 query and 8 key-value heads, BF16: 681 us at head size 128 (1,210
// TFLOP/s; tensor pipe 59 %, special function unit 52 %: neither waits for
// the other but for the hand-over of scores and weights), 502 us at 64 (the
// exponentials: one per 256 operations); 16 and 2 heads at 256: 714 us (1,155
// TFLOP/s, tensor pipe 55 %).  FP32, 2 x 2,048 behind 2,048, 16 and 4 heads:
// 2.06 ms at head size 128, 50 TFLOP/s, half of what three warp MMAs per
// product allow.
//
// Weights enter the BF16 product with V rounded to BF16, the tensor cores'
// operand type (2^-8 relative at most; their sum is of the unrounded ones):
// outputs are 2.3e-3 off the 64-bit ones, against 1.7e-3 for weights in FP32,
// which is the output's own rounding.
#include <algorithm>

#include "lq_attn_common.cuh"
#include "lq_tc.cuh"

namespace lq {
namespace {

// What a block works on: the heads of a tile one after the other.
struct BlockPlace {
    long long turn, tiles;
    int head;  // first of the block's heads
};
__device__ __forceinline__ BlockPlace place_of(const AttnArgs &a, int group_shift, int split) {
    const unsigned block = blockIdx.x / (unsigned)split, groups = (unsigned)a.Hq >> group_shift;
    const unsigned tiles = gridDim.x / ((unsigned)split * groups), t = block / groups;
    return BlockPlace{t, tiles, (int)((block - t * groups) << group_shift)};
}

// Few rows behind long contexts: the key tiles of a query tile are dealt out
// to the `split` blocks of a cluster.  Each leaves its rows' unnormalised
// outputs, maximum (in units of log2) and sum in its shared memory, rows
// D + 4 floats apart at `part`, and every block joins the rows whose number is
// its rank modulo the split, in the order of the ranks.
__device__ __forceinline__ void my_keys(int &k_first, int &n, int split, uint32_t rank) {
    const int first = (int)((long long)n * rank / split);
    n = (int)((long long)n * (rank + 1) / split) - first;
    k_first += first;
}

constexpr int kMaxSplit = 8;

template <int D, bool BF16>
__device__ __forceinline__ void join_split(uint32_t part, int rows, int group_shift, int split, uint32_t rank,
                                           const AttnArgs &a, const QueryTile &qt, int h0) {
    cluster_sync();
    constexpr int CH = D / 4;
    for (int i = threadIdx.x; i < (rows + split - 1) / split * CH; i += blockDim.x) {
        const int R = i / CH * split + (int)rank, ch = i % CH;
        if (R >= rows) continue;
        const uint32_t row = part + R * (D + 4) * 4;
        float2 ml[kMaxSplit];
        float4 o[kMaxSplit];
#pragma unroll
        for (int k = 0; k < kMaxSplit; ++k) {
            if (k >= split) break;
            const uint32_t at = peer_addr(row, k);
            ml[k] = peer_load2(at + D * 4);
            o[k] = peer_load4(at + ch * 16);
        }
        float top = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int k = 0; k < kMaxSplit; ++k)
            if (k < split) top = fmaxf(top, ml[k].x);
        if (top == -INFINITY) top = 0.0f;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < kMaxSplit; ++k) {
            if (k >= split) break;
            const float f = ex2(ml[k].x - top);
            sum = fmaf(ml[k].y, f, sum);
            v.x = fmaf(o[k].x, f, v.x), v.y = fmaf(o[k].y, f, v.y), v.z = fmaf(o[k].z, f, v.z), v.w = fmaf(o[k].w, f, v.w);
        }
        const float inv = 1.0f / sum;
        const size_t dst = ((size_t)(qt.base + qt.first + (R >> group_shift)) * a.Hq + h0 + (R & ((1 << group_shift) - 1))) * D + 4 * ch;
        if constexpr (BF16) {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x * inv, v.y * inv), hi = __floats2bfloat162_rn(v.z * inv, v.w * inv);
            *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.o) + dst) =
                make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
        } else {
            *reinterpret_cast<float4 *>(static_cast<float *>(a.o) + dst) = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
        }
    }
    cluster_sync();  // until then the peers read this block's shared memory
}

// Blocks of a cluster for a grid of `blocks` that leaves SMs idle (`slots`
// blocks fit at once), with at least a tile of 128 keys each if the contexts
// filled their block tables; tiles that turn out to have no more than
// kSplitMin keys are left to one of the blocks.  Clusters of 8 do not reach
// all SMs of a processing cluster, hence the eighth that is kept back.
// 16 new tokens behind 2,000, 20,000 and 100,000, 32 query and 8 key-value
// heads at head size 128, BF16: 33, 259 and 1261 us without, 13, 44 and 170
// us with clusters.
int split_of(const AttnArgs &a, long long blocks, int rows, long long slots) {
    long long reach = (long long)a.max_pages << a.page_shift;
    if (a.window > 0) reach = std::min(reach, (long long)a.window + rows);
    slots -= slots / 8;
    int split = 1;
    while (split < kMaxSplit && 2 * split * blocks <= slots && 2 * split * 128 <= reach) split *= 2;
    return split;
}

// Launch as clusters of `split` blocks.
template <typename... P, typename... A>
cudaError_t launch_split(void (*kern)(P...), long long blocks, int split, int threads, int smem, cudaStream_t stream, const A &...args) {
    if (blocks * split > 0x7fffffffLL) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(blocks * split));
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)split, attr.val.clusterDim.y = 1, attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = split > 1;
    return cudaLaunchKernelEx(&cfg, kern, P(args)...);
}

// ---------------------------------------------------------------------------
// FP32: warp MMAs on operands in two TF32 parts
// ---------------------------------------------------------------------------

template <int D, int KG>
struct F32 {
    static constexpr int kThreads = 128;
    static constexpr int kRowGroups = 4 / KG, kRows = 16 * kRowGroups;  // of 16 rows
    static constexpr int kKeys = D == 64 ? 32 : 16;         // keys of a tile
    static constexpr int kBoxes = D / 32;                   // 128-byte column blocks
    static constexpr int kBoxBytes = kKeys * 128;
    static constexpr int kHalfBytes = kBoxes * kBoxBytes;   // K of a tile, then V
    static constexpr int kLd = D + 4;                       // row stride of Q: rows on distinct banks
    static constexpr int kBufs = D < 256 && KG == 2 ? 2 : 1;         // tiles of K, and of V, that a key group holds
    static constexpr int kSmem = 1024 + 2 * KG * kBufs * kHalfBytes + kRows * kLd * 4;
    static constexpr int kBlocks = D == 64 ? 3 : D == 256 && KG == 4 ? 1 : 2;  // on an SM
    static constexpr int kSplitMin = 128;  // keys up to which a tile is not split (208: 17 -> 12 us at head size 128)
};

// One block: 16 or 32 rows, each a (token, head) pair of heads that share a
// key-value head (head fastest).  A warp takes 16 rows and every KG-th tile of
// keys, and the KG parts of a row's keys are joined at the end.  The warps of
// a key group share two buffers of K and V, or one, of which K's part is
// filled again while the weights meet V and V's part while the queries meet
// K: that leaves room for a second block on the SM (head size 256, 2 x 2048
// tokens on a prefix: 6.6 -> 4.9 ms).  Products of two-part operands:
// hi hi + hi lo + lo hi, 3 MMAs.
template <int D, int KG>
__global__ void __launch_bounds__(F32<D, KG>::kThreads, F32<D, KG>::kBlocks)
    attn_prefill_f32(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                     const AttnArgs a, const int group_shift, const int cluster) {
    using T = F32<D, KG>;
    constexpr int RG = T::kRowGroups, KT = T::kKeys, NB = T::kBoxes, NT = KT / 8, LD = T::kLd, NBUF = T::kBufs;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    float *qs = reinterpret_cast<float *>(ring + 2 * KG * NBUF * T::kHalfBytes);
    __shared__ uint64_t full[KG][2][2], empty[KG][2][2];  // [key group][K (and V with two buffers), V][buffer]
    __shared__ int find[T::kThreads / 32 + 6];
    __shared__ int sent[KG][2];  // tiles whose copies were issued, by the barrier they arrive at
    const BlockPlace at = place_of(a, group_shift, cluster);
    const QueryTile qt = find_query_tile<T::kThreads, (T::kBlocks > 1)>(a, T::kRows >> group_shift, at.turn, at.tiles, find);
    if (qt.rows <= 0) return;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int rg = warp % RG, kg = warp / RG;
    const int heads = 1 << group_shift, h0 = at.head, kv = h0 / (a.Hq / a.Hkv);
    const int p0 = qt.start + qt.first, len = p0 + qt.rows;  // keys any row sees: lo .. len - 1
    const int lo = a.window > 0 && p0 + 1 > a.window ? p0 + 1 - a.window : 0;
    int k_first = lo / KT, n = (len - 1) / KT - k_first + 1;
    __shared__ int split_of_tile;  // (not a register of the loop below)
    {
        const int split = n * KT > T::kSplitMin ? cluster : 1;
        const uint32_t rank = cluster > 1 ? cluster_rank() : 0;
        if (rank >= (uint32_t)split) return;
        if (split > 1) my_keys(k_first, n, split, rank);
        if (tid == 0) split_of_tile = split;
    }
    if (tid < 4 * KG) mbar_init(&full[0][0][0] + tid, 1), mbar_init(&empty[0][0][0] + tid, RG);
    __syncthreads();
    // One lane of a key group fills its buffers for the group's i-th tile: K
    // (v = 0) or V (1) where the group has one buffer of each, else both.
    auto issue = [&](int i, int v) {
        const int k0 = (k_first + KG * i + kg) * KT;
        uint64_t *bar = &full[kg][v][i % NBUF];
        unsigned char *kdst = ring + (2 * kg * NBUF + i % NBUF) * T::kHalfBytes, *vdst = kdst + NBUF * T::kHalfBytes;
        sent[kg][v] = i + 1;
        mbar_arrive_expect_tx(bar, NBUF > 1 ? 2 * T::kHalfBytes : T::kHalfBytes);
        for (int r = 0; r < KT; r += 16) {
            const int tok = k0 + r;
            int z = -1;  // rows past the visible keys are filled with zeros
            if (tok < len && tok + 16 > lo) {
                const int page = __ldg(a.block_table + (size_t)qt.b * a.max_pages + (tok >> a.page_shift));
                if (page >= 0 && page < a.num_pages) z = page * a.Hkv + kv;
                else atomicOr(&g_dev_error, kErrBadPage);
            }
            for (int x = 0; x < NB; ++x) {
                const int off = x * T::kBoxBytes + r * 128;
                if (NBUF > 1 || v == 0) tma_page_load(kdst + off, &kmap, 32 * x, tok & (a.page_size - 1), z, bar);
                if (NBUF > 1 || v == 1) tma_page_load(vdst + off, &vmap, 32 * x, tok & (a.page_size - 1), z, bar);
            }
        }
    };
    const int mine = kg < n ? (n - kg + KG - 1) / KG : 0;  // tiles of the group
    const bool producer = rg == 0 && lane == 0;
    for (int i = 0; producer && i < NBUF && i < mine; ++i) {
        issue(i, 0);
        if (NBUF == 1) issue(i, 1);
    }
    for (int i = tid; i < T::kRows * (D / 4); i += T::kThreads) {
        const int r = i / (D / 4), c = 4 * (i % (D / 4)), tok = r >> group_shift;
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (tok < qt.rows)
            x = *reinterpret_cast<const float4 *>(static_cast<const float *>(a.q) +
                                                  ((size_t)(qt.base + qt.first + tok) * a.Hq + h0 + (r & (heads - 1))) * D + c);
        *reinterpret_cast<float4 *>(qs + r * LD + c) = x;
    }
    __syncthreads();

    const SoftCap cap = soft_cap(a.scale, a.softcap);
    int pos[2];  // of rows g and g + 8 (rows past the last token see what it sees, no further keys)
    for (int r = 0; r < 2; ++r) pos[r] = min(p0 + ((16 * rg + g + 8 * r) >> group_shift), len - 1);
    const int pw0 = min(p0 + ((16 * rg) >> group_shift), len - 1), pw1 = min(p0 + ((16 * rg + 15) >> group_shift), len - 1);
    const float *qr = qs + (16 * rg + g) * LD;
    float o[NB][4][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
    for (int x = 0; x < NB; ++x)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[x][i][e] = 0.0f;
    bool ok = true;
    int it = 0;
    for (; it < mine; ++it) {
        const int k0 = (k_first + KG * it + kg) * KT;
        const int buf = it % NBUF, phase = it / NBUF & 1;
        const unsigned char *kbuf = ring + (2 * kg * NBUF + buf) * T::kHalfBytes;
        unsigned char *vbuf = ring + ((2 * kg + 1) * NBUF + buf) * T::kHalfBytes;
        // into the last tile's buffer, once both warps have left it
        if (it > 0 && it - 1 + NBUF < mine && producer) {
            const int last = (it - 1) % NBUF, left = (it - 1) / NBUF & 1;
            ok = bar_wait(&empty[kg][1][last], left);
            if (ok) issue(it - 1 + NBUF, NBUF == 1);
        }
        __syncwarp();
        ok = __all_sync(0xffffffffu, ok && bar_wait(&full[kg][0][buf], phase));
        if (!ok) break;
        // rows g, g (tokens 2t, 2t + 1), g + 8, g + 8; the large products of
        // the two K steps and the small ones are summed apart
        float s[NT][4], s1[NT][4], s2[NT][4];
#pragma unroll
        for (int k = 0; k < NT; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[k][e] = s1[k][e] = s2[k][e] = 0.0f;
        // a lane reads 16 bytes of channels at a time: lane t takes chunks 2t
        // and 2t + 1 of a box as two K steps
#pragma unroll
        for (int x = 0; x < NB; ++x)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float qa[8], qb[8];
                split_tf32(*reinterpret_cast<const float4 *>(qr + 32 * x + 4 * (2 * t + j)), qa);
                split_tf32(*reinterpret_cast<const float4 *>(qr + 8 * LD + 32 * x + 4 * (2 * t + j)), qb);
#pragma unroll
                for (int k = 0; k < NT; ++k) {
                    float kk[8];
                    split_tf32(*reinterpret_cast<const float4 *>(kbuf + x * T::kBoxBytes + (8 * k + g) * 128 + (((2 * t + j) ^ g) << 4)), kk);
#pragma unroll
                    for (int h = 0; h < 8; h += 4) {
                        mma_1688(h ? s1[k] : s[k], qa[h], qb[h], qa[h + 2], qb[h + 2], kk[h], kk[h + 2]);
                        mma_1688(s2[k], qa[h + 1], qb[h + 1], qa[h + 3], qb[h + 3], kk[h], kk[h + 2]);
                        mma_1688(s2[k], qa[h], qb[h], qa[h + 2], qb[h + 2], kk[h + 1], kk[h + 3]);
                    }
                }
            }
#pragma unroll
        for (int k = 0; k < NT; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[k][e] += s1[k][e] + s2[k][e];
        const bool masked = k0 + KT - 1 > pw0 || (a.window > 0 && k0 <= pw1 - a.window);
        auto seen = [&](int r, int k, int e) {
            const int tok = k0 + 8 * k + 2 * t + e;
            return !masked || (tok <= pos[r] && (a.window == 0 || tok > pos[r] - a.window));
        };
        bool odd = false;
#pragma unroll
        for (int k = 0; k < NT; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) odd = odd || (s[k][e] != s[k][e] && seen(e >> 1, k, e & 1));
        if (__any_sync(0xffffffffu, odd)) {
            // The split turns an infinity into NaN: such scores (and no
            // others, of whatever rows share the warp) are formed again, in FP32.
#pragma unroll 1
            for (int i = 0; i < 4 * NT; ++i) {
                const int tok = 8 * (i >> 2) + 2 * t + (i & 1);
                float v = 0.0f;
#pragma unroll 1
                for (int d = 0; d < D; ++d)
                    v = fmaf(qr[(i & 2) * 4 * LD + d], *reinterpret_cast<const float *>(kbuf + (d >> 5) * T::kBoxBytes + tok * 128 +
                                                                                     ((((d >> 2) & 7) ^ (tok & 7)) << 4) + 4 * (d & 3)), v);
#pragma unroll
                for (int k = 0; k < NT; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (4 * k + e == i && s[k][e] != s[k][e]) s[k][e] = v;
            }
        }
        if constexpr (NBUF == 1) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[kg][0][0]);
            // the next K at once
            if (it + 1 < mine && producer) {
                ok = bar_wait(&empty[kg][0][0], phase);
                if (ok) issue(it + 1, 0);
            }
            __syncwarp();
        }
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int k = 0; k < NT; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[k][e] = a.softcap > 0.0f ? capped_log2<false>(s[k][e], cap) : s[k][e] * (a.scale * kLog2e);
                if (!seen(e >> 1, k, e & 1)) s[k][e] = -INFINITY;
                mx[e >> 1] = fmaxf(mx[e >> 1], s[k][e]);
            }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
            mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
        }
        if (__any_sync(0xffffffffu, mx[0] > m[0] || mx[1] > m[1])) {
            float f[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float x = fmaxf(m[r], mx[r]);
                f[r] = x == -INFINITY ? 1.0f : ex2(m[r] - x);
                m[r] = x;
                l[r] *= f[r];
            }
#pragma unroll
            for (int x = 0; x < NB; ++x)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[x][i][e] *= f[e >> 1];
        }
        float w[NT][8];  // (hi, lo) of the four weights
#pragma unroll
        for (int k = 0; k < NT; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float v = ex2(s[k][e] - (m[e >> 1] == -INFINITY ? 0.0f : m[e >> 1]));
                l[e >> 1] += v;
                split_tf32(v, w[k][2 * e], w[k][2 * e + 1]);
            }
        if constexpr (NBUF == 1) {
            ok = __all_sync(0xffffffffu, ok && bar_wait(&full[kg][1][0], phase));
            if (!ok) break;
        }
        if (k0 < lo || k0 + KT > len) {
            // rows of V that no row sees may hold NaN: weight 0 would not
            // silence them (either warp of the tile clears them all)
            for (int r = 0; r < KT; ++r) {
                if (k0 + r >= lo && k0 + r < len) continue;
                for (int ch = lane; ch < D / 4; ch += 32)
                    *reinterpret_cast<uint4 *>(vbuf + (ch >> 3) * T::kBoxBytes + r * 128 + (ch & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();  // before the buffer's next TMA write
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
            for (int k = 0; k < NT; ++k) {
                const unsigned char *vp = vbuf + x * T::kBoxBytes + (8 * k + 2 * t) * 128;
                float v0[8], v1[8];
                split_tf32(*reinterpret_cast<const float4 *>(vp + ((g ^ (2 * t)) << 4)), v0);
                split_tf32(*reinterpret_cast<const float4 *>(vp + 128 + ((g ^ (2 * t + 1)) << 4)), v1);
#pragma unroll
                for (int i = 0; i < 4; ++i) mma_1688(c[i], w[k][0], w[k][4], w[k][2], w[k][6], v0[2 * i], v1[2 * i]);
#pragma unroll
                for (int i = 0; i < 4; ++i) mma_1688(c[i], w[k][1], w[k][5], w[k][3], w[k][7], v0[2 * i], v1[2 * i]);
#pragma unroll
                for (int i = 0; i < 4; ++i) mma_1688(c[i], w[k][0], w[k][4], w[k][2], w[k][6], v0[2 * i + 1], v1[2 * i + 1]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[x][i][e] += c[i][e];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[kg][1][buf]);
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    }
    // out of time: copies still in flight get theirs before the ring takes the parts
    for (int v = 0; !ok && producer && v < (NBUF > 1 ? 1 : 2); ++v)
        for (int i = it; i < sent[kg][v]; ++i) bar_wait(&full[kg][v][i % NBUF], i / NBUF & 1);
    // Join the groups' parts of the keys, which groups 1 and up hand over
    // through shared memory.  With one of the waits out of time the block's
    // rows are not valid: they are left out or, in a split call, NaN.
    ok = __syncthreads_and(ok);
    const int split = split_of_tile;
    constexpr int JLD = D + 2;
    float *jo = reinterpret_cast<float *>(ring) + rg * 16 * JLD;
    if (kg > 0) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float *row = jo + (kg - 1) * T::kRows * JLD + (g + 8 * r) * JLD;
#pragma unroll
            for (int x = 0; x < NB; ++x)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e) row[32 * x + 8 * t + 4 * e + i] = o[x][i][2 * r + e];
            if (t == 0) row[D] = m[r], row[D + 1] = l[r];
        }
    }
    __syncthreads();
    if (kg == 0) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int R = 16 * rg + g + 8 * r, tok = R >> group_shift;
            if (tok >= qt.rows) continue;
            const float *row = jo + (g + 8 * r) * JLD;
            float top = m[r], f[KG];
#pragma unroll
            for (int k = 1; k < KG; ++k) top = fmaxf(top, row[(k - 1) * T::kRows * JLD + D]);
            const float base = top == -INFINITY ? 0.0f : top;
            f[0] = ex2(m[r] - base);
            float sum = l[r] * f[0];
#pragma unroll
            for (int k = 1; k < KG; ++k) {
                f[k] = ex2(row[(k - 1) * T::kRows * JLD + D] - base);
                sum += row[(k - 1) * T::kRows * JLD + D + 1] * f[k];
            }
            // the row's output or, in a split call, its part
            const float inv = split > 1 ? 1.0f : 1.0f / sum;
            float *dst = split > 1 ? qs + R * LD
                                   : static_cast<float *>(a.o) + ((size_t)(qt.base + qt.first + tok) * a.Hq + h0 + (R & (heads - 1))) * D;
            if (split == 1 && !ok) continue;
#pragma unroll
            for (int x = 0; x < NB; ++x)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float v[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        v[i] = o[x][i][2 * r + e] * f[0];
#pragma unroll
                        for (int k = 1; k < KG; ++k) v[i] += row[(k - 1) * T::kRows * JLD + 32 * x + 8 * t + 4 * e + i] * f[k];
                        v[i] *= inv;
                    }
                    *reinterpret_cast<float4 *>(dst + 32 * x + 8 * t + 4 * e) = make_float4(v[0], v[1], v[2], v[3]);
                }
            if (split > 1 && t == 0) dst[D] = ok ? top : NAN, dst[D + 1] = sum;
        }
    }
    if (split > 1) join_split<D, false>(smem_u32(qs), qt.rows << group_shift, group_shift, split, cluster_rank(), a, qt, h0);
}

// log2 of the heads that share a block's rows: the power of two in Hq / Hkv, at most 32.
int group_shift_of(const AttnArgs &a) {
    int gs = 0;
    while (gs < 5 && ((a.Hq / a.Hkv) >> gs) % 2 == 0) ++gs;
    return gs;
}

template <int D, int KG>
cudaError_t launch_f32_kg(const AttnArgs &a, int sms, cudaStream_t stream) {
    using T = F32<D, KG>;
    static std::atomic<uint64_t> ready{0};
    auto kern = attn_prefill_f32<D, KG>;
    const cudaError_t e = allow_smem(kern, ready, T::kSmem);
    if (e != cudaSuccess) return e;
    const int gs = std::min(group_shift_of(a), KG == 2 ? 5 : 4);
    CUtensorMap km, vm;
    if (!page_map(&km, a.k_pages, D, a, false, 16) || !page_map(&vm, a.v_pages, D, a, false, 16)) return cudaErrorInvalidValue;
    const long long blocks = query_tiles(a, T::kRows >> gs) * (a.Hq >> gs);
    const int split = KG == 4 ? split_of(a, blocks, T::kRows >> gs, (long long)T::kBlocks * sms) : 1;
    return launch_split(kern, blocks, split, T::kThreads, T::kSmem, stream, km, vm, a, gs, split);
}

template <int D>
cudaError_t launch_f32(const AttnArgs &a, cudaStream_t stream) {
    const int gs = group_shift_of(a);
    int sms = 0;
    const cudaError_t e = device_sms(&sms);
    if (e != cudaSuccess) return e;
    // Calls whose blocks of 32 rows are resident at once anyway take blocks
    // of 16 rows and four groups of keys: half the time of the longest block
    // (8 heads, 475 new tokens: 49 -> 35 us at head size 128; 1400 at 64: 86
    // -> 66; past the bound 4 x 512 at 64 take 44 against 53, 3 x 512 at 128
    // 62 against 70).  At head size 256 one such block fills an SM (512
    // tokens: 100 -> 68 us, 2 x 512: 124 against 135).  Short windows leave
    // little to divide (2 x 600 tokens, window 200: 36 against 42 us).
    const long long limit = a.window > 0 && a.window <= 512 ? 1 : F32<D, 4>::kBlocks;
    if (query_tiles(a, 32 >> gs) * (a.Hq >> gs) <= limit * sms) return launch_f32_kg<D, 4>(a, sms, stream);
    return launch_f32_kg<D, 2>(a, sms, stream);
}

// ---------------------------------------------------------------------------
// BF16: tensor cores
// ---------------------------------------------------------------------------

// A row of 128, 64 or 16 consecutive TMEM columns for each of the warp's 32 lanes;
// the wait is part of the statement.
__device__ __forceinline__ void tmem_load_row(uint32_t taddr, float (&v)[128]) {
    uint32_t r[128];
    asm volatile(
        "{ tcgen05.ld.sync.aligned.32x32b.x128.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63,%64,%65,%66,%67,%68,%69,%70,%71,%72,%73,%74,%75,%76,%77,%78,%79,%80,%81,%82,%83,%84,%85,%86,%87,%88,%89,%90,%91,%92,%93,%94,%95,%96,%97,%98,%99,%100,%101,%102,%103,%104,%105,%106,%107,%108,%109,%110,%111,%112,%113,%114,%115,%116,%117,%118,%119,%120,%121,%122,%123,%124,%125,%126,%127}, [%128];\n\t"
        "tcgen05.wait::ld.sync.aligned; }"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63]), "=r"(r[64]), "=r"(r[65]), "=r"(r[66]), "=r"(r[67]), "=r"(r[68]), "=r"(r[69]), "=r"(r[70]), "=r"(r[71]), "=r"(r[72]), "=r"(r[73]), "=r"(r[74]), "=r"(r[75]), "=r"(r[76]), "=r"(r[77]), "=r"(r[78]), "=r"(r[79]), "=r"(r[80]), "=r"(r[81]), "=r"(r[82]), "=r"(r[83]), "=r"(r[84]), "=r"(r[85]), "=r"(r[86]), "=r"(r[87]), "=r"(r[88]), "=r"(r[89]), "=r"(r[90]), "=r"(r[91]), "=r"(r[92]), "=r"(r[93]), "=r"(r[94]), "=r"(r[95]), "=r"(r[96]), "=r"(r[97]), "=r"(r[98]), "=r"(r[99]), "=r"(r[100]), "=r"(r[101]), "=r"(r[102]), "=r"(r[103]), "=r"(r[104]), "=r"(r[105]), "=r"(r[106]), "=r"(r[107]), "=r"(r[108]), "=r"(r[109]), "=r"(r[110]), "=r"(r[111]), "=r"(r[112]), "=r"(r[113]), "=r"(r[114]), "=r"(r[115]), "=r"(r[116]), "=r"(r[117]), "=r"(r[118]), "=r"(r[119]), "=r"(r[120]), "=r"(r[121]), "=r"(r[122]), "=r"(r[123]), "=r"(r[124]), "=r"(r[125]), "=r"(r[126]), "=r"(r[127])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 128; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_load_row(uint32_t taddr, float (&v)[64]) { tmem_load64(taddr, v); }

__device__ __forceinline__ void tmem_store_row(uint32_t taddr, const float (&v)[32]) { tmem_store32(taddr, v); }
__device__ __forceinline__ void tmem_store_row(uint32_t taddr, const float (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
        "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
        : "memory");
}

__device__ __forceinline__ void tmem_load_row(uint32_t taddr, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "{ tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned; }"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// Maximum of three that keeps NaN.
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// 2^v of two values on the FMA pipe, for the weights that the special
// function unit has no time for: v = n + r with n the nearest integer (left
// in the low bits by adding 1.5 * 2^23) and |r| <= 1/2, 2^r by a cubic
// through 1 (least maximum relative error, 1.0e-4: a fortieth of the BF16
// rounding that follows), n added to the exponent.  From -127 down: 0.
// v <= 127.
__device__ __forceinline__ void ex2_fma(f32x2 v, float &a, float &b) {
    float x, y;
    apart(v, x, y);
    v = two(fmaxf(x, -127.0f), fmaxf(y, -127.0f));
    const f32x2 magic = two(12582912.0f, 12582912.0f), one = two(1.0f, 1.0f);
    const f32x2 t = add2(v, magic), n = add2(t, two(-12582912.0f, -12582912.0f));
    const f32x2 r = fma2(n, two(-1.0f, -1.0f), v);
    f32x2 p = fma2(r, two(0.05500893294811249f, 0.05500893294811249f), two(0.2422109693288803f, 0.2422109693288803f));
    p = fma2(p, r, two(0.6932829022407532f, 0.6932829022407532f));
    p = fma2(p, r, one);
    float pa, pb, ta, tb;
    apart(p, pa, pb);
    apart(t, ta, tb);
    a = __int_as_float(__float_as_int(pa) + (int)((unsigned)__float_as_int(ta) << 23));
    b = __int_as_float(__float_as_int(pb) + (int)((unsigned)__float_as_int(tb) << 23));
}

// cap tanh(z x) in units of log2 for |z x| <= 3/4, as x times a polynomial in
// x^2 whose coefficients hold z and the cap: tanh y = y + y^3 (c0 + c1 y^2 +
// c2 y^4), least maximum error 5.6e-6.  That error of a score grows with the
// cap: up to a cap of 100 it moves a weight by 5.6e-4 at most, a seventh of the
// BF16 rounding that follows.  The coefficients hold powers of z up to the 7th:
// with z between 2^-14 and 2^14 all of them are normal numbers.  Other caps and
// other z take capped_log2.
constexpr float kTanhReach = 0.75f, kPolyCap = 100.0f;
struct CapPoly {
    float k[4];
};
// |x| up to which the polynomial serves (-1: not at all).
__device__ __forceinline__ float cap_reach(float z, float cap) {
    z = fabsf(z);
    return cap <= kPolyCap && z >= 1.0f / 16384.0f && z <= 16384.0f ? kTanhReach / z : -1.0f;
}
__device__ __forceinline__ CapPoly cap_poly(float z, float out) {
    const float z3 = z * z * z, z5 = z3 * z * z, z7 = z5 * z * z;
    return CapPoly{{out * z, out * z3 * -0.3327198326587677f, out * z5 * 0.1272989809513092f, out * z7 * -0.03519973158836365f}};
}
__device__ __forceinline__ f32x2 capped(f32x2 x, const CapPoly &c) {
    const f32x2 u = mul2(x, x);
    f32x2 p = fma2(u, two(c.k[3], c.k[3]), two(c.k[2], c.k[2]));
    p = fma2(p, u, two(c.k[1], c.k[1]));
    p = fma2(p, u, two(c.k[0], c.k[0]));
    return mul2(p, x);
}

// Shared-memory operand descriptors as two words: all K steps of a tile share
// the upper word and add to the lower one.  K-major, 128-byte swizzle: 8-row
// atoms of 1024 bytes (the stride byte offset).  MN-major, 128-byte swizzle:
// blocks of 64 MN elements (128 bytes) by K rows, 8 K rows to an atom of 1024
// bytes, `block` bytes from one block to the next (the leading byte offset).
// Descriptors hold 18 bits of an address: above them the address of a block in
// a cluster has its rank.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_k(uint32_t saddr) { return (saddr & 0x3FFFFu) >> 4 | (1u << 16); }
__device__ __forceinline__ uint32_t desc_mn(uint32_t saddr, uint32_t block) {
    return (saddr & 0x3FFFFu) >> 4 | (block >> 4) << 16;
}

// D (TMEM) = A B (+ D when `add`), BF16, issued by one thread; A from shared
// memory or, with its weights, from TMEM.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{ .reg .pred p; .reg .b64 da, db; setp.ne.b32 p, %4, 0; mov.b64 da, {%1, %5}; mov.b64 db, {%2, %5}; "
        "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p; }" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)add), "n"(kDescHi)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{ .reg .pred p; .reg .b64 db; setp.ne.b32 p, %4, 0; mov.b64 db, {%2, %5}; "
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p; }" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)add), "n"(kDescHi)
        : "memory");
}

// NS query tiles of 128 rows ("streams") to a block.
template <int D, int NS>
struct Tc {
    static constexpr int kStreams = NS;
    static constexpr int kKeys = D == 128 ? 128 : 64;     // keys of a tile
    static constexpr int kTiles = D == 256 ? 2 : 1;  // score tiles of a stream in TMEM
    static constexpr int kHalves = D / 64;                // 128-byte column blocks
    static constexpr int kQBytes = 128 * D * 2;           // a query tile
    static constexpr int kSlotBytes = kKeys * D * 2;      // a tile of K or V
    static constexpr int kSlots = 5;
    static constexpr int kSoftWarps = 4 * kStreams;
    static constexpr int kMmaWarp = kSoftWarps, kLoadWarp = kSoftWarps + 1;
    static constexpr int kThreads = (kSoftWarps + 2) * 32;
    static constexpr int kSmem = 1024 + kStreams * kQBytes + kSlots * kSlotBytes;
    static_assert(kStreams * 128 * (D + 4) * 4 <= kSmem - 1024, "the parts of a split call take the operands' place");
    // TMEM columns: the score tiles, whose first half the weights overwrite,
    // then the outputs
    static constexpr uint32_t kColS = 0, kColO = kStreams * kTiles * kKeys;
    static constexpr uint32_t kCols = kColO + NS * D <= 256 ? 256 : 512;
    // At head size 64 half of TMEM is enough for a block, and a second block
    // on the SM keeps its softmax pipes busy (2 x 4096 tokens on a 4096-token
    // prefix, 32 heads: 752 -> 504 us; one block of four streams: 688).
    static constexpr int kBlocks = 512 / kCols;
    // keys up to which a tile is not split: a split costs 2 to 4 us (at head
    // size 128 it breaks even with 200 keys, and saves 3 of 16 us with 500)
    static constexpr int kSplitMin = 256;
};

struct TcBars {
    uint64_t q_full, kv_full[5], kv_empty[5], s_full[2], p_half[2], p_ready[2], o_done[2], tail, all_done;
};

// One block: 128 kStreams rows, each a (token, head) pair of `group` heads
// that share a key-value head (head fastest), against the tiles of keys.
template <int D, int NS, bool CAP>
__global__ void __launch_bounds__(Tc<D, NS>::kThreads, Tc<D, NS>::kBlocks)
    attn_prefill_tc(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                    const __grid_constant__ CUtensorMap vmap, const AttnArgs a, const int group_shift, const int box_shift,
                    const int cluster) {
    using T = Tc<D, NS>;
    constexpr int KT = T::kKeys, NH = T::kHalves;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *qs = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    unsigned char *ring = qs + NS * T::kQBytes;
    __shared__ TcBars bars;
    __shared__ uint32_t tmem_slot;
    __shared__ int find[T::kThreads / 32 + 6];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int tokens = 128 * NS >> group_shift;  // of a block
    if (warp == T::kMmaWarp) tmem_alloc(&tmem_slot, T::kCols);
    if (tid == 0) prefetch_map(&qmap), prefetch_map(&kmap), prefetch_map(&vmap);
    const BlockPlace at = place_of(a, group_shift, cluster);
    const QueryTile qt = find_query_tile<T::kThreads, (T::kBlocks > 1)>(a, tokens, at.turn, at.tiles, find);
    if (qt.rows <= 0) {
        __syncthreads();
        if (warp == T::kMmaWarp) tmem_dealloc(tmem_slot, T::kCols);
        return;
    }
    const int h0 = at.head, kv = h0 / (a.Hq / a.Hkv);
    const int p0 = qt.start + qt.first, len = p0 + qt.rows;  // keys any row sees: lo .. len - 1
    const int lo = a.window > 0 && p0 + 1 > a.window ? p0 + 1 - a.window : 0;
    // (streams without rows are left out)
    const int streams = (qt.rows * NS + tokens - 1) / tokens;
    int k_first = lo / KT, n = (len - 1) / KT - k_first + 1;
    const int split = n * KT > T::kSplitMin ? cluster : 1;
    const uint32_t rank = cluster > 1 ? cluster_rank() : 0;
    if (rank >= (uint32_t)split) {
        __syncthreads();
        if (warp == T::kMmaWarp) tmem_dealloc(tmem_slot, T::kCols);
        return;
    }
    if (split > 1) my_keys(k_first, n, split, rank);

    if (tid < (int)(sizeof(TcBars) / sizeof(uint64_t))) {
        // a thread per barrier (each initialisation ends in a fence)
        uint64_t *bar = reinterpret_cast<uint64_t *>(&bars) + tid;
        mbar_init(bar, bar >= bars.p_half && bar < bars.o_done ? 4 : 1);  // (the weights' barriers: a warp each)
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem_slot, 0);
    // the parts of a split call go in the operands' place: every warp passes
    // here once its copies and products are done
    auto operands_free = [] { asm volatile("bar.sync 1, %0;" ::"n"(T::kThreads) : "memory"); };

    if (warp == T::kLoadWarp) {
        // ------------------------------------------------------------ TMA
        if (lane == 0 && n > 0) {
            mbar_arrive_expect_tx(&bars.q_full, NS * T::kQBytes);
            const int t0 = (int)(qt.base + qt.first), per = 128 >> group_shift;
            for (int s = 0; s < NS; ++s)
                for (int x = 0; x < NH; ++x)
                    tma_page_load(qs + s * T::kQBytes + x * 16384, &qmap, 64 * x, h0, t0 + s * per, &bars.q_full);
        }
        // lane = (box of rows, column block) of a tile; boxes past the
        // visible keys are filled with zeros
        const int box_rows = 1 << box_shift, boxes = KT >> box_shift;
        const bool mine = lane < boxes * NH;
        const int bx = lane / NH, x = lane - bx * NH;
        int slot = 0, use = 0, tail_phase = 0;
        auto visible = [&](int j) {
            const int tok = (k_first + j) * KT + bx * box_rows;
            return mine && tok < len && tok + box_rows > lo;
        };
        // the block table is read a tile ahead of its use
        auto page_of = [&](int j) {
            const int tok = (k_first + j) * KT + bx * box_rows;
            return visible(j) ? __ldg(a.block_table + (size_t)qt.b * a.max_pages + (tok >> a.page_shift)) : -1;
        };
        auto map_row = [&](int j, int page) -> int {
            if (page >= 0 && page < a.num_pages) return page * a.Hkv + kv;
            if (visible(j)) atomicOr(&g_dev_error, kErrBadPage);
            return -1;
        };
        // tile j of K or V into the next slot
        auto load = [&](const CUtensorMap *map, int j, int z, bool is_v) {
            if (use > 0 && !warp_wait(&bars.kv_empty[slot], (use - 1) & 1)) return false;
            unsigned char *dst = ring + slot * T::kSlotBytes;
            const int k0 = (k_first + j) * KT;
            // V rows that no query row sees may hold NaN, which a weight of
            // zero does not silence: such a tile is cleared there first
            const bool clear = is_v && (k0 < lo || k0 + KT > len);
            uint64_t *bar = clear ? &bars.tail : &bars.kv_full[slot];
            if (lane == 0) mbar_arrive_expect_tx(bar, T::kSlotBytes);
            __syncwarp();
            if (mine)
                tma_page_load(dst + x * (KT * 128) + bx * box_rows * 128, map, 64 * x,
                              (k0 + bx * box_rows) & (a.page_size - 1), z, bar);
            if (clear) {
                if (!warp_wait(&bars.tail, tail_phase)) {
                    bar_wait(&bars.tail, tail_phase);  // (as below)
                    return false;
                }
                tail_phase ^= 1;
                for (int i = lane; i < KT * D / 8; i += 32) {
                    const int r = i / (D / 8), c = i - r * (D / 8);
                    if (k0 + r >= lo && k0 + r < len) continue;
                    *reinterpret_cast<uint4 *>(dst + (c >> 3) * (KT * 128) + r * 128 + (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.kv_full[slot]);
            }
            if (++slot == T::kSlots) slot = 0, ++use;
            return true;
        };
        // in the order the MMA lane takes them
        int z = map_row(0, page_of(0)), page = page_of(1);
        bool ok = n > 0 && load(&kmap, 0, z, false);
        for (int j = 0; ok && j < n; ++j) {
            const int zv = z;
            if (T::kTiles == 1) ok = load(&vmap, j, zv, true);
            if (ok && j + 1 < n) {
                z = map_row(j + 1, page);
                page = page_of(j + 2);
                ok = load(&kmap, j + 1, z, false);
            }
            if (ok && T::kTiles == 2) ok = load(&vmap, j, zv, true);
        }
        // Whoever gave up, the copies land (or get their time) before this
        // memory takes the parts of a split call or is freed.
        if (n > 0) {
            bar_wait(&bars.q_full, 0);
            const int fills = use * T::kSlots + slot;
            for (int i = max(0, fills - T::kSlots); i < fills; ++i) bar_wait(&bars.kv_full[i % T::kSlots], i / T::kSlots & 1);
        }
    } else if (warp == T::kMmaWarp) {
        // ------------------------------------------------------------ MMAs
        // The whole warp runs the loop, so that addresses stay uniform, and
        // one lane issues: with the loop inside that lane's branch an MMA
        // took about 90 cycles to issue, and the issue bounded the kernel.
        constexpr uint32_t id_qk = idesc_bf16(128, KT, false, false), id_pv = idesc_bf16(128, D, false, true);
        const uint32_t q_desc = desc_k(smem_u32(qs)), ring_addr = smem_u32(ring);
        int slot = 0, use = 0;
        auto take = [&](int &at) {
            at = slot;
            const bool ok = warp_wait(&bars.kv_full[slot], use & 1);
            if (++slot == T::kSlots) slot = 0, ++use;
            return ok;
        };
        // scores of one stream into its score tile at column col: the tile's
        // last weights were read by an earlier MMA of this thread
        auto qk = [&](int s, int at, uint32_t col) {
            const uint32_t k_desc = desc_k(ring_addr + at * T::kSlotBytes);
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
                mma_ss(col, q_desc + (s * T::kQBytes + (k >> 2) * 16384 + (k & 3) * 32) / 16,
                       k_desc + ((k >> 2) * (KT * 128) + (k & 3) * 32) / 16, id_qk, k > 0);
        };
        // half of the product with V
        auto pv = [&](int s, int at, uint32_t col, int half, bool add) {
            const uint32_t v_desc = desc_mn(ring_addr + at * T::kSlotBytes, KT * 128);
#pragma unroll
            for (int i = 0; i < KT / 32; ++i) {
                const int k = half * (KT / 32) + i;
                mma_ts(tm + T::kColO + s * D, col + 8 * k, v_desc + k * (2048 / 16), id_pv, add || i > 0);
            }
        };
        int ks = 0, vs = 0;
        bool ok = n > 0 && warp_wait(&bars.q_full, 0) && take(ks);
        tc_fence_after_sync();
        if (ok && elect_one()) {
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                if (s >= streams) break;
                qk(s, ks, tm + T::kColS + s * T::kTiles * KT);
                mma_commit(&bars.s_full[s * T::kTiles]);
            }
            mma_commit(&bars.kv_empty[ks]);
        }
        __syncwarp();
        for (int j = 0; ok && j < n; ++j) {
            const bool more = j + 1 < n;
            if constexpr (T::kTiles == 2) {
                // two score tiles: the next scores are made during this
                // tile's softmax
                if (more) {
                    ok = take(ks);
                    if (!ok) break;
                    tc_fence_after_sync();
                    if (elect_one()) {
#pragma unroll
                        for (int s = 0; s < NS; ++s) {
                            if (s >= streams) break;
                            qk(s, ks, tm + T::kColS + (2 * s + ((j + 1) & 1)) * KT);
                            mma_commit(&bars.s_full[2 * s + ((j + 1) & 1)]);
                        }
                        mma_commit(&bars.kv_empty[ks]);
                    }
                    __syncwarp();
                }
                ok = take(vs);
            } else {
                ok = take(vs) && (!more || take(ks));
            }
            for (int s = 0; ok && s < streams; ++s) {
                const uint32_t col = tm + T::kColS + (T::kTiles == 2 ? 2 * s + (j & 1) : s) * KT;
                ok = warp_wait(&bars.p_half[s], j & 1);
                if (!ok) break;
                tc_fence_after_sync();
                if (elect_one()) pv(s, vs, col, 0, j > 0);
                __syncwarp();
                ok = warp_wait(&bars.p_ready[s], j & 1);
                if (!ok) break;
                tc_fence_after_sync();
                if (elect_one()) {
                    pv(s, vs, col, 1, true);
                    if (T::kTiles == 2 || !more) mma_commit(&bars.o_done[s]);
                    if (s + 1 == streams) mma_commit(&bars.kv_empty[vs]);
                    if (T::kTiles == 1 && more) {
                        qk(s, ks, col);
                        mma_commit(&bars.s_full[s]);
                        if (s + 1 == streams) mma_commit(&bars.kv_empty[ks]);
                    }
                }
                __syncwarp();
            }
        }
        // the products issued so far as well
        if (n > 0) {
            if (elect_one()) mma_commit(&bars.all_done);
            __syncwarp();
            bar_wait(&bars.all_done, 0);
        }
    } else if (warp < 4 * streams) {
        // ------------------------------------------------------------ softmax: one row per thread
        const int s = warp >> 2, q4 = warp & 3;
        const int R = s * 128 + 32 * q4 + lane;
        const int tok = R >> group_shift, head = h0 + (R & ((1 << group_shift) - 1));
        const int p = p0 + tok;
        // positions of the warp's rows
        const int pw0 = p0 + ((s * 128 + 32 * q4) >> group_shift), pw1 = p0 + ((s * 128 + 32 * q4 + 31) >> group_shift);
        const uint32_t lanes = tm + ((uint32_t)(32 * q4) << 16);
        const uint32_t oa = lanes + T::kColO + s * D;
        // scores enter as 2^(c x): c = log2(e) |scale| (never 0, so that a
        // masked score stays -inf), or 1 for capped scores
        const float c = CAP ? 1.0f : fmaxf(fabsf(a.scale * kLog2e), 1e-30f);
        const SoftCap cap = soft_cap(a.scale, a.softcap);
        const CapPoly poly = cap_poly(cap.in, cap.out);
        const float in_reach = cap_reach(cap.in, a.softcap);
        float m = -INFINITY, l = 0.0f;
        bool ok = true;
        for (int j = 0; j < n; ++j) {
            const int buf = T::kTiles == 2 ? 2 * s + (j & 1) : s;
            const uint32_t sa = lanes + T::kColS + buf * KT;
            if (!warp_wait(&bars.s_full[buf], T::kTiles == 2 ? (j >> 1) & 1 : j & 1)) { ok = false; break; }
            tc_fence_after_sync();
            float x[KT];
            tmem_load_row(sa, x);
            const int k0 = (k_first + j) * KT;
            // the row sees x[first .. last] of the tile
            const bool edge = k0 + KT - 1 > pw0, early = a.window > 0 && k0 <= pw1 - a.window;
            const int last = p - k0, first = early ? p - a.window + 1 - k0 : 0;
            if constexpr (CAP) {
                // Scores well inside the cap, as they mostly are, take a
                // polynomial on the FMA pipe; two special functions else.  A
                // row chooses by the scores that it sees and by no others, so
                // that nothing else has a part in its output: where some score
                // of the warp is outside, those that a row does not see are
                // cleared and its others looked at again.  (Rows that differ
                // take both ways in turn: 2 x 2,048 tokens behind 2,048, cap
                // 50, scores around 15, 490 us at head size 64 and 573 at 128,
                // against 413 and 489 with one choice for the warp; scores
                // around 1, 215 and 246 against 210 and 245.)
                auto inside = [&] {
                    float big0 = 0.0f, big1 = 0.0f;
#pragma unroll
                    for (int i = 0; i < KT; i += 4) {
                        big0 = max3(big0, fabsf(x[i]), fabsf(x[i + 1]));
                        big1 = max3(big1, fabsf(x[i + 2]), fabsf(x[i + 3]));
                    }
                    return big0 <= in_reach && big1 <= in_reach;
                };
                auto small = [&] {
#pragma unroll
                    for (int i = 0; i < KT; i += 2) apart(capped(two(x[i], x[i + 1]), poly), x[i], x[i + 1]);
                };
                if (__all_sync(0xffffffffu, inside())) {
                    small();
                } else {
                    if (edge || early) {
#pragma unroll
                        for (int i = 0; i < KT; ++i) x[i] = (edge && i > last) || (early && i < first) ? 0.0f : x[i];
                    }
                    if (inside()) {
                        small();
                    } else {
#pragma unroll
                        for (int i = 0; i < KT; ++i) x[i] = capped_log2<true>(x[i], cap);
                    }
                }
            } else if (a.scale < 0.0f) {
#pragma unroll
                for (int i = 0; i < KT; ++i) x[i] = -x[i];
            }
            if (edge) {
#pragma unroll
                for (int i = 0; i < KT; ++i) x[i] = i > last ? -INFINITY : x[i];
            }
            if (early) {
#pragma unroll
                for (int i = 0; i < KT; ++i) x[i] = i < first ? -INFINITY : x[i];
            }
            float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
            for (int i = 4; i < KT - 4; i += 8) {
#pragma unroll
                for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], x[i + 2 * e], x[i + 2 * e + 1]);
            }
            const float tile_max = max3(max3(mx[0], x[KT - 4], x[KT - 3]), max3(mx[1], x[KT - 2], x[KT - 1]), max3(mx[2], mx[3], mx[3]));
            // The reference maximum moves only when weights would pass 2^8, so
            // that the output in TMEM is rescaled in few of the steps.
            // (a NaN becomes the maximum, and so the row's output)
            const bool grow = !(tile_max <= m) && (m == -INFINITY || !((tile_max - m) * c <= 8.0f));
            if (__any_sync(0xffffffffu, grow)) {
                const float f = grow ? ex2((m - tile_max) * c) : 1.0f;  // m = -inf: 0
                if (grow) m = tile_max, l *= f;
                if (j > 0) {
                    // (with one score tile, these scores followed that product)
                    if (T::kTiles == 2) {
                        if (!warp_wait(&bars.o_done[s], (j - 1) & 1)) { ok = false; break; }
                        tc_fence_after_sync();
                    }
#pragma unroll 1
                    for (int k = 0; k < D; k += 16) {
                        float o[16];
                        tmem_load_row(oa + k, o);
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] *= f;
                        tmem_store_row(oa + k, o);
                    }
                }
            }
            const float base = m == -INFINITY ? 0.0f : m * c;
            const f32x2 c2 = two(c, c), base2 = two(-base, -base);
            f32x2 sum0 = two(0.0f, 0.0f), sum1 = sum0;
            // with two score tiles, the barriers' phase of the tile before
            // must have been passed before they are arrived at again
            if (T::kTiles == 2 && j > 0 && !warp_wait(&bars.o_done[s], (j - 1) & 1)) { ok = false; break; }
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                constexpr int HW = KT / 4;  // words of half a tile's weights
                // of 8 pairs of weights, those exponentiated on the FMA pipe
                constexpr int kFmaOf8 = CAP ? 0 : 1;
                float w[HW];
#pragma unroll
                for (int i = 0; i < HW; ++i) {
                    const int k = half * (KT / 2) + 2 * i;
                    const f32x2 v = fma2(two(x[k], x[k + 1]), c2, base2);
                    float e0, e1;
                    if (i % 8 < kFmaOf8) {
                        ex2_fma(v, e0, e1);
                    } else {
                        apart(v, e0, e1);
                        e0 = ex2(e0), e1 = ex2(e1);
                    }
                    if (i & 1) sum1 = add2(sum1, two(e0, e1));
                    else sum0 = add2(sum0, two(e0, e1));
                    const __nv_bfloat162 h = __floats2bfloat162_rn(e0, e1);
                    w[i] = __uint_as_float(*reinterpret_cast<const uint32_t *>(&h));
                }
                tmem_store_row(sa + half * HW, w);
                tmem_wait_st();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(half ? &bars.p_ready[s] : &bars.p_half[s]);
            }
            float sa0, sb0;
            apart(add2(sum0, sum1), sa0, sb0);
            l += sa0 + sb0;
        }
        ok = ok && (n == 0 || warp_wait(&bars.o_done[s], T::kTiles == 2 ? (n - 1) & 1 : 0));
        tc_fence_after_sync();
        if (split > 1) {
            operands_free();
            float *row = reinterpret_cast<float *>(qs) + R * (D + 4);
#pragma unroll 1
            for (int k = 0; k < D; k += 16) {
                float o[16];
                if (n > 0) tmem_load_row(oa + k, o);
#pragma unroll
                for (int i = 0; i < 16; i += 4)
                    *reinterpret_cast<float4 *>(row + k + i) =
                        n > 0 ? make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
            // (out of time: NaN)
            row[D] = ok ? m * c : NAN;
            row[D + 1] = l;
        } else if (ok) {
            const float f = 1.0f / l;
            __nv_bfloat16 *op = static_cast<__nv_bfloat16 *>(a.o) + ((size_t)(qt.base + qt.first + tok) * a.Hq + head) * D;
#pragma unroll 1
            for (int k = 0; k < D; k += 32) {
                float o[32];
                tmem_load32(oa + k, o);
                if (tok < qt.rows) {
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const __nv_bfloat162 h = __floats2bfloat162_rn(o[i + 2 * e] * f, o[i + 2 * e + 1] * f);
                            w[e] = *reinterpret_cast<const uint32_t *>(&h);
                        }
                        *reinterpret_cast<uint4 *>(op + k + i) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            }
        }
    }
    if (split > 1) {
        __syncwarp();
        if (warp >= 4 * streams) operands_free();
        join_split<D, true>(smem_u32(qs), qt.rows << group_shift, group_shift, split, rank, a, qt, h0);
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == T::kMmaWarp) {
        tc_fence_after_sync();
        tmem_dealloc(tm, T::kCols);
    }
}

// Map of q [tokens, Hq, D]: boxes of 64 channels x `heads` heads x 128 / heads tokens.
bool query_map(CUtensorMap *m, const AttnArgs &a, int D, int heads) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)a.Hq, (cuuint64_t)a.tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)a.Hq * D * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)heads, (cuuint32_t)(128 / heads)};
    const cuuint32_t one[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(a.q), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int NS, bool CAP>
cudaError_t launch_tc(const AttnArgs &a, cudaStream_t stream) {
    using T = Tc<D, NS>;
    static std::atomic<uint64_t> ready{0};
    auto kern = attn_prefill_tc<D, NS, CAP>;
    const cudaError_t e = allow_smem(kern, ready, T::kSmem);
    if (e != cudaSuccess) return e;
    const int gs = group_shift_of(a);
    int bs = a.page_shift;
    while ((1 << bs) > T::kKeys) --bs;
    CUtensorMap qm, km, vm;
    if (!query_map(&qm, a, D, 1 << gs) || !page_map(&km, a.k_pages, D, a, true, 1 << bs) ||
        !page_map(&vm, a.v_pages, D, a, true, 1 << bs))
        return cudaErrorInvalidValue;
    int sms = 0;
    const cudaError_t es = device_sms(&sms);
    if (es != cudaSuccess) return es;
    const long long blocks = query_tiles(a, 128 * NS >> gs) * (a.Hq >> gs);
    const int split = split_of(a, blocks, 128 * NS >> gs, (long long)T::kBlocks * sms);
    return launch_split(kern, blocks, split, T::kThreads, T::kSmem, stream, qm, km, vm, a, gs, bs, split);
}

template <int D>
cudaError_t launch_tc_d(const AttnArgs &a, cudaStream_t stream) {
    constexpr int NS = D == 256 ? 1 : 2;
    return a.softcap > 0.0f ? launch_tc<D, NS, true>(a, stream) : launch_tc<D, NS, false>(a, stream);
}

}  // namespace

cudaError_t launch_attn_prefill(const AttnArgs &a, int D, bool bf16, cudaStream_t stream) {
    switch (D) {
        case 64: return bf16 ? launch_tc_d<64>(a, stream) : launch_f32<64>(a, stream);
        case 128: return bf16 ? launch_tc_d<128>(a, stream) : launch_f32<128>(a, stream);
        case 256: return bf16 ? launch_tc_d<256>(a, stream) : launch_f32<256>(a, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace lq
