// lq_attn_common.cuh -- device and host helpers shared by the attention
// kernels over the paged cache.
#pragma once

#include <atomic>

#include "lq_attn.h"
#include "lq_common.cuh"
#include "lq_kernels.h"

namespace lq {

// Two FP32 values in one 64-bit register: one instruction for both.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 two(float a, float b) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void apart(f32x2 v, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
constexpr float kLog2e = 1.4426950408889634f;

// Waits for phase `parity` of `bar` like mbar_wait_bounded, for loops that pass
// many barriers which are mostly complete already: the test without a
// suspend-time hint takes 14 cycles on a complete phase, with one 46 to 124.
__device__ __forceinline__ bool bar_test(uint64_t *bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
        : "=r"(done)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return done != 0;
}
__device__ __forceinline__ bool bar_wait(uint64_t *bar, uint32_t parity) {
    if (bar_test(bar, parity)) return true;
    const unsigned long long t0 = global_ns();
    for (;;) {
        // the clock is read once every 32 tests
        for (int k = 0; k < 32; ++k)
            if (bar_test(bar, parity)) return true;
        if (global_ns() - t0 > kWaitLimitNs) {
            atomicOr(&g_dev_error, kErrWaitTimeout);
            return false;
        }
    }
}

// The same for a converged warp, with one outcome for all of its lanes: each
// lane reads the clock for itself, and warp-wide instructions follow a wait.
// (A vote after every test instead: BF16 prefill at head size 64, 2 x 4,096
// tokens behind 4,096, 537 against 502 us.)
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity) {
    if (__all_sync(0xffffffffu, bar_test(bar, parity))) return true;
    return __all_sync(0xffffffffu, bar_wait(bar, parity)) != 0;
}

// One lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(r));
    return r != 0;
}

// Box load of a 3-D map ([pages * heads][page_size][D]; no multicast).  A
// coordinate outside the map fills zeros.
__device__ __forceinline__ void tma_page_load(void *dst, const CUtensorMap *map, int c0, int c1, int c2,
                                              uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
        "%4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
        : "memory");
}

// Brings a map near before its first use.
__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// The same with shared-memory addresses, and the bytes that a barrier expects.
__device__ __forceinline__ void tma_page_load_at(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
        "%4}], [%5];" ::"r"(dst),
        "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void expect_bytes(uint32_t bar, uint32_t bytes) {
    asm volatile("{ .reg .b64 st; mbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1; }" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldsm_x4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// D += A B, 16 x 8 x 16, BF16 operands, FP32 sums.
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// FP32 operands of TF32 MMAs in two parts: x = hi + lo, hi rounded to 11 bits
// (half away from zero), so that lo has either sign and what the MMA drops of
// it (at most 2^-22 of x) cancels over a sum; cut off instead, hi would leave
// every product short in the same direction.  An infinity becomes (inf, NaN);
// a NaN leaves a NaN in lo.
__device__ __forceinline__ void split_tf32(float x, float &hi, float &lo) {
    hi = __uint_as_float((__float_as_uint(x) + 0x1000u) & 0xFFFFE000u);
    lo = x - hi;
}
// (hi, lo) of four values.
__device__ __forceinline__ void split_tf32(const float4 &x, float (&v)[8]) {
    split_tf32(x.x, v[0], v[1]), split_tf32(x.y, v[2], v[3]), split_tf32(x.z, v[4], v[5]), split_tf32(x.w, v[6], v[7]);
}

// D += A B, 16 x 8 x 8, TF32 operands, FP32 sums.  The sum is cut off, not
// rounded: over a chain of n of these it ends about n / 2 steps of FP32 short,
// so chains are kept to 16 and joined by rounded additions (outputs summed in
// the MMAs alone over 100000 tokens came out 6e-6 small).
__device__ __forceinline__ void mma_1688(float (&d)[4], float a0, float a1, float a2, float a3, float b0, float b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(__float_as_uint(a0)), "r"(__float_as_uint(a1)), "r"(__float_as_uint(a2)), "r"(__float_as_uint(a3)),
          "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)));
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// cap tanh(scale s / cap) in units of log2.  FP32 outputs take tanhf.  For
// BF16 ones tanh y = 1 - 2 / (1 + e^{2y}), and below 1/4, where the difference
// loses digits that a large cap would bring back, the series to y^7.
struct SoftCap {
    float in, out;  // scale / cap and log2(e) cap
};

__device__ __forceinline__ SoftCap soft_cap(float scale, float cap) { return SoftCap{scale / cap, kLog2e * cap}; }

template <bool BF16>
__device__ __forceinline__ float capped_log2(float s, const SoftCap &c) {
    const float y = s * c.in;
    if constexpr (BF16) {
        const float u = y * y;
        const float near = y * fmaf(u, fmaf(u, fmaf(u, -17.0f / 315.0f, 2.0f / 15.0f), -1.0f / 3.0f), 1.0f);
        const float far = fmaf(-2.0f, rcp(1.0f + ex2(2.0f * kLog2e * y)), 1.0f);
        return c.out * (fabsf(y) < 0.25f ? near : far);
    } else {
        return c.out * tanhf(y);
    }
}

// Programmatic dependent launch: lets the next launch of the stream start,
// and waits for the previous one's results.
__device__ __forceinline__ void pdl_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Thread-block clusters: rank, barrier over all of their threads, and reads
// of a peer block's shared memory.
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ float4 peer_load4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float2 peer_load2(uint32_t addr) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}

// A tile of query rows of one sequence: rows first .. first + rows - 1 of its
// new tokens, in rows base + first .. of q and o; `start` tokens were in the
// cache before.
struct QueryTile {
    int b, first, rows, start;
    long long base;
};

// The turn-th tile of `rows` query rows in the order that the grid takes them,
// rows == 0 past the last one; `tiles` is the count that the grid was made
// for.  All NT threads of the block take part.  The order is from the last
// sequence's last tile to the first one's first or, with LEVELS and at most 32
// sequences, by the tiles' place in their sequence, the last ones first, so
// that the last blocks to start are short ones.  LEVELS is for kernels with
// several blocks on an SM: nine BF16 runs of 200 to 1,300 tokens at head size
// 64 take 71 -> 65 us by levels, three FP32 runs of 350 to 740 at 128 83 -> 77;
// one block to an SM gains nothing (BF16 at 128: 91 against 95 us).
// Sequence lengths come from cu_tokens (or are all tokens / B); an idle
// slot has no tiles, rows that would lie outside [0, tokens) or at positions
// past the block table are cut off, the latter with the device error word set.
template <int NT, bool LEVELS>
__device__ __forceinline__ QueryTile find_query_tile(const AttnArgs &a, int rows, long long turn, long long tiles,
                                                     int *smem /* NT / 32 + 6 */) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cap = a.max_pages << a.page_shift;
    auto rows_of = [&](int b, long long &base, int &start) -> int {
        start = __ldg(a.pos + b);
        long long n;
        if (a.cu) {
            base = __ldg(a.cu + b);
            n = __ldg(a.cu + b + 1) - base;
        } else {
            n = a.tokens / a.B;
            base = b * n;
        }
        if (start < 0 || base < 0) return 0;
        if (n > a.tokens - base) n = a.tokens - base;
        if (n > (long long)cap - start) {
            if (turn == 0 && n > 0) atomicOr(&g_dev_error, kErrBadPosition);
            n = (long long)cap - start;
        }
        return n > 0 ? (int)n : 0;
    };
    long long base = 0;
    int start = 0, n = 0;
    QueryTile q;
    if (LEVELS && a.B <= 32) {
        // a sequence per lane, every warp for itself; the tiles of a sequence
        // are at levels e .. e + t - 1
        if (lane < a.B) n = rows_of(lane, base, start);
        const int t = (n + rows - 1) / rows, e = start / rows;
        auto from = [&](int level) {  // tiles at this level or above
            return (long long)__reduce_add_sync(0xffffffffu, max(0, min(t, e + t - level)));
        };
        int lo = 0, hi = __reduce_max_sync(0xffffffffu, t > 0 ? e + t - 1 : 0);
        if (turn >= from(0)) {
            q.b = q.first = q.rows = q.start = 0, q.base = 0;
            return q;
        }
        while (lo < hi) {  // the highest level with the tile at or above it
            const int mid = (lo + hi + 1) >> 1;
            if (from(mid) > turn) lo = mid;
            else hi = mid - 1;
        }
        const int nth = (int)(turn - from(lo + 1));
        const bool here = e <= lo && lo < e + t;
        const unsigned all = __ballot_sync(0xffffffffu, here);
        const unsigned one = __ballot_sync(0xffffffffu, here && __popc(all & ((1u << lane) - 1)) == nth);
        q.b = __ffs(one) - 1;
        q.first = (lo - __shfl_sync(0xffffffffu, e, q.b)) * rows;
        q.rows = min(rows, __shfl_sync(0xffffffffu, n, q.b) - q.first);
        q.start = __shfl_sync(0xffffffffu, start, q.b);
        q.base = __shfl_sync(0xffffffffu, base, q.b);
        return q;
    }
    const long long tile_index = tiles - 1 - turn;
    // a thread's sequences; with at most NT of them it keeps what it read
    const int chunk = (a.B + NT - 1) / NT;
    int mine = 0;
    for (int i = 0; i < chunk; ++i) {
        const int b = tid * chunk + i;
        if (b >= a.B) break;
        n = rows_of(b, base, start);
        mine += (n + rows - 1) / rows;
    }
    int incl = mine;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, s);
        if (lane >= s) incl += y;
    }
    if (lane == 31) smem[warp] = incl;
    int *found = smem + NT / 32;
    if (tid == 0) found[2] = 0;
    __syncthreads();
    long long at = incl - mine;
    for (int w = 0; w < warp; ++w) at += smem[w];
    if (tile_index >= at && tile_index < at + mine) {
        for (int i = 0; i < chunk; ++i) {
            const int b = tid * chunk + i;
            if (chunk > 1) n = rows_of(b, base, start);
            const int t = (n + rows - 1) / rows;
            if (tile_index < at + t) {
                const int first = (int)(tile_index - at) * rows;
                found[0] = b;
                found[1] = first;
                found[2] = min(rows, n - first);
                found[3] = start;
                found[4] = (int)base;
                break;
            }
            at += t;
        }
    }
    __syncthreads();
    q.b = found[0], q.first = found[1], q.rows = found[2], q.start = found[3], q.base = found[4];
    return q;
}

// Tiles of `rows` query rows that `tokens` rows of B sequences can have.
inline long long query_tiles(const AttnArgs &a, int rows) {
    if (!a.cu) return (long long)a.B * ((a.tokens / a.B + rows - 1) / rows);
    return (long long)a.tokens / rows + (a.B < a.tokens ? a.B : a.tokens);
}

// Map of the cache pages as [num_pages * Hkv][page_size][D], boxes of 128
// bytes x `rows` tokens stored with the 128-byte swizzle.
inline bool page_map(CUtensorMap *m, const void *base, int D, const AttnArgs &a, bool bf16, int rows) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t es = bf16 ? 2 : 4;
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)a.page_size, (cuuint64_t)a.num_pages * a.Hkv};
    const cuuint64_t strides[2] = {D * es, D * es * a.page_size};
    const cuuint32_t box[3] = {(cuuint32_t)(128 / es), (cuuint32_t)rows, 1};
    const cuuint32_t one[3] = {1, 1, 1};
    return enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3,
               const_cast<void *>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// SM count of the current device, looked up once per device.
inline cudaError_t device_sms(int *sms) {
    static std::atomic<int> count[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    int n = count[dev & 63].load(std::memory_order_relaxed);
    if (n == 0) {
        e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        count[dev & 63].store(n, std::memory_order_relaxed);
    }
    *sms = n;
    return cudaSuccess;
}

// Raises a kernel's shared-memory limit once per device.
template <typename K>
cudaError_t allow_smem(K kern, std::atomic<uint64_t> &done, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_acq_rel);
    return e;
}

}  // namespace lq
