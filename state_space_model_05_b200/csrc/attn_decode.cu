// Causal softmax attention of one token per sequence against its cache.
//
//     o = sum_s p_s v_s / sum_s p_s,   p_s = 2^(c q.k_s - m),   c = scale log2(e),   s = 0 .. len
//
// Bound by memory: the cached rows, read once.  All (batch row, key/value head, block of
// query heads) units are laid end to end in tiles of 64 positions, as many as each row's length
// needs, and every CTA takes an equal contiguous range of tiles, so that one long cache fills the
// GPU as well as many short ones do, whatever the capacity.  A unit inside one CTA's range
// is written at once; the pieces of a unit that is cut go to the workspace with their maxima
// and sums, and a second kernel joins them in the order of the CTAs (the same on every run).
//
// bf16: one warp streams tiles into a ring by TMA; four warps take 16 positions of each tile, the
// query heads (up to 16) as the rows of mma.sync products, with a softmax state of their own
// that is merged where a unit ends.  mma.sync is enough: 16 positions are 32 instructions, a
// fifth of the time their 8 KB take to arrive, and up to 16 rows would leave a 128-row
// tcgen05 tile nearly empty.  fp32: the same ranges on the CUDA cores, a tile at a time: load, barrier,
// scores, barrier, softmax, barrier, products, with no loads in flight behind them, 128 columns and 8 query
// heads whatever the sizes.  That is the simplest right form, bound by the latency of those steps: one
// cache of 64999, 32/8 heads of 128, 532 MB: 287 us = 1.85 TB/s, where the bytes take 82 us.
//
// Measured, 32/8 heads of 128: one cache of 64999, 266 MB: 52 us = 5.1 TB/s; 32 caches of up to 4096, 246 MB: 53 us
// = 4.7 TB/s, of which the join's loads and the start take about 8 us.  Units of at most 8 rows skip the
// upper half of the products' rows (32 x 2000, groups of 4: 49.2 us, 50.5 us with it); heads of up to 64
// dimensions have tiles of 64 (64 x 1500, 16 heads: 78.7 us, 83.9 us on tiles of 128).
#include <cuda.h>

#include "mixers.cuh"
#include "prefill_tc.h"
#include "ptx.cuh"

namespace ssd {

using namespace ptx;

namespace {

constexpr float kLog2e = 1.44269504088896341f;
constexpr int kTile = 64;                                  // positions per tile

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

__device__ __forceinline__ int row_tiles(int len, int capacity) { return len < 0 || len >= capacity ? 0 : len / kTile + 1; }

// Query heads of one unit, and the floats of one piece: O, then m and l of every row.
template <int kRows> constexpr int kPiece = kRows * (kMixMaxDim + 2);

// The work's shape: the units of one batch row.
struct Units {
    int group, blocks, per_row;
    __host__ __device__ Units(int hq, int hkv, int rows) : group(hq / hkv), blocks((hq / hkv + rows - 1) / rows), per_row(hkv * blocks) {}
};

// ---- ranges of tiles -----------------------------------------------------------------
// a / b, in 32 bits where both fit (a 64-bit division is a hundred instructions, cold ones here).
__device__ __forceinline__ long long quotient(long long a, long long b)
{
    return (a | b) >> 32 ? a / b : (long long)((unsigned)a / (unsigned)b);
}

// W tiles over at most `ctas` CTAs: the first W mod G take one more than the others, and no
// range is empty.
struct Ranges {
    long long W, each;
    int G, more;
    __device__ __forceinline__ Ranges(long long tiles, int ctas) : W(tiles), each(0), G((int)min((long long)ctas, tiles)), more(0)
    {
        if (G > 0) {
            each = quotient(W, G);
            more = (int)(W - each * G);
        }
    }
    __device__ __forceinline__ long long first(int c) const { return each * c + min(c, more); }
    __device__ __forceinline__ int owner(long long t) const         // the CTA whose range holds tile t
    {
        const long long longer = (each + 1) * more;
        return (int)(t < longer ? quotient(t, each + 1) : more + quotient(t - longer, each));
    }
};

// Tiles of all rows and of those before one row, found by the threads of a CTA together.
struct Located { int b; long long before, total; };

// Sums the rows' tiles; `want(total)` then names a tile of the batch whose rows' tiles repeat
// `units` times, and its row is returned (by_row: the row itself).
template <int kThreads, typename F>
__device__ __forceinline__ Located locate(const int* __restrict__ lens, int batch, int capacity, int units, bool by_row,
                                          int* err, F want)
{
    __shared__ long long warp_sum[kThreads / 32];
    __shared__ Located found;
    const int tid = threadIdx.x, lane = tid & 31, per = (batch + kThreads - 1) / kThreads;
    const int b0 = min(batch, tid * per), b1 = min(batch, b0 + per);
    long long sum = 0;
    bool bad = false;
    for (int b = b0; b < b1; ++b) {
        const int len = lens[b];
        bad |= len >= capacity;
        sum += row_tiles(len, capacity);
    }
    if (bad && err) record_error(err, SSD_ERR_SHAPE);
    long long upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
    }
    if (lane == 31) warp_sum[tid >> 5] = upto;
    __syncthreads();
    long long before = upto - sum, total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < (tid >> 5)) before += warp_sum[w];
        total += warp_sum[w];
    }
    const long long x = want(total);
    if (tid == 0) found = Located{batch, total, total};
    __syncthreads();
    if (by_row ? (x >= b0 && x < b1) : (x >= before * units && x < (before + sum) * units)) {
        for (int b = b0; b < b1; ++b) {
            const int n = row_tiles(lens[b], capacity);
            if (by_row ? b == x : x < (before + n) * units) {
                found = Located{b, before, total};
                break;
            }
            before += n;
        }
    }
    __syncthreads();
    return found;
}

// A range's tiles in order.
struct Cursor {
    int b, u, tile, n, len;                                // row, unit of the row, tile of the unit, the unit's tiles
    __device__ __forceinline__ void start(const int* lens, int capacity, const Located& at, long long x, int units)
    {
        b = at.b;
        len = lens[b];
        n = row_tiles(len, capacity);
        const long long y = x - at.before * units;
        u = (int)quotient(y, n);
        tile = (int)(y - (long long)u * n);
    }
    __device__ __forceinline__ void next(const int* lens, int capacity, int units, bool more)
    {
        if (++tile < n) return;
        tile = 0;
        if (++u < units || !more) return;
        u = 0;
        do {
            len = lens[++b];
            n = row_tiles(len, capacity);
        } while (n == 0);
    }
};

// ================================================================ bf16
constexpr int kRows = 16;                                  // query heads per unit
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32 + 32;                 // and the warp that loads

template <int D>
struct Cfg {
    static constexpr int kHalf = kTile * 128;              // 64 dimensions of a tile's rows
    static constexpr int kSide = D / 64 * kHalf;           // keys (or values) of a tile
    static constexpr int kStages = D == 128 ? 3 : 6;
    static constexpr int kO = kStages * 2 * kSide;         // merged output rows
    static constexpr int kLdO = D + 8;
    static constexpr int kStat = kO + kRows * kLdO * 4;    // m, l per warp and row
    static constexpr int kBar = kStat + 2 * kWarps * kRows * 4;
    static constexpr int kAbort = kBar + 2 * kStages * 8;
    static constexpr int kBytes = kAbort + 16 + 1024;
    static_assert(2 * (kBytes + 1024) <= 228 * 1024, "two CTAs per SM");
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

struct CacheMaps { CUtensorMap k, v; };

// kHigh: units have more than 8 rows (rows 8 .. 15 of the products are used).
template <int D, bool kHigh>
__global__ void __launch_bounds__(kThreads, 2)
attn_decode_bf16_kernel(const __grid_constant__ CacheMaps maps, const AttnDecodeArgs a, float* __restrict__ pieces, int* err)
{
    using L = Cfg<D>;
    using T = __nv_bfloat16;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* sO = reinterpret_cast<float*>(sm + L::kO);
    float* sM = reinterpret_cast<float*>(sm + L::kStat);
    float* sL = sM + kWarps * kRows;
    uint64_t *full = reinterpret_cast<uint64_t*>(sm + L::kBar), *empty = full + L::kStages;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::kAbort);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kWarps);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    griddep_wait();                                        // every input may come from the kernel before
    griddep_launch_dependents();                           // (only now: the join reads the lengths at once)
    const Units un(a.hq, a.hkv, kRows);
    const int c = blockIdx.x;
    const Located at = locate<kThreads>(a.lens, a.batch, a.capacity, un.per_row, false, c == 0 ? err : nullptr,
                                        [&](long long total) {
                                            const Ranges r(total * un.per_row, gridDim.x);
                                            return c < r.G ? r.first(c) : -1;
                                        });
    const Ranges ranges(at.total * un.per_row, gridDim.x);
    if (c >= ranges.G) return;
    const long long x0 = ranges.first(c), x1 = ranges.first(c + 1);
    Cursor cur;
    cur.start(a.lens, a.capacity, at, x0, un.per_row);
    auto wait = [&](uint64_t* bar, int phase) { return mbar_wait_compact(bar, phase & 1, err, abort_flag); };

    if (warp == kWarps) {
        if (lane == 0) {
            for (long long x = x0; x < x1; ++x) {
                const int i = (int)(x - x0), s = i % L::kStages;
                if (i >= L::kStages && !wait(&empty[s], i / L::kStages - 1)) break;
                const int hk = cur.u / un.blocks;
                uint8_t* st = sm + s * 2 * L::kSide;
                mbar_expect_tx(&full[s], 2 * L::kSide);
                for (int d = 0; d < D; d += 64) {
                    tma_load_4d(st + d / 64 * L::kHalf, &maps.k, d, hk, cur.tile * kTile, cur.b, &full[s]);
                    tma_load_4d(st + L::kSide + d / 64 * L::kHalf, &maps.v, d, hk, cur.tile * kTile, cur.b, &full[s]);
                }
                cur.next(a.lens, a.capacity, un.per_row, x + 1 < x1);
            }
            settle(abort_flag);
        }
        return;
    }

    // ---- four warps; a thread holds rows lane / 4 and lane / 4 + 8 of its warp's products
    const int r0 = lane >> 2, qd = 2 * (lane & 3);
    const float c2 = a.scale * kLog2e;
    bool from_start = cur.tile == 0, fresh = true;
    uint32_t q[D / 16][4];
    float o[D / 8][4], m[2], l[2];
    for (long long x = x0; x < x1; ++x) {
        const int i = (int)(x - x0), s = i % L::kStages;
        const int hk = cur.u / un.blocks, first = (cur.u - hk * un.blocks) * kRows;
        const int h0 = hk * un.group + first, rows = min(kRows, un.group - first);
        if (fresh) {
            const T* src = static_cast<const T*>(a.q) + ((size_t)cur.b * a.hq + h0) * a.dim;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int row = r0 + (e & 1) * 8, d = ks * 16 + qd + (e >> 1) * 8;
                    q[ks][e] = row < rows && d < a.dim ? *reinterpret_cast<const uint32_t*>(src + (size_t)row * a.dim + d) : 0u;
                }
#pragma unroll
            for (int e = 0; e < D / 8; ++e) o[e][0] = o[e][1] = o[e][2] = o[e][3] = 0.f;
            m[0] = m[1] = neg_inf();
            l[0] = l[1] = 0.f;
            fresh = false;
        }
        wait(&full[s], i / L::kStages);                    // on expiry the abort flag ends every wait of the CTA
        __syncwarp();
        uint8_t* keys = sm + s * 2 * L::kSide;
        uint8_t* values = keys + L::kSide;
        const bool ends = cur.tile == cur.n - 1;
        const int p0 = cur.tile * kTile + warp * 16;       // this warp's first position
        if (ends && p0 + 15 >= cur.len) {
            // the new token's row comes from the inputs and joins the cache; rows behind it, which may
            // hold anything, are zeroed among the values (0 x inf is not 0) and masked among the keys
            for (int j = lane; j < 16 * (D / 8); j += 32) {
                const int row = j / (D / 8), ch = j % (D / 8), pos = p0 + row, at_row = warp * 16 + row;
                if (pos < cur.len) continue;
                const int off = (ch >> 3) * L::kHalf + at_row * 128 + (((ch & 7) ^ (at_row & 7)) << 4);
                uint4 kk = make_uint4(0u, 0u, 0u, 0u), vv = kk;
                if (pos == cur.len && ch * 8 < a.dim) {
                    const size_t in = ((size_t)cur.b * a.hkv + hk) * a.dim + ch * 8;
                    kk = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.k) + in);
                    vv = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.v) + in);
                    if (first == 0) {
                        const size_t row_at = (((size_t)cur.b * a.capacity + pos) * a.hkv + hk) * a.dim + ch * 8;
                        *reinterpret_cast<uint4*>(static_cast<T*>(a.k_cache) + row_at) = kk;
                        *reinterpret_cast<uint4*>(static_cast<T*>(a.v_cache) + row_at) = vv;
                    }
                }
                *reinterpret_cast<uint4*>(keys + off) = kk;
                *reinterpret_cast<uint4*>(values + off) = vv;
            }
            fence_proxy_async_smem();                      // the slot's next load overwrites these rows
            __syncwarp();
        }
        if (p0 <= cur.len) {
            // ldmatrix addresses: lane's row of the four 8 x 8 matrices, and its 16-byte chunk
            const int krow = warp * 16 + (lane & 7) + ((lane >> 4) << 3), kch = (lane >> 3) & 1;
            const int vrow = warp * 16 + (lane & 15), vch = lane >> 4;
            float sc[2][4] = {};
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                uint32_t b[4];
                ldsm4(b, smem_u32(keys + (ks >> 2) * L::kHalf + krow * 128 + ((((ks & 3) * 2 + kch) ^ (krow & 7)) << 4)));
                mma16816(sc[0], q[ks], b[0], b[1]);
                mma16816(sc[1], q[ks], b[2], b[3]);
            }
            uint32_t p[4] = {0u, 0u, 0u, 0u};
            const int left = cur.len - p0 - qd;            // positions past the new token's are masked
#pragma unroll
            for (int half = 0; half < (kHigh ? 2 : 1); ++half) {
                float y[4] = {sc[0][2 * half] * c2, sc[0][2 * half + 1] * c2, sc[1][2 * half] * c2, sc[1][2 * half + 1] * c2};
                if (ends) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if ((e & 1) + (e >> 1) * 8 > left) y[e] = neg_inf();
                }
                float top = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // the maximum moves only when exceeded by 2^8: p stays below that until then
                float keep = 1.f;
                if (top > m[half] + 8.f) {
                    keep = ex2(m[half] - top);
                    m[half] = top;
                }
                if (__any_sync(0xffffffffu, keep != 1.f)) {
                    l[half] *= keep;
#pragma unroll
                    for (int e = 0; e < D / 8; ++e) {
                        o[e][2 * half] *= keep;
                        o[e][2 * half + 1] *= keep;
                    }
                }
                const float base = m[half] == neg_inf() ? 0.f : m[half];
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = ex2(y[e] - base);
                l[half] += (y[0] + y[1]) + (y[2] + y[3]);
                p[half] = pack_bf16x2(y[0], y[1]);         // P is rounded to bf16, the operand type; its sum is not
                p[2 + half] = pack_bf16x2(y[2], y[3]);
            }
#pragma unroll
            for (int nd = 0; nd < D / 16; ++nd) {
                uint32_t b[4];
                ldsm4_t(b, smem_u32(values + (nd >> 2) * L::kHalf + vrow * 128 + ((((nd & 3) * 2 + vch) ^ (vrow & 7)) << 4)));
                mma16816(o[2 * nd], p, b[0], b[1]);
                mma16816(o[2 * nd + 1], p, b[2], b[3]);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[s]);

        if (ends || x + 1 == x1) {
            // the four warps' states, merged in their order
#pragma unroll
            for (int half = 0; half < (kHigh ? 2 : 1); ++half) {
                l[half] += __shfl_xor_sync(0xffffffffu, l[half], 1);
                l[half] += __shfl_xor_sync(0xffffffffu, l[half], 2);
                if ((lane & 3) == 0) {
                    sM[warp * kRows + r0 + 8 * half] = m[half];
                    sL[warp * kRows + r0 + 8 * half] = l[half];
                }
            }
            named_bar_sync(1, kWarps * 32);
            float top[2], sum[2];
#pragma unroll
            for (int half = 0; half < (kHigh ? 2 : 1); ++half) {
                top[half] = neg_inf();
                sum[half] = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) top[half] = fmaxf(top[half], sM[w * kRows + r0 + 8 * half]);
                const float base = top[half] == neg_inf() ? 0.f : top[half];
#pragma unroll
                for (int w = 0; w < kWarps; ++w)
                    sum[half] = fmaf(sL[w * kRows + r0 + 8 * half], ex2(sM[w * kRows + r0 + 8 * half] - base), sum[half]);
                const float mul = ex2(m[half] - base);
#pragma unroll
                for (int e = 0; e < D / 8; ++e) {
                    o[e][2 * half] *= mul;
                    o[e][2 * half + 1] *= mul;
                }
            }
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                if (warp == w) {
#pragma unroll
                    for (int half = 0; half < (kHigh ? 2 : 1); ++half)
#pragma unroll
                        for (int e = 0; e < D / 8; ++e) {
                            float2* at_o = reinterpret_cast<float2*>(sO + (r0 + 8 * half) * L::kLdO + 8 * e + qd);
                            if (w > 0) {
                                const float2 z = *at_o;
                                o[e][2 * half] += z.x;
                                o[e][2 * half + 1] += z.y;
                            }
                            if (w < kWarps - 1) *at_o = make_float2(o[e][2 * half], o[e][2 * half + 1]);
                        }
                }
                if (w < kWarps - 1) named_bar_sync(1, kWarps * 32);
            }
            if (warp == kWarps - 1) {
                const bool whole = ends && from_start;
                float* piece = pieces + (size_t)(2 * c + (from_start ? 1 : 0)) * kPiece<kRows>;
#pragma unroll
                for (int half = 0; half < (kHigh ? 2 : 1); ++half) {
                    const int row = r0 + 8 * half;
                    if (row >= rows) continue;
                    if (whole) {
                        const float inv = 1.f / sum[half];
                        T* out = static_cast<T*>(a.out) + ((size_t)cur.b * a.hq + h0 + row) * a.dim;
#pragma unroll
                        for (int e = 0; e < D / 8; ++e)
                            if (8 * e < a.dim)
                                *reinterpret_cast<uint32_t*>(out + 8 * e + qd) = pack_bf16x2(o[e][2 * half] * inv, o[e][2 * half + 1] * inv);
                    } else {
#pragma unroll
                        for (int e = 0; e < D / 8; ++e)
                            *reinterpret_cast<float2*>(piece + row * kMixMaxDim + 8 * e + qd) = make_float2(o[e][2 * half], o[e][2 * half + 1]);
                        if ((lane & 3) == 0) {
                            piece[kRows * kMixMaxDim + row] = top[half];
                            piece[kRows * kMixMaxDim + kRows + row] = sum[half];
                        }
                    }
                }
            }
            fresh = true;
            from_start = true;
        }
        cur.next(a.lens, a.capacity, un.per_row, x + 1 < x1);
    }
}

// ================================================================ fp32, on the CUDA cores
constexpr int kRows32 = 8;
constexpr int kThreads32 = 128;
constexpr int kLd = kMixMaxDim + 4;
constexpr int kLdP = kTile + 4;
constexpr int kBytes32 = (2 * kTile * kLd + kRows32 * kMixMaxDim + kRows32 * kLdP) * 4;

__global__ void __launch_bounds__(kThreads32)
attn_decode_f32_kernel(const AttnDecodeArgs a, float* __restrict__ pieces, int* err)
{
    extern __shared__ float smf[];
    float *sk = smf, *sv = sk + kTile * kLd, *sq = sv + kTile * kLd, *sp = sq + kRows32 * kMixMaxDim;
    __shared__ float sm_m[kRows32], sm_l[kRows32], sm_keep[kRows32];
    griddep_wait();                                        // every input may come from the kernel before
    griddep_launch_dependents();                           // (only now: the join reads the lengths at once)
    const int tid = threadIdx.x, c = blockIdx.x;
    const Units un(a.hq, a.hkv, kRows32);
    const Located at = locate<kThreads32>(a.lens, a.batch, a.capacity, un.per_row, false, c == 0 ? err : nullptr,
                                        [&](long long total) {
                                            const Ranges r(total * un.per_row, gridDim.x);
                                            return c < r.G ? r.first(c) : -1;
                                        });
    const Ranges ranges(at.total * un.per_row, gridDim.x);
    if (c >= ranges.G) return;
    const long long x0 = ranges.first(c), x1 = ranges.first(c + 1);
    Cursor cur;
    cur.start(a.lens, a.capacity, at, x0, un.per_row);
    bool from_start = cur.tile == 0, fresh = true;
    float acc[kRows32];
    for (long long x = x0; x < x1; ++x) {
        const int hk = cur.u / un.blocks, first = (cur.u - hk * un.blocks) * kRows32, len = cur.len, b = cur.b;
        const int h0 = hk * un.group + first, rows = min(kRows32, un.group - first);
        __syncthreads();
        if (fresh) {
            for (int i = tid; i < kRows32 * kMixMaxDim; i += kThreads32) {
                const int r = i / kMixMaxDim, d = i % kMixMaxDim;
                sq[i] = (r < rows && d < a.dim)
                            ? static_cast<const float*>(a.q)[((size_t)b * a.hq + h0 + r) * a.dim + d] * (a.scale * kLog2e) : 0.f;
            }
            if (tid < kRows32) {
                sm_m[tid] = neg_inf();
                sm_l[tid] = 0.f;
            }
#pragma unroll
            for (int r = 0; r < kRows32; ++r) acc[r] = 0.f;
            fresh = false;
        }
        // keys and values of the tile; the new token's come from the inputs and join the cache
        const int p0 = cur.tile * kTile, np = min(kTile, len + 1 - p0);
        for (int i = tid; i < kTile * (kMixMaxDim / 4); i += kThreads32) {
            const int r = i / (kMixMaxDim / 4), d = 4 * (i % (kMixMaxDim / 4)), pos = p0 + r;
            float4 kk = make_float4(0.f, 0.f, 0.f, 0.f), vv = kk;
            if (r < np && d < a.dim) {
                const size_t row = (((size_t)b * a.capacity + pos) * a.hkv + hk) * a.dim + d;
                const size_t in = ((size_t)b * a.hkv + hk) * a.dim + d;
                kk = *reinterpret_cast<const float4*>(pos < len ? static_cast<const float*>(a.k_cache) + row : static_cast<const float*>(a.k) + in);
                vv = *reinterpret_cast<const float4*>(pos < len ? static_cast<const float*>(a.v_cache) + row : static_cast<const float*>(a.v) + in);
                if (pos == len && first == 0) {
                    *reinterpret_cast<float4*>(static_cast<float*>(a.k_cache) + row) = kk;
                    *reinterpret_cast<float4*>(static_cast<float*>(a.v_cache) + row) = vv;
                }
            }
            *reinterpret_cast<float4*>(sk + r * kLd + d) = kk;
            *reinterpret_cast<float4*>(sv + r * kLd + d) = vv;
        }
        __syncthreads();
        // scores: position tid % 64, query heads 4 (tid / 64) .. + 3
        {
            const int pos = tid % kTile, r0 = tid / kTile * (kRows32 / 2);
            float s[kRows32 / 2] = {};
            for (int d = 0; d < a.dim; d += 4) {
                const float4 y = *reinterpret_cast<const float4*>(sk + pos * kLd + d);
#pragma unroll
                for (int r = 0; r < kRows32 / 2; ++r) {
                    const float4 z = *reinterpret_cast<const float4*>(sq + (r0 + r) * kMixMaxDim + d);
                    s[r] = fmaf(z.x, y.x, fmaf(z.y, y.y, fmaf(z.z, y.z, fmaf(z.w, y.w, s[r]))));
                }
            }
#pragma unroll
            for (int r = 0; r < kRows32 / 2; ++r) sp[(r0 + r) * kLdP + pos] = pos < np ? s[r] : neg_inf();
        }
        __syncthreads();
        // running maximum and sum: warp w takes rows 2 w, 2 w + 1
        for (int r = tid / 32 * 2; r < tid / 32 * 2 + 2; ++r) {
            const int lane = tid & 31;
            const float s0 = sp[r * kLdP + lane], s1 = sp[r * kLdP + 32 + lane];
            float top = fmaxf(s0, s1);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float old = sm_m[r];
            top = fmaxf(top, old);
            const float base = top == neg_inf() ? 0.f : top;
            const float e0 = exp2f(s0 - base), e1 = exp2f(s1 - base);
            sp[r * kLdP + lane] = e0;
            sp[r * kLdP + 32 + lane] = e1;
            float sum = e0 + e1;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            __syncwarp();
            if (lane == 0) {
                const float keep = exp2f(old - base);
                sm_keep[r] = keep;
                sm_m[r] = top;
                sm_l[r] = fmaf(sm_l[r], keep, sum);
            }
        }
        __syncthreads();
        // thread: dimension tid of every row
#pragma unroll
        for (int r = 0; r < kRows32; ++r) acc[r] *= sm_keep[r];
        for (int s = 0; s < np; ++s) {
            const float y = sv[s * kLd + tid];
#pragma unroll
            for (int r = 0; r < kRows32; ++r) acc[r] = fmaf(sp[r * kLdP + s], y, acc[r]);
        }
        const bool ends = cur.tile == cur.n - 1;
        if (ends || x + 1 == x1) {
            if (ends && from_start) {
                if (tid < a.dim)
                    for (int r = 0; r < rows; ++r)
                        static_cast<float*>(a.out)[((size_t)b * a.hq + h0 + r) * a.dim + tid] = acc[r] / sm_l[r];
            } else {
                float* p = pieces + (size_t)(2 * c + (from_start ? 1 : 0)) * kPiece<kRows32>;
#pragma unroll
                for (int r = 0; r < kRows32; ++r) p[r * kMixMaxDim + tid] = acc[r];
                if (tid < kRows32) {
                    p[kRows32 * kMixMaxDim + tid] = sm_m[tid];
                    p[kRows32 * kMixMaxDim + kRows32 + tid] = sm_l[tid];
                }
            }
            fresh = true;
            from_start = true;
        }
        cur.next(a.lens, a.capacity, un.per_row, x + 1 < x1);
    }
}

// ================================================================ cut units
// Joins the pieces of a unit that more than one CTA worked on: one CTA per unit and query
// head, one thread per dimension, the pieces in the order of their CTAs.  A long row is cut
// into hundreds of pieces: their weights are formed side by side first, so that the sum's loads
// do not wait for one another; up to kFew pieces are loaded at once with their maxima and sums
// (32 rows of up to 4096 positions: 54.5 us -> 52.9 us for both kernels).  (`pieces` is written while
// this kernel already runs, so it is not declared as read-only.)
constexpr int kFew = 4;

template <typename T, int kUnitRows>
__global__ void __launch_bounds__(kMixMaxDim)
attn_decode_join_kernel(const AttnDecodeArgs a, const float* pieces, int max_ctas)
{
    extern __shared__ float weight[];                      // [max_ctas]
    __shared__ float red[2][kMixMaxDim / 32];
    const Units un(a.hq, a.hkv, kUnitRows);
    const int b = blockIdx.x / a.hq, h = blockIdx.x - b * a.hq, d = threadIdx.x;
    const int hk = h / un.group, r = (h - hk * un.group) % kUnitRows, u = hk * un.blocks + (h - hk * un.group) / kUnitRows;
    const Located at = locate<kMixMaxDim>(a.lens, a.batch, a.capacity, un.per_row, true, nullptr, [&](long long) { return (long long)b; });
    const int n = row_tiles(a.lens[b], a.capacity);
    if (n == 0) {
        griddep_wait();                                    // also where nothing is to join: this grid ends after the one before
        return;
    }
    const Ranges ranges(at.total * un.per_row, max_ctas);
    const long long t0 = at.before * un.per_row + (long long)u * n, t1 = t0 + n;
    const int c0 = ranges.owner(t0), c1 = ranges.owner(t1 - 1);
    griddep_wait();
    if (c0 == c1) return;
    // the piece that starts at its unit's start lies in its CTA's second slot
    auto piece = [&](int c) { return pieces + (size_t)(2 * c + (c == c0 ? 1 : 0)) * kPiece<kUnitRows>; };
    if (c1 - c0 < kFew) {                                  // all loads at once, every thread forms the weights
        if (d >= a.dim) return;
        float m[kFew], l[kFew], o[kFew];
#pragma unroll
        for (int i = 0; i < kFew; ++i) {
            const float* p = piece(min(c0 + i, c1));
            m[i] = c0 + i <= c1 ? p[kUnitRows * kMixMaxDim + r] : neg_inf();
            l[i] = p[kUnitRows * kMixMaxDim + kUnitRows + r];
            o[i] = p[r * kMixMaxDim + d];
        }
        float top = m[0];
#pragma unroll
        for (int i = 1; i < kFew; ++i) top = fmaxf(top, m[i]);
        const float base = top == neg_inf() ? 0.f : top;
        float sum = 0.f, all = 0.f;
#pragma unroll
        for (int i = 0; i < kFew; ++i)
            if (c0 + i <= c1) {
                const float w = exp2f(m[i] - base);
                sum = fmaf(w, l[i], sum);
                all = fmaf(w, o[i], all);
            }
        Elem<T>::store(static_cast<T*>(a.out) + ((size_t)b * a.hq + h) * a.dim + d, all / sum);
        return;
    }
    float top = neg_inf();
    for (int c = c0 + d; c <= c1; c += kMixMaxDim) top = fmaxf(top, piece(c)[kUnitRows * kMixMaxDim + r]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if ((d & 31) == 0) red[0][d >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kMixMaxDim / 32; ++w) top = fmaxf(top, red[0][w]);
    const float base = top == neg_inf() ? 0.f : top;
    float l = 0.f;
    for (int c = c0 + d; c <= c1; c += kMixMaxDim) {
        const float* p = piece(c) + kUnitRows * kMixMaxDim;
        const float w = exp2f(p[r] - base);
        weight[c - c0] = w;
        l = fmaf(w, p[kUnitRows + r], l);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    if ((d & 31) == 0) red[1][d >> 5] = l;
    __syncthreads();
    if (d >= a.dim) return;
    l = red[1][0];
#pragma unroll
    for (int w = 1; w < kMixMaxDim / 32; ++w) l += red[1][w];
    float o = piece(c0)[r * kMixMaxDim + d] * weight[0];
#pragma unroll 8
    for (int c = c0 + 1; c <= c1; ++c)
        o = fmaf(pieces[(size_t)(2 * c) * kPiece<kUnitRows> + r * kMixMaxDim + d], weight[c - c0], o);
    Elem<T>::store(static_cast<T*>(a.out) + ((size_t)b * a.hq + h) * a.dim + d, o / l);
}

// CTAs of the decode kernel: as many as fit the GPU at once, no more than there can be tiles.
int decode_ctas(int batch, int capacity, int hq, int hkv, bool bf16)
{
    const Units un(hq, hkv, bf16 ? kRows : kRows32);
    const long long tiles = (long long)batch * un.per_row * ((capacity - 1) / kTile + 1);
    const long long fit = (long long)tc_sm_count() * (bf16 ? 2 : 3);
    return (int)(tiles < fit ? tiles : fit);
}

// [batch][capacity][heads][dim] bf16 in boxes of 64 dimensions x 64 positions of one head.  L2 fetches
// 256 bytes at a time only where they are one head's: with heads of at most 128 bytes the other half
// is another CTA's, perhaps much later (64 rows of 1500 positions, 16 heads of 64: 105 us -> 81 us;
// heads of 128 dimensions: 54.4 us at 256 and 54.5 us at 128).
bool cache_map(CUtensorMap* m, const void* p, const AttnDecodeArgs& a)
{
    const uint64_t row = (uint64_t)a.dim * 2, pos = row * a.hkv;
    const uint64_t dims[4] = {(uint64_t)a.dim, (uint64_t)a.hkv, (uint64_t)a.capacity, (uint64_t)a.batch};
    const uint64_t strides[3] = {row, pos, pos * a.capacity};
    const uint32_t box[4] = {64, 1, kTile, 1};
    return tc_encode_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, p, dims, strides, box, true,
                         a.dim <= 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

template <typename T, int kUnitRows>
cudaError_t launch_join(const AttnDecodeArgs& a, const float* pieces, int G, cudaStream_t s)
{
    return launch_dependent(attn_decode_join_kernel<T, kUnitRows>, dim3((unsigned)(a.batch * a.hq)), dim3(kMixMaxDim),
                            (size_t)G * sizeof(float), s, a, pieces, G);
}

template <int D, bool kHigh>
cudaError_t launch_bf16(const AttnDecodeArgs& a, float* pieces, cudaStream_t s)
{
    CacheMaps maps;
    if (!cache_map(&maps.k, a.k_cache, a) || !cache_map(&maps.v, a.v_cache, a)) return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(attn_decode_bf16_kernel<D, kHigh>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kBytes);
    if (e != cudaSuccess) return e;
    const int G = decode_ctas(a.batch, a.capacity, a.hq, a.hkv, true);
    e = launch_dependent(attn_decode_bf16_kernel<D, kHigh>, dim3(G), dim3(kThreads), Cfg<D>::kBytes, s, maps, a, pieces, device_error_word());
    return e != cudaSuccess ? e : launch_join<__nv_bfloat16, kRows>(a, pieces, G, s);
}

}  // namespace

size_t attn_decode_workspace(int batch, int capacity, int hq, int hkv, ssd_dtype_t dtype)
{
    const bool bf16 = dtype == SSD_BF16;
    return (size_t)decode_ctas(batch, capacity, hq, hkv, bf16) * 2 * (bf16 ? kPiece<kRows> : kPiece<kRows32>) * sizeof(float);
}

cudaError_t launch_attn_decode(const AttnDecodeArgs& a, ssd_dtype_t dtype, void* workspace, cudaStream_t s)
{
    float* pieces = static_cast<float*>(workspace);
    const bool high = a.hq / a.hkv > 8;
    if (dtype == SSD_BF16) {
        if (a.dim <= 64) return high ? launch_bf16<64, true>(a, pieces, s) : launch_bf16<64, false>(a, pieces, s);
        return high ? launch_bf16<128, true>(a, pieces, s) : launch_bf16<128, false>(a, pieces, s);
    }
    cudaError_t e = cudaFuncSetAttribute(attn_decode_f32_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes32);
    if (e != cudaSuccess) return e;
    const int G = decode_ctas(a.batch, a.capacity, a.hq, a.hkv, false);
    e = launch_dependent(attn_decode_f32_kernel, dim3(G), dim3(kThreads32), kBytes32, s, a, pieces, device_error_word());
    return e != cudaSuccess ? e : launch_join<float, kRows32>(a, pieces, G, s);
}

}  // namespace ssd
