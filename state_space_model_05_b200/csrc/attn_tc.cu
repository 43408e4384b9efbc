// Causal softmax attention over packed prompts on the tensor cores (bf16, sm_100a):
// tcgen05.mma with scores, probabilities and outputs in TMEM, operands staged by TMA.
//
//     o_t = sum_{s<=t} p_s v_s / sum_{s<=t} p_s,   p_s = 2^(c q_t.k_s - m),   c = scale log2(e)
//
// A CTA takes 256 query rows of one key/value head at a time, as two tiles of 128 rows.  A row is a
// (token, query head of the group) pair, so the heads that share a key/value head share its
// loads and a tile spans 128 / group tokens, which also keeps the masked part of the last key
// tile small.  Keys are visited 128 at a time.  Per key tile i and query tile j:
//     S = Q_j K_i^T  (TMEM)  ->  softmax warps: row maximum, P = 2^(c S - m) as bf16 over S
//     O_j += P V_i   (TMEM, A operand from TMEM)
// Roles: four softmax warps per query tile (one thread per row), one warp that issues each
// tile's products, one TMA warp and one warp that looks after the values of the masked key tiles.
// While one tile's softmax runs, the tensor cores work for the other tile: the tiles take turns
// at the exponentials, since side by side both would wait for those and then for the products.
//
// The running maximum moves only when a row's scores exceed it by 2^8: until then p stays
// below 2^8 and nothing has to be rescaled; the sum and O use the same m, so the quotient is
// exact.  A move rescales O in TMEM by its own warp, which is safe because the barrier that
// announces S_i also covers P V_(i-1), issued before it.  P is rounded to bf16 (the operand type; its sum is
// taken before the rounding, in fp32), as is the output; everything else is fp32.
//
// Bound by the products and the exponentials together: per 128 x 128 scores the products took 770
// clocks at 64 dimensions and 1460 at 128 when timed alone, and 16384 exponentials take 1024 at 16 a
// clock.  Measured, 16384 tokens, 16/4 heads of 128: 832 us = 1.32 PFLOP/s at 1.9 GHz, 1.0 ms =
// 1.10 PFLOP/s under the power limit (a large library matrix product: 1.67 and 1.43).  32 x 512 tokens,
// 32/8 heads of 64: 93 us, 116 us at the clocks where one block per CTA took 164.  Without turns at the
// exponentials: 903 us instead of 832, 98 instead of 93.  Heads of up to 64 dimensions have tiles of 64,
// which leaves room for twice the slots: 8192 tokens, 32/8 heads: 370 us, 413 us on the tiles of 128.
#include <cuda.h>

#include "mixers.cuh"
#include "prefill_tc.h"
#include "ptx.cuh"

namespace ssd {

using namespace ptx;

namespace {

constexpr int kRows = 128;                                 // query rows per tile
constexpr int kKeys = 128;                                 // keys per tile
constexpr int kHalf = kKeys * 128;                         // one 64-dimension half of a tile, 128-byte rows
constexpr int kThreads = 384;                              // 8 softmax warps, TMA, 2 MMA, values
constexpr int kWarpTma = 8, kWarpMma = 9, kWarpValues = 11;
constexpr int kMaxMasked = 3;                              // key tiles that hold a diagonal of the block
constexpr int kFixedBars = 16 + 4 * kMaxMasked;            // barriers before those of the K and V tiles
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kSlack = 8.f;                              // log2 of the largest p before the maximum moves

template <int D>
struct Cfg {
    static constexpr int kHalves = D / 64;
    static constexpr int kTile = kHalves * kHalf;          // bytes of a Q, K or V tile
    static constexpr int kSlots = D == 128 ? 4 : 8;        // K and V tiles in flight
    static constexpr int kKv = 2 * kTile;
    static constexpr int kStage = kKv + kSlots * kTile;    // outputs on their way: 4 KB per softmax warp
    static constexpr int kBar = kStage + 8 * 4096;
    static constexpr int kItems = kBar + 48 * 8;           // the blocks being worked on
    static constexpr int kNext = kItems + 2 * 48;          // the launch control's answers
    static constexpr int kTm = kNext + 2 * 16;
    static constexpr int kBytes = kTm + 16 + 1024;
    // TMEM columns: two score tiles, two outputs
    static constexpr uint32_t kS = 0, kO = 256;
    static_assert(kBytes <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// Zeroes value rows from `rows` on (another sequence's) and looks for values that are not
// finite among the others: 0 x inf would carry them into rows that must not see them.  Those
// are zeroed too and reported, and the epilogue adds them where they belong.  A lane takes one
// 16-byte chunk of every fourth row (the swizzle permutes chunks within a row).
template <int D>
__device__ __forceinline__ bool fix_values(uint8_t* sv, int rows, int lane)
{
    const __nv_bfloat162 zero = __float2bfloat162_rn(0.f);
    __nv_bfloat162 acc[4] = {zero, zero, zero, zero};      // NaN as soon as one of its values is not finite
#pragma unroll 1
    for (int h = 0; h < D / 64; ++h) {
        uint4* p = reinterpret_cast<uint4*>(sv + h * kHalf) + lane;
        const int full = rows / 4;                         // groups of four rows that all count
#pragma unroll 8
        for (int k = 0; k < full; ++k) {
            const uint4 u = p[32 * k];
            const __nv_bfloat162* x = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[j] = __hfma2(x[j], zero, acc[j]);
        }
#pragma unroll 2
        for (int k = full; k < kKeys / 4; ++k) {
            if (4 * k + (lane >> 3) >= rows) {
                p[32 * k] = make_uint4(0u, 0u, 0u, 0u);
            } else {
                const uint4 u = p[32 * k];
                const __nv_bfloat162* x = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[j] = __hfma2(x[j], zero, acc[j]);
            }
        }
    }
    const __nv_bfloat162 all = __hadd2(__hadd2(acc[0], acc[1]), __hadd2(acc[2], acc[3]));
    const bool any = __any_sync(0xffffffffu, __hisnan(all.x) || __hisnan(all.y));
    if (any) {
#pragma unroll 1
        for (int i = lane; i < kKeys * (D / 8); i += 32) {
            uint4* p = reinterpret_cast<uint4*>(sv) + i;
            uint4 u = *p;
            uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if ((w[j] & 0x7F80u) == 0x7F80u) w[j] &= 0xFFFF0000u;
                if ((w[j] & 0x7F800000u) == 0x7F800000u) w[j] &= 0xFFFFu;
            }
            *p = u;
        }
    }
    return any;
}

constexpr float kNone = -__builtin_inff();

// One row's scores made ready for row_tile where they need it: keys past `limit` masked, and all
// times `c` (whole: every score, not only where the mask reaches).  A short loop of its own, so that
// row_tile's long code exists once: short prompts run it cold.
__device__ __forceinline__ void prepare_scores(uint32_t tS, float c, bool whole, int limit)
{
#pragma unroll 1
    for (int q = 0; q < kKeys / 32; ++q) {
        const int first = 32 * q;
        if (!whole && __all_sync(0xffffffffu, limit >= first + 31)) continue;
        uint32_t s[32];
        if (whole || __any_sync(0xffffffffu, limit >= first)) {
            tmem_ld32(tS + first, s);
            tmem_wait_ld();
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) s[e] = __float_as_uint(e <= limit - first ? __uint_as_float(s[e]) * c : kNone);
        tmem_st16(tS + first, reinterpret_cast<uint32_t(&)[16]>(s[0]));
        tmem_st16(tS + first + 16, reinterpret_cast<uint32_t(&)[16]>(s[16]));
    }
    tmem_wait_st();
}

// One row's softmax over one key tile: maximum, then P as bf16 over the scores in two parts
// of 64 keys, announced on p_full[0] and p_full[1]; m and l are the row's running maximum and sum.
// turn / next: named barriers before and after the exponentials (0: none).
template <int D>
__device__ __forceinline__ void row_tile(uint32_t tS, uint32_t tO, bool started, float mul, float& m, float& l, uint64_t* p_full,
                                         int turn, int next)
{
    uint32_t s[kKeys];
#pragma unroll
    for (int q = 0; q < 4; ++q) tmem_ld32(tS + 32 * q, reinterpret_cast<uint32_t(&)[32]>(s[32 * q]));
    tmem_wait_ld();
    float* x = reinterpret_cast<float*>(s);
    float top[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        top[q] = fmaxf(x[q], x[q + 8]);
#pragma unroll
        for (int e = 16; e < kKeys; e += 16) top[q] = max3(top[q], x[e + q], x[e + q + 8]);
    }
    const float now = max3(max3(top[0], top[1], top[2]), max3(top[3], top[4], top[5]), fmaxf(top[6], top[7])) * mul;
    float keep = 1.f;
    if (now > m + kSlack) {
        keep = ex2(m - now);                               // 0 from the initial -inf
        m = now;
        l *= keep;
    }
    if (started && __any_sync(0xffffffffu, keep != 1.f)) {
#pragma unroll 1
        for (int q = 0; q < D / 16; ++q) {
            uint32_t o[16];
            tmem_ld16(tO + 16 * q, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * keep);
            tmem_st16(tO + 16 * q, o);
        }
    }
    const float base = m == kNone ? 0.f : m;               // a row of -inf so far keeps p = 0
    const float2 mul2 = make_float2(mul, mul), base2 = make_float2(-base, -base);
    float2 sum[2] = {make_float2(l, 0.f), make_float2(0.f, 0.f)};
    if (turn) named_bar_sync(turn, 2 * kRows);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        uint32_t p[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const int k = 32 * q + 2 * e;
            float2 y = ffma2(make_float2(x[k], x[k + 1]), mul2, base2);
            y.x = ex2(y.x);
            y.y = ex2(y.y);
            sum[e & 1] = add2(sum[e & 1], y);
            p[e] = pack_bf16x2(y.x, y.y);
        }
        tmem_st16(tS + 16 * q, p);
        if (q == 2 && next) named_bar_arrive(next, 2 * kRows);
        if (q & 1) {
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&p_full[q >> 1]);
        }
    }
    const float2 both = add2(sum[0], sum[1]);
    l = both.x + both.y;
}

struct AttnMaps { CUtensorMap q, k, v; };

// Adds to eight outputs of a row (from dimension d0) the values that are not finite and that its
// token t may see, which were taken out of the masked key tiles named in `bad`: p > 0 times one
// of them is that value, whatever p is.
__device__ __noinline__ uint4 add_bad_values(const AttnArgs& a, uint4 out, int bad, int masked, int first, int t, int hk, int d0)
{
    uint32_t w[4] = {out.x, out.y, out.z, out.w};
    for (int i = masked; bad >> (i - masked); ++i) {
        if (!(bad >> (i - masked) & 1)) continue;
        for (int s = i * kKeys; s <= min(t, i * kKeys + kKeys - 1); ++s) {
            const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.v) +
                                                            (size_t)(first + s) * a.v_stride + (size_t)hk * a.dim + d0);
            const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float lo = bf16lo(x[e]), hi = bf16hi(x[e]), inf = __int_as_float(0x7f800000);
                if (!(fabsf(lo) < inf) || !(fabsf(hi) < inf))
                    w[e] = pack_bf16x2(bf16lo(w[e]) + (fabsf(lo) < inf ? 0.f : lo), bf16hi(w[e]) + (fabsf(hi) < inf ? 0.f : hi));
            }
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// One block of work: 2 x span tokens of one sequence, for one key/value head.
struct Item {
    int first, len;                                        // the sequence's first row and its length
    int t0, hk;                                            // first token, within the sequence; key/value head
    int nk0, nk1, masked;                                  // key tiles of the two query tiles; the first that reaches past some row's diagonal
    int bad;                                               // masked tiles (from `masked`) with values that are not finite
    int live;                                              // 0: no more work
};

// A CTA takes a block of work for its own number and then, one by one, blocks whose CTAs have not
// been launched yet (cluster launch control cancels their launch and hands over their numbers):
// the work stays balanced by the hardware, while the next block's loads and first scores run
// behind the current one's end.
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
attn_prefill_tc_kernel(const __grid_constant__ AttnMaps maps, const __grid_constant__ AttnArgs a, int group, int span, const Divisor block_div,
                       const Divisor hkv_div, int* err)
{
    using L = Cfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::kBar);
    uint64_t *item_full = bars, *item_empty = bars + 2, *q_empty = bars + 4, *next_full = bars + 5, *s_full = bars + 6,
             *p_full = bars + 8, *o_full = bars + 12, *o_free = bars + 14, *v_in = bars + 16, *v_ok = v_in + 2 * kMaxMasked,
             *full = bars + kFixedBars, *empty = full + L::kSlots;
    static_assert(kFixedBars + 2 * L::kSlots <= 48, "barriers");
    Item* items = reinterpret_cast<Item*>(sm + L::kItems);
    uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + L::kTm);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::kTm + 4);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (warp == kWarpTma) {
        if (lane < 3) prefetch_tensor_map(lane == 0 ? &maps.q : lane == 1 ? &maps.k : &maps.v);
        // arrivals per phase: an item's 8 softmax warps, 2 issuing threads and the values warp; a
        // tile's rows for P and for O's release; a thread per query tile for the loads' release
        for (int i = lane; i < kFixedBars + 2 * L::kSlots; i += 32)
            mbar_init(&bars[i], i == 2 || i == 3 ? 11 : i == 4 ? 2 : (i >= 8 && i < 12) || i == 14 || i == 15 ? kRows
                                : i >= kFixedBars + L::kSlots ? 2 : 1);
        if (lane == 0) *abort_flag = 0;
        fence_mbar_init();
    }
    // every input may come from the kernel before (and TMEM is not held while it may still need some)
    griddep_wait();
    if (warp == kWarpMma) {
        tmem_alloc(tslot, 512);
        tmem_relinquish();
    }
    if (blockIdx.x == 0) check_offsets(a.cu, a.nseq, a.total, err);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    auto kv = [&](int n) { return sm + L::kKv + (n % L::kSlots) * L::kTile; };   // tiles in the order of their loads: K_0 V_0 K_1 ..
    auto wait = [&](uint64_t* bar, int phase) { return mbar_wait_compact(bar, phase & 1, err, abort_flag); };
    auto poll = [&](uint64_t* bar, int phase) { return mbar_wait_compact<true>(bar, phase & 1, err, abort_flag); };

    // the softmax threads hold a row of scores each: 216 registers for them, 72 for the other
    // warps (together the 384 x 168 that the CTA was launched with)
    if (warp >= kWarpTma) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == kWarpTma) {
        // ---------------------------------------------------------------- blocks of work, and their loads
        const bool leader = elect_one();
        uint4* next = reinterpret_cast<uint4*>(sm + L::kNext);
        int cta = blockIdx.x, it = 0, n = 0;
        bool ok = true;
#pragma unroll 1
        for (int asked = 0; cta >= 0 && ok; ++asked) {
            // blocks with the most keys first, the key/value heads side by side
            const int place = gridDim.x - 1 - cta, blk = hkv_div.d > 1 ? hkv_div.div(place) : place, hk = place - blk * a.hkv;
            int seq, j0, first, len;
            const bool valid = packed_block(a.cu, a.nseq, a.total, block_div, blk, err, &seq, &j0, &first, &len);
            if (valid && (long long)j0 * 2 * span < len) {
                const int t0 = j0 * 2 * span;
                const int nk0 = (min(t0 + span, len) - 1) / kKeys + 1;
                const int nk1 = t0 + span < len ? (min(t0 + 2 * span, len) - 1) / kKeys + 1 : 0;
                const int nk = max(nk0, nk1), masked = (t0 + 1) / kKeys, slot = it & 1;
                ok = __all_sync(0xffffffffu, (it < 2 || wait(&item_empty[slot], it / 2 - 1)) && (it < 1 || wait(q_empty, it - 1)));
                if (ok && leader) {
                    items[slot] = Item{first, len, t0, hk, nk0, nk1, masked, 0, 1};
                    const int tiles = nk1 > 0 ? 2 : 1;
                    mbar_expect_tx(&item_full[slot], tiles * L::kHalves * 128 * group * span);
#pragma unroll 1
                    for (int j = 0; j < tiles; ++j)
                        for (int h = 0; h < L::kHalves; ++h)
                            tma_load_3d(sm + j * L::kTile + h * kHalf, &maps.q, 64 * h, hk * group, first + t0 + j * span, &item_full[slot]);
#pragma unroll 1
                    for (int k = 0; k < 2 * nk; ++k, ++n) {
                        uint64_t* turn = &full[n % L::kSlots];
                        if (n >= L::kSlots && !wait(&empty[n % L::kSlots], n / L::kSlots - 1)) {
                            ok = false;
                            break;
                        }
                        // a masked tile's values go to the values warp first, on barriers of their own, so
                        // that it need not follow the slots' phases (`full` then only marks the turn)
                        const bool to_fix = (k & 1) && (k >> 1) >= masked;
                        uint64_t* bar = to_fix ? &v_in[slot * kMaxMasked + (k >> 1) - masked] : turn;
                        mbar_expect_tx(bar, L::kTile);
                        for (int h = 0; h < L::kHalves; ++h)
                            tma_load_3d(kv(n) + h * kHalf, k & 1 ? &maps.v : &maps.k, 64 * h, hk, first + (k >> 1) * kKeys, bar);
                        if (to_fix) mbar_arrive(turn);
                    }
                }
                ok = __all_sync(0xffffffffu, ok);
                ++it;
            }
            if (!ok) break;
            // (asked for only now, with this block's loads under way: a block held in reserve any longer
            // would be missing where a CTA has run out of work)
            if (leader) {
                mbar_expect_tx(next_full, 16);
                launch_control_next(&next[asked & 1], next_full);
            }
            ok = __all_sync(0xffffffffu, wait(next_full, asked)) && ok;
            cta = ok ? launch_control_cta(next[asked & 1]) : -1;
        }
        // the end, as a block of its own (its place is free once the roles are done with what it held)
        const int slot = it & 1;
        ok = ok && __all_sync(0xffffffffu, it < 2 || wait(&item_empty[slot], it / 2 - 1));
        settle(abort_flag);
        if (ok) {
            if (leader) {
                items[slot].live = 0;
                mbar_arrive(&item_full[slot]);
            }
        }
    } else if (warp == kWarpMma || warp == kWarpMma + 1) {
        // A thread per query tile issues that tile's products: most of a thread's time goes into
        // the waits between them, which the other tile's products fill.
        if (elect_one()) {
            constexpr uint32_t idS = idesc_bf16_f32(128, kKeys, false, false);
            constexpr uint32_t idO = idesc_bf16_f32(128, D, false, true);
            const int j = warp - kWarpMma;
            const uint32_t tS = tmem + L::kS + j * 128, tO = tmem + L::kO + j * 128;
            const uint64_t dQ = smem_desc_sw128(smem_u32(sm + j * L::kTile), 16, 1024);
            int n = 0, scores = 0, outputs = 0;            // loads, score tiles and outputs so far
            uint32_t fixed = 0;                            // phase of each masked tile's barrier
            bool ok = true;
#pragma unroll 1
            for (int it = 0; ok; ++it) {
                ok = poll(&item_full[it & 1], it / 2);
                if (!ok || !items[it & 1].live) break;
                const Item& x = items[it & 1];
                const int nk = max(x.nk0, x.nk1), own = j ? x.nk1 : x.nk0, masked = x.masked;
                if (own == 0) mbar_arrive(q_empty);
#pragma unroll 1
                for (int i = -1; i < nk && ok; ++i) {
                    // V_i and K_(i+1), waited for before P_i is
                    const int nV = n + 2 * i + 1, nK = nV + 1;
                    const bool has_v = i >= 0, has_k = i + 1 < nk;
                    if (has_v) ok = poll(&full[nV % L::kSlots], nV / L::kSlots);
                    if (has_k) ok = ok && poll(&full[nK % L::kSlots], nK / L::kSlots);
                    if (has_v && i >= masked) {            // (by both threads, so that neither misses a phase)
                        const int k = (it & 1) * kMaxMasked + i - masked;
                        ok = ok && poll(&v_ok[k], fixed >> k);
                        fixed ^= 1u << k;
                    }
                    const uint64_t dK = smem_desc_sw128(smem_u32(kv(nK)), 16, 1024);
                    const uint64_t dV = smem_desc_sw128(smem_u32(kv(has_v ? nV : nK)), kHalf, 1024);
                    if (has_v && i < own) {                // O += P V_i, P in two parts of 64 keys
                        // (the block before's outputs have been read)
                        if (i == 0 && outputs > 0) ok = ok && poll(&o_free[j], outputs - 1);
#pragma unroll 1
                        for (int part = 0; part < 2; ++part) {
                            ok = ok && poll(&p_full[2 * j + part], scores);
                            if (!ok) break;
                            tc_fence_after();
#pragma unroll
                            for (int ks = 0; ks < kKeys / 32; ++ks)
                                umma_f16_ts(tO, tS + part * 32 + ks * 8, desc_advance(dV, part * 8192 + ks * 2048), idO,
                                            (i > 0 || part > 0 || ks > 0) ? 1u : 0u);
                        }
                        ++scores;
                    }
                    if (!ok) break;
                    if (i + 1 < own) {                     // S = Q K_(i+1)^T
                        // S over P: products of one thread run in the order of issue, so the one that
                        // reads P is done with it
                        tc_fence_after();
#pragma unroll
                        for (int ks = 0; ks < D / 16; ++ks) {
                            const uint32_t off = (ks >> 2) * kHalf + (ks & 3) * 32;
                            umma_f16(tS, desc_advance(dQ, off), desc_advance(dK, off), idS, ks > 0 ? 1u : 0u);
                        }
                        umma_commit(&s_full[j]);
                        if (i + 2 == own) umma_commit(q_empty);
                    }
                    if (has_v) umma_commit(&empty[nV % L::kSlots]);
                    if (has_k) umma_commit(&empty[nK % L::kSlots]);
                    if (has_v && i == own - 1) umma_commit(&o_full[j]);
                }
                n += 2 * nk;
                if (own > 0) ++outputs;
                mbar_arrive(&item_empty[it & 1]);
            }
            // no TMEM is released with products in flight
            if (outputs > 0) wait(&o_full[j], outputs - 1);
        }
    } else {
        // ---------------------------------------------------------------- values of masked tiles
        int n = 0;
        uint32_t fixed = 0;                                // phase of each masked tile's barrier
#pragma unroll 1
        for (int it = 0;; ++it) {
            if (!__all_sync(0xffffffffu, wait(&item_full[it & 1], it / 2)) || !items[it & 1].live) break;
            Item* x = &items[it & 1];
            const int nk = max(x->nk0, x->nk1), masked = x->masked, len = x->len;
            bool ok = true;
#pragma unroll 1
            for (int i = masked; i < nk && ok; ++i) {
                const int k = (it & 1) * kMaxMasked + i - masked;
                ok = __all_sync(0xffffffffu, wait(&v_in[k], fixed >> k));
                if (!ok) break;
                fixed ^= 1u << k;
                const bool bad = fix_values<D>(kv(n + 2 * i + 1), min(kKeys, len - i * kKeys), lane);
                if (bad && lane == 0) x->bad |= 1 << (i - masked);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&v_ok[k]);
            }
            if (!ok) break;
            n += 2 * nk;
            __syncwarp();
            if (lane == 0) mbar_arrive(&item_empty[it & 1]);
        }
    }
    } else {
        // ---------------------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int j = warp >> 2, r = tid & 127;            // query tile, row
        const int tok = r / group;                         // the row's token, within the tile
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lanes + L::kS + j * 128, tO = tmem + lanes + L::kO + j * 128;
        const float c = a.scale * kLog2e;
        const bool positive = c > 0.f;
        uint8_t* stage = sm + L::kStage + warp * 4096;
        int scores = 0, outputs = 0;                       // score tiles and outputs so far
        // A warp that gives up a wait does no more work but goes on taking its turns, block by
        // block, so that the other tile's warps are not left at a named barrier; for the same reason
        // the wait for a block does not end early when another wait has expired.
        bool ok = true;
#pragma unroll 1
        for (int it = 0;; ++it) {
            if (!__all_sync(0xffffffffu, mbar_wait(&item_full[it & 1], (it / 2) & 1, err)) || !items[it & 1].live) break;
            const Item* x = &items[it & 1];
            const int nk0 = x->nk0, nk1 = x->nk1, masked = x->masked, n_own = j ? nk1 : nk0;
            const int t = x->t0 + j * span + tok;          // the row's token, within the sequence
            const bool live = tok < span && t < x->len;
            float m = kNone, l = 0.f;
            // turns at the exponentials: tile 0 first, then 1, .. while both have key tiles left
            if (j == 1 && nk1 > 0) named_bar_arrive(1, 2 * kRows);
#pragma unroll 1
            for (int i = 0; i < n_own; ++i) {
                const int turn = nk1 > 0 && i < nk0 ? 1 + j : 0;
                const int next = nk1 > 0 && (j == 0 || i + 1 < nk0) ? 2 - j : 0;
                ok = ok && __all_sync(0xffffffffu, wait(&s_full[j], scores));
                ++scores;
                if (!ok) {
                    if (turn) named_bar_sync(turn, 2 * kRows);
                    if (next) named_bar_arrive(next, 2 * kRows);
                    continue;
                }
                tc_fence_after();
                // (a scale that is not positive is applied before the maximum)
                if (i >= masked || !positive) prepare_scores(tS, positive ? 1.f : c, !positive, i < masked ? kKeys : t - i * kKeys);
                row_tile<D>(tS, tO, i > 0, positive ? c : 1.f, m, l, &p_full[2 * j], turn, next);
            }
            if (n_own > 0) ok = ok && __all_sync(0xffffffffu, wait(&o_full[j], outputs++));
            if (n_own > 0 && ok) {
                tc_fence_after();
                const float inv = 1.f / l;
                const int bad = x->bad, first = x->first, hk = x->hk;
                // rows of the tile start at this (token, head); a row's place after it fits 32 bits
                // (128 tokens of 65535 heads of 128)
                const int to_row = live ? tok * a.hq + (r - tok * group) : -1;
                __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) +
                                     ((size_t)(first + x->t0 + j * span) * a.hq + (size_t)hk * group) * a.dim + 8 * (lane & 7);
                // 64 dimensions at a time go through shared memory, a row per thread, so that the global
                // stores are whole rows; 16-byte chunks are permuted by the row
#pragma unroll 1
                for (int h = 0; h < L::kHalves; ++h) {
#pragma unroll 1
                    for (int q = 0; q < 2; ++q) {
                        uint32_t o[32];
                        tmem_ld32(tO + 64 * h + 32 * q, o);
                        tmem_wait_ld();
                        float y[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) y[e] = __uint_as_float(o[e]) * inv;
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
                            *reinterpret_cast<uint4*>(stage + lane * 128 + (((4 * q + e / 8) ^ (lane & 7)) << 4)) =
                                make_uint4(pack_bf16x2(y[e], y[e + 1]), pack_bf16x2(y[e + 2], y[e + 3]),
                                           pack_bf16x2(y[e + 4], y[e + 5]), pack_bf16x2(y[e + 6], y[e + 7]));
                    }
                    if (h == L::kHalves - 1) {             // O may be replaced
                        tc_fence_before();
                        mbar_arrive(&o_free[j]);
                    }
                    if (bad) {
                        // (rare: the staged rows are corrected where they lie)
#pragma unroll 1
                        for (int c8 = 0; c8 < 8 && 64 * h + 8 * c8 < a.dim; ++c8) {
                            uint4* p = reinterpret_cast<uint4*>(stage + lane * 128 + ((c8 ^ (lane & 7)) << 4));
                            if (live) *p = add_bad_values(a, *p, bad, masked, first, t, hk, 64 * h + 8 * c8);
                        }
                    }
                    __syncwarp();
                    const bool inside = 64 * h + 8 * (lane & 7) < a.dim;
#pragma unroll 2
                    for (int k = 0; k < 8; ++k) {
                        const int row = 4 * k + (lane >> 3), to = __shfl_sync(0xffffffffu, to_row, row);
                        const uint4 v = *reinterpret_cast<const uint4*>(stage + row * 128 + (((lane & 7) ^ (row & 7)) << 4));
                        if (to >= 0 && inside) *reinterpret_cast<uint4*>(out + 64 * h + (size_t)(unsigned)(to * a.dim)) = v;
                    }
                    __syncwarp();
                }
            }
            if (lane == 0) mbar_arrive(&item_empty[it & 1]);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// [tokens][heads][dim] bf16 with `stride` elements between tokens, read in boxes of 64
// dimensions x `heads_box` heads x `tokens_box` tokens; what lies outside reads as zero.
bool token_map(CUtensorMap* m, const void* p, int dim, int heads, int tokens, long long stride, int heads_box, int tokens_box)
{
    const uint64_t dims[3] = {(uint64_t)dim, (uint64_t)heads, (uint64_t)tokens};
    const uint64_t strides[2] = {(uint64_t)dim * 2, (uint64_t)stride * 2};
    const uint32_t box[3] = {64, (uint32_t)heads_box, (uint32_t)tokens_box};
    return tc_encode_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, p, dims, strides, box, true);
}

template <int D>
cudaError_t launch_t(const AttnArgs& a, cudaStream_t s)
{
    const int group = a.hq / a.hkv, span = kRows / group;
    AttnMaps maps;
    if (!token_map(&maps.q, a.q, a.dim, a.hq, a.total, a.q_stride, group, span) ||
        !token_map(&maps.k, a.k, a.dim, a.hkv, a.total, a.k_stride, 1, kKeys) ||
        !token_map(&maps.v, a.v, a.dim, a.hkv, a.total, a.v_stride, 1, kKeys))
        return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(attn_prefill_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kBytes);
    if (e != cudaSuccess) return e;
    const long long grid = (long long)packed_blocks(a.total, a.nseq, 2 * span) * a.hkv;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    return launch_dependent(attn_prefill_tc_kernel<D>, dim3((unsigned)grid), dim3(kThreads), Cfg<D>::kBytes, s, maps, a, group, span,
                            Divisor(2 * span), Divisor(a.hkv), device_error_word());
}

}  // namespace

bool attn_tc_supported(const AttnArgs& a) { return a.hq / a.hkv <= kRows; }

cudaError_t launch_attn_prefill_tc(const AttnArgs& a, cudaStream_t s)
{
    return a.dim <= 64 ? launch_t<64>(a, s) : launch_t<128>(a, s);
}

}  // namespace ssd
