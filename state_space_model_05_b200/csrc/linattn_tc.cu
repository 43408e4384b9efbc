// Linear attention with a decay per head over packed prompts on the tensor cores (bf16,
// sm_100a): tcgen05.mma with accumulators in TMEM, operands staged by TMA.
//
//     S_t = g S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t,   g = exp(log_decay[h])
//
// in blocks of n <= 128 tokens with the carried state S (dk x dv) at the block's start:
//     o_t = scale (sum_{s<=t} g^(t-s) (q_t.k_s) v_s + g^(t+1) S^T q_t)
//     S  <- g^n S + sum_s k_s (g^(n-1-s) v_s)^T
// The decay does not depend on the tokens, so every factor comes from one table g^0 .. g^128.
//
// linattn_output_kernel: one CTA walks the blocks of one (segment, value head), the state in
// the state warps' registers (fp32).  A segment is a sequence, or `blocks` blocks of a long
// one; linattn_segment_kernel, launched before it when a sequence can be that long, forms
// every segment's own state from zero, and the walk starts from
// S = g^L (.. (g^L S_0 + U_0) ..) + U_(j-1).  Splitting costs a second read of k and v and
// buys segments for all SMs; the host picks the length (segment_blocks).
//
// Per block: S = Q K^T, masked and decayed into P (bf16, over S in TMEM), Yd = P V; Yo = Q S from
// the state's bf16 image; U = K^T V~ with V~ = g^(n-1-s) v_s.  V~ is carried as the sum of three
// bf16 numbers (24 bits), so that the state keeps fp32 accuracy; P and the state's image are
// rounded to bf16 once, each by at most half the output's own rounding step.
//
// Bound by the chain of one block's steps, of which an SM has one at a time: V~, U, the state, its image, Q S,
// the outputs.  No unit is full meanwhile (issue slots 49%, tensor pipe 25%, DRAM 32% in the output kernel):
// the roles wait for one another.  8192 tokens, 32 heads of 128 x 128: 129 to 132 us (segment kernel 44, output
// kernel 97, overlapped); all tensors once take 42 us.  dk and dv of up to 64 have kernels of their own: 8 x 1024
// tokens, 32 heads of 64 x 64: 68 us, 91 us on the ones for 128.
#include <cuda.h>

#include <cmath>

#include "mixers.cuh"
#include "prefill_tc.h"
#include "ptx.cuh"

namespace ssd {

using namespace ptx;

namespace {

constexpr int kBlk = 128;                                  // tokens per block
constexpr int kHalf = kBlk * 128;                          // 64 dimensions of a block's rows
constexpr int kConvThreads = 256;                          // threads that form a piece of V~
// Tokens of V~ formed at a time: a 16-byte chunk per thread.
template <int DV> constexpr int kPiece = kConvThreads * 8 / DV;
template <int DV> constexpr int kPieces = kBlk / kPiece<DV>;
constexpr int kPart = kConvThreads * 16;                   // bytes of one part of a piece: [dv / 64][tokens][128 bytes]
constexpr int kSlot = 3 * kPart;

// g^0 .. g^128 and, reversed, g^31 .. g^0
constexpr int kSub = 32;
struct Powers { float up[kBlk + 4]; float down[kSub]; };

__device__ __forceinline__ void fill_powers(Powers* p, float ld, int tid, int threads)
{
    for (int i = tid; i <= kBlk; i += threads) p->up[i] = decay_pow(ld, i);
    for (int i = tid; i < kSub; i += threads) p->down[i] = decay_pow(ld, kSub - 1 - i);
}

// A thread's chunk (eight elements of one token, s) of a piece of V, times w, as three bf16 parts:
// the product's 24 bits in three cuts of 8, so that the parts' sum is exactly the fp32 product.  (One
// that is not finite leaves NaN in the lower parts: own_state.)
__device__ __forceinline__ void split3(uint4 (&part)[3], const uint4& v, float w)
{
    const uint32_t in[4] = {v.x, v.y, v.z, v.w};
    uint32_t out[3][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float2 x = fmul2(make_float2(bf16lo(in[j]), bf16hi(in[j])), make_float2(w, w));
#pragma unroll
        for (int q = 0; q < 3; ++q) {
            const uint32_t a = __float_as_uint(x.x), b = __float_as_uint(x.y);
            out[q][j] = __byte_perm(a, b, 0x7632);         // the upper halves of both
            if (q < 2) x = ffma2(make_float2(__uint_as_float(a & 0xFFFF0000u), __uint_as_float(b & 0xFFFF0000u)), make_float2(-1.f, -1.f), x);
        }
    }
#pragma unroll
    for (int q = 0; q < 3; ++q) part[q] = make_uint4(out[q][0], out[q][1], out[q][2], out[q][3]);
}

// Where a thread's chunk of piece p lies in a block's tile (the swizzle permutes chunks within a
// row by the row's number mod 8, which the piece keeps), and the chunk's token.
template <int DV>
__device__ __forceinline__ uint4* piece_chunk(uint8_t* values, int p, int tid, int* token)
{
    constexpr int kRowChunks = kPiece<DV> * 8;             // chunks of a 64-dimension half
    const int half = tid / kRowChunks, i = tid % kRowChunks;
    *token = p * kPiece<DV> + (i >> 3);
    return reinterpret_cast<uint4*>(values + half * kHalf + p * kPiece<DV> * 128 + i * 16);
}

__device__ __forceinline__ void write_piece(uint8_t* slot, const uint4 (&part)[3], int tid)
{
#pragma unroll
    for (int q = 0; q < 3; ++q) *reinterpret_cast<uint4*>(slot + q * kPart + tid * 16) = part[q];
}

// The products of one piece: U (+)= K^T V~ over its tokens.
template <int DK, int DV>
__device__ __forceinline__ void issue_state(uint32_t tU, uint32_t keys, uint32_t conv, int p, bool fresh)
{
    constexpr uint32_t id = idesc_bf16_f32(128, DV, true, true);
    // (dk = 64: rows 64 .. 127 of the product, from what lies behind the keys, are never read)
    const uint64_t dK = smem_desc_sw128(keys + p * kPiece<DV> * 128, kHalf, 1024);
    const uint64_t dV = smem_desc_sw128(conv, kPiece<DV> * 128, 1024);
#pragma unroll
    for (int q = 0; q < 3; ++q)
#pragma unroll
        for (int ks = 0; ks < kPiece<DV> / 16; ++ks)
            umma_f16(tU, desc_advance(dK, ks * 2048), desc_advance(dV, q * kPart + ks * 2048), id, (fresh && q == 0 && ks == 0) ? 0u : 1u);
}

struct LinattnMaps { CUtensorMap q, k, v, out; };

// The segment of this CTA: sequence, segment within it, its first token and number of tokens.
struct Segment { int seq, j, first, start, len, seq_len; };

__device__ __forceinline__ bool this_segment(const LinattnArgs& a, int blocks, const Divisor& len_div, int unit, int* err, Segment* s)
{
    int first, len;
    if (!packed_block(a.cu, a.nseq, a.total, len_div, unit, err, &s->seq, &s->j, &first, &len)) return false;
    if (s->j > 0 && (long long)s->j * blocks * kBlk >= len) return false;
    s->start = s->j * blocks * kBlk;
    s->seq_len = len;
    s->len = min(blocks * kBlk, len - s->start);
    s->first = first + s->start;
    return true;
}

// Of a bf16 number in the lower 16 bits, or of an fp32 number's upper 16.
__device__ __forceinline__ bool not_finite(uint32_t bf16_bits) { return (bf16_bits & 0x7F80u) == 0x7F80u; }

// ---- states with infinities
// A product of an infinite value (whose lower parts are NaN) or key (which meets lower parts of zero) is
// NaN where the recurrence has an infinity.  So where four columns of a row of U are not all finite, they
// are formed again in fp32 on the CUDA cores, by one thread:
//     U = sum_s g^(n-1-s) (k_s v_s^T)   over n tokens from `first`.
// Rows and columns of the padding are zero.  Bound by the loads' latency, two tokens' at a time (four would
// cost the output kernel's state warps registers): about 25 us for a block with one such column.
__device__ __forceinline__ float4 own_state(const LinattnArgs& a, const Powers* pw, float ld, size_t first, int n, int h, int row, int col)
{
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row >= a.dk || col >= a.dv) return x;
    const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(a.k) + first * a.k_stride + (size_t)(h / (a.hv / a.hq)) * a.dk + row;
    const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.v) + first * a.v_stride + (size_t)h * a.dv + col;
    constexpr int kAtOnce = 2;
    float behind = 1.f;                                    // the decay over the whole blocks behind a token's
    int at = -1;                                           // their number
#pragma unroll 1
    for (int s0 = 0; s0 < n; s0 += kAtOnce) {
        float kk[kAtOnce];
        uint2 y[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const size_t s = min(s0 + i, n - 1);
            kk[i] = __bfloat162float(k[s * a.k_stride]);
            y[i] = *reinterpret_cast<const uint2*>(v + s * a.v_stride);
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int left = n - 1 - s0 - i;
            if (left < 0) break;
            if (left / kBlk != at) {
                at = left / kBlk;
                behind = decay_pow(ld, at * kBlk);
            }
            const float w = pw->up[left % kBlk] * behind;
            x.x = fmaf(w, kk[i] * bf16lo(y[i].x), x.x);
            x.y = fmaf(w, kk[i] * bf16hi(y[i].x), x.y);
            x.z = fmaf(w, kk[i] * bf16lo(y[i].y), x.z);
            x.w = fmaf(w, kk[i] * bf16hi(y[i].y), x.w);
        }
        if (x.x != x.x && x.y != x.y && x.z != x.z && x.w != x.w) break;
    }
    return x;
}

__device__ __forceinline__ bool finite4(const uint32_t (&u)[4])
{
    return !not_finite(u[0] >> 16) && !not_finite(u[1] >> 16) && !not_finite(u[2] >> 16) && !not_finite(u[3] >> 16);
}

// `columns` columns of U in TMEM, from `col` on, put right; a row per lane, by whole warps.
template <int DK, int columns>
__device__ __forceinline__ void mend_state(uint32_t tU, const LinattnArgs& a, const Powers* pw, float ld, size_t first, int n, int h, int row,
                                           int col)
{
#pragma unroll 1
    for (int c = 0; c < columns; c += 4) {
        uint32_t u[4];
        tmem_ld4(tU + c, u);
        tmem_wait_ld();
        if (row < DK && !finite4(u)) {
            const float4 x = own_state(a, pw, ld, first, n, h, row, col + c);
            u[0] = __float_as_uint(x.x); u[1] = __float_as_uint(x.y); u[2] = __float_as_uint(x.z); u[3] = __float_as_uint(x.w);
        }
        __syncwarp();
        tmem_st4(tU + c, u);
    }
    tmem_wait_st();
}

// Out of the way of the code that runs, where the registers allow a call (31 prompts of 128 x 64: 166 us with
// it in line, 163 us so).
template <int DK, int columns>
__device__ __noinline__ void mend_state_apart(uint32_t tU, const LinattnArgs& a, const Powers* pw, float ld, size_t first, int n, int h,
                                              int row, int col)
{
    mend_state<DK, columns>(tU, a, pw, ld, first, n, h, row, col);
}

// ================================================================ a segment's own state
constexpr int kSegThreads = 128 + 2 * kConvThreads, kSegStages = 2, kSegSlots = 4;   // two groups take turns at the pieces

template <int DK, int DV>
struct SegCfg {
    static constexpr int kKeys = DK / 64 * kHalf, kValues = DV / 64 * kHalf;
    static constexpr int kStage = kKeys + kValues;
    static constexpr int kConv = kSegStages * kStage;
    static constexpr int kPow = kConv + kSegSlots * kSlot;
    static constexpr int kBar = (kPow + (int)sizeof(Powers) + 7) / 8 * 8;
    static constexpr int kTm = kBar + (2 * kSegStages + 2 * kSegSlots + 1) * 8;
    static constexpr int kBytes = kTm + 16 + 1024;
    static_assert(kBytes <= 227 * 1024, "shared memory");
};

template <int DK, int DV>
__global__ void __launch_bounds__(kSegThreads, 1)
linattn_segment_kernel(const __grid_constant__ LinattnMaps maps, const __grid_constant__ LinattnArgs a, int blocks, const Divisor seg_div,
                       const Divisor hv_div, float4* __restrict__ states, int* err)
{
    using L = SegCfg<DK, DV>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::kBar);
    uint64_t *full = bars, *empty = full + kSegStages, *conv_full = empty + kSegStages, *conv_empty = conv_full + kSegSlots,
             *done = conv_empty + kSegSlots;
    uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + L::kTm);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::kTm + 4);
    Powers* pw = reinterpret_cast<Powers*>(sm + L::kPow);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int unit = hv_div.d > 1 ? hv_div.div(blockIdx.x) : (int)blockIdx.x, h = blockIdx.x - unit * a.hv;
    griddep_wait();                                        // every input may come from the kernel before
    Segment sg;
    if (!this_segment(a, blocks, seg_div, unit, err, &sg)) return;
    if (sg.seq_len - sg.start <= blocks * kBlk) {
        // the last segment of a sequence hands its state to no one; where the final states replace the
        // initial ones, it keeps the sequence's for the segments, some of which may start after
        // another has written the final state
        if (sg.j > 0 && a.init_states == a.final_states) {
            const size_t elems = (size_t)a.dk * a.dv;
            const float4* src = reinterpret_cast<const float4*>(a.init_states + ((size_t)sg.seq * a.hv + h) * elems);
            for (int i = threadIdx.x; i < (int)(elems / 4); i += kSegThreads) states[(size_t)blockIdx.x * (DK * DV / 4) + i] = src[i];
        }
        return;
    }

    if (tid == 0) {
        for (int s = 0; s < kSegStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < kSegSlots; ++s) {
            mbar_init(&conv_full[s], kConvThreads / 32);
            mbar_init(&conv_empty[s], 1);
        }
        mbar_init(done, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    const float ld = a.log_decay[h];
    fill_powers(pw, ld, tid, kSegThreads);
    if (warp == 1) {
        tmem_alloc(tslot, 128);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // (with this kernel's TMEM in hand: a CTA of the output kernel that shares the SM takes all that
    // is left of it and then waits for this kernel's end)
    griddep_launch_dependents();
    const uint32_t tmem = *tslot;
    auto wait = [&](uint64_t* bar, int phase) { return mbar_wait_compact(bar, phase & 1, err, abort_flag); };
    auto conv = [&](int n) { return sm + L::kConv + (n % kSegSlots) * kSlot; };

    if (warp == 0) {
        if (lane == 0) {
            const int hq = h / (a.hv / a.hq);
            for (int c = 0; c < blocks; ++c) {
                const int s = c % kSegStages;
                if (c >= kSegStages && !wait(&empty[s], c / kSegStages - 1)) break;
                uint8_t* st = sm + s * L::kStage;
                mbar_expect_tx(&full[s], L::kStage);
                for (int x = 0; x < DK; x += 64) tma_load_3d(st + x / 64 * kHalf, &maps.k, x, hq, sg.first + c * kBlk, &full[s]);
                for (int x = 0; x < DV; x += 64)
                    tma_load_3d(st + L::kKeys + x / 64 * kHalf, &maps.v, x, h, sg.first + c * kBlk, &full[s]);
            }
        }
    } else if (warp == 1) {
        if (elect_one()) {
            bool ok = true;
            for (int n = 0; n < blocks * kPieces<DV> && ok; ++n) {
                const int c = n / kPieces<DV>, p = n % kPieces<DV>;
                ok = wait(&conv_full[n % kSegSlots], n / kSegSlots);
                if (!ok) break;
                tc_fence_after();
                issue_state<DK, DV>(tmem, smem_u32(sm + (c % kSegStages) * L::kStage), smem_u32(conv(n)), p, n == 0);
                umma_commit(&conv_empty[n % kSegSlots]);
                if (p == kPieces<DV> - 1) umma_commit(&empty[c % kSegStages]);
            }
            umma_commit(done);
            wait(done, 0);                                 // no TMEM is released with products in flight
        }
    } else if (warp >= 4) {
        const int group = (tid - 128) / kConvThreads, ctid = (tid - 128) % kConvThreads;
        bool ok = true;
        for (int c = 0; c < blocks && ok; ++c) {
            ok = __all_sync(0xffffffffu, wait(&full[c % kSegStages], c / kSegStages));
            // weights from the segment's end: the products accumulate over all its blocks
            const float extra = decay_pow(ld, (blocks - 1 - c) * kBlk);
#pragma unroll 1
            for (int p = group; p < kPieces<DV>; p += 2) {
                const int n = c * kPieces<DV> + p;
                int t;
                uint4 part[3];
                const uint4 v = *piece_chunk<DV>(sm + (c % kSegStages) * L::kStage + L::kKeys, p, ctid, &t);
                split3(part, v, pw->up[kBlk - 1 - t] * extra);
                ok = ok && (n < kSegSlots || __all_sync(0xffffffffu, wait(&conv_empty[n % kSegSlots], n / kSegSlots - 1)));
                if (!ok) break;
                write_piece(conv(n), part, ctid);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&conv_full[n % kSegSlots]);
            }
        }
        if (__all_sync(0xffffffffu, ok && wait(done, 0))) {
            tc_fence_after();
            // quads of columns as [column quad][row]: consecutive lanes write consecutive quads
            const int row = (warp & 3) * 32 + lane, c0 = ((warp - 4) >> 2) * (DV / 4);
            float4* dst = states + (size_t)blockIdx.x * (DK * DV / 4);
#pragma unroll
            for (int q = 0; q < DV / 64; ++q) {
                uint32_t v[16];
                const uint32_t tU = tmem + ((uint32_t)((warp & 3) * 32) << 16) + c0 + 16 * q;
                tmem_ld16(tU, v);
                tmem_wait_ld();
                bool fine = true;
#pragma unroll
                for (int e = 0; e < 16; ++e) fine = fine && !not_finite(v[e] >> 16);
                if (__any_sync(0xffffffffu, row < DK && !fine)) {
                    mend_state<DK, 16>(tU, a, pw, ld, sg.first, blocks * kBlk, h, row, c0 + 16 * q);
                    tmem_ld16(tU, v);
                    tmem_wait_ld();
                }
                if (row < DK) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        dst[(c0 / 4 + 4 * q + e) * DK + row] =
                            make_float4(__uint_as_float(v[4 * e]), __uint_as_float(v[4 * e + 1]),
                                        __uint_as_float(v[4 * e + 2]), __uint_as_float(v[4 * e + 3]));
                }
            }
        }
    }
    settle(abort_flag);
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 128);
    }
}

// ================================================================ outputs and final states
constexpr int kOutThreads = 768;                           // TMA, 3 MMA, 8 + 8 for V~ (the latter for the state, too), 4 output warps
constexpr int kWarpConv = 4, kWarpState = 12, kWarpOut = 20;
constexpr int kConvSlots = 2;

template <int DK, int DV>
struct OutCfg {
    static constexpr int kKeys = DK / 64 * kHalf, kValues = DV / 64 * kHalf;
    static constexpr int kImage = DV / 64 * DK * 128;      // state as [dv / 64][dk rows][128 bytes]
    static constexpr int kQSlots = DK + DV <= 192 ? 2 : 1;
    static constexpr int kK = kQSlots * kKeys, kV = kK + 2 * kKeys, kImg = kV + 2 * kValues;
    static constexpr int kConv = kImg + kImage;
    static constexpr int kPow = kConv + kConvSlots * kSlot;
    static constexpr int kBar = (kPow + (int)sizeof(Powers) + 7) / 8 * 8;
    static constexpr int kTm = kBar + 32 * 8;
    static constexpr int kBytes = kTm + 64 + 1024;
    static_assert(kBytes <= 227 * 1024, "shared memory");
    // TMEM columns: scores (then P), the block's part, the carried part, the block's state
    static constexpr uint32_t kS = 0, kYd = 128, kYo = 256, kU = 384;
};

// Takes the values that are not finite out of a thread's chunks of a block's tile and marks their tokens
// (a bit each): P's zeros would not hide them from the rows before them.
template <int DV>
__device__ __forceinline__ void take_out_bad_values(uint8_t* values, int odd, int gt, unsigned* tokens)
{
#pragma unroll 1
    for (int p = odd; p < kPieces<DV>; p += 2) {
        int t;
        uint4* at = piece_chunk<DV>(values, p, gt, &t);
        const uint4 u = *at;
        uint32_t w[4] = {u.x, u.y, u.z, u.w}, fine = ~0u;
#pragma unroll
        for (int j = 0; j < 4; ++j) {                      // x 0 = 0: all ones in a finite half
            const __nv_bfloat162 zero = __float2bfloat162_rn(0.f);
            const uint32_t mask = __heq2_mask(__hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w[j]), zero), zero);
            w[j] &= mask;
            fine &= mask;
        }
        if (fine != ~0u) {
            *at = make_uint4(w[0], w[1], w[2], w[3]);
            atomicOr(&tokens[t >> 5], 1u << (t & 31));
        }
    }
}

// Adds those values, times their scores, to the staged outputs of row r (`row`, its 16-byte chunks
// permuted by the row): g^(r-s) (q_r.k_s) v_s from the tokens s <= r marked in `tokens`.  Only the sign
// of a score matters, or that it is zero.  Rare, and called by whole warps.
template <int DV>
__device__ __noinline__ void add_bad_values(const LinattnArgs& a, const Powers* pw, uint8_t* row, const unsigned* tokens, size_t base,
                                            int r, int rows, int h)
{
    auto chunk = [&](int ch) { return reinterpret_cast<uint4*>(row + (ch >> 3) * kHalf + (((ch & 7) ^ (r & 7)) << 4)); };
    // where every output is NaN already (a state that holds NaN), there is nothing to add
    bool all = true;
#pragma unroll 1
    for (int ch = 0; 8 * ch < a.dv && r < rows; ++ch) {
        const uint4 u = *chunk(ch);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) all = all && (w[j] & 0x7FFFu) > 0x7F80u && (w[j] >> 16 & 0x7FFFu) > 0x7F80u;
    }
    if (__all_sync(0xffffffffu, all)) return;
    const size_t hq = (size_t)(h / (a.hv / a.hq)) * a.dk;
    const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + (base + r) * a.q_stride + hq;
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
#pragma unroll 1
        for (unsigned left = tokens[i]; left; left &= left - 1) {
            const int s = 32 * i + __ffs(left) - 1;
            if (s > r || r >= rows) continue;
            const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(a.k) + (base + s) * a.k_stride + hq;
            const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.v) + (base + s) * a.v_stride + (size_t)h * a.dv;
            float score = 0.f;                             // formed where an infinity needs it
            bool formed = false;
#pragma unroll 1
            for (int ch = 0; 8 * ch < a.dv; ++ch) {
                const uint4 vv = *reinterpret_cast<const uint4*>(v + 8 * ch);
                const uint32_t x[4] = {vv.x, vv.y, vv.z, vv.w};
                bool any = false, inf = false;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    any |= not_finite(x[j]) || not_finite(x[j] >> 16);
                    inf |= (x[j] & 0x7FFFu) == 0x7F80u || (x[j] >> 16 & 0x7FFFu) == 0x7F80u;
                }
                if (!any) continue;
                if (inf && !formed) {
#pragma unroll 1
                    for (int d = 0; d < a.dk; d += 8) {
                        const uint4 qq = *reinterpret_cast<const uint4*>(q + d), kk = *reinterpret_cast<const uint4*>(k + d);
                        const uint32_t y[4] = {qq.x, qq.y, qq.z, qq.w}, z[4] = {kk.x, kk.y, kk.z, kk.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) score = fmaf(bf16hi(y[j]), bf16hi(z[j]), fmaf(bf16lo(y[j]), bf16lo(z[j]), score));
                    }
                    score *= pw->up[r - s];
                    formed = true;
                }
                uint4* at = chunk(ch);
                const uint4 u = *at;
                uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float lo = not_finite(x[j]) ? score * bf16lo(x[j]) * a.scale : 0.f;
                    const float hi = not_finite(x[j] >> 16) ? score * bf16hi(x[j]) * a.scale : 0.f;
                    w[j] = pack_bf16x2(bf16lo(w[j]) + lo, bf16hi(w[j]) + hi);
                }
                *at = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    }
}

template <int DK, int DV>
__global__ void __launch_bounds__(kOutThreads, 1)
linattn_output_kernel(const __grid_constant__ LinattnMaps maps, const __grid_constant__ LinattnArgs a, int blocks, const Divisor seg_div,
                      const Divisor hv_div, const float4* states, int* err)
{
    using L = OutCfg<DK, DV>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::kBar);
    uint64_t *q_full = bars, *q_empty = bars + 2, *k_full = bars + 4, *k_empty = bars + 6, *v_full = bars + 8,
             *v_empty = bars + 10, *v_ok = bars + 12, *s_full = bars + 14, *p_full = bars + 15, *yd_full = bars + 16,
             *yd_free = bars + 17, *yo_full = bars + 18, *yo_free = bars + 19, *img_full = bars + 20, *u_full = bars + 21,
             *u_free = bars + 22, *conv_full = bars + 23, *conv_empty = bars + 25, *v_used = bars + 27;
    uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + L::kTm);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::kTm + 4);
    volatile int* bad_block = reinterpret_cast<volatile int*>(sm + L::kTm + 8);      // [4], by block mod 4: something is not finite
    unsigned* bad_tokens = reinterpret_cast<unsigned*>(sm + L::kTm + 24);            // [2][4], by block mod 2
    Powers* pw = reinterpret_cast<Powers*>(sm + L::kPow);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int unit = hv_div.d > 1 ? hv_div.div(blockIdx.x) : (int)blockIdx.x, h = blockIdx.x - unit * a.hv;
    // after a segment kernel, first segments start while its last ones run; without one, every input may
    // come from the kernel before
    if (a.total <= blocks * kBlk) griddep_wait();
    if (blockIdx.x == 0) check_offsets(a.cu, a.nseq, a.total, err);
    Segment sg;
    if (!this_segment(a, blocks, seg_div, unit, err, &sg)) {
        griddep_wait();                                    // this grid ends after the one before, here and below
        return;
    }
    const int nb = (sg.len + kBlk - 1) / kBlk;             // 0 for an empty sequence
    const int last = sg.len - (nb - 1) * kBlk;             // tokens of the last block
    const bool ends = sg.start + sg.len >= sg.seq_len;     // this segment writes the final state

    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&q_full[s], 1);
            mbar_init(&q_empty[s], 2);
            mbar_init(&k_full[s], 1);
            mbar_init(&k_empty[s], 2);
            mbar_init(&v_full[s], 1);
            mbar_init(&v_empty[s], 1);
            mbar_init(&v_ok[s], 2 * kConvThreads / 32);
            mbar_init(&v_used[s], 1);
        }
        mbar_init(s_full, 1);
        mbar_init(p_full, 128);
        mbar_init(yd_full, 1);
        mbar_init(yd_free, 128);
        mbar_init(yo_full, 1);
        mbar_init(yo_free, 128);
        mbar_init(img_full, 8);
        mbar_init(u_full, 1);
        mbar_init(u_free, 8);
        for (int s = 0; s < kConvSlots; ++s) {
            mbar_init(&conv_full[s], kConvThreads / 32);
            mbar_init(&conv_empty[s], 1);
        }
        *abort_flag = 0;
        for (int i = 0; i < 4; ++i) bad_block[i] = 0;
        for (int i = 0; i < 8; ++i) bad_tokens[i] = 0u;
        fence_mbar_init();
    }
    const float ld = a.log_decay[h];
    fill_powers(pw, ld, tid, kOutThreads);
    if (warp == 1) {
        tmem_alloc(tslot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    auto wait = [&](uint64_t* bar, int phase) { return mbar_wait_compact(bar, phase & 1, err, abort_flag); };
    auto wait_warp = [&](uint64_t* bar, int phase) { return (bool)__all_sync(0xffffffffu, wait(bar, phase)); };
    auto qslot = [&](int c) { return sm + (c % L::kQSlots) * L::kKeys; };
    auto kslot = [&](int c) { return sm + L::kK + (c & 1) * L::kKeys; };
    auto vslot = [&](int c) { return sm + L::kV + (c & 1) * L::kValues; };
    auto tokens = [&](int c) { return c == nb - 1 ? last : kBlk; };
    constexpr int QS = L::kQSlots;
    // The pieces of block c's V~ whose number is `odd` mod 2, formed by 256 threads.  On the way the
    // values themselves are looked after: rows behind the sequence's end are another's and zeroed,
    // since 0 x inf is not 0; values that are not finite are taken out and left to the output warps, as
    // P's zeros would not hide them.
    auto weighted_values = [&](int c, int odd, int gt) {
        const int rows = tokens(c);
        const __nv_bfloat162 zero = __float2bfloat162_rn(0.f);
        __nv_bfloat162 acc[4] = {zero, zero, zero, zero};  // NaN as soon as one of its weighted values is not finite
        if (!wait_warp(&v_full[c & 1], c / 2)) return false;
        uint8_t* slot = sm + L::kConv + odd * kSlot;
#pragma unroll 1
        for (int p = odd; p < kPieces<DV>; p += 2) {
            int t;
            uint4* at = piece_chunk<DV>(vslot(c), p, gt, &t);
            uint4 v = *at, part[3];
            if (t >= rows) {
                v = make_uint4(0u, 0u, 0u, 0u);
                *at = v;
            }
            if (p * kPiece<DV> >= rows) continue;          // (the same for all threads)
            split3(part, v, t < rows ? pw->up[rows - 1 - t] : 0.f);
            const __nv_bfloat162* x = reinterpret_cast<const __nv_bfloat162*>(&part[0]);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] = __hfma2(x[e], zero, acc[e]);
            const int use = c * (kPieces<DV> / 2) + p / 2;
            if (use > 0 && !wait_warp(&conv_empty[odd], use - 1)) return false;
            write_piece(slot, part, gt);
            const int cut = (p + 1) * kPiece<DV> - rows;   // the piece's keys behind the sequence's end, zeroed alike
            if (cut > 0) {
                if (!wait_warp(&k_full[c & 1], c / 2)) return false;
                for (int i = gt; i < cut * (DK / 8); i += kConvThreads) {
                    const int ch = i % (DK / 8), row = rows + i / (DK / 8);
                    *reinterpret_cast<uint4*>(kslot(c) + (ch >> 3) * kHalf + row * 128 + (ch & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&conv_full[odd]);
        }
        const __nv_bfloat162 all = __hadd2(__hadd2(acc[0], acc[1]), __hadd2(acc[2], acc[3]));
        if (__builtin_expect(__hisnan(all.x) || __hisnan(all.y), 0)) {
            bad_block[c & 3] = c + 1;
            take_out_bad_values<DV>(vslot(c), odd, gt, bad_tokens + 4 * (c & 1));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_ok[c & 1]);
        return true;
    };

    // registers by role, together the 768 x 80 that the CTA was launched with
    if (warp < kWarpConv) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 0) {
        // ---------------------------------------------------------------- loads
        if (elect_one()) {
            const int hq = h / (a.hv / a.hq);
            auto load_kv = [&](int c) {
                const int row = sg.first + c * kBlk, s = c & 1;
                mbar_expect_tx(&k_full[s], L::kKeys);
                for (int x = 0; x < DK; x += 64) tma_load_3d(kslot(c) + x / 64 * kHalf, &maps.k, x, hq, row, &k_full[s]);
                mbar_expect_tx(&v_full[s], L::kValues);
                for (int x = 0; x < DV; x += 64) tma_load_3d(vslot(c) + x / 64 * kHalf, &maps.v, x, h, row, &v_full[s]);
                if (c >= QS)                               // queries that wait for their slot wait in the L2
                    for (int x = 0; x < DK; x += 64) tma_prefetch_3d(&maps.q, x, hq, row);
            };
            // a block's queries replace the block before's once its scores and carried part are formed,
            // which is before that block's keys and values make room for the next one's
            if (nb > 0) load_kv(0);
#pragma unroll 1
            for (int c = 0; c < nb; ++c) {
                if (c >= QS && !wait(&q_empty[c % QS], c / QS - 1)) break;
                mbar_expect_tx(&q_full[c % QS], L::kKeys);
                for (int x = 0; x < DK; x += 64)
                    tma_load_3d(qslot(c) + x / 64 * kHalf, &maps.q, x, hq, sg.first + c * kBlk, &q_full[c % QS]);
                if (c + 1 == nb) break;
                if (c >= 1 && !(wait(&k_empty[(c + 1) & 1], (c + 1) / 2 - 1) && wait(&v_empty[(c + 1) & 1], (c + 1) / 2 - 1))) break;
                load_kv(c + 1);
            }
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------- S = Q K^T, Yd = P V
        if (elect_one()) {
            constexpr uint32_t idS = idesc_bf16_f32(128, kBlk, false, false), idY = idesc_bf16_f32(128, DV, false, true);
            bool ok = true;
            for (int c = 0; c < nb && ok; ++c) {
                ok = wait(&q_full[c % QS], c / QS) && wait(&k_full[c & 1], c / 2) && (c == 0 || wait(yd_full, c - 1));
                if (!ok) break;
                tc_fence_after();
                const uint64_t dQ = smem_desc_sw128(smem_u32(qslot(c)), 16, 1024), dK = smem_desc_sw128(smem_u32(kslot(c)), 16, 1024);
#pragma unroll 1
                for (int ks = 0; ks < DK / 16; ++ks) {
                    const uint32_t off = (ks >> 2) * kHalf + (ks & 3) * 32;
                    umma_f16(tmem + L::kS, desc_advance(dQ, off), desc_advance(dK, off), idS, ks > 0 ? 1u : 0u);
                }
                umma_commit(&k_empty[c & 1]);
                umma_commit(&q_empty[c % QS]);
                umma_commit(s_full);
                ok = wait(&v_ok[c & 1], c / 2) && wait(p_full, c) && (c == 0 || wait(yd_free, c - 1));
                if (!ok) break;
                tc_fence_after();
                const uint64_t dV = smem_desc_sw128(smem_u32(vslot(c)), kHalf, 1024);
#pragma unroll 1
                for (int ks = 0; ks < kBlk / 16; ++ks)
                    umma_f16_ts(tmem + L::kYd, tmem + L::kS + ks * 8, desc_advance(dV, ks * 2048), idY, ks > 0 ? 1u : 0u);
                umma_commit(yd_full);
            }
            if (ok && nb > 0) wait(yd_full, nb - 1);       // no TMEM is released with products in flight
        }
    } else if (warp == 2) {
        // ---------------------------------------------------------------- Yo = Q S
        if (elect_one()) {
            constexpr uint32_t id = idesc_bf16_f32(128, DV, false, true);
            bool ok = true;
            for (int c = 0; c < nb && ok; ++c) {
                ok = wait(&q_full[c % QS], c / QS) && wait(img_full, c) && (c == 0 || wait(yo_free, c - 1));
                if (!ok) break;
                tc_fence_after();
                const uint64_t dQ = smem_desc_sw128(smem_u32(qslot(c)), 16, 1024);
                const uint64_t dS = smem_desc_sw128(smem_u32(sm + L::kImg), DK * 128, 1024);
#pragma unroll 1
                for (int ks = 0; ks < DK / 16; ++ks)
                    umma_f16(tmem + L::kYo, desc_advance(dQ, (ks >> 2) * kHalf + (ks & 3) * 32), desc_advance(dS, ks * 2048), id,
                             ks > 0 ? 1u : 0u);
                umma_commit(&q_empty[c % QS]);
                umma_commit(yo_full);
            }
            if (ok && nb > 0) wait(yo_full, nb - 1);
        }
    } else if (warp == 3) {
        // ---------------------------------------------------------------- U = K~^T V
        if (elect_one()) {
            bool ok = true;
            for (int c = 0; c < nb && ok; ++c) {
                const int pieces = (tokens(c) + kPiece<DV> - 1) / kPiece<DV>;
                ok = wait(&k_full[c & 1], c / 2);
#pragma unroll 1
                for (int p = 0; p < pieces; ++p) {         // piece p comes through slot p mod 2
                    ok = ok && wait(&conv_full[p & 1], c * (kPieces<DV> / 2) + p / 2) && (p > 0 || c == 0 || wait(u_free, c - 1));
                    if (!ok) break;
                    tc_fence_after();
                    issue_state<DK, DV>(tmem + L::kU, smem_u32(kslot(c)), smem_u32(sm + L::kConv + (p & 1) * kSlot), p, p == 0);
                    umma_commit(&conv_empty[p & 1]);
                }
                if (!ok) break;
                umma_commit(&k_empty[c & 1]);
                umma_commit(&v_used[c & 1]);
                ok = wait(&v_ok[c & 1], c / 2);            // what V~'s threads found is known before U is read
                if (!ok) break;
                umma_commit(u_full);
            }
            if (ok && nb > 0) wait(u_full, nb - 1);
        }
    }
    } else if (warp < kWarpState) {
        // ---------------------------------------------------------------- V~, even pieces
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        for (int c = 0; c < nb; ++c)
            if (!weighted_values(c, 0, tid - kWarpConv * 32)) break;
    } else if (warp < kWarpOut) {
        // ---------------------------------------------------------------- V~, odd pieces; the carried state
        asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
        constexpr int NC = DV / 2;                         // columns per thread
        const int quarter = warp & 3, row = quarter * 32 + lane, c0 = ((warp - kWarpState) >> 2) * NC;
        const bool mine = row < a.dk;
        float S[NC];
        const size_t at = (((size_t)sg.seq * a.hv + h) * a.dk + row) * a.dv + c0;
        const float* init = a.init_states ? a.init_states + at : nullptr;
        if (init && a.init_states == a.final_states && sg.seq_len > blocks * kBlk) {
            griddep_wait();                                // kept in the last segment's place (linattn_segment_kernel)
            const size_t place = blockIdx.x + (size_t)((sg.seq_len - 1) / (blocks * kBlk) - sg.j) * a.hv;
            init = reinterpret_cast<const float*>(states + place * (DK * DV / 4)) + (size_t)row * a.dv + c0;
        }
#pragma unroll
        for (int e = 0; e < NC; e += 4) {
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (init && mine && c0 + e < a.dv) x = *reinterpret_cast<const float4*>(init + e);
            S[e] = x.x; S[e + 1] = x.y; S[e + 2] = x.z; S[e + 3] = x.w;
        }
        if (sg.j > 0) {
            griddep_wait();                                // the segments' states come from the kernel before
            const float g = decay_pow(ld, blocks * kBlk);
            const float4* src = states + (size_t)(blockIdx.x - sg.j * a.hv) * (DK * DV / 4) + (c0 / 4) * DK + row;
            for (int i = 0; i < sg.j; ++i, src += (size_t)a.hv * (DK * DV / 4)) {
#pragma unroll
                for (int e = 0; e < NC; e += 4) {
                    const float4 u = row < DK ? src[e / 4 * DK] : make_float4(0.f, 0.f, 0.f, 0.f);
                    S[e] = fmaf(g, S[e], u.x);
                    S[e + 1] = fmaf(g, S[e + 1], u.y);
                    S[e + 2] = fmaf(g, S[e + 2], u.z);
                    S[e + 3] = fmaf(g, S[e + 3], u.w);
                }
            }
        }
        // bf16 image: row `row` of each 64-column half, 16-byte chunks permuted by the row
        auto write_image = [&]() {
            if (row < DK) {
#pragma unroll
                for (int e = 0; e < NC; e += 8) {
                    const int col = c0 + e;
                    *reinterpret_cast<uint4*>(sm + L::kImg + (col >> 6) * (DK * 128) + row * 128 + (((col & 63) >> 3) ^ (row & 7)) * 16) =
                        make_uint4(pack_bf16x2(S[e], S[e + 1]), pack_bf16x2(S[e + 2], S[e + 3]),
                                   pack_bf16x2(S[e + 4], S[e + 5]), pack_bf16x2(S[e + 6], S[e + 7]));
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(img_full);
        };
        if (nb > 0) write_image();
        bool ok = true;
        for (int c = 0; c < nb; ++c) {
            ok = weighted_values(c, 1, tid - kWarpState * 32) && wait_warp(u_full, c);
            if (!ok) break;
            tc_fence_after();
            // (a key that is not finite leaves a whole row of U so: one element tells)
            uint32_t one;
            tmem_ld1(tmem + ((uint32_t)(quarter * 32) << 16) + L::kU + c0, one);
            tmem_wait_ld();
            if (__builtin_expect(bad_block[c & 3] == c + 1 || __any_sync(0xffffffffu, row < DK && not_finite(one >> 16)), 0)) {
                const uint32_t tU = tmem + ((uint32_t)(quarter * 32) << 16) + L::kU + c0;
                const size_t base = sg.first + (size_t)c * kBlk;
                if constexpr (NC == 32)
                    mend_state_apart<DK, NC>(tU, a, pw, ld, base, tokens(c), h, row, c0);
                else
                    mend_state<DK, NC>(tU, a, pw, ld, base, tokens(c), h, row, c0);
            }
            const float g = pw->up[tokens(c)];
#pragma unroll
            for (int q = 0; q < NC / 16; ++q) {
                uint32_t v[16];
                tmem_ld16(tmem + ((uint32_t)(quarter * 32) << 16) + L::kU + c0 + 16 * q, v);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) S[16 * q + e] = fmaf(g, S[16 * q + e], __uint_as_float(v[e]));
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(u_free);
            if (c + 1 < nb) {
                ok = wait_warp(yo_full, c);                // the product that reads the image has completed
                if (!ok) break;
                write_image();
            }
        }
        if (ok && ends && mine) {
#pragma unroll
            for (int e = 0; e < NC; e += 4)
                if (c0 + e < a.dv)
                    *reinterpret_cast<float4*>(a.final_states + at + e) = make_float4(S[e], S[e + 1], S[e + 2], S[e + 3]);
        }
    } else {
        // ---------------------------------------------------------------- P, and the outputs
        asm volatile("setmaxnreg.inc.sync.aligned.u32 88;");
        const int quarter = warp & 3, r = quarter * 32 + lane;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        const float g_out = pw->up[r + 1];
        const bool leader = warp == kWarpOut && lane == 0;
        for (int c = 0; c < nb; ++c) {
            bool ok = wait_warp(s_full, c);
            tc_fence_after();
#pragma unroll 1
            for (int kc = 0; kc < 4; ++kc) {
                uint32_t pk[16];
                if (kc <= quarter) {                       // the same for the warp's 32 rows
                    uint32_t v[32];
                    tmem_ld32(tmem + lanes + L::kS + 32 * kc, v);
                    tmem_wait_ld();
                    if (kc < quarter) {
                        // g^(t-s) = g^(t-e) g^(e-s), e the last of these 32 columns
                        const float u = pw->up[r - 32 * kc - 31];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float4 w = *reinterpret_cast<const float4*>(&pw->down[4 * e]);
                            pk[2 * e] = pack_bf16x2(__uint_as_float(v[4 * e]) * (u * w.x), __uint_as_float(v[4 * e + 1]) * (u * w.y));
                            pk[2 * e + 1] = pack_bf16x2(__uint_as_float(v[4 * e + 2]) * (u * w.z), __uint_as_float(v[4 * e + 3]) * (u * w.w));
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float x = 2 * e <= lane ? __uint_as_float(v[2 * e]) * pw->up[lane - 2 * e] : 0.f;
                            const float y = 2 * e + 1 <= lane ? __uint_as_float(v[2 * e + 1]) * pw->up[lane - 2 * e - 1] : 0.f;
                            pk[e] = pack_bf16x2(x, y);
                        }
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) pk[e] = 0u;
                }
                // P over S: this warp has read these columns, and the ones after them lie further on
                tmem_st16(tmem + lanes + L::kS + 16 * kc, pk);
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(p_full);
            if (leader && c > 0) {                         // the last block's values may be replaced once its outputs are read
                bulk_wait_group_read0();
                mbar_arrive(&v_empty[(c - 1) & 1]);
            }
            // (after the block's state product, too, its values are not needed any more: a barrier
            // per value slot says so, as u_full may be a block further on by now)
            ok = ok && wait_warp(yd_full, c) && wait_warp(yo_full, c) && wait_warp(&v_used[c & 1], c / 2);
            tc_fence_after();
            const bool bad = bad_block[c & 3] == c + 1;
            const int rows = sg.len - c * kBlk;            // rows from here on belong to another sequence
            const size_t base = sg.first + (size_t)c * kBlk;
            // the outputs go over the block's values, in the layout that they were loaded in
            uint8_t* stage = vslot(c) + r * 128;
#pragma unroll 1
            for (int q = 0; q < DV / 32; ++q) {
                uint32_t yd[32], yo[32];
                tmem_ld32(tmem + lanes + L::kYd + 32 * q, yd);
                tmem_ld32(tmem + lanes + L::kYo + 32 * q, yo);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    uint32_t o[4];
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        const float2 y = fmul2(ffma2(make_float2(g_out, g_out),
                                                     make_float2(__uint_as_float(yo[e + 2 * z]), __uint_as_float(yo[e + 2 * z + 1])),
                                                     make_float2(__uint_as_float(yd[e + 2 * z]), __uint_as_float(yd[e + 2 * z + 1]))),
                                               make_float2(a.scale, a.scale));
                        o[z] = pack_bf16x2(y.x, y.y);
                    }
                    *reinterpret_cast<uint4*>(stage + (q >> 1) * kHalf + ((((q & 1) * 4 + e / 8) ^ (r & 7)) << 4)) =
                        make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
            if (__builtin_expect(bad, 0)) add_bad_values<DV>(a, pw, stage, bad_tokens + 4 * (c & 1), base, r, rows, h);
            tc_fence_before();
            mbar_arrive(yd_free);
            mbar_arrive(yo_free);
            fence_proxy_async_smem();
            if (!named_bar_and(1, 128, ok)) break;         // all four warps have staged theirs, or all stop
            if (__builtin_expect(bad && leader, 0))                             // (the slot's next values come once it has released it, below)
                for (int i = 0; i < 4; ++i) bad_tokens[4 * (c & 1) + i] = 0u;
            if (rows >= kBlk) {
                if (leader) {
                    for (int x = 0; x < DV; x += 64) tma_store_3d(&maps.out, x, h, (int)base, vslot(c) + x / 64 * kHalf);
                    bulk_commit_group();
                }
            } else {
                // the sequence's last rows: whole rows at a time
                constexpr int kChunks = DV / 8;
                const int ch = lane % kChunks;
#pragma unroll 2
                for (int k = 0; k < kChunks; ++k) {
                    const int row = quarter * 32 + k * (32 / kChunks) + lane / kChunks;
                    const uint4 v = *reinterpret_cast<const uint4*>(vslot(c) + (ch >> 3) * kHalf + row * 128 + (((ch & 7) ^ (row & 7)) << 4));
                    if (row < rows && 8 * ch < a.dv)
                        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + ((base + row) * a.hv + h) * a.dv + 8 * ch) = v;
                }
            }
        }
        if (leader) bulk_wait_group0();
    }
    settle(abort_flag);
    tc_fence_before();
    __syncthreads();
    griddep_wait();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------- host side
// Blocks per segment: the length that costs least.  Us of a CTA, all SMs busy: a block of 128 tokens
// 2.5 in the output kernel and 1.75 in the segment kernel, 6 and 2 more to start and end, 1 for a
// CTA that finds nothing to do, 1 to add a segment's state to the next one's.
// One sequence: whole waves of equal CTAs.  More: the host knows only their average length and takes
// the lengths as exponentially spread (a sequence goes on past k segments with probability
// e^(-k len / avg), the longest of n has avg (ln n + 0.6)); a kernel then takes its work shared
// evenly and a fifth of its longest CTA, at least that CTA.
// The costs are those of 128 x 128, taken for the other sizes too.  Measured, 128 x 128 in graphs: 1024 tokens,
// 8 heads: 23 us at the chosen 1 block, 43 us unsplit; 8192 tokens, 32 heads: 126 us at 16, 301 us unsplit; 31
// sequences cut at random from 16384 tokens, 32 heads: 233 us at 40, 223 us unsplit.  Of 27 shapes, 13 get the
// best of the lengths tried and 11 lose up to 11%; 64 sequences and 8 heads lose 13 to 21%, as the
// sequences alone would fill the SMs.
int segment_blocks(int nseq, int total, int hv)
{
    constexpr double kOut = 2.5, kOutCta = 6, kSeg = 1.75, kSegCta = 2, kIdle = 1, kJoin = 1, kTail = 0.2;
    const double sms = tc_sm_count();
    const long long all = max(1LL, ((long long)total + kBlk - 1) / kBlk), avg = max(1LL, ((long long)total / nseq + kBlk - 1) / kBlk);
    auto cost = [&](long long len) {
        const double launched = ((double)(total / (kBlk * len)) + nseq) * hv;      // CTAs, of either kernel
        const bool split = total > len * kBlk;
        double us;
        if (nseq == 1) {
            const double segs = (double)((avg + len - 1) / len);
            us = std::ceil(segs * hv / sms) * (kOut * min(len, avg) + kOutCta) + (segs - 1) * kJoin;
            if (split) us += std::ceil((segs - 1) * hv / sms) * (kSeg * len + kSegCta);
        } else {
            const double inner = (double)nseq * hv / (std::exp((double)len / avg) - 1), units = (double)nseq * hv + inner;
            auto even = [&](double work, double longest) { return max(work / sms + kTail * longest, longest); };
            us = even(all * hv * kOut + units * kOutCta + max(0.0, launched - units) * kIdle,
                      kOut * min((double)len, avg * (std::log((double)nseq) + 0.6)) + kOutCta) +
                 (avg + len - 1) / len * kJoin;
            if (split)
                us += even(inner * (kSeg * len + kSegCta) + max(0.0, launched - inner) * kIdle, min(1.0, inner / hv) * (kSeg * len + kSegCta));
        }
        return us;
    };
    long long best = avg;
    double least = cost(best);
    auto consider = [&](long long len) {
        const double us = cost(len);
        if (us < least) {
            least = us;
            best = len;
        }
    };
    // an average sequence in 2, 3, .. equal segments, each length once
    for (long long len = avg; len > 1;) {
        const long long segs = (avg + len - 2) / (len - 1);
        len = (avg + segs - 1) / segs;
        consider(len);
    }
    // and segments of several average sequences, while a sequence much longer than the others would
    // not keep one CTA at work for much longer than an SM's share of all blocks takes
    for (int m : {2, 3, 4, 6, 8, 12, 16})
        if (nseq > 1 && (m == 2 || avg * m * sms <= 1.5 * (double)all * hv)) consider(min(all, avg * m));
    return (int)best;
}

bool token_map(CUtensorMap* m, const void* p, int dim, int heads, int tokens, long long stride)
{
    const uint64_t dims[3] = {(uint64_t)dim, (uint64_t)heads, (uint64_t)tokens};
    const uint64_t strides[2] = {(uint64_t)dim * 2, (uint64_t)stride * 2};
    const uint32_t box[3] = {64, 1, kBlk};
    return tc_encode_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, p, dims, strides, box, true);
}

template <int DK, int DV>
cudaError_t launch_t(const LinattnArgs& a, float4* states, cudaStream_t s)
{
    LinattnMaps maps = {};
    if (a.total > 0 && (!token_map(&maps.q, a.q, a.dk, a.hq, a.total, a.q_stride) ||
                        !token_map(&maps.k, a.k, a.dk, a.hq, a.total, a.k_stride) ||
                        !token_map(&maps.v, a.v, a.dv, a.hv, a.total, a.v_stride) ||
                        !token_map(&maps.out, a.out, a.dv, a.hv, a.total, (long long)a.hv * a.dv)))
        return cudaErrorInvalidValue;
    const int blocks = segment_blocks(a.nseq, a.total, a.hv);
    const long long grid = (long long)packed_blocks(a.total, a.nseq, blocks * kBlk) * a.hv;
    if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
    const Divisor seg_div(blocks * kBlk), hv_div(a.hv);
    int* err = device_error_word();
    cudaError_t e = cudaSuccess;
    if (a.total > blocks * kBlk) {
        e = cudaFuncSetAttribute(linattn_segment_kernel<DK, DV>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 SegCfg<DK, DV>::kBytes);
        if (e != cudaSuccess) return e;
        e = launch_dependent(linattn_segment_kernel<DK, DV>, dim3((unsigned)grid), dim3(kSegThreads), SegCfg<DK, DV>::kBytes, s, maps, a,
                             blocks, seg_div, hv_div, states, err);
        if (e != cudaSuccess) return e;
    }
    e = cudaFuncSetAttribute(linattn_output_kernel<DK, DV>, cudaFuncAttributeMaxDynamicSharedMemorySize, OutCfg<DK, DV>::kBytes);
    if (e != cudaSuccess) return e;
    return launch_dependent(linattn_output_kernel<DK, DV>, dim3((unsigned)grid), dim3(kOutThreads), OutCfg<DK, DV>::kBytes, s, maps, a,
                            blocks, seg_div, hv_div, states, err);
}

}  // namespace

size_t linattn_tc_workspace(int nseq, int total, int hv, int dk, int dv)
{
    const int blocks = segment_blocks(nseq, total, hv);
    if (total <= blocks * kBlk) return 0;
    return (size_t)packed_blocks(total, nseq, blocks * kBlk) * hv * (dk <= 64 ? 64 : 128) * (dv <= 64 ? 64 : 128) * sizeof(float);
}

cudaError_t launch_linattn_prefill_tc(const LinattnArgs& a, void* workspace, cudaStream_t s)
{
    float4* states = static_cast<float4*>(workspace);
    if (a.dk <= 64) return a.dv <= 64 ? launch_t<64, 64>(a, states, s) : launch_t<64, 128>(a, states, s);
    return a.dv <= 64 ? launch_t<128, 64>(a, states, s) : launch_t<128, 128>(a, states, s);
}

}  // namespace ssd
