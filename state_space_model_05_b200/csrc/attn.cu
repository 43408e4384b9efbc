// Causal softmax attention with grouped heads over packed prompts on the CUDA cores, in fp32
// arithmetic: fp32 tensors, and bf16 ones with more than 128 query heads per key/value head.
//
//     o_t = sum_{s<=t} p_s v_s / sum_{s<=t} p_s,   p_s = exp(scale q_t.k_s - m),   m = max_s scale q_t.k_s
//
// Query head h reads key/value head h / (hq / hkv).  Keys are visited tile by tile with the
// running maximum m and sum of each row (one pass); exponentials are taken in base 2, with
// log2(e) folded into the scale.
//
// Bound by the fp32 units and by the shared memory that feeds them: a CTA takes 32 queries of one
// head, a thread 4 of them with 4 (of heads over 64 dimensions: 8) output columns, in packed pairs.  Tiles of 32
// queries rather than 64 fill the SMs with short prompts (1031 tokens, 8/2 heads of 64, two sequences:
// 47 us a call; floor 8 us at 72 TFLOP/s).  With ten times the tokens: 1.78 ms = 30.6 TFLOP/s, 43% of that rate,
// as a tile's loads and products take turns between barriers.  Heads of up to 64 dimensions on the kernel for 64: 83 us for one
// sequence of 1031, 117 us on the one for 128.
#include "mixers.cuh"
#include "prefill_tc.h"
#include "ptx.cuh"

namespace ssd {

namespace {

constexpr float kLog2e = 1.44269504088896341f;

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

// ================================================================ packed prompts, CUDA cores
// A CTA takes 32 queries of one head and walks the keys up to its diagonal, 64 at a time: small
// enough that a few hundred tokens fill the GPU and four CTAs share an SM, which hides the loads
// of one behind the products of another.  Products run on packed fp32 pairs: the scores' over
// pairs of dimensions, the outputs' over pairs of columns.
constexpr int kRows = 32;
constexpr int kKeys = 64;
constexpr int kThreads = 128;
constexpr int kLdP = kKeys + 4;

// `rows` rows of `cols` elements (a multiple of 4) as fp32 into padded shared rows, zeros past
// them.  (Rows of D + 4 floats: 16-byte reads of 8 rows hit 8 different bank quads.)
template <typename T, int D, int kCount>
__device__ __forceinline__ void load_rows(float* dst, const T* src, long long stride, int rows, int cols, float mul)
{
#pragma unroll 8
    for (int i = threadIdx.x; i < kCount * (D / 4); i += kThreads) {
        const int r = i / (D / 4), c = 4 * (i % (D / 4));
        float4 x = (r < rows && c < cols) ? load4<T>(src + (size_t)r * stride + c) : make_float4(0.f, 0.f, 0.f, 0.f);
        x.x *= mul; x.y *= mul; x.z *= mul; x.w *= mul;
        *reinterpret_cast<float4*>(dst + r * (D + 4) + c) = x;
    }
}

__device__ __forceinline__ float2 lo2(const float4& x) { return make_float2(x.x, x.y); }
__device__ __forceinline__ float2 hi2(const float4& x) { return make_float2(x.z, x.w); }

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
attn_prefill_kernel(const AttnArgs a, const Divisor block, int* err)
{
    constexpr int kLd = D + 4, kCols = D / 64;             // output columns per thread: 4 kCols
    extern __shared__ float sm[];
    float *sq = sm, *sk = sq + kRows * kLd, *sv = sk + kKeys * kLd, *sp = sv + kKeys * kLd;
    const int h = blockIdx.y, tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    ptx::griddep_wait();                                   // every input may come from the kernel before
    if (blockIdx.x == 0 && h == 0) check_offsets(a.cu, a.nseq, a.total, err);
    int seq, j, first, len;
    // the blocks with the most keys first
    if (!packed_block(a.cu, a.nseq, a.total, block, gridDim.x - 1 - blockIdx.x, err, &seq, &j, &first, &len)) return;
    if ((long long)j * kRows >= len) return;
    const int q0 = j * kRows, n = min(kRows, len - q0);
    const size_t t0 = (size_t)first + q0;
    const int hk = h / (a.hq / a.hkv), tiles = (q0 + n - 1) / kKeys + 1;
    load_rows<T, D, kRows>(sq, static_cast<const T*>(a.q) + t0 * a.q_stride + (size_t)h * a.dim, a.q_stride, n, a.dim,
                           a.scale * kLog2e);
    // thread: rows 4 ty + i, score columns tx + 16 jj, output columns 4 tx .. + 3 (and 64 more)
    float m[4], l[4];
    float2 acc[4][kCols][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = neg_inf();
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < kCols; ++c) acc[i][c][0] = acc[i][c][1] = make_float2(0.f, 0.f);
    }
    for (int kb = 0; kb < tiles; ++kb) {
        const size_t s0 = (size_t)first + (size_t)kb * kKeys;
        const int ns = min(kKeys, len - kb * kKeys);
        __syncthreads();
        load_rows<T, D, kKeys>(sk, static_cast<const T*>(a.k) + s0 * a.k_stride + (size_t)hk * a.dim, a.k_stride, ns, a.dim, 1.f);
        load_rows<T, D, kKeys>(sv, static_cast<const T*>(a.v) + s0 * a.v_stride + (size_t)hk * a.dim, a.v_stride, ns, a.dim, 1.f);
        __syncthreads();
        float2 p2[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int jj = 0; jj < 4; ++jj) p2[i][jj] = make_float2(0.f, 0.f);
#pragma unroll 2
        for (int d = 0; d < a.dim; d += 4) {
            float4 x[4], y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(sq + (4 * ty + i) * kLd + d);
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = *reinterpret_cast<const float4*>(sk + (tx + 16 * i) * kLd + d);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int jj = 0; jj < 4; ++jj)
                    p2[i][jj] = ptx::ffma2(hi2(x[i]), hi2(y[jj]), ptx::ffma2(lo2(x[i]), lo2(y[jj]), p2[i][jj]));
        }
        const int diag = q0 - kb * kKeys;                  // key s is seen from row t on: s <= t + diag
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = 4 * ty + i;
            float p[4], top = m[i];
#pragma unroll
            for (int jj = 0; jj < 4; ++jj) {
                p[jj] = tx + 16 * jj <= t + diag ? p2[i][jj].x + p2[i][jj].y : neg_inf();
                top = fmaxf(top, p[jj]);
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float base = top == neg_inf() ? 0.f : top;       // a row of -inf so far keeps p = 0
            const float keep = exp2f(m[i] - base);
            m[i] = top;
            float sum = 0.f;
#pragma unroll
            for (int jj = 0; jj < 4; ++jj) {
                const float x = exp2f(p[jj] - base);
                sum += x;
                sp[t * kLdP + tx + 16 * jj] = x;
            }
            l[i] = fmaf(l[i], keep, sum);
#pragma unroll
            for (int c = 0; c < kCols; ++c) {
                acc[i][c][0] = ptx::fmul2(acc[i][c][0], make_float2(keep, keep));
                acc[i][c][1] = ptx::fmul2(acc[i][c][1], make_float2(keep, keep));
            }
        }
        __syncwarp();                                              // a row's 16 threads are of one warp
        // keys that every row of the tile sees, four at a time; then those that some rows do not,
        // where a masked key's value must not be touched (0 x inf is not 0)
        const int whole = min(kKeys, max(0, diag + 1)) & ~3, last = min(ns, diag + n);
        int s = 0;
#pragma unroll 2
        for (; s < whole; s += 4) {
            float4 x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(sp + (4 * ty + i) * kLdP + s);
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int c = 0; c < kCols; ++c) {
                    const float4 v = *reinterpret_cast<const float4*>(sv + (s + e) * kLd + 64 * c + 4 * tx);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float w = e == 0 ? x[i].x : e == 1 ? x[i].y : e == 2 ? x[i].z : x[i].w;
                        acc[i][c][0] = ptx::ffma2(make_float2(w, w), lo2(v), acc[i][c][0]);
                        acc[i][c][1] = ptx::ffma2(make_float2(w, w), hi2(v), acc[i][c][1]);
                    }
                }
        }
        for (; s < last; ++s) {
#pragma unroll
            for (int c = 0; c < kCols; ++c) {
                const float4 v = *reinterpret_cast<const float4*>(sv + s * kLd + 64 * c + 4 * tx);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (s <= 4 * ty + i + diag) {
                        const float w = sp[(4 * ty + i) * kLdP + s];
                        acc[i][c][0] = ptx::ffma2(make_float2(w, w), lo2(v), acc[i][c][0]);
                        acc[i][c][1] = ptx::ffma2(make_float2(w, w), hi2(v), acc[i][c][1]);
                    }
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
        const float inv = 1.f / l[i];
        if (4 * ty + i < n) {
            T* o = static_cast<T*>(a.out) + ((t0 + 4 * ty + i) * a.hq + h) * a.dim;
#pragma unroll
            for (int c = 0; c < kCols; ++c) {
                const int col = 64 * c + 4 * tx;
                if (col < a.dim) {
                    Elem<T>::store(o + col + 0, inv * acc[i][c][0].x);
                    Elem<T>::store(o + col + 1, inv * acc[i][c][0].y);
                    Elem<T>::store(o + col + 2, inv * acc[i][c][1].x);
                    Elem<T>::store(o + col + 3, inv * acc[i][c][1].y);
                }
            }
        }
    }
}

template <typename T, int D>
cudaError_t prefill_d(const AttnArgs& a, cudaStream_t s)
{
    constexpr int kBytes = ((kRows + 2 * kKeys) * (D + 4) + kRows * kLdP) * 4;
    cudaError_t e = cudaFuncSetAttribute(attn_prefill_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)packed_blocks(a.total, a.nseq, kRows), (unsigned)a.hq);
    return launch_dependent(attn_prefill_kernel<T, D>, grid, dim3(kThreads), kBytes, s, a, Divisor(kRows), device_error_word());
}

template <typename T>
cudaError_t prefill_t(const AttnArgs& a, cudaStream_t s)
{
    return a.dim <= 64 ? prefill_d<T, 64>(a, s) : prefill_d<T, 128>(a, s);
}

}  // namespace

cudaError_t launch_attn_prefill_simt(const AttnArgs& a, ssd_dtype_t dtype, cudaStream_t s)
{
    return dtype == SSD_F32 ? prefill_t<float>(a, s) : prefill_t<__nv_bfloat16>(a, s);
}

}  // namespace ssd
