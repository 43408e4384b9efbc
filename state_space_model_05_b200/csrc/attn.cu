// Causal softmax attention with grouped heads over packed prompts on the CUDA cores, in fp32
// arithmetic: fp32 tensors, and bf16 ones with more than 128 query heads per key/value head.
//
//     o_t = sum_{s<=t} p_s v_s / sum_{s<=t} p_s,   p_s = exp(scale q_t.k_s - m),   m = max_s scale q_t.k_s
//
// Query head h reads key/value head h / (hq / hkv).  Keys are visited tile by tile with the
// running maximum m and sum of each row (one pass); exponentials are taken in base 2, with
// log2(e) folded into the scale.
#include "mixers.cuh"

namespace ssd {

namespace {

constexpr float kLog2e = 1.44269504088896341f;

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

// ================================================================ packed prompts, CUDA cores
// A CTA takes 64 queries of one head and walks the keys up to its diagonal, 64 at a time.
constexpr int kTok = 64;
constexpr int kThreads = 256;
constexpr int kLd = kMixMaxDim + 4;
constexpr int kLdP = kTok + 4;

template <typename T>
__device__ __forceinline__ void load_rows(float* dst, const T* src, long long stride, int rows, int cols, float mul)
{
    for (int i = threadIdx.x; i < kTok * (kMixMaxDim / 4); i += kThreads) {
        const int r = i / (kMixMaxDim / 4), c = 4 * (i % (kMixMaxDim / 4));
        float4 x = (r < rows && c < cols) ? load4<T>(src + (size_t)r * stride + c) : make_float4(0.f, 0.f, 0.f, 0.f);
        x.x *= mul; x.y *= mul; x.z *= mul; x.w *= mul;
        *reinterpret_cast<float4*>(dst + r * kLd + c) = x;
    }
}

__device__ __forceinline__ void fma4(float4& a, float s, const float4& b)
{
    a.x = fmaf(s, b.x, a.x); a.y = fmaf(s, b.y, a.y); a.z = fmaf(s, b.z, a.z); a.w = fmaf(s, b.w, a.w);
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
attn_prefill_kernel(const AttnArgs a, const Divisor block, int* err)
{
    extern __shared__ float sm[];
    float *sq = sm, *sk = sq + kTok * kLd, *sv = sk + kTok * kLd, *sp = sv + kTok * kLd;
    const int h = blockIdx.y, tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    if (blockIdx.x == 0 && h == 0) check_offsets(a.cu, a.nseq, a.total, err);
    int seq, j, first, len;
    // the blocks with the most keys first
    if (!packed_block(a.cu, a.nseq, a.total, block, gridDim.x - 1 - blockIdx.x, err, &seq, &j, &first, &len)) return;
    const int n = min(kTok, len - j * kTok);
    if (n <= 0) return;
    const size_t t0 = (size_t)first + (size_t)j * kTok;
    const int hk = h / (a.hq / a.hkv);
    load_rows<T>(sq, static_cast<const T*>(a.q) + t0 * a.q_stride + (size_t)h * a.dim, a.q_stride, n, a.dim,
                 a.scale * kLog2e);
    // thread: rows 4 ty + i, score columns tx + 16 jj, output columns 4 tx .. + 3 (and 64 more)
    float m[4], l[4];
    float4 acc[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = neg_inf();
        l[i] = 0.f;
        acc[i][0] = acc[i][1] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int kb = 0; kb <= j; ++kb) {
        const size_t s0 = (size_t)first + (size_t)kb * kTok;
        const int ns = min(kTok, len - kb * kTok);
        __syncthreads();
        load_rows<T>(sk, static_cast<const T*>(a.k) + s0 * a.k_stride + (size_t)hk * a.dim, a.k_stride, ns, a.dim, 1.f);
        load_rows<T>(sv, static_cast<const T*>(a.v) + s0 * a.v_stride + (size_t)hk * a.dim, a.v_stride, ns, a.dim, 1.f);
        __syncthreads();
        float p[4][4] = {};
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
                    p[i][jj] = fmaf(x[i].x, y[jj].x, fmaf(x[i].y, y[jj].y, fmaf(x[i].z, y[jj].z, fmaf(x[i].w, y[jj].w, p[i][jj]))));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = 4 * ty + i;
            float top = m[i];
#pragma unroll
            for (int jj = 0; jj < 4; ++jj) {
                if (kb == j && tx + 16 * jj > t) p[i][jj] = neg_inf();
                top = fmaxf(top, p[i][jj]);
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float base = top == neg_inf() ? 0.f : top;       // a row of -inf so far keeps p = 0
            const float keep = exp2f(m[i] - base);
            m[i] = top;
            float sum = 0.f;
#pragma unroll
            for (int jj = 0; jj < 4; ++jj) {
                const float x = exp2f(p[i][jj] - base);
                sum += x;
                sp[t * kLdP + tx + 16 * jj] = x;
            }
            l[i] = fmaf(l[i], keep, sum);
#pragma unroll
            for (int jj = 0; jj < 2; ++jj) {
                acc[i][jj].x *= keep; acc[i][jj].y *= keep; acc[i][jj].z *= keep; acc[i][jj].w *= keep;
            }
        }
        __syncwarp();                                              // a row's 16 threads are of one warp
        const int last = kb == j ? min(n, 4 * ty + 4) : kTok;
        for (int s = 0; s < last; ++s) {
            const float4 v0 = *reinterpret_cast<const float4*>(sv + s * kLd + 4 * tx);
            const float4 v1 = *reinterpret_cast<const float4*>(sv + s * kLd + 64 + 4 * tx);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (kb < j || s <= 4 * ty + i) {
                    const float x = sp[(4 * ty + i) * kLdP + s];
                    fma4(acc[i][0], x, v0);
                    fma4(acc[i][1], x, v1);
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
            for (int jj = 0; jj < 2; ++jj) {
                const int c = 64 * jj + 4 * tx;
                if (c < a.dim) {
                    Elem<T>::store(o + c + 0, inv * acc[i][jj].x);
                    Elem<T>::store(o + c + 1, inv * acc[i][jj].y);
                    Elem<T>::store(o + c + 2, inv * acc[i][jj].z);
                    Elem<T>::store(o + c + 3, inv * acc[i][jj].w);
                }
            }
        }
    }
}

template <typename T>
cudaError_t prefill_t(const AttnArgs& a, cudaStream_t s)
{
    constexpr int kBytes = (3 * kTok * kLd + kTok * kLdP) * 4;
    cudaError_t e = cudaFuncSetAttribute(attn_prefill_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    if (e != cudaSuccess) return e;
    const dim3 grid((unsigned)packed_blocks(a.total, a.nseq, kTok), (unsigned)a.hq);
    attn_prefill_kernel<T><<<grid, kThreads, kBytes, s>>>(a, Divisor(kTok), device_error_word());
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_prefill_simt(const AttnArgs& a, ssd_dtype_t dtype, cudaStream_t s)
{
    return dtype == SSD_F32 ? prefill_t<float>(a, s) : prefill_t<__nv_bfloat16>(a, s);
}

}  // namespace ssd
