// Linear attention with a decay per head on the CUDA cores: the single-token step on the
// state, and the chunked prefill of fp32 tensors (bf16: linattn_tc.cu).
//
//     S_t = g S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t,   g = exp(log_decay[h])
//
// with S a dk x dv matrix per value head; value head h reads query/key head h / (hv / hq).
#include "mixers.cuh"

namespace ssd {

namespace {

// ================================================================ single-token step
// Bound by memory: 8 bytes of state traffic per element against 4 flops.  The columns of S
// are independent, so a CTA takes one (batch row, value head, block of columns); a thread
// owns 16 rows of 4 columns, issues those 16-byte loads before using any of them, updates
// and writes them back, and the partial sums of S^T q cross the row groups through shared
// memory once.
constexpr int kStepRows = 16;                              // rows per thread

template <typename T, int kCols>
__global__ void __launch_bounds__(kCols / 4 * (kMixMaxDim / kStepRows))
linattn_decode_kernel(float* __restrict__ state, const T* __restrict__ q, const T* __restrict__ k,
                      const T* __restrict__ v, const float* __restrict__ log_decay, T* __restrict__ out, int hq,
                      int hv, int dk, int dv, float scale)
{
    constexpr int kQuads = kCols / 4;
    constexpr int kGroups = kMixMaxDim / kStepRows;
    __shared__ float4 red[kGroups][kQuads];
    const int unit = blockIdx.x, b = unit / hv, h = unit - b * hv;
    const int cq = threadIdx.x % kQuads, rg = threadIdx.x / kQuads;
    const int c0 = blockIdx.y * kCols + 4 * cq, i0 = rg * kStepRows;
    const bool col = c0 < dv;
    float* S = state + (size_t)unit * dk * dv + c0;
    float4 s[kStepRows];
#pragma unroll
    for (int r = 0; r < kStepRows; ++r)
        s[r] = (col && i0 + r < dk) ? *reinterpret_cast<const float4*>(S + (size_t)(i0 + r) * dv)
                                    : make_float4(0.f, 0.f, 0.f, 0.f);
    const size_t qk = ((size_t)b * hq + h / (hv / hq)) * dk;
    const float g = expf(log_decay[h]);
    const float4 vv = col ? load4<T>(v + (size_t)unit * dv + c0) : make_float4(0.f, 0.f, 0.f, 0.f);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int r4 = 0; r4 < kStepRows; r4 += 4) {
        if (i0 + r4 < dk) {                                // dk is a multiple of 8
            const float4 k4 = load4<T>(k + qk + i0 + r4), q4 = load4<T>(q + qk + i0 + r4);
            const float kk[4] = {k4.x, k4.y, k4.z, k4.w}, qq[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float4& x = s[r4 + r];
                x.x = fmaf(kk[r], vv.x, g * x.x);
                x.y = fmaf(kk[r], vv.y, g * x.y);
                x.z = fmaf(kk[r], vv.z, g * x.z);
                x.w = fmaf(kk[r], vv.w, g * x.w);
                o.x = fmaf(qq[r], x.x, o.x);
                o.y = fmaf(qq[r], x.y, o.y);
                o.z = fmaf(qq[r], x.z, o.z);
                o.w = fmaf(qq[r], x.w, o.w);
                if (col) *reinterpret_cast<float4*>(S + (size_t)(i0 + r4 + r) * dv) = x;
            }
        }
    }
    red[rg][cq] = o;
    __syncthreads();
    if (rg == 0 && col) {
        float4 t = red[0][cq];
#pragma unroll
        for (int w = 1; w < kGroups; ++w) {
            const float4 a = red[w][cq];
            t.x += a.x; t.y += a.y; t.z += a.z; t.w += a.w;
        }
        T* p = out + (size_t)unit * dv + c0;
        Elem<T>::store(p + 0, scale * t.x);
        Elem<T>::store(p + 1, scale * t.y);
        Elem<T>::store(p + 2, scale * t.z);
        Elem<T>::store(p + 3, scale * t.w);
    }
}

template <typename T>
cudaError_t decode_t(float* state, const void* q, const void* k, const void* v, const float* log_decay, void* out,
                     int batch, int hq, int hv, int dk, int dv, float scale, cudaStream_t s)
{
    constexpr int kCols = 64;
    const dim3 grid((unsigned)(batch * hv), (unsigned)((dv + kCols - 1) / kCols));
    linattn_decode_kernel<T, kCols><<<grid, kCols / 4 * (kMixMaxDim / kStepRows), 0, s>>>(
        state, static_cast<const T*>(q), static_cast<const T*>(k), static_cast<const T*>(v), log_decay,
        static_cast<T*>(out), hq, hv, dk, dv, scale);
    return cudaGetLastError();
}

// ================================================================ chunked prefill, CUDA cores
// Blocks of 64 tokens in three launches: every block's own state U = sum_s g^(len-1-s) k_s v_s^T
// (all blocks in parallel), a scan that turns the U into start states and writes the final
// states, and every block's output  o_t = g^(t+1) S^T q_t + sum_{s<=t} g^(t-s) (q_t.k_s) v_s.
constexpr int kTok = 64;                                   // tokens per block
constexpr int kThreads = 256;
constexpr int kLd = kMixMaxDim + 4;                        // padded rows: 16-byte reads of 8 rows hit 8 bank quads
constexpr int kLdP = kTok + 4;

// `rows` rows of `cols` elements (a multiple of 4) into padded shared rows as fp32, zeros
// past them up to 64 x `width`.
template <typename T>
__device__ __forceinline__ void load_rows(float* dst, const T* src, long long stride, int rows, int cols, int width)
{
    const int quads = width / 4;
    for (int i = threadIdx.x; i < kTok * quads; i += kThreads) {
        const int r = i / quads, c = 4 * (i - r * quads);
        const float4 x = (r < rows && c < cols) ? load4<T>(src + (size_t)r * stride + c) : make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<float4*>(dst + r * kLd + c) = x;
    }
}

__device__ __forceinline__ void fma4(float4& a, float s, const float4& b)
{
    a.x = fmaf(s, b.x, a.x); a.y = fmaf(s, b.y, a.y); a.z = fmaf(s, b.z, a.z); a.w = fmaf(s, b.w, a.w);
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
linattn_block_state_kernel(const LinattnArgs a, const Divisor block, float* __restrict__ states, int* err)
{
    extern __shared__ float sm[];
    float *sk = sm, *sv = sm + kTok * kLd;
    const int h = blockIdx.y, tid = threadIdx.x;
    if (blockIdx.x == 0 && h == 0) check_offsets(a.cu, a.nseq, a.total, err);
    int seq, j, first, len;
    if (!packed_block(a.cu, a.nseq, a.total, block, blockIdx.x, err, &seq, &j, &first, &len)) return;
    const int n = min(kTok, len - j * kTok);
    if (n <= 0) return;
    const size_t t0 = (size_t)first + (size_t)j * kTok;
    const float ld = a.log_decay[h];
    load_rows<T>(sk, static_cast<const T*>(a.k) + t0 * a.k_stride + (size_t)(h / (a.hv / a.hq)) * a.dk, a.k_stride, n,
                 a.dk, kMixMaxDim);
    load_rows<T>(sv, static_cast<const T*>(a.v) + t0 * a.v_stride + (size_t)h * a.dv, a.v_stride, n, a.dv, kMixMaxDim);
    __syncthreads();
    // thread: rows 8 ty .. + 7, columns 4 tx .. + 3 and 64 + 4 tx .. + 3
    const int tx = tid & 15, ty = tid >> 4;
    float4 acc[8][2];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i][0] = acc[i][1] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s = 0; s < n; ++s) {
        const float w = decay_pow(ld, n - 1 - s);
        const float4 k0 = *reinterpret_cast<const float4*>(sk + s * kLd + 8 * ty);
        const float4 k1 = *reinterpret_cast<const float4*>(sk + s * kLd + 8 * ty + 4);
        const float4 v0 = *reinterpret_cast<const float4*>(sv + s * kLd + 4 * tx);
        const float4 v1 = *reinterpret_cast<const float4*>(sv + s * kLd + 64 + 4 * tx);
        const float kk[8] = {k0.x, k0.y, k0.z, k0.w, k1.x, k1.y, k1.z, k1.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            fma4(acc[i][0], w * kk[i], v0);
            fma4(acc[i][1], w * kk[i], v1);
        }
    }
    float* U = states + ((size_t)blockIdx.x * a.hv + h) * a.dk * a.dv;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = 8 * ty + i;
        if (r < a.dk) {
            if (4 * tx < a.dv) *reinterpret_cast<float4*>(U + (size_t)r * a.dv + 4 * tx) = acc[i][0];
            if (64 + 4 * tx < a.dv) *reinterpret_cast<float4*>(U + (size_t)r * a.dv + 64 + 4 * tx) = acc[i][1];
        }
    }
}

// Start state of every block (over its U) and the final state, four elements a thread.
__global__ void __launch_bounds__(kThreads)
linattn_scan_kernel(const LinattnArgs a, float* __restrict__ states, int* err)
{
    const int seq = blockIdx.x / a.hv, h = blockIdx.x - seq * a.hv;
    const int e = (blockIdx.y * kThreads + threadIdx.x) * 4, elems = a.dk * a.dv;
    if (e >= elems) return;
    const int first = a.cu[seq], len = a.cu[seq + 1] - first;
    if (first < 0 || len < 0 || first + len > a.total) return;      // reported by the blocks
    const float ld = a.log_decay[h];
    const size_t base = (size_t)blockIdx.x * elems + e;
    float4 H = a.init_states ? *reinterpret_cast<const float4*>(a.init_states + base) : make_float4(0.f, 0.f, 0.f, 0.f);
    float* U = states + ((size_t)(first / kTok + seq) * a.hv + h) * elems + e;
    const size_t step = (size_t)a.hv * elems;
    for (int t = 0; t < len; t += kTok, U += step) {
        const float4 u = *reinterpret_cast<const float4*>(U);
        *reinterpret_cast<float4*>(U) = H;
        const float g = decay_pow(ld, min(kTok, len - t));
        H.x = fmaf(g, H.x, u.x); H.y = fmaf(g, H.y, u.y); H.z = fmaf(g, H.z, u.z); H.w = fmaf(g, H.w, u.w);
    }
    *reinterpret_cast<float4*>(a.final_states + base) = H;
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
linattn_block_output_kernel(const LinattnArgs a, const Divisor block, const float* __restrict__ states, int* err)
{
    extern __shared__ float sm[];
    float *sq = sm, *sk = sq + kTok * kLd, *sv = sk + kTok * kLd, *sp = sv + kTok * kLd;
    const int h = blockIdx.y, tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    int seq, j, first, len;
    if (!packed_block(a.cu, a.nseq, a.total, block, blockIdx.x, err, &seq, &j, &first, &len)) return;
    const int n = min(kTok, len - j * kTok);
    if (n <= 0) return;
    const size_t t0 = (size_t)first + (size_t)j * kTok;
    const float ld = a.log_decay[h];
    const size_t hk = (size_t)(h / (a.hv / a.hq)) * a.dk;
    load_rows<T>(sq, static_cast<const T*>(a.q) + t0 * a.q_stride + hk, a.q_stride, n, a.dk, kMixMaxDim);
    load_rows<T>(sk, static_cast<const T*>(a.k) + t0 * a.k_stride + hk, a.k_stride, n, a.dk, kMixMaxDim);
    load_rows<T>(sv, static_cast<const T*>(a.v) + t0 * a.v_stride + (size_t)h * a.dv, a.v_stride, n, a.dv, kMixMaxDim);
    __syncthreads();
    // scores: thread rows t = 4 ty + i, columns s = tx + 16 jj
    float p[4][4] = {};
    for (int d = 0; d < a.dk; d += 4) {
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
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
            const int t = 4 * ty + i, s = tx + 16 * jj;
            sp[t * kLdP + s] = s <= t ? p[i][jj] * decay_pow(ld, t - s) : 0.f;
        }
    // the carried part: acc = S^T q, 64 rows of S at a time in the keys' place
    const float* S = states + ((size_t)blockIdx.x * a.hv + h) * a.dk * a.dv;
    float4 acc[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i][0] = acc[i][1] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int d0 = 0; d0 < a.dk; d0 += kTok) {
        __syncthreads();
        load_rows<float>(sk, S + (size_t)d0 * a.dv, a.dv, min(kTok, a.dk - d0), a.dv, kMixMaxDim);
        __syncthreads();
        for (int d = 0; d < min(kTok, a.dk - d0); ++d) {
            const float4 v0 = *reinterpret_cast<const float4*>(sk + d * kLd + 4 * tx);
            const float4 v1 = *reinterpret_cast<const float4*>(sk + d * kLd + 64 + 4 * tx);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = sq[(4 * ty + i) * kLd + d0 + d];
                fma4(acc[i][0], x, v0);
                fma4(acc[i][1], x, v1);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float g = decay_pow(ld, 4 * ty + i + 1);
#pragma unroll
        for (int jj = 0; jj < 2; ++jj) {
            float4& x = acc[i][jj];
            x.x *= g; x.y *= g; x.z *= g; x.w *= g;
        }
    }
    // the block's own part: rows s <= t of v
    for (int s = 0; s < min(n, 4 * ty + 4); ++s) {
        const float4 v0 = *reinterpret_cast<const float4*>(sv + s * kLd + 4 * tx);
        const float4 v1 = *reinterpret_cast<const float4*>(sv + s * kLd + 64 + 4 * tx);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (s <= 4 * ty + i) {
                const float x = sp[(4 * ty + i) * kLdP + s];
                fma4(acc[i][0], x, v0);
                fma4(acc[i][1], x, v1);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (4 * ty + i < n) {
            T* o = static_cast<T*>(a.out) + ((t0 + 4 * ty + i) * a.hv + h) * a.dv;
#pragma unroll
            for (int jj = 0; jj < 2; ++jj) {
                const int c = 64 * jj + 4 * tx;
                if (c < a.dv) {
                    Elem<T>::store(o + c + 0, a.scale * acc[i][jj].x);
                    Elem<T>::store(o + c + 1, a.scale * acc[i][jj].y);
                    Elem<T>::store(o + c + 2, a.scale * acc[i][jj].z);
                    Elem<T>::store(o + c + 3, a.scale * acc[i][jj].w);
                }
            }
        }
    }
}

template <typename T>
cudaError_t prefill_t(const LinattnArgs& a, float* states, cudaStream_t s)
{
    constexpr int kStateBytes = 2 * kTok * kLd * 4, kOutBytes = (3 * kTok * kLd + kTok * kLdP) * 4;
    cudaError_t e = cudaFuncSetAttribute(linattn_block_state_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kStateBytes);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(linattn_block_output_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kOutBytes);
    if (e != cudaSuccess) return e;
    int* err = device_error_word();
    const dim3 grid((unsigned)packed_blocks(a.total, a.nseq, kTok), (unsigned)a.hv);
    linattn_block_state_kernel<T><<<grid, kThreads, kStateBytes, s>>>(a, Divisor(kTok), states, err);
    const dim3 scan((unsigned)(a.nseq * a.hv), (unsigned)((a.dk * a.dv + 4 * kThreads - 1) / (4 * kThreads)));
    linattn_scan_kernel<<<scan, kThreads, 0, s>>>(a, states, err);
    if (a.total > 0) linattn_block_output_kernel<T><<<grid, kThreads, kOutBytes, s>>>(a, Divisor(kTok), states, err);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_linattn_decode(ssd_dtype_t dtype, float* state, const void* q, const void* k, const void* v,
                                  const float* log_decay, void* out, int batch, int hq, int hv, int dk, int dv,
                                  float scale, cudaStream_t s)
{
    return dtype == SSD_F32 ? decode_t<float>(state, q, k, v, log_decay, out, batch, hq, hv, dk, dv, scale, s)
                            : decode_t<__nv_bfloat16>(state, q, k, v, log_decay, out, batch, hq, hv, dk, dv, scale, s);
}

size_t linattn_simt_workspace(int nseq, int total, int hv, int dk, int dv)
{
    return (size_t)packed_blocks(total, nseq, kTok) * hv * dk * dv * sizeof(float);
}

cudaError_t launch_linattn_prefill_simt(const LinattnArgs& a, void* workspace, cudaStream_t s)
{
    return prefill_t<float>(a, static_cast<float*>(workspace), s);
}

}  // namespace ssd
