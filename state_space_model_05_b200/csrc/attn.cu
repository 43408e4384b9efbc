// Causal softmax attention with grouped heads on the CUDA cores: packed prompts in fp32
// arithmetic, and one token per sequence against a cache.
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
attn_prefill_kernel(const AttnArgs a, int* err)
{
    extern __shared__ float sm[];
    float *sq = sm, *sk = sq + kTok * kLd, *sv = sk + kTok * kLd, *sp = sv + kTok * kLd;
    const int h = blockIdx.y, tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    if (blockIdx.x == 0 && h == 0) check_offsets(a.cu, a.nseq, a.total, err);
    int seq, j, first, len;
    // the blocks with the most keys first
    if (!packed_block(a.cu, a.nseq, a.total, kTok, gridDim.x - 1 - blockIdx.x, err, &seq, &j, &first, &len)) return;
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
    attn_prefill_kernel<T><<<grid, kThreads, kBytes, s>>>(a, device_error_word());
    return cudaGetLastError();
}

// ================================================================ one token against a cache
// The work is the cached rows, read once.  All (row b, key/value head, block of query heads)
// units are laid end to end in tiles of 64 positions, as many as each row's length needs, and
// every CTA takes an equal contiguous range of tiles, so that one long cache fills the GPU as
// well as many short ones do, whatever the capacity.  A unit inside one CTA's range is written
// at once; the pieces of a unit that is cut go to the workspace, with their maxima and sums,
// and a second kernel joins them in the order of the CTAs (the same order on every run).
constexpr int kTile = 64;                                  // positions per tile
constexpr int kDecThreads = 128;
constexpr int kDecRows = 8;                                // query heads per unit
constexpr int kPiece = kDecRows * (kMixMaxDim + 2);        // floats of one piece: O, then m, l per row
constexpr int kMaxCtas = 148 * 4;

__device__ __forceinline__ int row_tiles(int len, int capacity) { return len < 0 || len >= capacity ? 0 : len / kTile + 1; }

// Tiles of the rows before the row looked for, over the whole batch, found by the CTA's
// threads together.
struct Located { int b; long long before, total; };

// The row b that `want` names (by_row), or the row whose tiles hold tile `want` of the batch
// when every row's tiles are repeated `units` times.
__device__ inline Located locate(const int* __restrict__ lens, int batch, int capacity, int units, long long want,
                                 bool by_row, int* err)
{
    __shared__ long long part[kDecThreads];
    __shared__ Located found;
    const int tid = threadIdx.x, per = (batch + kDecThreads - 1) / kDecThreads;
    const int b0 = min(batch, tid * per), b1 = min(batch, b0 + per);
    long long sum = 0;
    bool bad = false;
    for (int b = b0; b < b1; ++b) {
        bad |= lens[b] >= capacity;
        sum += row_tiles(lens[b], capacity);
    }
    if (bad && err) record_error(err, SSD_ERR_SHAPE);
    part[tid] = sum;
    __syncthreads();
    long long before = 0, total = 0;
    for (int t = 0; t < kDecThreads; ++t) {
        if (t < tid) before += part[t];
        total += part[t];
    }
    if (tid == 0) found = Located{batch, total, total};
    __syncthreads();
    for (int b = b0; b < b1; ++b) {
        const int n = row_tiles(lens[b], capacity);
        if (by_row ? b == want : (want >= before * units && want < (before + n) * units)) found = Located{b, before, total};
        before += n;
    }
    __syncthreads();
    return found;
}

template <typename T>
__global__ void __launch_bounds__(kDecThreads)
attn_decode_kernel(const AttnDecodeArgs a, float* __restrict__ pieces, int* err)
{
    extern __shared__ float sm[];
    float *sk = sm, *sv = sk + kTile * kLd, *sq = sv + kTile * kLd, *sp = sq + kDecRows * kMixMaxDim;
    __shared__ float sm_m[kDecRows], sm_l[kDecRows], sm_keep[kDecRows];
    const int tid = threadIdx.x, group = a.hq / a.hkv, blocks = (group + kDecRows - 1) / kDecRows;
    const int units = a.hkv * blocks, c = blockIdx.x;
    // the range: total first, then the row of its first tile
    Located at = locate(a.lens, a.batch, a.capacity, units, 0, true, c == 0 ? err : nullptr);
    const long long W = at.total * units, G = min((long long)gridDim.x, W);   // no CTA's range is empty
    if (c >= G) return;
    const long long x0 = W * c / G, x1 = W * (c + 1) / G;
    __syncthreads();
    at = locate(a.lens, a.batch, a.capacity, units, x0, false, nullptr);
    int b = at.b;
    int len = a.lens[b], n = row_tiles(len, a.capacity);
    int u = (int)((x0 - at.before * units) / n), tile = (int)((x0 - at.before * units) % n);
    bool from_start = tile == 0;                           // the unit's first tile is in this range
    bool fresh = true;
    float acc[kDecRows];
    for (long long x = x0; x < x1; ++x) {
        const int hk = u / blocks, h0 = hk * group + (u % blocks) * kDecRows, rows = min(kDecRows, group - (u % blocks) * kDecRows);
        __syncthreads();
        if (fresh) {
            for (int i = tid; i < kDecRows * kMixMaxDim; i += kDecThreads) {
                const int r = i / kMixMaxDim, d = i % kMixMaxDim;
                sq[i] = (r < rows && d < a.dim)
                            ? Elem<T>::load(static_cast<const T*>(a.q) + ((size_t)b * a.hq + h0 + r) * a.dim + d) * (a.scale * kLog2e) : 0.f;
            }
            if (tid < kDecRows) {
                sm_m[tid] = neg_inf();
                sm_l[tid] = 0.f;
            }
#pragma unroll
            for (int r = 0; r < kDecRows; ++r) acc[r] = 0.f;
            fresh = false;
        }
        // keys and values of the tile; the new token's come from the inputs and join the cache
        const int p0 = tile * kTile, np = min(kTile, len + 1 - p0);
        for (int i = tid; i < kTile * (kMixMaxDim / 4); i += kDecThreads) {
            const int r = i / (kMixMaxDim / 4), d = 4 * (i % (kMixMaxDim / 4)), pos = p0 + r;
            float4 kk = make_float4(0.f, 0.f, 0.f, 0.f), vv = kk;
            if (r < np && d < a.dim) {
                const size_t row = (((size_t)b * a.capacity + pos) * a.hkv + hk) * a.dim + d;
                const size_t in = ((size_t)b * a.hkv + hk) * a.dim + d;
                kk = pos < len ? load4<T>(static_cast<const T*>(a.k_cache) + row) : load4<T>(static_cast<const T*>(a.k) + in);
                vv = pos < len ? load4<T>(static_cast<const T*>(a.v_cache) + row) : load4<T>(static_cast<const T*>(a.v) + in);
                if (pos == len && u % blocks == 0) {
                    T* kc = static_cast<T*>(a.k_cache) + row;
                    T* vc = static_cast<T*>(a.v_cache) + row;
                    Elem<T>::store(kc, kk.x); Elem<T>::store(kc + 1, kk.y); Elem<T>::store(kc + 2, kk.z); Elem<T>::store(kc + 3, kk.w);
                    Elem<T>::store(vc, vv.x); Elem<T>::store(vc + 1, vv.y); Elem<T>::store(vc + 2, vv.z); Elem<T>::store(vc + 3, vv.w);
                }
            }
            *reinterpret_cast<float4*>(sk + r * kLd + d) = kk;
            *reinterpret_cast<float4*>(sv + r * kLd + d) = vv;
        }
        __syncthreads();
        // scores: position tid % 64, query heads 4 (tid / 64) .. + 3
        {
            const int pos = tid % kTile, r0 = tid / kTile * (kDecRows / 2);
            float s[kDecRows / 2] = {};
            for (int d = 0; d < a.dim; d += 4) {
                const float4 y = *reinterpret_cast<const float4*>(sk + pos * kLd + d);
#pragma unroll
                for (int r = 0; r < kDecRows / 2; ++r) {
                    const float4 z = *reinterpret_cast<const float4*>(sq + (r0 + r) * kMixMaxDim + d);
                    s[r] = fmaf(z.x, y.x, fmaf(z.y, y.y, fmaf(z.z, y.z, fmaf(z.w, y.w, s[r]))));
                }
            }
#pragma unroll
            for (int r = 0; r < kDecRows / 2; ++r) sp[(r0 + r) * kLdP + pos] = pos < np ? s[r] : neg_inf();
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
        for (int r = 0; r < kDecRows; ++r) acc[r] *= sm_keep[r];
        for (int s = 0; s < np; ++s) {
            const float y = sv[s * kLd + tid];
#pragma unroll
            for (int r = 0; r < kDecRows; ++r) acc[r] = fmaf(sp[r * kLdP + s], y, acc[r]);
        }
        // the unit's end, or the range's
        const bool ends = tile == n - 1;
        if (ends || x + 1 == x1) {
            if (ends && from_start) {
                if (tid < a.dim)
                    for (int r = 0; r < rows; ++r)
                        Elem<T>::store(static_cast<T*>(a.out) + ((size_t)b * a.hq + h0 + r) * a.dim + tid, acc[r] / sm_l[r]);
            } else {
                float* p = pieces + (size_t)(2 * c + (from_start ? 1 : 0)) * kPiece;
#pragma unroll
                for (int r = 0; r < kDecRows; ++r) p[r * kMixMaxDim + tid] = acc[r];
                if (tid < kDecRows) {
                    p[kDecRows * kMixMaxDim + tid] = sm_m[tid];
                    p[kDecRows * kMixMaxDim + kDecRows + tid] = sm_l[tid];
                }
            }
            fresh = true;
            from_start = true;
        }
        if (++tile == n) {
            tile = 0;
            if (++u == units && x + 1 < x1) {
                u = 0;
                do ++b; while (row_tiles(a.lens[b], a.capacity) == 0);
                len = a.lens[b];
                n = row_tiles(len, a.capacity);
            }
        }
    }
}

// Joins the pieces of a unit that more than one CTA worked on.
template <typename T>
__global__ void __launch_bounds__(kDecThreads)
attn_decode_join_kernel(const AttnDecodeArgs a, const float* __restrict__ pieces, int ctas)
{
    const int group = a.hq / a.hkv, blocks = (group + kDecRows - 1) / kDecRows, units = a.hkv * blocks;
    const int b = blockIdx.x / units, u = blockIdx.x - b * units, tid = threadIdx.x;
    const Located at = locate(a.lens, a.batch, a.capacity, units, b, true, nullptr);
    const int n = row_tiles(a.lens[b], a.capacity);
    if (n == 0) return;
    const long long W = at.total * units, G = min((long long)ctas, W), t0 = at.before * units + (long long)u * n, t1 = t0 + n;
    auto owner = [&](long long t) {                        // the CTA whose range holds tile t
        long long c = t * G / W;
        while (W * (c + 1) / G <= t) ++c;
        return (int)c;
    };
    const int c0 = owner(t0), c1 = owner(t1 - 1);
    if (c0 == c1) return;
    const int h0 = (u / blocks) * group + (u % blocks) * kDecRows, rows = min(kDecRows, group - (u % blocks) * kDecRows);
    for (int r = 0; r < rows; ++r) {
        float m = neg_inf(), l = 0.f, o = 0.f;
        for (int c = c0; c <= c1; ++c) {
            // the piece that starts at its unit's start lies in its CTA's second slot
            const float* p = pieces + (size_t)(2 * c + (c == c0 ? 1 : 0)) * kPiece;
            const float pm = p[kDecRows * kMixMaxDim + r], pl = p[kDecRows * kMixMaxDim + kDecRows + r];
            const float top = fmaxf(m, pm), base = top == neg_inf() ? 0.f : top;
            const float keep = exp2f(m - base), add = exp2f(pm - base);
            o = o * keep + p[r * kMixMaxDim + tid] * add;
            l = l * keep + pl * add;
            m = top;
        }
        if (tid < a.dim) Elem<T>::store(static_cast<T*>(a.out) + ((size_t)b * a.hq + h0 + r) * a.dim + tid, o / l);
    }
}

// CTAs of the decode kernel: enough to fill the GPU, no more than there can be tiles.
int decode_ctas(int batch, int capacity, int hq, int hkv)
{
    const int group = hq / hkv;
    const long long tiles = (long long)batch * hkv * ((group + kDecRows - 1) / kDecRows) * ((capacity + kTile - 1) / kTile);
    return (int)(tiles < kMaxCtas ? tiles : kMaxCtas);
}

template <typename T>
cudaError_t decode_t(const AttnDecodeArgs& a, float* pieces, cudaStream_t s)
{
    constexpr int kBytes = (2 * kTile * kLd + kDecRows * kMixMaxDim + kDecRows * kLdP) * 4;
    cudaError_t e = cudaFuncSetAttribute(attn_decode_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    if (e != cudaSuccess) return e;
    const int G = decode_ctas(a.batch, a.capacity, a.hq, a.hkv), group = a.hq / a.hkv;
    attn_decode_kernel<T><<<G, kDecThreads, kBytes, s>>>(a, pieces, device_error_word());
    const unsigned units = (unsigned)(a.batch * a.hkv * ((group + kDecRows - 1) / kDecRows));
    attn_decode_join_kernel<T><<<units, kDecThreads, 0, s>>>(a, pieces, G);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_prefill_simt(const AttnArgs& a, ssd_dtype_t dtype, cudaStream_t s)
{
    return dtype == SSD_F32 ? prefill_t<float>(a, s) : prefill_t<__nv_bfloat16>(a, s);
}

size_t attn_decode_workspace(int batch, int capacity, int hq, int hkv, int dim)
{
    (void)dim;
    return (size_t)decode_ctas(batch, capacity, hq, hkv) * 2 * kPiece * sizeof(float);
}

cudaError_t launch_attn_decode(const AttnDecodeArgs& a, ssd_dtype_t dtype, void* workspace, cudaStream_t s)
{
    float* pieces = static_cast<float*>(workspace);
    return dtype == SSD_F32 ? decode_t<float>(a, pieces, s) : decode_t<__nv_bfloat16>(a, pieces, s);
}

}  // namespace ssd
