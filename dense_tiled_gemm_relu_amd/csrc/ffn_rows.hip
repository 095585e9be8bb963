// Row-wise and element-wise kernels of the feed-forward operators: layer norm
// forward and backward, the gated projections' element-wise gradient, and the
// quantisation of rows to 8 bits.
#include "ffn.hpp"

namespace gemm_relu_hip {

namespace {

constexpr int kThreads = 256;

template <int DT> struct Elem;
template <> struct Elem<DT_F16> {
    using T = _Float16;
};
template <> struct Elem<DT_BF16> {
    using T = __bf16;
};
template <> struct Elem<DT_F32> {
    using T = float;
};

// Sum over the workgroup, the same value in every thread.
__device__ __forceinline__ float block_sum(float v, float* lds)
{
#pragma unroll
    for (int s = 32; s > 0; s >>= 1) v += __shfl_xor(v, s);
    __syncthreads();                      // earlier reads of lds are done
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}
__device__ __forceinline__ float block_max(float v, float* lds)
{
#pragma unroll
    for (int s = 32; s > 0; s >>= 1) v = fmaxf(v, __shfl_xor(v, s));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    return fmaxf(fmaxf(lds[0], lds[1]), fmaxf(lds[2], lds[3]));
}

// ------------------------------------------------------------- layer norm
// One workgroup per row: the mean, then the squares around it (so a large
// common offset costs no digits), then the output.
template <int DT, int WDT> __global__ void __launch_bounds__(kThreads) layer_norm_kernel(NormArgs a)
{
    using T = typename Elem<DT>::T;
    using W = typename Elem<WDT>::T;
    __shared__ float lds[4];
    const W* w = static_cast<const W*>(a.w);
    const W* b = static_cast<const W*>(a.b);
    for (size_t row = blockIdx.x; row < (size_t)a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * (size_t)a.x_stride;
    T* y = static_cast<T*>(a.y) + row * (size_t)a.cols;
    float s = 0.0f;
    for (int j = threadIdx.x; j < a.cols; j += kThreads) s += (float)x[j];
    const float mean = block_sum(s, lds) / (float)a.cols;
    float v = 0.0f;
    for (int j = threadIdx.x; j < a.cols; j += kThreads) {
        const float d = (float)x[j] - mean;
        v += d * d;
    }
    const float rstd = 1.0f / sqrtf(block_sum(v, lds) / (float)a.cols + a.eps);
    for (int j = threadIdx.x; j < a.cols; j += kThreads)
        y[j] = (T)(((float)x[j] - mean) * rstd * (float)w[j] + (b ? (float)b[j] : 0.0f));
    if (threadIdx.x == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
    }
    }
}

template <int DT, int WDT> __global__ void __launch_bounds__(kThreads) layer_norm_dx_kernel(NormArgs a)
{
    using T = typename Elem<DT>::T;
    using W = typename Elem<WDT>::T;
    __shared__ float lds[4];
    const W* w = static_cast<const W*>(a.w);
    for (size_t row = blockIdx.x; row < (size_t)a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * (size_t)a.x_stride;
    const T* dy = static_cast<const T*>(a.dy) + row * (size_t)a.dy_stride;
    T* dx = static_cast<T*>(a.dx) + row * (size_t)a.cols;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float s0 = 0.0f, s1 = 0.0f;
    for (int j = threadIdx.x; j < a.cols; j += kThreads) {
        const float c = (float)dy[j] * (float)w[j];
        s0 += c;
        s1 += c * (((float)x[j] - mean) * rstd);
    }
    s0 = block_sum(s0, lds) / (float)a.cols;
    s1 = block_sum(s1, lds) / (float)a.cols;
    for (int j = threadIdx.x; j < a.cols; j += kThreads) {
        const float c = (float)dy[j] * (float)w[j];
        dx[j] = (T)(rstd * (c - s0 - ((float)x[j] - mean) * rstd * s1));
    }
    }
}

// Column sums of one strip of rows: thread per column.
template <int DT> __global__ void __launch_bounds__(kThreads) layer_norm_strip_kernel(NormArgs a, int strip_rows)
{
    using T = typename Elem<DT>::T;
    const int j = blockIdx.x * kThreads + threadIdx.x;
    if (j >= a.cols) return;
    const int r0 = blockIdx.y * strip_rows, r1 = min(a.rows, r0 + strip_rows);
    float dw = 0.0f, db = 0.0f;
    for (int r = r0; r < r1; ++r) {
        const float g = (float)static_cast<const T*>(a.dy)[(size_t)r * (size_t)a.dy_stride + j];
        const float v = (float)static_cast<const T*>(a.x)[(size_t)r * (size_t)a.x_stride + j];
        dw += g * ((v - a.mean[r]) * a.rstd[r]);
        db += g;
    }
    float* p = a.partial + (size_t)blockIdx.y * 2 * (size_t)a.cols;
    p[j] = dw;
    p[a.cols + j] = db;
}

template <int WDT> __global__ void __launch_bounds__(kThreads) layer_norm_join_kernel(NormArgs a, int strips)
{
    using W = typename Elem<WDT>::T;
    const int j = blockIdx.x * kThreads + threadIdx.x;
    if (j >= a.cols) return;
    float dw = 0.0f, db = 0.0f;
    for (int s = 0; s < strips; ++s) {
        const float* p = a.partial + (size_t)s * 2 * (size_t)a.cols;
        dw += p[j];
        db += p[a.cols + j];
    }
    static_cast<W*>(a.dw)[j] = (W)dw;
    if (a.db) static_cast<W*>(a.db)[j] = (W)db;
}

// --------------------------------------------- gradient of act(g) u
// A 64 x 64 tile of (rows, hidden): dg and du go out row-major, and transposed
// through LDS.
template <int DT> __global__ void __launch_bounds__(kThreads) gated_grad_kernel(GatedGradArgs a)
{
    using T = typename Elem<DT>::T;
    __shared__ T tile[2][64][66];
    const int htiles = (a.hidden + 63) / 64;
    const int h0 = (int)(blockIdx.x % htiles) * 64, r0 = (int)(blockIdx.x / htiles) * 64;
    const int c = threadIdx.x & 63, q = threadIdx.x >> 6;
    if (a.flags && blockIdx.x == 0)
        for (int k = threadIdx.x; k < kSplitkFlagWords; k += kThreads) a.flags[k] = 0u;
    for (int k = q; k < 64; k += 4) {
        const int r = r0 + k, h = h0 + c;
        T dg = (T)0.0f, du = (T)0.0f;
        if (r < a.rows && h < a.hidden) {
            const float* gu = a.gu + (size_t)r * 2 * (size_t)a.hidden;
            const float d = (float)static_cast<const T*>(a.dh)[(size_t)r * (size_t)a.dh_stride + h];
            float value, slope;
            activation_slope(gu[h], a.act, value, slope);
            dg = (T)(d * gu[a.hidden + h] * slope);
            du = (T)(d * value);
            T* out = static_cast<T*>(a.dgu) + (size_t)r * (size_t)a.ld;
            out[h] = dg;
            out[a.hidden + h] = du;
        }
        tile[0][c][k] = dg;
        tile[1][c][k] = du;
    }
    __syncthreads();
    for (int k = q; k < 64; k += 4) {
        const int h = h0 + k, r = r0 + c;
        if (r < a.rows && h < a.hidden) {
            T* out = static_cast<T*>(a.dgu_t);
            out[(size_t)h * (size_t)a.ld_t + r] = tile[0][k][c];
            out[(size_t)(a.hidden + h) * (size_t)a.ld_t + r] = tile[1][k][c];
        }
    }
}

// ------------------------------------------------------- quantisation
// 127 x / max is formed as one fp32 division of the product 127 x.  For 16-bit x
// the product is exact and the quotient's distance from a rounding border is
// either zero or more than half an fp32 step, so the result is that of exact
// arithmetic.  A row whose largest value is near the top of the fp32 range is
// scaled down by a power of two first, so that 127 x stays finite.
template <int DT>
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(const void* xs, int64_t x_stride,
                                                                 signed char* qs, float* scale, int rows, int cols)
{
    using T = typename Elem<DT>::T;
    __shared__ float lds[4];
    for (size_t row = blockIdx.x; row < (size_t)rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(xs) + row * (size_t)x_stride;
    signed char* q = qs + row * (size_t)cols;
    float top = 0.0f, bad = 0.0f;
    for (int j = threadIdx.x; j < cols; j += kThreads) {
        const float v = fabsf((float)x[j]);
        top = fmaxf(top, v);
        bad = v < INFINITY ? bad : 1.0f;
    }
    top = block_max(top, lds);
    bad = block_max(bad, lds);
    const bool empty = bad > 0.0f || top == 0.0f;
    const float down = top > 0x1p120f ? 0x1p-8f : 1.0f;
    for (int j = threadIdx.x; j < cols; j += kThreads)
        q[j] = empty ? (signed char)0 : (signed char)(int)rintf(127.0f * ((float)x[j] * down) / (top * down));
    if (threadIdx.x == 0) scale[row] = bad > 0.0f ? NAN : top / 127.0f;
    }
}

template <class... A> hipError_t start(void (*kernel)(A...), dim3 grid, hipStream_t stream, A... args)
{
    void* params[] = {&args...};
    return hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, dim3(kThreads), params, 0, stream);
}

constexpr int kStripRows = 64, kMaxStrips = 1024;
constexpr int kMaxRowGrid = 1 << 20;     // workgroups of a row kernel; each takes rows that far apart
int row_grid(int rows) { return rows < kMaxRowGrid ? rows : kMaxRowGrid; }

}  // namespace

hipError_t launch_layer_norm(const NormArgs& a, int dt, int wdt, hipStream_t stream)
{
    const dim3 grid(row_grid(a.rows));
    if (dt == DT_F32) return start(&layer_norm_kernel<DT_F32, DT_F32>, grid, stream, a);
    if (dt == DT_F16)
        return wdt == DT_F32 ? start(&layer_norm_kernel<DT_F16, DT_F32>, grid, stream, a)
                             : start(&layer_norm_kernel<DT_F16, DT_F16>, grid, stream, a);
    return wdt == DT_F32 ? start(&layer_norm_kernel<DT_BF16, DT_F32>, grid, stream, a)
                         : start(&layer_norm_kernel<DT_BF16, DT_BF16>, grid, stream, a);
}

// strips of at least kStripRows rows, at most kMaxStrips of them
int layer_norm_strips(int64_t rows)
{
    const int64_t n = (rows + kStripRows - 1) / kStripRows;
    return (int)(n < kMaxStrips ? n : kMaxStrips);
}

hipError_t launch_layer_norm_backward(const NormArgs& a, int dt, int wdt, hipStream_t stream)
{
    const int strips = layer_norm_strips(a.rows), colblocks = (a.cols + kThreads - 1) / kThreads;
    hipError_t e = hipSuccess;
    if (a.rows > 0) {
        const dim3 grid(row_grid(a.rows)), sgrid(colblocks, strips);
        const int strip_rows = (a.rows + strips - 1) / strips;
        if (dt == DT_F32) {
            e = start(&layer_norm_dx_kernel<DT_F32, DT_F32>, grid, stream, a);
            if (e == hipSuccess) e = start(&layer_norm_strip_kernel<DT_F32>, sgrid, stream, a, strip_rows);
        } else if (dt == DT_F16) {
            e = wdt == DT_F32 ? start(&layer_norm_dx_kernel<DT_F16, DT_F32>, grid, stream, a)
                              : start(&layer_norm_dx_kernel<DT_F16, DT_F16>, grid, stream, a);
            if (e == hipSuccess) e = start(&layer_norm_strip_kernel<DT_F16>, sgrid, stream, a, strip_rows);
        } else {
            e = wdt == DT_F32 ? start(&layer_norm_dx_kernel<DT_BF16, DT_F32>, grid, stream, a)
                              : start(&layer_norm_dx_kernel<DT_BF16, DT_BF16>, grid, stream, a);
            if (e == hipSuccess) e = start(&layer_norm_strip_kernel<DT_BF16>, sgrid, stream, a, strip_rows);
        }
        if (e != hipSuccess) return e;
    }
    const dim3 jgrid(colblocks);
    if (wdt == DT_F32) return start(&layer_norm_join_kernel<DT_F32>, jgrid, stream, a, strips);
    if (wdt == DT_F16) return start(&layer_norm_join_kernel<DT_F16>, jgrid, stream, a, strips);
    return start(&layer_norm_join_kernel<DT_BF16>, jgrid, stream, a, strips);
}

hipError_t launch_gated_grad(const GatedGradArgs& a, int dt, hipStream_t stream)
{
    const dim3 grid((unsigned)((a.hidden + 63) / 64) * (unsigned)((a.rows + 63) / 64));
    return dt == DT_F16 ? start(&gated_grad_kernel<DT_F16>, grid, stream, a)
                        : start(&gated_grad_kernel<DT_BF16>, grid, stream, a);
}

hipError_t launch_quantize_rows(const void* x, int64_t x_stride, signed char* q, float* scale, int rows,
                                int cols, int dt, hipStream_t stream)
{
    const dim3 grid(row_grid(rows));
    if (dt == DT_F32) return start(&quantize_rows_kernel<DT_F32>, grid, stream, x, x_stride, q, scale, rows, cols);
    if (dt == DT_F16) return start(&quantize_rows_kernel<DT_F16>, grid, stream, x, x_stride, q, scale, rows, cols);
    return start(&quantize_rows_kernel<DT_BF16>, grid, stream, x, x_stride, q, scale, rows, cols);
}

}  // namespace gemm_relu_hip
