// Orthogonalisation of a matrix by Newton-Schulz steps X <- a X + (b A + c A^2) X with
// A = X X^T, from X = G / (|G| + eps): the passes over the matrix before and after, and
// the three products of a step on the tile kernel.
//
// Precision.  X is the sum of two float16, x = xh + xl (22 bits: fp32 would be 2 bytes more
// to write), and the diagonals of A and of B = b A + c A^2 are fp32; the other values of A
// and B are float16 operands, and A is made of xh alone.  A step multiplies small singular
// values by a (485 times over five steps of a = 3.4445), so a rounding of X would grow as
// much.  B multiplies xh and xl: so every rounding in A and B is a factor (a + B + error) on
// X's left, and takes the same share of a small singular direction as of a large one.  B xh
// alone would leave B xl out, whose right side is any direction; with A's rounding, whose
// left side is, it couples the small directions among each other, which a then multiplies:
// off by 2e-2 after five steps of 16 x 16 of one direction over noise of 1e-3, by 0.3 after
// eight.  As it is, over spectra from flat to six decades, 2e-4 to 2e-3 (shorter sides from
// 16 on) after five or six.  The diagonals are where A and B are largest near the end (A
// tends to the identity), and rounding them would lose the most.
#include "block.hpp"
#include "linear_tiles.hpp"
#include "row_common.hpp"

namespace gemm_relu_hip {

namespace {

// ------------------------------------------------------- before the steps
// Sums of squares in binary64 (the values may be any fp32 ones): workgroups take rows in
// turns, 16 bytes a thread; of short rows up to four turns each (8 of 1792 x 36 bf16 in 32
// workgroups each 5 us, 10 in 256 of which 144 have nothing).
constexpr int kSquareThreads = 1024;
// threads that share a row of so many pieces of 16 bytes
__host__ __device__ constexpr int square_threads(int chunks) { return chunks + 64 < kSquareThreads ? (chunks + 64) / 64 * 64 : kSquareThreads; }
template <class T> __global__ void __launch_bounds__(kSquareThreads) ortho_squares_kernel(OrthoArgs a)
{
    constexpr int N = Chunk<T>::N;
    using X = typename Chunk<T>::Vec;
    __shared__ double part[kSquareThreads / 64];
    const T* g = static_cast<const T*>(a.g) + (size_t)blockIdx.y * (size_t)a.g_batch;
    double s = 0.0;
    const auto add = [&](float v) { s = fma((double)v, (double)v, s); };
    // short rows: several at a time
    const int chunks = a.cols / N, wide = square_threads(chunks), rows_here = kSquareThreads / wide;
    const int t = (int)threadIdx.x % wide, own = (int)threadIdx.x / wide;
    for (int64_t r = (int64_t)blockIdx.x * rows_here + own; own < rows_here && r < a.rows; r += (int64_t)gridDim.x * rows_here) {
        const T* row = g + (size_t)r * (size_t)a.g_stride;
        constexpr int AHEAD = 4;
        int j = t;
        for (; j + (AHEAD - 1) * wide < chunks; j += AHEAD * wide) {
            X v[AHEAD];
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) v[u] = load_vec<X>(row + (size_t)(j + u * wide) * N);
#pragma unroll
            for (int u = 0; u < AHEAD; ++u)
#pragma unroll
                for (int e = 0; e < N; ++e) add((float)v[u][e]);
        }
        for (; j < chunks; j += wide) {
            const X v = load_vec<X>(row + (size_t)j * N);
#pragma unroll
            for (int e = 0; e < N; ++e) add((float)v[e]);
        }
        if (t < a.cols - chunks * N) add((float)row[(size_t)chunks * N + t]);
    }
#pragma unroll
    for (int step = 1; step < 64; step *= 2) s += __shfl_xor(s, step);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int k = 1; k < kSquareThreads / 64; ++k) s += part[k];
        a.squares[(size_t)blockIdx.y * kOrthoParts + blockIdx.x] = s;
    }
}

// X, 64 x 64 a workgroup, transposed where the matrix is tall, with zeros in the padding.
// Four rows of four elements a thread, all loads in flight together.  Bound by HBM: 8192 x
// 8192 bf16, 0.4 GB.
template <class T> __global__ void __launch_bounds__(kThreads) ortho_start_kernel(OrthoArgs a)
{
    typedef T T4 __attribute__((ext_vector_type(4)));
    typedef _Float16 H4 __attribute__((ext_vector_type(4)));
    constexpr int ROWS = 64 * 16 / kThreads;
    __shared__ float tile[64][65];
    const size_t batch = blockIdx.y;
    const int lane = (int)(threadIdx.x & 63), c4 = (int)(threadIdx.x & 15) * 4, row = (int)(threadIdx.x >> 4);
    const int tiles = a.Q / 64, p0 = (int)(blockIdx.x / tiles) * 64, q0 = (int)(blockIdx.x % tiles) * 64;
    const T* g = static_cast<const T*>(a.g) + batch * (size_t)a.g_batch;
    const bool tall = a.rows > a.cols;
    const int r0 = tall ? q0 : p0, c = (tall ? p0 : q0) + c4;
    // the arrival counters of a K split that follows
    if (blockIdx.x == 0)
        for (int k = threadIdx.x; k < a.nflags; k += kThreads) a.flags[batch * (size_t)a.nflags + k] = 0u;
    T4 raw[ROWS];
    if (c + 4 <= a.cols) {
#pragma unroll
        for (int k = 0; k < ROWS; ++k)
            raw[k] = load_vec<T4>(g + (size_t)min(r0 + row + 64 / ROWS * k, a.rows - 1) * (size_t)a.g_stride + c);
    } else {
#pragma unroll
        for (int k = 0; k < ROWS; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                raw[k][e] = g[(size_t)min(r0 + row + 64 / ROWS * k, a.rows - 1) * (size_t)a.g_stride + min(c + e, a.cols - 1)];
    }
    double s = 0.0;
#pragma unroll
    for (int k = 0; k < kOrthoParts; k += 64) s += k + lane < a.parts ? a.squares[batch * kOrthoParts + k + lane] : 0.0;
#pragma unroll
    for (int step = 1; step < 64; step *= 2) s += __shfl_xor(s, step);
    // the scale as an fp32 number times a power of two: it may be past fp32's range, and
    // values below the normal range take the power first, while they are exact
    int power;
    const float factor = (float)frexp((double)kOrthoX / (sqrt(s) + (double)a.eps), &power);
    _Float16* xh = static_cast<_Float16*>(a.xh) + batch * 2 * (size_t)a.P * (size_t)a.Q;
    _Float16* xl = static_cast<_Float16*>(a.xl) + batch * 2 * (size_t)a.P * (size_t)a.Q;
    const auto put = [&](int p, int q, const float(&v)[4]) {
        const size_t at = (size_t)p * (size_t)a.Q + q;
        H4 hi, lo;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            hi[e] = (_Float16)v[e];
            lo[e] = (_Float16)((v[e] - (float)hi[e]) * kLowScale);
        }
        *reinterpret_cast<H4*>(xh + at) = hi;
        *reinterpret_cast<H4*>(xl + at) = lo;
    };
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
        const int r = row + 64 / ROWS * k;
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[e] = r0 + r < a.rows && c + e < a.cols ? ldexpf((float)raw[k][e], power) * factor : 0.0f;
        if (tall) {
#pragma unroll
            for (int e = 0; e < 4; ++e) tile[r][c4 + e] = v[e];
        } else {
            put(p0 + r, q0 + c4, v);
        }
    }
    if (!tall) return;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
        const int p = row + 64 / ROWS * k;
        const float v[4] = {tile[c4][p], tile[c4 + 1][p], tile[c4 + 2][p], tile[c4 + 3][p]};
        put(p0 + p, q0 + c4, v);
    }
}

// ------------------------------------------------------- without any step
__global__ void __launch_bounds__(kThreads) ortho_copy_kernel(OrthoArgs a)
{
    __shared__ float tile[64][65];
    const size_t batch = blockIdx.y;
    const int lane = (int)(threadIdx.x & 63), wave = (int)(threadIdx.x >> 6);
    const int tiles = a.Q / 64, p0 = (int)(blockIdx.x / tiles) * 64, q0 = (int)(blockIdx.x % tiles) * 64;
    const bool tall = a.rows > a.cols;
    const _Float16* xh = static_cast<const _Float16*>(a.xh) + batch * 2 * (size_t)a.P * (size_t)a.Q;
    const _Float16* xl = static_cast<const _Float16*>(a.xl) + batch * 2 * (size_t)a.P * (size_t)a.Q;
    __bf16* out = static_cast<__bf16*>(a.out) + batch * (size_t)a.rows * (size_t)a.cols;
    for (int k = wave; k < 64; k += kThreads / 64) {
        const int p = p0 + k, q = q0 + lane;
        const size_t at = (size_t)p * (size_t)a.Q + q;
        const float v = fmaf((float)xl[at], 1.0f / kLowScale, (float)xh[at]) / kOrthoX;
        if (tall)
            tile[k][lane] = v;
        else if (p < a.p && q < a.q)
            out[(size_t)p * (size_t)a.cols + q] = (__bf16)v;
    }
    if (!tall) return;
    __syncthreads();
    for (int k = wave; k < 64; k += kThreads / 64)
        if (q0 + k < a.q && p0 + lane < a.p) out[(size_t)(q0 + k) * (size_t)a.cols + p0 + lane] = (__bf16)tile[lane][k];
}

// ------------------------------------------------------------ the products
// B X is one product over 2 P values of K: [B / kLowScale, B] [xl; xh], the lesser terms first
// (xl holds kLowScale times what xh loses, B / kLowScale loses nothing that counts beside B
// xh).  What a step of 8192 x 8192 takes: A 475 us and A^2 509 (half of their products; 1160
// and 1080 TFLOP/s for those), B X 1652 (1330 TFLOP/s; 895 without xl), whose epilogue
// reads and writes 8 bytes an element while the matrix units wait: one tile fills a CU.  8 x
// 1024 x 2048: 43, 35 and 88 us (63 without xl), of which 25 are such an epilogue (one round
// of tiles); with X in fp32 it was the same.
template <class C> __global__ void __launch_bounds__(C::NTHREADS, 1) ortho_product_kernel(OrthoProduct p)
{
    __shared__ __attribute__((aligned(1024))) unsigned char smem_raw[C::LDS_BYTES];
    KernelArgs args = p.k;
    const uint64_t batch = blockIdx.y;
    args.A += batch * p.a;
    args.B += batch * p.b;
    args.C += batch * p.c;
    args.R += batch * p.r;
    args.L += batch * p.r;
    args.low += batch * p.low;
    args.diag += batch * p.diag;
    args.diag_out += batch * p.diag;
    args.ws += batch * p.ws;
    args.flags += batch * p.flags;
    // a K split's workgroups take part wg / tiles of tile wg % tiles
    const int wg = (int)blockIdx.x, tiles = C::SPLITK ? (int)gridDim.x / args.splits : 1;
    gemm_relu_tile<C>(args, C::SPLITK ? wg % tiles : wg, (GR_LDS unsigned char*)(smem_raw), nullptr,
                      Region{args.tiles_m, args.tiles_n, args.panel, 0, C::SPLITK ? wg / tiles : 0});
}
template <class C> hipError_t launch_product(const OrthoProduct& p, int tiles, int batch, hipStream_t stream)
{
    void* params[] = {const_cast<OrthoProduct*>(&p)};
    return hipLaunchKernel(reinterpret_cast<const void*>(&ortho_product_kernel<C>), dim3(tiles, batch), dim3(C::NTHREADS), params,
                           0, stream);
}
template <int EPI> OrthoLaunchFn pick_product(int cfg)
{
    constexpr int OUT = EPI == EPI_LAST ? DT_BF16 : DT_F16;
    switch (cfg) {
    case LIN_256: return &launch_product<typename LinearCfg<DT_F16, OUT, EPI, LIN_256>::type>;
    case LIN_128: return &launch_product<typename LinearCfg<DT_F16, OUT, EPI, LIN_128>::type>;
    case LIN_128X2: return &launch_product<typename LinearCfg<DT_F16, OUT, EPI, LIN_128X2>::type>;
    case LIN_64: return &launch_product<typename LinearCfg<DT_F16, OUT, EPI, LIN_64>::type>;
    default: return nullptr;
    }
}

}  // namespace

OrthoLaunchFn launcher_ortho(int epi, int cfg)
{
    switch (epi) {
    case EPI_GRAM: return pick_product<EPI_GRAM>(cfg);
    case EPI_POLY: return pick_product<EPI_POLY>(cfg);
    case EPI_STEP: return pick_product<EPI_STEP>(cfg);
    case EPI_LAST: return pick_product<EPI_LAST>(cfg);
    default: return nullptr;
    }
}

int ortho_square_parts(int64_t rows, int64_t cols, int dt)
{
    const int rows_here = kSquareThreads / square_threads(int(cols / (16 / elem_size(dt))));
    int64_t parts = ceil_div(rows, rows_here);
    if (rows_here >= 4 && parts > 32) parts = std::max<int64_t>(32, ceil_div(parts, 4));
    return int(std::min<int64_t>(parts, kOrthoParts));
}

hipError_t launch_ortho_squares(const OrthoArgs& a, int dt, hipStream_t stream)
{
    return with_types(dt, dt, [&](auto x, auto) {
        using T = decltype(x);
        return start(&ortho_squares_kernel<T>, dim3(a.parts, a.batch), kSquareThreads, stream, a);
    });
}

hipError_t launch_ortho_start(const OrthoArgs& a, int dt, hipStream_t stream)
{
    const hipError_t e = launch_ortho_squares(a, dt, stream);
    if (e != hipSuccess) return e;
    return with_types(dt, dt, [&](auto x, auto) {
        using T = decltype(x);
        return start(&ortho_start_kernel<T>, dim3((unsigned)(a.P / 64) * (unsigned)(a.Q / 64), a.batch), kThreads, stream, a);
    });
}

hipError_t launch_ortho_copy(const OrthoArgs& a, hipStream_t stream)
{
    return start(&ortho_copy_kernel, dim3((unsigned)(a.P / 64) * (unsigned)(a.Q / 64), a.batch), kThreads, stream, a);
}

}  // namespace gemm_relu_hip
