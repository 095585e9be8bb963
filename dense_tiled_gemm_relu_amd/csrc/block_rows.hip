// Row-wise and element-wise kernels around the half layer: the gradient of an
// activation, and the sums over rows.
#include <algorithm>
#include <type_traits>

#include "api_common.hpp"
#include "block.hpp"
#include "row_common.hpp"

namespace gemm_relu_hip {

namespace {

// The strips' sums, in order: 64 columns a workgroup, each of 16 waves takes every
// 16th strip.
template <class W> __global__ void __launch_bounds__(1024) join_kernel(JoinArgs a)
{
    __shared__ float part[16][64];
    const int lane = (int)(threadIdx.x & 63), wave = (int)(threadIdx.x >> 6);
    const int64_t all = (int64_t)a.sums * a.cols;
    for (int64_t j0 = (int64_t)blockIdx.x * 64; j0 < all; j0 += (int64_t)gridDim.x * 64) {
        const int64_t j = j0 + lane;
        float s = 0.0f;
        if (j < all) {
            // a wave's strips in batches of 8, all loads of one in flight together
            // (strips past the end are the last one's, and count for nothing)
            for (int k = wave; k < a.strips; k += 16 * 8) {
                float v[8];
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    v[u] = a.partial[(size_t)min(k + 16 * u, a.strips - 1) * (size_t)all + j];
#pragma unroll
                for (int u = 0; u < 8; ++u) s += k + 16 * u < a.strips ? v[u] : 0.0f;
            }
        }
        part[wave][lane] = s;
        __syncthreads();
        if (!wave && j < all) {
#pragma unroll
            for (int k = 1; k < 16; ++k) s += part[k][lane];
            int64_t c = j;
#pragma unroll
            for (int k = 0; k < kMaxSums; ++k) {
                if (c >= 0 && c < a.cols && a.out[k]) static_cast<W*>(a.out[k])[c] = (W)s;
                c -= a.cols;
            }
        }
        __syncthreads();
    }
}

// ---------------------------------------------------- gradient of act(z)
// A 64 x 64 tile of (rows, n), 2 x 4 elements a thread with all loads issued before
// the first is used: dz goes out row-major, and transposed through LDS.  Both outputs'
// rows are padded to 16 bytes with zeros, so that the products may read them in whole
// pieces.  Bound by HBM.
template <int DT, int ACT> __global__ void __launch_bounds__(kActGradThreads) act_grad_kernel(ActGradArgs a)
{
    using T = typename Elem<DT>::T;
    typedef T T4 __attribute__((ext_vector_type(4)));
    typedef T T2 __attribute__((ext_vector_type(2)));
    constexpr int ROWS = 64 * 16 / kActGradThreads, WAVES = kActGradThreads / 64;
    constexpr int PITCH = 68;                      // elements of a transposed row: 8-byte pieces on spread banks
    static_assert(ROWS == 2, "a pair of rows a thread");
    __shared__ __attribute__((aligned(16))) T tile[64][PITCH];
    __shared__ float sums[WAVES][64];
    const int tiles = (a.n + 63) / 64;
    const int n0 = (int)(blockIdx.x % tiles) * 64, tr = (int)(blockIdx.x / tiles), r0 = tr * 64;
    if (blockIdx.x == 0)
        for (int k = threadIdx.x; k < a.nflags; k += kActGradThreads) a.flags[k] = 0u;
    const int c = (int)(threadIdx.x & 15) * 4, n = n0 + c, q = (int)(threadIdx.x >> 4) * ROWS;
    const bool whole = n + 4 <= a.n;
    f32x4_t z[ROWS];
    T4 d[ROWS];
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
        z[k] = f32x4_t{};
        d[k] = T4{};
        const int r = r0 + q + k;
        if (r >= a.rows) continue;
        const float* zr = a.z + (size_t)r * (size_t)a.n + n;
        const T* dy = static_cast<const T*>(a.dy) + (size_t)r * (size_t)a.dy_stride + n;
        if (whole) {
            if (ACT != ACT_NONE) z[k] = load_vec<f32x4_t>(zr);
            d[k] = load_vec<T4>(dy);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (n + e < a.n) {
                    if (ACT != ACT_NONE) z[k][e] = zr[e];
                    d[k][e] = dy[e];
                }
        }
    }
    T4 dz[ROWS];
    f32x4_t column = {};
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float value, slope;
            activation_slope<ACT>(z[k][e], value, slope);
            const float g = (float)d[k][e] * slope;
            column[e] += g;
            dz[k][e] = (T)(g * a.scale);
        }
        const int r = r0 + q + k;
        if (r >= a.rows || !a.dz) continue;
        T* out = static_cast<T*>(a.dz) + (size_t)r * (size_t)a.ld + n;
        if (whole) {
            __builtin_memcpy(out, &dz[k], 8);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (n + e < a.n) out[e] = dz[k][e];
        }
        // the row's padding, by the thread behind its last tile column
        if (n0 + 64 >= a.n && c == 60)
            for (int j = a.n; j < a.ld; ++j) static_cast<T*>(a.dz)[(size_t)r * (size_t)a.ld + j] = (T)0.0f;
    }
    // rows past the edge hold d = 0: their dz is the transposed padding, and adds nothing
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const T2 x = {dz[0][e], dz[1][e]};
        *reinterpret_cast<T2*>(&tile[c + e][q]) = x;
    }
    if (a.sums) {
        // the four row pairs of a wave, then the waves in order
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            column[e] += __shfl_xor(column[e], 16);
            column[e] += __shfl_xor(column[e], 32);
        }
        if ((threadIdx.x & 63) < 16) *reinterpret_cast<f32x4_t*>(&sums[threadIdx.x >> 6][c]) = column;
    }
    __syncthreads();
    if (a.sums && threadIdx.x < 64 && n0 + (int)threadIdx.x < a.n) {
        float s = sums[0][threadIdx.x];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) s += sums[w][threadIdx.x];
        a.sums[(size_t)tr * (size_t)a.n + n0 + threadIdx.x] = s;
    }
    const int hh = (int)threadIdx.x >> 3, rr = ((int)threadIdx.x & 7) * 8;
    if (n0 + hh >= a.n || r0 + rr >= a.rows) return;
    const T4* from = reinterpret_cast<const T4*>(&tile[hh][rr]);
    T* out = static_cast<T*>(a.dz_t) + (size_t)(n0 + hh) * (size_t)a.ld_t + r0 + rr;
    const T4 lo = from[0], hi = from[1];
    __builtin_memcpy(out, &lo, 8);
    __builtin_memcpy(out + 4, &hi, 8);
}

}  // namespace

hipError_t launch_join(const JoinArgs& a, int out_dt, hipStream_t stream)
{
    const dim3 grid((unsigned)std::min<int64_t>(ceil_div((int64_t)a.sums * a.cols, 64), kMaxRowGrid));
    switch (out_dt) {
    case DT_F32: return start(&join_kernel<float>, grid, 1024, stream, a);
    case DT_F16: return start(&join_kernel<_Float16>, grid, 1024, stream, a);
    default: return start(&join_kernel<__bf16>, grid, 1024, stream, a);
    }
}

hipError_t launch_act_grad(const ActGradArgs& a, int dt, hipStream_t stream)
{
    const dim3 grid((unsigned)((a.n + 63) / 64) * (unsigned)((a.rows + 63) / 64));
    const auto go = [&](auto act) {
        constexpr int ACT = decltype(act)::value;
        return start(dt == DT_F16 ? &act_grad_kernel<DT_F16, ACT> : &act_grad_kernel<DT_BF16, ACT>, grid, kActGradThreads,
                     stream, a);
    };
    switch (a.act) {
    case ACT_SILU: return go(std::integral_constant<int, ACT_SILU>{});
    case ACT_GELU: return go(std::integral_constant<int, ACT_GELU>{});
    case ACT_GELU_TANH: return go(std::integral_constant<int, ACT_GELU_TANH>{});
    case ACT_RELU: return go(std::integral_constant<int, ACT_RELU>{});
    default: return go(std::integral_constant<int, ACT_NONE>{});
    }
}

}  // namespace gemm_relu_hip
