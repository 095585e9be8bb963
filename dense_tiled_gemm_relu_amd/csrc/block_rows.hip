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
    const int blocks = (int)(((int64_t)a.cols + 63) / 64);
    for (int64_t u = blockIdx.x; u < (int64_t)a.results * blocks; u += gridDim.x) {
        const int k = (int)(u / blocks);
        const JoinArgs::Result r = a.result[k];
        if (!r.out) continue;
        const int64_t c = u % blocks * 64 + lane, j = (int64_t)r.of * a.cols + c;
        float s = 0.0f;
        if (c < a.cols) {
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
        if (!wave && c < a.cols) {
#pragma unroll
            for (int k = 1; k < 16; ++k) s += part[k][lane];
            s *= r.scale;
            if (r.factor) s *= (float)static_cast<const W*>(r.factor)[c];
            static_cast<W*>(r.out)[c] = (W)s;
        }
        __syncthreads();
    }
}

// ---------------------------------------------------- gradient of act(z)
// A 64 x 64 tile of (rows, n), 2 x 4 elements a thread with all loads issued before
// the first is used: dz goes out row-major, and transposed through LDS.  Both outputs'
// rows are padded to 16 bytes with zeros, so that the products may read them in whole
// pieces.  Bound by HBM: 4096 x 4096 bf16, 0.17 GB in 30 us, 5.6 TB/s.
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
            activation_slope<ACT, true>(z[k][e], value, slope);
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

// ------------------------------------------------- residual sum and norms
typedef float Stats __attribute__((ext_vector_type(4), aligned(4)));       // a row's statistics, at any float's address

// One read of x and the residual, one write of s and y: the row stays in registers
// between its sums; the next row is loaded meanwhile, and what is the same for all rows
// stays in registers, gate, post_weight and scale as one product.  One wave a row and four
// rows a workgroup, or `waves` waves a row: one chunk a thread (two where 16 waves would
// not hold the row).  Bound by HBM where there is one norm (16384 x 8192 bf16 194 us, 5.5
// TB/s); with layer norms on both sides the waves wait half of their time, a row's four
// barriers among it, and the vector unit is busy for the other half (40 instructions an
// element; 4097 x 3001 fp16 27 us, 3.6 TB/s).
template <class T, class W, bool ONE, int V>
__global__ void __launch_bounds__(ONE ? kThreads : 1024) add_norm_kernel(AddNormArgs a, int waves)
{
    constexpr int N = Chunk<T>::N;
    using X = typename Chunk<T>::Vec;
    using WV = typename VecN<W, N>::Vec;
    __shared__ float lds[2][4][16];
    const int lane = (int)(threadIdx.x & 63), wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const RowMap<T, V> map(a.cols, ONE ? lane : (int)threadIdx.x, ONE ? 64 : 64 * waves);
    // whether a lane of the wave holds elements that its neighbour owns: only then do the
    // sums look at each element's owner
    const bool edge = __any(map.skip != 0);
    const bool element_gate = a.gate && a.gate_stride, channel_gate = a.gate && !a.gate_stride;
    WV w[V], b[V];
    float k[V][N];                // scale gate post_weight
#pragma unroll
    for (int v = 0; v < V; ++v) {
        w[v] = b[v] = WV{};
        WV pw = WV{}, gate = WV{};
        if (map.has(v)) {
            if (a.w) w[v] = load_vec<WV>(static_cast<const W*>(a.w) + map.start[v]);
            if (a.b) b[v] = load_vec<WV>(static_cast<const W*>(a.b) + map.start[v]);
            if (a.pw) pw = load_vec<WV>(static_cast<const W*>(a.pw) + map.start[v]);
            if (channel_gate) gate = load_vec<WV>(static_cast<const W*>(a.gate) + map.start[v]);
        }
#pragma unroll
        for (int e = 0; e < N; ++e) k[v][e] = a.scale * (channel_gate ? (float)gate[e] : 1.0f) * (a.pw ? (float)pw[e] : 1.0f);
    }
    constexpr int ROWS = ONE ? kThreads / 64 : 1;
    const int step = (int)gridDim.x * ROWS;
    int64_t row = (int64_t)blockIdx.x * ROWS + (ONE ? wave : 0);          // 64 bits: the last row's successor may pass 2^31
    X nx[V], nr[V], ng[V];
    auto fetch = [&](int64_t at) {
        const T* x = static_cast<const T*>(a.x) + (size_t)at * (size_t)a.x_stride;
        const T* r = static_cast<const T*>(a.r) + (size_t)at * (size_t)a.r_stride;
        const T* g = static_cast<const T*>(a.gate) + (size_t)at * (size_t)a.gate_stride;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (map.has(v)) {
                nx[v] = load_vec<X>(x + map.start[v]);
                nr[v] = load_vec<X>(r + map.start[v]);
                if (element_gate) ng[v] = load_vec<X>(g + map.start[v]);
            }
    };
#pragma unroll
    for (int v = 0; v < V; ++v) nx[v] = nr[v] = ng[v] = X{};
    if (row < a.rows) fetch(row);
    const float n = (float)a.cols;
    // the sum over the row; the waves alternate between buffers, so that whoever writes one
    // again has passed the barrier of another, behind every read
    auto row_sum = [&](float v, float(&buffer)[16]) {
        v = wave_all<Sum>(v);
        if constexpr (!ONE) {
            if (lane == 0) buffer[wave] = v;
            __syncthreads();
            const int j = lane & 15;
            v = row16_sum(j < waves ? buffer[j] : 0.0f);
        }
        return v;
    };
    // f((its elements as they count in sums))
    auto each = [&](auto&& f) {
        if (edge) {
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int e = 0; e < N; ++e) f(v, e, map.owns(v, e));
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int e = 0; e < N; ++e) f(v, e, true);
        }
    };
    // mean (0 for the root mean square) and 1 / deviation of f
    auto statistics = [&](const float(&f)[V][N], float(&buffers)[4][16], int first, float& mean, float& rstd) {
        float sum = 0.0f;
        mean = 0.0f;
        if (a.layer) {
            each([&](int v, int e, bool own) { sum += own ? f[v][e] : 0.0f; });
            mean = row_sum(sum, buffers[first]) / n;
            sum = 0.0f;
        }
        each([&](int v, int e, bool own) {
            const float d = own ? f[v][e] - mean : 0.0f;
            sum = fmaf(d, d, sum);
        });
        rstd = 1.0f / sqrtf(row_sum(sum, buffers[first + 1]) / n + a.eps);
    };
    for (int turn = 0; row < a.rows; row += step, turn ^= 1) {
        float f[V][N];
        X r[V], g[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            r[v] = nr[v];
            g[v] = ng[v];
#pragma unroll
            for (int e = 0; e < N; ++e) f[v][e] = (float)nx[v][e];
        }
        if (row < a.rows - step) fetch(row + step);
        f32x4_t stats = {0.0f, 1.0f, 0.0f, 1.0f};
        if (a.pw) {
            float mean, rstd;
            statistics(f, lds[turn], 0, mean, rstd);
            stats[0] = mean;
            stats[1] = rstd;
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int e = 0; e < N; ++e) f[v][e] = (f[v][e] - mean) * rstd;
        }
        if (element_gate) {
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int e = 0; e < N; ++e) f[v][e] *= (float)g[v][e];
        }
        T* s = static_cast<T*>(a.s) + (size_t)row * (size_t)a.cols;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            X out;
#pragma unroll
            for (int e = 0; e < N; ++e) {
                f[v][e] = fmaf(k[v][e], f[v][e], (float)r[v][e]);
                out[e] = (T)f[v][e];
            }
            if (map.has(v)) __builtin_memcpy(s + map.start[v], &out, sizeof out);
        }
        if (a.w) {
            float mean, rstd;
            statistics(f, lds[turn], 2, mean, rstd);
            stats[2] = mean;
            stats[3] = rstd;
            T* y = static_cast<T*>(a.y) + (size_t)row * (size_t)a.cols;
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (map.has(v)) {
                    X out;
#pragma unroll
                    for (int e = 0; e < N; ++e) out[e] = (T)fmaf((f[v][e] - mean) * rstd, (float)w[v][e], (float)b[v][e]);
                    __builtin_memcpy(y + map.start[v], &out, sizeof out);
                }
        }
        if (a.stats && (ONE ? lane : (int)threadIdx.x) == 0) *reinterpret_cast<Stats*>(a.stats + 4 * (size_t)row) = stats;
    }
}

// The backward pass in one read of its inputs: s is computed again, the row's two sums
// give dresidual, two more dx.  A workgroup takes rows in turns, `waves` waves a row and
// as many rows at a time as 16 waves hold, and leaves one strip of sums over its rows; the
// join kernel adds the strips in order.
//
// A thread's own sums over rows stand in LDS: three fp32 sums an element beside five
// streams, the next row's among them, do not fit the 128 registers that 16 waves a CU
// leave.  They are nobody else's, so they need no barrier, and they take a sixth of LDS's
// rate.  16-bit rows of more than 1024 chunks have more than LDS holds: their sums over
// rows are left to add_norm_strip_any_kernel.  A chunk
// moved back inside the row has its weights cleared where its neighbour owns the element:
// the row's sums then need no test, and only what it owns is stored.  Bound by HBM:
// 16384 x 4096 bf16, eight streams, 200 us (5.4 TB/s; 440 with the sums in registers, which
// spill); with layer norms on both sides by its waits, more than half of the waves' time, the
// vector unit busy for 38 % (45 instructions an element; 4097 x 3001 fp16 37 us, 4.0 TB/s: six
// waves a row, so 12 of the 16 that fit).
template <class T, class W, int V>
__global__ void __launch_bounds__(1024) add_norm_backward_kernel(AddNormArgs a, int waves)
{
    constexpr int N = Chunk<T>::N;
    using X = typename Chunk<T>::Vec;
    using WV = typename VecN<W, N>::Vec;
    constexpr bool SUMS = V * N <= 8;
    constexpr int QUADS = V * N / 4;                  // of a thread's elements
    __shared__ float lds[2][4][16];
    __shared__ __attribute__((aligned(16))) f32x4_t sums_raw[SUMS ? kNormSums * QUADS * 1024 : 1];
    const int lane = (int)(threadIdx.x & 63), wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int groups = (int)(blockDim.x >> 6) / waves, group = wave / waves, in_row = wave - group * waves;
    const RowMap<T, V> map(a.cols, in_row * 64 + lane, 64 * waves);
    const bool element_gate = a.gate && a.gate_stride, channel_gate = a.gate && !a.gate_stride;
    WV w[V];
    float k[V][N];                // scale gate post_weight
#pragma unroll
    for (int v = 0; v < V; ++v) {
        w[v] = WV{};
        WV pw = WV{}, gate = WV{};
        if (a.w) w[v] = load_vec<WV>(static_cast<const W*>(a.w) + map.start[v]);
        if (a.pw) pw = load_vec<WV>(static_cast<const W*>(a.pw) + map.start[v]);
        if (channel_gate) gate = load_vec<WV>(static_cast<const W*>(a.gate) + map.start[v]);
#pragma unroll
        for (int e = 0; e < N; ++e) {
            k[v][e] = a.scale * (channel_gate ? (float)gate[e] : 1.0f) * (a.pw ? (float)pw[e] : 1.0f);
            if (!map.owns(v, e)) {
                w[v][e] = (W)0.0f;
                k[v][e] = 0.0f;
            }
        }
    }
    // sum `which` of the thread's quad q of elements
    const auto sum_at = [&](int which, int q) -> f32x4_t& { return sums_raw[(which * QUADS + q) * 1024 + (int)threadIdx.x]; };
    if constexpr (SUMS) {
#pragma unroll
        for (int which = 0; which < kNormSums; ++which)
#pragma unroll
            for (int q = 0; q < QUADS; ++q) sum_at(which, q) = f32x4_t{};
    }
    const int64_t step = (int64_t)gridDim.x * groups;
    const int64_t first_row = (int64_t)blockIdx.x * groups;
    int64_t row = first_row + group;
    // a missing chunk is the row's last, a row past the end the last one
    X nx[V], nr[V], ny[V], nd[V], ng[V];
    auto fetch = [&](int64_t to) {
        const size_t at = (size_t)min(to, (int64_t)a.rows - 1);
        const T* x = static_cast<const T*>(a.x) + at * (size_t)a.x_stride;
        const T* r = static_cast<const T*>(a.r) + at * (size_t)a.r_stride;
        const T* y = static_cast<const T*>(a.dy) + at * (size_t)a.dy_stride;
        const T* d = static_cast<const T*>(a.ds) + at * (size_t)a.ds_stride;
        const T* g = static_cast<const T*>(a.gate) + at * (size_t)a.gate_stride;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            nx[v] = load_vec<X>(x + map.start[v]);
            if (a.w) nr[v] = load_vec<X>(r + map.start[v]);
            if (a.w) ny[v] = load_vec<X>(y + map.start[v]);
            if (a.ds) nd[v] = load_vec<X>(d + map.start[v]);
            if (element_gate) ng[v] = load_vec<X>(g + map.start[v]);
        }
    };
#pragma unroll
    for (int v = 0; v < V; ++v) nx[v] = nr[v] = ny[v] = nd[v] = ng[v] = X{};
    fetch(row);
    const float inv_n = 1.0f / (float)a.cols;
    // one value for the whole wave: read through the scalar cache
    typedef const __attribute__((address_space(4))) Stats* Scalars;
    const Scalars all_stats = (Scalars)(uintptr_t)a.stats;
    // means over the row of p (0 for the root mean square) and q
    auto means = [&](float& p, float& q, float(&buffers)[4][16], int first) {
        q = wave_all<Sum>(q);
        if (a.layer) p = wave_all<Sum>(p);
        if (waves > 1) {
            if (lane == 0) {
                buffers[first][wave] = p;
                buffers[first + 1][wave] = q;
            }
            __syncthreads();
            // 16 lanes each add the waves'
            const int j = lane & 15;
            if (a.layer) p = row16_sum(j < waves ? buffers[first][group * waves + j] : 0.0f);
            q = row16_sum(j < waves ? buffers[first + 1][group * waves + j] : 0.0f);
        }
        p = a.layer ? p * inv_n : 0.0f;
        q *= inv_n;
    };
    // the row's values f of an output
    auto store = [&](void* out, size_t at, const float(&f)[V][N]) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            X packed;
#pragma unroll
            for (int e = 0; e < N; ++e) packed[e] = (T)f[v][e];
            T* to = static_cast<T*>(out) + at + map.start[v];
            if (v < V - 1 || map.skip == 0) {
                __builtin_memcpy(to, &packed, sizeof packed);
            } else {
#pragma unroll
                for (int e = 0; e < N; ++e)
                    if (e >= map.skip) to[e] = packed[e];
            }
        }
    };
    // all rows of a workgroup meet at its barriers, so a row past the end runs along
    // with nothing to add and nothing to store
    for (int turn = 0; row - group < a.rows; row += step, turn ^= 1) {
        const bool live = row < a.rows;
        const size_t at = (size_t)row * (size_t)a.cols;
        const Stats stats = all_stats[min(row, (int64_t)a.rows - 1)];
        float xhat[V][N], dr[V][N];
        X g[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            g[v] = ng[v];
#pragma unroll
            for (int e = 0; e < N; ++e) {
                xhat[v][e] = ((float)nx[v][e] - stats[0]) * stats[1];
                dr[v][e] = (float)nd[v][e];
            }
        }
        if (a.w) {
            // c = dy weight
            float shat[V][N], c[V][N], p = 0.0f, q = 0.0f;
            X y[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                y[v] = ny[v];
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const float gated = element_gate ? xhat[v][e] * (float)g[v][e] : xhat[v][e];
                    shat[v][e] = (fmaf(k[v][e], gated, (float)nr[v][e]) - stats[2]) * stats[3];
                    c[v][e] = (float)y[v][e] * (float)w[v][e];
                    p += c[v][e];
                    q = fmaf(c[v][e], shat[v][e], q);
                }
            }
            fetch(row + step);
            means(p, q, lds[turn], 0);
            if (!SUMS && live && in_row == 0 && lane == 0) {
                a.row_sums[2 * row] = p;
                a.row_sums[2 * row + 1] = q;
            }
            p *= -stats[3];
            q *= -stats[3];
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int e = 0; e < N; ++e) dr[v][e] = fmaf(shat[v][e], q, fmaf(c[v][e], stats[3], dr[v][e] + p));
            if constexpr (SUMS) {
#pragma unroll
                for (int v = 0; v < V; ++v)
#pragma unroll
                for (int h = 0; h < N / 4; ++h) {
                    f32x4_t dw = sum_at(0, v * (N / 4) + h);
#pragma unroll
                    for (int u = 0; u < 4; ++u) dw[u] = fmaf((float)y[v][4 * h + u], shat[v][4 * h + u], dw[u]);
                    if (live) sum_at(0, v * (N / 4) + h) = dw;
                    if (a.db) {
                        f32x4_t db = sum_at(1, v * (N / 4) + h);
#pragma unroll
                        for (int u = 0; u < 4; ++u) db[u] += (float)y[v][4 * h + u];
                        if (live) sum_at(1, v * (N / 4) + h) = db;
                    }
                }
            }
        } else {
            fetch(row + step);
        }
        if (a.dr && live) store(a.dr, at, dr);
        if (element_gate) {
            // t's other factor beside xhat, and dt without the rest of it
            float dg[V][N];
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    dg[v][e] = dr[v][e] * xhat[v][e] * k[v][e];
                    dr[v][e] *= (float)g[v][e];
                }
            if (a.dgate && live) store(a.dgate, at, dg);
        }
        float p = 0.0f, q = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int h = 0; h < N / 4; ++h) {
                if (SUMS && (a.gate || a.pw)) {
                    f32x4_t sum = sum_at(2, v * (N / 4) + h);
#pragma unroll
                    for (int u = 0; u < 4; ++u) sum[u] = fmaf(dr[v][4 * h + u], xhat[v][4 * h + u], sum[u]);
                    if (live) sum_at(2, v * (N / 4) + h) = sum;
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int e = 4 * h + u;
                    dr[v][e] *= k[v][e];
                    p += dr[v][e];
                    q = fmaf(dr[v][e], xhat[v][e], q);
                }
            }
        if (a.pw) {
            means(p, q, lds[turn], 2);
            p *= -stats[1];
            q *= -stats[1];
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int e = 0; e < N; ++e) dr[v][e] = fmaf(xhat[v][e], q, fmaf(dr[v][e], stats[1], p));
        }
        if (a.dx && live) store(a.dx, at, dr);
    }
    // the groups' sums join first, in order
    if constexpr (!SUMS) return;
    __syncthreads();
    if (group) return;
    float* strip = a.partial + (size_t)blockIdx.x * kNormSums * (size_t)a.cols;
#pragma unroll
    for (int which = 0; which < kNormSums; ++which) {
        if (!(which == 0 ? a.w != nullptr : which == 1 ? a.db != nullptr : a.gate || a.pw)) continue;
#pragma unroll
        for (int q = 0; q < QUADS; ++q) {
            f32x4_t s = sum_at(which, q);
            for (int j = 1; j < groups; ++j) s += sums_raw[(which * QUADS + q) * 1024 + j * 64 * waves + (int)threadIdx.x];
            const int v = q / (N / 4), e = 4 * (q % (N / 4));
            float* to = strip + (size_t)which * (size_t)a.cols + map.start[v] + e;
            if (v < V - 1 || map.skip == 0) {
                __builtin_memcpy(to, &s, 16);
            } else {
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (e + u >= map.skip) to[u] = s[u];
            }
        }
    }
}

// ---- rows of any length: one workgroup a row, read once per use.  Forward, x and the residual
// are read three times for a root mean square norm of s, four for a layer norm, and x
// once or twice more for a norm of its own: 1024 x 65536 bf16, rms, 463 us forward and 862 backward
// (its bytes' share 101 and 127), with post norm and gate 676 and 2142; 2048 x 32768 fp32 552
// and 873, 822 and 2043.
template <class T, class W> struct AnyRow {
    const AddNormArgs& a;
    const T *x, *r;
    const T* g;
    const W *pw, *gc;
    float mean, rstd;          // of x
    __device__ __forceinline__ AnyRow(const AddNormArgs& args, size_t row)
        : a(args), x(static_cast<const T*>(args.x) + row * (size_t)args.x_stride),
          r(static_cast<const T*>(args.r) + row * (size_t)args.r_stride),
          g(args.gate && args.gate_stride ? static_cast<const T*>(args.gate) + row * (size_t)args.gate_stride : nullptr),
          pw(static_cast<const W*>(args.pw)), gc(args.gate && !args.gate_stride ? static_cast<const W*>(args.gate) : nullptr),
          mean(0.0f), rstd(1.0f)
    {
    }
    __device__ __forceinline__ float gate(int64_t j) const { return g ? (float)g[j] : gc ? (float)gc[j] : 1.0f; }
    __device__ __forceinline__ float xhat(int64_t j) const { return ((float)x[j] - mean) * rstd; }
    __device__ __forceinline__ float t(int64_t j) const { return pw ? xhat(j) * (float)pw[j] : xhat(j); }
    __device__ __forceinline__ float s(int64_t j) const { return fmaf(a.scale, t(j) * gate(j), (float)r[j]); }
};
template <class T, class W, bool SHORT> __global__ void __launch_bounds__(kThreads) add_norm_any_kernel(AddNormArgs a)
{
    __shared__ RowSums<1> lds[2][4][kThreads / 64];
    const W* w = static_cast<const W*>(a.w);
    const W* b = static_cast<const W*>(a.b);
    int turn = 0;
    for (size_t row = blockIdx.x; row < (size_t)a.rows; row += gridDim.x, turn ^= 1) {
        AnyRow<T, W> in(a, row);
        auto statistics = [&](auto&& at, int first, float& mean, float& rstd) {
            float m = 0.0f;
            if (a.layer) m = row_means<SHORT, 1>(a.cols, [&](int64_t j) { return Values<1>{at(j)}; }, lds[turn][first]).v[0];
            const auto square = [&](int64_t j) {
                const float d = at(j) - m;
                return Values<1>{d * d};
            };
            rstd = 1.0f / sqrtf(row_means<SHORT, 1>(a.cols, square, lds[turn][first + 1]).v[0] + a.eps);
            mean = m;
        };
        if (a.pw) {
            float mean, rstd;
            statistics([&](int64_t j) { return (float)in.x[j]; }, 0, mean, rstd);
            in.mean = mean;
            in.rstd = rstd;
        }
        T* s = static_cast<T*>(a.s) + row * (size_t)a.cols;
        each_column<SHORT>(a.cols, [&](int64_t j) { return (T)in.s(j); }, [&](int64_t j, T v) { s[j] = v; });
        float mean = 0.0f, rstd = 1.0f;
        if (w) {
            statistics([&](int64_t j) { return in.s(j); }, 2, mean, rstd);
            T* y = static_cast<T*>(a.y) + row * (size_t)a.cols;
            each_column<SHORT>(
                a.cols, [&](int64_t j) { return (T)((in.s(j) - mean) * rstd * (float)w[j] + (b ? (float)b[j] : 0.0f)); },
                [&](int64_t j, T v) { y[j] = v; });
        }
        if (a.stats && threadIdx.x == 0) {
            const f32x4_t stats = {in.mean, in.rstd, mean, rstd};
            *reinterpret_cast<Stats*>(a.stats + 4 * row) = stats;
        }
    }
}
// dresidual's value at column j of a row, given the means of c = dy weight and of c shat
template <class T, class W> struct AnyGrad : AnyRow<T, W> {
    const T *dy, *ds;
    const W* w;
    float smean, srstd, p, q;
    __device__ __forceinline__ AnyGrad(const AddNormArgs& a, size_t row)
        : AnyRow<T, W>(a, row), dy(a.w ? static_cast<const T*>(a.dy) + row * (size_t)a.dy_stride : nullptr),
          ds(a.ds ? static_cast<const T*>(a.ds) + row * (size_t)a.ds_stride : nullptr), w(static_cast<const W*>(a.w)), p(0.0f),
          q(0.0f)
    {
        const f32x4_t stats = *reinterpret_cast<const Stats*>(a.stats + 4 * row);
        this->mean = stats[0];
        this->rstd = stats[1];
        smean = stats[2];
        srstd = stats[3];
    }
    __device__ __forceinline__ float shat(int64_t j) const { return (this->s(j) - smean) * srstd; }
    __device__ __forceinline__ float dr(int64_t j) const
    {
        const float d = ds ? (float)ds[j] : 0.0f;
        return w ? fmaf(srstd, fmaf(-shat(j), q, fmaf((float)dy[j], (float)w[j], -p)), d) : d;
    }
};
template <class T, class W, bool SHORT> __global__ void __launch_bounds__(kThreads) add_norm_dx_any_kernel(AddNormArgs a)
{
    __shared__ RowSums<2> lds[2][2][kThreads / 64];
    int turn = 0;
    for (size_t row = blockIdx.x; row < (size_t)a.rows; row += gridDim.x, turn ^= 1) {
        AnyGrad<T, W> in(a, row);
        if (a.w) {
            const auto terms = [&](int64_t j) {
                const float c = (float)in.dy[j] * (float)in.w[j];
                return Values<2>{c, c * in.shat(j)};
            };
            const Values<2> m = row_means<SHORT, 2>(a.cols, terms, lds[turn][0]);
            in.p = a.layer ? m.v[0] : 0.0f;
            in.q = m.v[1];
        }
        if (a.w && threadIdx.x == 0) {
            a.row_sums[2 * row] = in.p;
            a.row_sums[2 * row + 1] = in.q;
        }
        const size_t at = row * (size_t)a.cols;
        T *dr = static_cast<T*>(a.dr), *dg = in.g ? static_cast<T*>(a.dgate) : nullptr, *dx = static_cast<T*>(a.dx);
        if (dr) each_column<SHORT>(a.cols, [&](int64_t j) { return (T)in.dr(j); }, [&](int64_t j, T v) { dr[at + j] = v; });
        if (dg)
            each_column<SHORT>(
                a.cols, [&](int64_t j) { return (T)(a.scale * in.dr(j) * in.t(j)); }, [&](int64_t j, T v) { dg[at + j] = v; });
        if (!dx) continue;
        const auto c2 = [&](int64_t j) { return a.scale * in.gate(j) * in.dr(j) * (in.pw ? (float)in.pw[j] : 1.0f); };
        float p = 0.0f, q = 0.0f;
        if (in.pw) {
            const auto terms = [&](int64_t j) {
                const float c = c2(j);
                return Values<2>{c, c * in.xhat(j)};
            };
            const Values<2> m = row_means<SHORT, 2>(a.cols, terms, lds[turn][1]);
            p = a.layer ? m.v[0] : 0.0f;
            q = m.v[1];
        }
        each_column<SHORT>(
            a.cols, [&](int64_t j) { return (T)(in.pw ? in.rstd * fmaf(-in.xhat(j), q, c2(j) - p) : c2(j)); },
            [&](int64_t j, T v) { dx[at + j] = v; });
    }
}
// Column sums of one strip of rows: thread per column.
template <class T, class W>
__global__ void __launch_bounds__(kThreads) add_norm_strip_any_kernel(AddNormArgs a, int strip_rows)
{
    const int64_t j = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (j >= a.cols) return;
    const int64_t r0 = (int64_t)blockIdx.y * strip_rows, r1 = min((int64_t)a.rows, r0 + strip_rows);
    float dw = 0.0f, db = 0.0f, sum = 0.0f;
#pragma unroll 4
    for (int64_t r = r0; r < r1; ++r) {
        AnyGrad<T, W> in(a, (size_t)r);
        if (a.w) {
            in.p = a.row_sums[2 * (size_t)r];
            in.q = a.row_sums[2 * (size_t)r + 1];
        }
        if (a.w) {
            const float d = (float)in.dy[j];
            dw = fmaf(d, in.shat(j), dw);
            db += d;
        }
        if (in.gc || in.pw) sum = fmaf(in.g ? in.dr(j) * in.gate(j) : in.dr(j), in.xhat(j), sum);
    }
    float* p = a.partial + (size_t)blockIdx.y * kNormSums * (size_t)a.cols + j;
    p[0] = dw;
    p[(size_t)a.cols] = db;
    p[2 * (size_t)a.cols] = sum;
}

}  // namespace

hipError_t launch_join(const JoinArgs& a, int out_dt, hipStream_t stream)
{
    const dim3 grid((unsigned)std::min<int64_t>(a.results * ceil_div(a.cols, 64), kMaxRowGrid));
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

hipError_t launch_add_norm(const AddNormArgs& a, int dt, int wdt, hipStream_t stream)
{
    return with_types(dt, wdt, [&](auto x, auto w) {
        using T = decltype(x);
        using W = decltype(w);
        const int chunks = row_chunks(a.cols, sizeof(T)), waves = (int)ceil_div(chunks, 64);
        if (chunks == 0 || waves > 32)
            return start(a.cols <= kThreads ? &add_norm_any_kernel<T, W, true> : &add_norm_any_kernel<T, W, false>,
                         dim3(any_grid(a.rows)), kThreads, stream, a);
        // as many workgroups as a device holds of these kernels' 20 waves a CU (4097 x 3001
        // fp16 29.5 us; with four times as many, each of fewer rows, 34; 16384 x 8192 bf16
        // 194 and 217)
        const auto go = [&](auto kernel, int rows_here, int row_waves) {
            const int grid = even_grid(a.rows, rows_here, kNumCUs * std::max(1, 20 / (rows_here * row_waves)));
            return start(kernel, dim3(grid), 64 * rows_here * row_waves, stream, a, row_waves);
        };
        return waves == 1    ? go(&add_norm_kernel<T, W, true, 1>, kThreads / 64, 1)
               : waves <= 16 ? go(&add_norm_kernel<T, W, false, 1>, 1, waves)
                             : go(&add_norm_kernel<T, W, false, 2>, 1, (waves + 1) / 2);
    });
}

// Workgroups of the backward pass, each of which leaves one strip of sums: one a CU, whatever
// the rows' length.  (Of short rows a workgroup takes up to 16 at a time, so that of a few
// hundred rows some have none and leave zeros.)
int add_norm_strips(int64_t rows)
{
    return rows == 0 ? 0 : even_grid(rows, 1, 256);
}

hipError_t launch_add_norm_backward(const AddNormArgs& a, int dt, int wdt, hipStream_t stream)
{
    if (a.rows == 0) return hipSuccess;
    const int strips = add_norm_strips(a.rows);
    return with_types(dt, wdt, [&](auto x, auto w) {
        using T = decltype(x);
        using W = decltype(w);
        const int chunks = row_chunks(a.cols, sizeof(T)), waves = (int)ceil_div(chunks, 64);
        if (chunks > 0 && waves <= 16)
            return start(&add_norm_backward_kernel<T, W, 1>, dim3(strips), 64 * waves * (16 / waves), stream, a, waves);
        hipError_t e;
        if (chunks > 0 && waves <= 32) {
            e = start(&add_norm_backward_kernel<T, W, 2>, dim3(strips), 64 * ((waves + 1) / 2), stream, a, (waves + 1) / 2);
            if (sizeof(T) == 4) return e;
        } else {
            e = start(a.cols <= kThreads ? &add_norm_dx_any_kernel<T, W, true> : &add_norm_dx_any_kernel<T, W, false>,
                      dim3(any_grid(a.rows)), kThreads, stream, a);
        }
        if (e == hipSuccess && (a.w || a.gate || a.pw))
            e = start(&add_norm_strip_any_kernel<T, W>, dim3((unsigned)ceil_div(a.cols, kThreads), strips), kThreads, stream, a,
                      (int)ceil_div(a.rows, strips));
        return e;
    });
}

}  // namespace gemm_relu_hip
