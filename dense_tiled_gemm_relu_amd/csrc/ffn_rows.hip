// Row-wise and element-wise kernels of the feed-forward operators: layer norm
// forward and backward, the gated projections' element-wise gradient, and the
// quantisation of rows to 8 bits.
#include <algorithm>
#include <type_traits>

#include "api_common.hpp"
#include "ffn.hpp"
#include "row_common.hpp"

namespace gemm_relu_hip {

namespace {

// ------------------------------------------------------------- layer norm
// One read and one write of the row: it stays in registers between the mean,
// the squares around it (so a large common offset costs no digits) and the
// output; the next row of the group is loaded meanwhile, and the weight and the
// bias stay in registers over all of its rows.  Bound by HBM: 16384 x 8192 bf16 in
// 92.5 us, 5.8 TB/s (a plain copy of 512 MB runs at 5.55); odd rows too: 4097 x 3001
// fp16 10.4 us, 4.7 TB/s.
template <class T, class W, int G, int V> __global__ void __launch_bounds__(kGroupThreads<G>) layer_norm_kernel(NormArgs a)
{
    constexpr int N = Chunk<T>::N;
    using X = typename Chunk<T>::Vec;
    using WV = typename VecN<W, N>::Vec;
    __shared__ float lds[2][G / 64];
    const RowMap<T, V> map(a.cols, (int)threadIdx.x % G, G);
    WV w[V], b[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        w[v] = b[v] = WV{};
        if (map.has(v)) {
            w[v] = load_vec<WV>(static_cast<const W*>(a.w) + map.start[v]);
            if (a.b) b[v] = load_vec<WV>(static_cast<const W*>(a.b) + map.start[v]);
        }
    }
    const int step = (int)gridDim.x * kGroups<G>;
    int64_t row = group_index<G>();          // 64 bits: the last row's successor may pass 2^31
    X next[V];
    auto fetch = [&](int64_t r) {
        const T* x = static_cast<const T*>(a.x) + (size_t)r * (size_t)a.x_stride;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (map.has(v)) next[v] = load_vec<X>(x + map.start[v]);
    };
#pragma unroll
    for (int v = 0; v < V; ++v) next[v] = X{};
    if (row < a.rows) fetch(row);
    const float n = (float)a.cols;
    for (; row < a.rows; row += step) {
        X x[V];
#pragma unroll
        for (int v = 0; v < V; ++v) x[v] = next[v];
        if (row < a.rows - step) fetch(row + step);
        float s = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int e = 0; e < N; ++e) s += map.owns(v, e) ? (float)x[v][e] : 0.0f;
        const float mean = group_all<G, Sum>(s, lds[0]) / n;
        s = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float d = map.owns(v, e) ? (float)x[v][e] - mean : 0.0f;
                s += d * d;
            }
        const float rstd = 1.0f / sqrtf(group_all<G, Sum>(s, lds[1]) / n + a.eps);
        T* y = static_cast<T*>(a.y) + (size_t)row * (size_t)a.cols;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (map.has(v)) {
                X out;
#pragma unroll
                for (int e = 0; e < N; ++e)
                    out[e] = (T)(((float)x[v][e] - mean) * rstd * (float)w[v][e] + (float)b[v][e]);
                __builtin_memcpy(y + map.start[v], &out, sizeof out);
            }
        if (threadIdx.x % G == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
    }
}

// The backward pass in one read of dy and x: the row's two sums and dx, and the
// thread's columns of dweight and dbias, summed in registers over its rows.  A
// workgroup leaves one strip of partial sums; a second kernel joins the strips in
// order.  ONE: four rows a workgroup, one wave each; else `waves` waves a row, as
// many as it has chunks for, and as many rows at a time as 16 waves hold.
//
// A row takes a trip to memory, two sums over the group and a store, and a CU
// holds few rows at a time (the sums fill its registers), so the rows to come are
// copied ahead into LDS, RING of them: each lane's own 16 bytes, which no other
// lane reads, so the only wait is the wave's own.  Large batches are bound by HBM
// (16384 x 8192 bf16 155 us with the join, 5.2 TB/s), smaller ones by the rows a
// workgroup takes in turn and by starting, leaving and joining the strips (4097 x
// 3001 fp16 22 us with the join, 3.4 TB/s).
template <class T, class W, bool ONE, int V>
__global__ void __launch_bounds__(ONE ? kThreads : 1024) __attribute__((amdgpu_waves_per_eu(4)))
layer_norm_backward_kernel(NormArgs a, int waves)
{
    constexpr int N = Chunk<T>::N;
    using X = typename Chunk<T>::Vec;
    using WV = typename VecN<W, N>::Vec;
    constexpr int RING = V == 1 ? 4 : 2, ROW_BYTES = 2 * V * 1024;       // of a wave
    constexpr int RINGS = ONE ? kThreads / 64 : 16;
    __shared__ __attribute__((aligned(1024))) unsigned char rows_raw[RINGS * RING * ROW_BYTES];
    __shared__ float lds[2][2][16];
    static_assert(RINGS * 64 * N * V * 4 <= RINGS * RING * ROW_BYTES, "the waves' sums fit the rings");
    const int lane = (int)(threadIdx.x & 63), wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int groups = ONE ? RINGS : (int)(blockDim.x >> 6) / waves, group = ONE ? wave : wave / waves;
    const int in_row = ONE ? 0 : wave - group * waves;                    // the wave's place in its row
    const RowMap<T, V> map(a.cols, in_row * 64 + lane, ONE ? 64 : 64 * waves);
    WV w[V];
    float dw[V][N], db[V][N];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        w[v] = load_vec<WV>(static_cast<const W*>(a.w) + map.start[v]);
#pragma unroll
        for (int e = 0; e < N; ++e) dw[v][e] = db[v][e] = 0.0f;
    }
    const int64_t step = (int64_t)gridDim.x * groups;
    int64_t row = (int64_t)blockIdx.x * groups + group;
    const int64_t first_row = row - group;
    GR_LDS unsigned char* const ring = (GR_LDS unsigned char*)rows_raw + wave * RING * ROW_BYTES;
    // row r (the last one in place of those past it) to a slot; a missing chunk is
    // the row's last
    auto fetch = [&](int64_t r, int slot) {
        const size_t at = (size_t)min(r, (int64_t)a.rows - 1);
        const T* x = static_cast<const T*>(a.x) + at * (size_t)a.x_stride;
        const T* d = static_cast<const T*>(a.dy) + at * (size_t)a.dy_stride;
        const uint32_t to = lds_addr(ring) + slot * ROW_BYTES;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            copy_to_lds(reinterpret_cast<const unsigned char*>(x + map.start[v]), to + 2 * v * 1024);
            copy_to_lds(reinterpret_cast<const unsigned char*>(d + map.start[v]), to + (2 * v + 1) * 1024);
        }
    };
#pragma unroll
    for (int k = 0; k < RING; ++k) fetch(row + k * step, k);
    // the weight has arrived here, so that no load but the copies is waited for below
#pragma unroll
    for (int v = 0; v < V; ++v) stay_packed(w[v]);
    const float inv_n = 1.0f / (float)a.cols;
    // one value for the whole wave: read through the scalar cache
    typedef const __attribute__((address_space(4))) float* Scalars;
    const Scalars means = (Scalars)(uintptr_t)a.mean, rstds = (Scalars)(uintptr_t)a.rstd;
    int slot = 0;
    // all rows of a workgroup meet at one barrier, so a row past the end runs along
    // with nothing to add and nothing to store
    const int64_t behind = ONE ? 0 : row - first_row;
    for (int turn = 0; row - behind < a.rows; row += step, turn ^= 1) {
        const bool live = ONE || row < a.rows;
        const int64_t at = min(row, (int64_t)a.rows - 1);
        const float mean = means[at], rstd = rstds[at];
        // behind this row's copies are those of RING - 1 rows; the stores between
        // them only make the wait stricter
        __builtin_amdgcn_s_waitcnt(waitcnt_vm((RING - 1) * 2 * V));
        asm volatile("" ::: "memory");
        X x[V], d[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const GR_LDS unsigned char* from = ring + slot * ROW_BYTES + 2 * v * 1024 + lane * 16;
            x[v] = __builtin_bit_cast(X, lds_read_b128(from));
            d[v] = __builtin_bit_cast(X, lds_read_b128(from + 1024));
            stay_packed(x[v]);
            stay_packed(d[v]);
            if (V > 1) stay_packed(w[v]);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");      // read, so the slot is free
        fetch(row + RING * step, slot);
        slot = slot == RING - 1 ? 0 : slot + 1;
        // c = dy weight: s0 = sum c, s1 = sum c xhat.  Elements that the neighbour
        // owns count in its sums only (and its columns: these are not stored).
        float s0 = 0.0f, s1 = 0.0f, xhat[V][N], c[V][N];
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float g = (float)d[v][e];
                xhat[v][e] = ((float)x[v][e] - mean) * rstd;
                c[v][e] = g * (float)w[v][e];
                if (live) {
                    dw[v][e] = fmaf(g, xhat[v][e], dw[v][e]);
                    db[v][e] += g;
                }
                const float own = map.owns(v, e) ? c[v][e] : 0.0f;
                s0 += own;
                s1 = fmaf(own, map.owns(v, e) ? xhat[v][e] : 0.0f, s1);
            }
        // both sums at once: s0 in the lower half of the wave, s1 in the upper
        const auto p = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(unsigned, s0), __builtin_bit_cast(unsigned, s1),
                                                        false, false);
        float s = __builtin_bit_cast(float, (unsigned)p[0]) + __builtin_bit_cast(float, (unsigned)p[1]);
        const auto q = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, s), __builtin_bit_cast(unsigned, s),
                                                        false, false);
        s = row16_sum(__builtin_bit_cast(float, (unsigned)q[0]) + __builtin_bit_cast(float, (unsigned)q[1]));
        if constexpr (!ONE) {
            // lane 0 and lane 32 hold the wave's; 16 lanes each add the waves'
            if ((lane & 31) == 0) lds[turn][lane >> 5][wave] = s;
            __syncthreads();
            const int k = lane & 15;
            s = row16_sum(k < waves ? lds[turn][lane >> 5][group * waves + k] : 0.0f);
        }
        s0 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, s), 0)) * inv_n * rstd;
        s1 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, s), 32)) * inv_n * rstd;
        T* dx = static_cast<T*>(a.dx) + (size_t)row * (size_t)a.cols;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (map.has(v) && live) {
                X out;
#pragma unroll
                for (int e = 0; e < N; ++e) out[e] = (T)fmaf(-xhat[v][e], s1, fmaf(c[v][e], rstd, -s0));
                __builtin_memcpy(dx + map.start[v], &out, sizeof out);
            }
    }
    // the ring's last copies, of rows past the end, land before its memory is used
    // again or given back
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
    asm volatile("" ::: "memory");
    // the groups' sums join first, in order
    GR_LDS float* const part = (GR_LDS float*)rows_raw;
    const int per_row = ONE ? 1 : waves;
    float* strip = a.partial + (size_t)blockIdx.x * 2 * (size_t)a.cols;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        float(&own)[V][N] = half ? db : dw;
        __syncthreads();
        if (group) {
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int e = 0; e < N; ++e) part[((wave * V + v) * N + e) * 64 + lane] = own[v][e];
        }
        __syncthreads();
        if (group) continue;
        for (int k = 1; k < groups; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int e = 0; e < N; ++e) own[v][e] += part[(((k * per_row + in_row) * V + v) * N + e) * 64 + lane];
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (map.has(v)) {
                float* to = strip + (size_t)half * a.cols + map.start[v];
                if (v < V - 1 || map.skip == 0) {
#pragma unroll
                    for (int e = 0; e < N; e += 4) {
                        const f32x4_t four = {own[v][e], own[v][e + 1], own[v][e + 2], own[v][e + 3]};
                        __builtin_memcpy(to + e, &four, 16);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < N; ++e)
                        if (e >= map.skip) to[e] = own[v][e];
                }
            }
    }
}

// Few rows: the whole backward pass in one launch, since a second one would take
// longer than the work (256 x 4096 bf16 4.1 us against 8.7 in two launches; 512 x
// 1001 5.4 against 8.0; 1024 x 256 8.1 against 6.3).  The first workgroups take rows (as many waves a row as it
// has chunks for, rounded up to a power of two) and write dx; the others take 64
// columns each over all rows, which they read a second time from the L2, and write
// dweight and dbias.
constexpr int kFewRows = 512;
template <class T, class W, int V>
__global__ void __launch_bounds__(1024) layer_norm_backward_few_kernel(NormArgs a, int row_blocks, int waves)
{
    constexpr int N = Chunk<T>::N;
    using X = typename Chunk<T>::Vec;
    using WV = typename VecN<W, N>::Vec;
    __shared__ float lds[2][16][64];
    const int lane = (int)(threadIdx.x & 63), wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    typedef const __attribute__((address_space(4))) float* Scalars;
    const Scalars means = (Scalars)(uintptr_t)a.mean, rstds = (Scalars)(uintptr_t)a.rstd;
    if ((int)blockIdx.x < row_blocks) {
        const int rows_here = 16 / waves, first = wave & ~(waves - 1);
        const int wanted = (int)blockIdx.x * rows_here + wave / waves, row = min(wanted, a.rows - 1);
        const RowMap<T, V> map(a.cols, (wave - first) * 64 + lane, 64 * waves);
        const T* x = static_cast<const T*>(a.x) + (size_t)row * (size_t)a.x_stride;
        const T* d = static_cast<const T*>(a.dy) + (size_t)row * (size_t)a.dy_stride;
        float xhat[V][N], c[V][N], s0 = 0.0f, s1 = 0.0f;
        const float mean = means[row], rstd = rstds[row];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const X xv = load_vec<X>(x + map.start[v]), dv = load_vec<X>(d + map.start[v]);
            const WV w = load_vec<WV>(static_cast<const W*>(a.w) + map.start[v]);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                xhat[v][e] = ((float)xv[e] - mean) * rstd;
                c[v][e] = (float)dv[e] * (float)w[e];
                const float own = map.owns(v, e) ? c[v][e] : 0.0f;
                s0 += own;
                s1 = fmaf(own, map.owns(v, e) ? xhat[v][e] : 0.0f, s1);
            }
        }
        s0 = wave_all<Sum>(s0);
        s1 = wave_all<Sum>(s1);
        if (lane == 0) {
            lds[0][wave][0] = s0;
            lds[1][wave][0] = s1;
        }
        __syncthreads();
        s0 = s1 = 0.0f;
        for (int k = 0; k < waves; ++k) {
            s0 += lds[0][first + k][0];
            s1 += lds[1][first + k][0];
        }
        const float inv_n = 1.0f / (float)a.cols;
        s0 *= inv_n * rstd;
        s1 *= inv_n * rstd;
        T* dx = static_cast<T*>(a.dx) + (size_t)row * (size_t)a.cols;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (map.has(v) && wanted < a.rows) {
                X out;
#pragma unroll
                for (int e = 0; e < N; ++e) out[e] = (T)fmaf(-xhat[v][e], s1, fmaf(c[v][e], rstd, -s0));
                __builtin_memcpy(dx + map.start[v], &out, sizeof out);
            }
        return;
    }
    const int j = ((int)blockIdx.x - row_blocks) * 64 + lane, col = min(j, a.cols - 1);
    float dw = 0.0f, db = 0.0f;
#pragma unroll 4
    for (int r = wave; r < a.rows; r += 16) {
        const float g = (float)static_cast<const T*>(a.dy)[(size_t)r * (size_t)a.dy_stride + col];
        const float v = (float)static_cast<const T*>(a.x)[(size_t)r * (size_t)a.x_stride + col];
        dw = fmaf(g, (v - means[r]) * rstds[r], dw);
        db += g;
    }
    lds[0][wave][lane] = dw;
    lds[1][wave][lane] = db;
    __syncthreads();
    if (wave > 1 || j >= a.cols) return;
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < 16; ++k) s += lds[wave][k][lane];
    if (wave == 0)
        static_cast<W*>(a.dw)[j] = (W)s;
    else if (a.db)
        static_cast<W*>(a.db)[j] = (W)s;
}

template <class T, class W, bool SHORT> __global__ void __launch_bounds__(kThreads) layer_norm_any_kernel(NormArgs a)
{
    __shared__ RowSums<1> lds[2][kThreads / 64];
    const W* w = static_cast<const W*>(a.w);
    const W* b = static_cast<const W*>(a.b);
    for (size_t row = blockIdx.x; row < (size_t)a.rows; row += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + row * (size_t)a.x_stride;
        T* y = static_cast<T*>(a.y) + row * (size_t)a.cols;
        const float mean = row_means<SHORT, 1>(a.cols, [&](int64_t j) { return Values<1>{(float)x[j]}; }, lds[0]).v[0];
        const auto square = [&](int64_t j) {
            const float d = (float)x[j] - mean;
            return Values<1>{d * d};
        };
        const float rstd = 1.0f / sqrtf(row_means<SHORT, 1>(a.cols, square, lds[1]).v[0] + a.eps);
        each_column<SHORT>(
            a.cols, [&](int64_t j) { return (T)(((float)x[j] - mean) * rstd * (float)w[j] + (b ? (float)b[j] : 0.0f)); },
            [&](int64_t j, T v) { y[j] = v; });
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[row] = mean;
            if (a.rstd) a.rstd[row] = rstd;
        }
    }
}
template <class T, class W, bool SHORT> __global__ void __launch_bounds__(kThreads) layer_norm_dx_any_kernel(NormArgs a)
{
    __shared__ RowSums<2> lds[2][kThreads / 64];
    const W* w = static_cast<const W*>(a.w);
    int turn = 0;
    for (size_t row = blockIdx.x; row < (size_t)a.rows; row += gridDim.x, turn ^= 1) {
        const T* x = static_cast<const T*>(a.x) + row * (size_t)a.x_stride;
        const T* dy = static_cast<const T*>(a.dy) + row * (size_t)a.dy_stride;
        T* dx = static_cast<T*>(a.dx) + row * (size_t)a.cols;
        const float mean = a.mean[row], rstd = a.rstd[row];
        const auto c_xhat = [&](int64_t j) { return Values<2>{(float)dy[j] * (float)w[j], ((float)x[j] - mean) * rstd}; };
        const auto terms = [&](int64_t j) {
            const Values<2> v = c_xhat(j);
            return Values<2>{v.v[0], v.v[0] * v.v[1]};
        };
        const Values<2> s = row_means<SHORT, 2>(a.cols, terms, lds[turn]);
        const float s0 = s.v[0], s1 = s.v[1];
        each_column<SHORT>(a.cols, c_xhat, [&](int64_t j, Values<2> v) { dx[j] = (T)(rstd * (v.v[0] - s0 - v.v[1] * s1)); });
    }
}
// Column sums of one strip of rows: thread per column.
template <class T, class W>
__global__ void __launch_bounds__(kThreads) layer_norm_strip_any_kernel(NormArgs a, int strip_rows)
{
    const int j = blockIdx.x * kThreads + threadIdx.x;
    if (j >= a.cols) return;
    const int64_t r0 = (int64_t)blockIdx.y * strip_rows, r1 = min((int64_t)a.rows, r0 + strip_rows);
    float dw = 0.0f, db = 0.0f;
    for (int64_t r = r0; r < r1; ++r) {
        const float g = (float)static_cast<const T*>(a.dy)[(size_t)r * (size_t)a.dy_stride + j];
        const float v = (float)static_cast<const T*>(a.x)[(size_t)r * (size_t)a.x_stride + j];
        dw += g * ((v - a.mean[r]) * a.rstd[r]);
        db += g;
    }
    float* p = a.partial + (size_t)blockIdx.y * 2 * (size_t)a.cols;
    p[j] = dw;
    p[(size_t)a.cols + j] = db;
}

// The strips' sums, in order: 64 columns a workgroup, each of 16 waves takes every
// 16th strip.
template <class W> __global__ void __launch_bounds__(1024) layer_norm_join_kernel(NormArgs a, int strips)
{
    __shared__ float part[16][64];
    const int lane = (int)(threadIdx.x & 63), wave = (int)(threadIdx.x >> 6);
    const int64_t all = 2 * (int64_t)a.cols;
    for (int64_t j0 = (int64_t)blockIdx.x * 64; j0 < all; j0 += (int64_t)gridDim.x * 64) {
        const int64_t j = j0 + lane;
        float s = 0.0f;
        if (j < all) {
            // a wave's strips in batches of 8, all loads of one in flight together
            // (strips past the end are the last one's, and count for nothing)
            for (int k = wave; k < strips; k += 16 * 8) {
                float v[8];
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    v[u] = a.partial[(size_t)min(k + 16 * u, strips - 1) * (size_t)all + j];
#pragma unroll
                for (int u = 0; u < 8; ++u) s += k + 16 * u < strips ? v[u] : 0.0f;
            }
        }
        part[wave][lane] = s;
        __syncthreads();
        if (!wave && j < all) {
#pragma unroll
            for (int k = 1; k < 16; ++k) s += part[k][lane];
            if (j < a.cols)
                static_cast<W*>(a.dw)[j] = (W)s;
            else if (a.db)
                static_cast<W*>(a.db)[j - a.cols] = (W)s;
        }
        __syncthreads();
    }
}

// --------------------------------------------- gradient of act(g) u
// A 64 x 64 tile of (rows, hidden), 2 x 4 elements a thread (more would only make
// its code longer, and a short call waits for code too) with all loads issued
// before the first is used: dg and du go out row-major, and transposed through
// LDS.  Both outputs' rows are padded to 16 bytes with zeros, so that the
// products may read them in whole pieces.  Bound by HBM: 4096 x 7168 bf16 reads and
// writes 0.53 GB in 89 us, 5.9 TB/s.
//
// A finite value whose rounding to float16 is an infinity is noted, for
// gated_repair_kernel.
constexpr float kHalfOver = 65520.0f;              // half a step above the largest float16, the first that rounds up
__device__ __forceinline__ bool passes_half(float v) { return fabsf(v) >= kHalfOver && fabsf(v) < INFINITY; }
template <int ACT> __device__ __forceinline__ void gated_slopes(float d, float g, float u, float& dg, float& du)
{
    float value, slope;
    activation_slope<ACT>(g, value, slope);
    dg = d * u * slope;
    du = d * value;
}
template <int DT, int ACT> __global__ void __launch_bounds__(kGradThreads) gated_grad_kernel(GatedGradArgs a)
{
    using T = typename Elem<DT>::T;
    typedef T T4 __attribute__((ext_vector_type(4)));
    typedef T T2 __attribute__((ext_vector_type(2)));
    constexpr int ROWS = 64 * 16 / kGradThreads;
    constexpr int PITCH = 68;                      // elements of a transposed row: 8-byte pieces on spread banks
    __shared__ __attribute__((aligned(16))) T tile[2][64][PITCH];
    __shared__ GradMask over[3];
    if constexpr (DT == DT_F16) {
        if (threadIdx.x < 3) over[threadIdx.x] = 0;
        __syncthreads();
    }
    const int htiles = (a.hidden + 63) / 64;
    const int h0 = (int)(blockIdx.x % htiles) * 64, r0 = (int)(blockIdx.x / htiles) * 64;
    if (blockIdx.x == 0)
        for (int k = threadIdx.x; k < a.nflags; k += kGradThreads) a.flags[k] = 0u;
    const int c = (int)(threadIdx.x & 15) * 4, h = h0 + c, q = (int)(threadIdx.x >> 4) * ROWS;
    const bool whole = h + 4 <= a.hidden;
    f32x4_t g[ROWS], u[ROWS];
    T4 d[ROWS];
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
        g[k] = u[k] = f32x4_t{};
        d[k] = T4{};
        const int r = r0 + q + k;
        if (r >= a.rows) continue;
        const float* gu = a.gu + (size_t)r * 2 * (size_t)a.hidden + h;
        const T* dh = static_cast<const T*>(a.dh) + (size_t)r * (size_t)a.dh_stride + h;
        if (whole) {
            g[k] = load_vec<f32x4_t>(gu);
            u[k] = load_vec<f32x4_t>(gu + a.hidden);
            d[k] = load_vec<T4>(dh);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (h + e < a.hidden) {
                    g[k][e] = gu[e];
                    u[k][e] = gu[a.hidden + e];
                    d[k][e] = dh[e];
                }
        }
    }
    T4 dg[ROWS], du[ROWS];
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
        float gate[4], up[4], top = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            gated_slopes<ACT>((float)d[k][e], g[k][e], u[k][e], gate[e], up[e]);
            dg[k][e] = (T)gate[e];
            du[k][e] = (T)up[e];
            top = fmaxf(top, fmaxf(fabsf(gate[e]), fabsf(up[e])));
        }
        if (DT == DT_F16 && top >= kHalfOver) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool in_gate = passes_half(gate[e]), in_up = passes_half(up[e]);
                if (in_gate) atomicOr(&over[1], 1ull << (c + e));
                if (in_up) atomicOr(&over[2], 1ull << (c + e));
                if (in_gate || in_up) atomicOr(&over[0], 1ull << (q + k));
            }
        }
        const int r = r0 + q + k;
        if (r >= a.rows) continue;
        T* out = static_cast<T*>(a.dgu) + (size_t)r * (size_t)a.ld + h;
        if (whole) {
            __builtin_memcpy(out, &dg[k], 8);
            __builtin_memcpy(out + a.hidden, &du[k], 8);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (h + e < a.hidden) {
                    out[e] = dg[k][e];
                    out[a.hidden + e] = du[k][e];
                }
        }
        // the row's padding, by the thread behind its last tile column
        if (h0 + 64 >= a.hidden && c == 60)
            for (int j = 2 * a.hidden; j < a.ld; ++j) static_cast<T*>(a.dgu)[(size_t)r * (size_t)a.ld + j] = (T)0.0f;
    }
    // rows past the edge hold d = 0: their dg and du are the transposed padding
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const T2 x = {dg[0][e], dg[1][e]}, y = {du[0][e], du[1][e]};
        *reinterpret_cast<T2*>(&tile[0][c + e][q]) = x;
        *reinterpret_cast<T2*>(&tile[1][c + e][q]) = y;
    }
    __syncthreads();
    if constexpr (DT == DT_F16)
        if (threadIdx.x < 3) a.over[(size_t)threadIdx.x * gridDim.x + blockIdx.x] = over[threadIdx.x];
#pragma unroll
    for (int k = 0; k < 1024 / kGradThreads; ++k) {
        const int p = k * kGradThreads + (int)threadIdx.x, half = p >> 9, hh = (p >> 3) & 63, rr = (p & 7) * 8;
        if (h0 + hh >= a.hidden || r0 + rr >= a.rows) continue;
        const T4* from = reinterpret_cast<const T4*>(&tile[half][hh][rr]);
        T* out = static_cast<T*>(a.dgu_t) + ((size_t)(h0 + hh) + (half ? (size_t)a.hidden : 0)) * (size_t)a.ld_t + r0 + rr;
        const T4 lo = from[0], hi = from[1];
        __builtin_memcpy(out, &lo, 8);
        __builtin_memcpy(out + 4, &hi, 8);
    }
}

// ---- where float16 cannot hold dg or du
// The products' operands are 16-bit, so a finite dg or du above 65504 has become an
// infinity, and with it its row of dx and its row of dweight, whose own values may
// be far inside the range (weights are small).  These rows are summed here once more,
// in fp32 from dg and du as they are.  A row counts if any of its elements passes the
// range; the others keep the products' results, whatever shares their tile.
//
// One launch more for float16, whose workgroups read the notes of all tiles and end
// there, 4 us (5 at 4096 x 7168 x 4096), but for gradients that large.  Then it takes
// 0.5 ms (one element) to 1 ms at 1027 x 2003 x 1501, 3.3 to 26 at 4096 x 7168 x 4096,
// bound by its steps' latency: 64 x 64 outputs a workgroup, 4 x 4 a thread, 16 K elements
// of both operands a step in LDS, for a case that a loss scale meets once in a while.
// Pieces are dealt out singly so that one large element occupies the device (with a few
// workgroups a block of rows it took 6.6 ms, and 13 us where there is nothing to do).
constexpr int kRepairK = 16;
__device__ __forceinline__ GradMask group_or(GradMask v, GradMask* lds)
{
#pragma unroll
    for (int step = 1; step < 64; step *= 2) v |= __shfl_xor(v, step);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    return lds[0] | lds[1] | lds[2] | lds[3];
}
template <int ACT> __global__ void __launch_bounds__(kThreads) gated_repair_kernel(GatedGradArgs a)
{
    using T = _Float16;
    __shared__ GradMask masks[2][kThreads / 64];
    __shared__ float left[2][kRepairK][64], right[2][kRepairK][64];
    const int tid = (int)threadIdx.x, htiles = (a.hidden + 63) / 64, rtiles = (a.rows + 63) / 64, tiles = htiles * rtiles;
    GradMask any = 0;
#pragma unroll 8
    for (int t = tid; t < tiles; t += kThreads) any |= a.over[t];
    if (!group_or(any, masks[0])) return;

    // 64 columns of 64 rows of dx, or of a 64-unit block of dweight, at a time
    const int col_tiles = (int)(((int64_t)a.cols + 63) / 64);
    const int64_t pieces = (int64_t)(rtiles + htiles) * col_tiles;
    for (int64_t piece = blockIdx.x; piece < pieces; piece += gridDim.x) {
        const int block = (int)(piece / col_tiles);
        const int64_t n0 = piece % col_tiles * 64;
        const bool of_dx = block < rtiles;
        const int m0 = 64 * (of_dx ? block : block - rtiles);       // its first row of dx, or unit
        // what the tiles along the other side found
        GradMask gate = 0, up = 0;
        if (of_dx) {
            for (int t = tid; t < htiles; t += kThreads) gate |= a.over[(size_t)block * htiles + t];
        } else {
            for (int t = tid; t < rtiles; t += kThreads) {
                const size_t at = (size_t)t * htiles + (block - rtiles);
                gate |= a.over[tiles + at];
                up |= a.over[2 * (size_t)tiles + at];
            }
        }
        __syncthreads();                        // the last piece's masks have been read
        gate = group_or(gate, masks[0]);
        up = group_or(up, masks[1]);
        if (!(gate | up)) continue;

        const int K = of_dx ? a.hidden : a.rows, mi = (tid >> 4) * 4, ni = (tid & 15) * 4;
        constexpr int NL = 64 * kRepairK / kThreads, NR = 2 * NL;
        float sums[2][4][4] = {};           // dx: the first only
        for (int k0 = 0; k0 < K; k0 += kRepairK) {
            __syncthreads();                // the last step's reads are done
            // all loads in flight together: what lies past an edge is the last one's, and
            // counts as zero
            float g[NL], u[NL], d[NL], other[NR];
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                const int e = i * kThreads + tid;
                // units are the fastest in memory
                const int m = of_dx ? e / kRepairK : e % 64, k = of_dx ? e % kRepairK : e / 64;
                const size_t row = (size_t)min(of_dx ? m0 + m : k0 + k, a.rows - 1);
                const size_t unit = (size_t)min(of_dx ? k0 + k : m0 + m, a.hidden - 1);
                g[i] = a.gu[row * 2 * (size_t)a.hidden + unit];
                u[i] = a.gu[row * 2 * (size_t)a.hidden + (size_t)a.hidden + unit];
                d[i] = (float)static_cast<const T*>(a.dh)[row * (size_t)a.dh_stride + unit];
            }
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const int e = i * kThreads + tid, k = (e / 64) % kRepairK, half = e / (64 * kRepairK);
                const size_t row = (size_t)min(k0 + k, K - 1) + (of_dx && half ? (size_t)a.hidden : 0);
                const size_t col = (size_t)min(n0 + e % 64, (int64_t)a.cols - 1);
                other[i] = (float)static_cast<const T*>(of_dx ? a.w : a.x)[row * (size_t)(of_dx ? a.w_stride : a.x_stride) + col];
            }
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                const int e = i * kThreads + tid;
                const int m = of_dx ? e / kRepairK : e % 64, k = of_dx ? e % kRepairK : e / 64;
                float dg, du;
                gated_slopes<ACT>(d[i], g[i], u[i], dg, du);
                left[0][k][m] = k0 + k < K ? dg : 0.0f;
                left[1][k][m] = k0 + k < K ? du : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const int e = i * kThreads + tid, k = (e / 64) % kRepairK;
                right[e / (64 * kRepairK)][k][e % 64] = k0 + k < K ? other[i] : 0.0f;
            }
            __syncthreads();
            auto add = [&](int k, int half, float(&s)[4][4]) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[i][j] = fmaf(left[half][k][mi + i], right[half][k][ni + j], s[i][j]);
            };
            for (int k = 0; k < kRepairK; ++k) {
                add(k, 0, sums[0]);
                if (of_dx)
                    add(k, 1, sums[0]);
                else
                    add(k, 1, sums[1]);
            }
        }
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (!((half ? up : gate) >> (mi + i) & 1)) continue;      // of dx: no up
                T* out = static_cast<T*>(of_dx ? a.dx : a.dw) +
                         ((size_t)(m0 + mi + i) + (half ? (size_t)a.hidden : 0)) * (size_t)a.cols + n0 + ni;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (n0 + ni + j < a.cols) out[j] = (T)sums[half][i][j];
            }
    }
}

// ------------------------------------------------------- quantisation
// The largest magnitude is taken over the values' bits without the sign, whose
// order as whole numbers is that of the values with infinities and NaN on top.
// The row is scaled by a power of two (exactly) so that its largest value m is in
// [1/2, 1); then 127 x / m is a product with the reciprocal and one step that adds
// the exact remainder's share, which costs half of a division.  For 16-bit x the
// products and the remainder are exact, the quotient's distance from a rounding
// border is either zero or more than 2^-20 of it, and a quotient on a border,
// being a short number, comes out exactly: the result is that of exact arithmetic.
struct Quantiser {
    int down;
    float m, r;
    __device__ __forceinline__ Quantiser(float top)
    {
        down = -__builtin_amdgcn_frexp_expf(top);
        m = ldexpf(top, down);
        r = __builtin_amdgcn_rcpf(m);
    }
    __device__ __forceinline__ signed char operator()(float x) const
    {
        const float v = 127.0f * ldexpf(x, down), p = v * r;
        return (signed char)(int)rintf(fmaf(fmaf(-p, m, v), r, p));
    }
};
template <class T> __device__ __forceinline__ unsigned magnitude(T x)
{
    if constexpr (sizeof(T) == 2)
        return __builtin_bit_cast(unsigned short, x) & 0x7fffu;
    else
        return __builtin_bit_cast(unsigned, x) & 0x7fffffffu;
}
template <class T> __device__ __forceinline__ float from_magnitude(unsigned m)
{
    if constexpr (sizeof(T) == 2)
        return (float)__builtin_bit_cast(T, (unsigned short)m);
    else
        return __builtin_bit_cast(float, m);
}
struct QuantArgs {
    const void* x;
    signed char* q;
    float* scale;
    int64_t x_stride;
    int rows, cols;
};

// The row stays in registers between its largest value and its quotients.  Bound by
// HBM: 16384 x 8192 bf16 in 81 us, 5.0 TB/s (89 us with a division an element).
template <class T, int G, int V> __global__ void __launch_bounds__(kGroupThreads<G>) quantize_rows_kernel(QuantArgs a)
{
    constexpr int N = Chunk<T>::N;
    using X = typename Chunk<T>::Vec;
    using Q = typename VecN<signed char, N>::Vec;
    __shared__ unsigned lds[2][G / 64];
    const RowMap<T, V> map(a.cols, (int)threadIdx.x % G, G);
    const int step = (int)gridDim.x * kGroups<G>;
    int64_t row = group_index<G>();          // 64 bits: the last row's successor may pass 2^31
    X next[V];
    auto fetch = [&](int64_t r) {
        const T* x = static_cast<const T*>(a.x) + (size_t)r * (size_t)a.x_stride;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (map.has(v)) next[v] = load_vec<X>(x + map.start[v]);
    };
#pragma unroll
    for (int v = 0; v < V; ++v) next[v] = X{};
    if (row < a.rows) fetch(row);
    for (int turn = 0; row < a.rows; row += step, turn ^= 1) {
        X x[V];
#pragma unroll
        for (int v = 0; v < V; ++v) x[v] = next[v];
        if (row < a.rows - step) fetch(row + step);
        unsigned most = 0;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int e = 0; e < N; ++e) most = Max::of(most, magnitude<T>(x[v][e]));
        const float top = from_magnitude<T>(group_all<G, Max>(most, lds[turn]));
        const bool bad = !(top < INFINITY), empty = bad || top == 0.0f;
        const Quantiser quantise(top);
        signed char* q = a.q + (size_t)row * (size_t)a.cols;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (map.has(v)) {
                Q out = Q{};
                if (!empty) {
#pragma unroll
                    for (int e = 0; e < N; ++e) out[e] = quantise((float)x[v][e]);
                }
                __builtin_memcpy(q + map.start[v], &out, sizeof out);
            }
        if (threadIdx.x % G == 0) a.scale[row] = bad ? NAN : top / 127.0f;
    }
}
template <class T, bool SHORT> __global__ void __launch_bounds__(kThreads) quantize_rows_any_kernel(QuantArgs a)
{
    __shared__ unsigned lds[2][4];
    int turn = 0;
    for (size_t row = blockIdx.x; row < (size_t)a.rows; row += gridDim.x, turn ^= 1) {
        const T* x = static_cast<const T*>(a.x) + row * (size_t)a.x_stride;
        signed char* q = a.q + row * (size_t)a.cols;
        unsigned most = 0;
        each_column<SHORT>(
            a.cols, [&](int64_t j) { return x[j]; }, [&](int64_t, T v) { most = Max::of(most, magnitude<T>(v)); });
        const float top = from_magnitude<T>(group_all<kThreads, Max>(most, lds[turn]));
        const bool bad = !(top < INFINITY), empty = bad || top == 0.0f;
        const Quantiser quantise(top);
        each_column<SHORT>(
            a.cols, [&](int64_t j) { return x[j]; },
            [&](int64_t j, T v) { q[j] = empty ? (signed char)0 : quantise((float)v); });
        if (threadIdx.x == 0) a.scale[row] = bad ? NAN : top / 127.0f;
    }
}

}  // namespace

hipError_t launch_layer_norm(const NormArgs& a, int dt, int wdt, hipStream_t stream)
{
    const RowShape s = row_shape(a.cols, elem_size(dt));
    return with_types(dt, wdt, [&](auto x, auto w) {
        using T = decltype(x);
        using W = decltype(w);
        if (!s.g)
            return start(a.cols <= kThreads ? &layer_norm_any_kernel<T, W, true> : &layer_norm_any_kernel<T, W, false>,
                         dim3(any_grid(a.rows)), kThreads, stream, a);
        return with_shape(s, [&](auto g, auto v) {
            constexpr int G = decltype(g)::value;
            const int grid = even_grid(a.rows, kGroups<G>, row_groups(a.rows, a.cols, sizeof(T), kGroupThreads<G>));
            return start(&layer_norm_kernel<T, W, G, decltype(v)::value>, dim3(grid), kGroupThreads<G>, stream, a);
        });
    });
}

// Workgroups of the backward pass, each of which leaves one strip of sums: one a
// CU (4097 x 3001 25 us, 32 with two), and two where a wave holds a row, 1024 bytes
// (12000 x 300 bf16 13.5 us, 14.0 with one; 50000 x 300 27.8 and 38.4; but fp32, two
// waves a row, 19.5 and 15.2).
int layer_norm_strips(int64_t rows, int64_t cols, int bytes)
{
    const bool wave = cols * bytes <= 1024;
    return rows == 0 ? 0 : even_grid(rows, wave ? 4 : 2, wave ? 512 : 256);
}

hipError_t launch_layer_norm_backward(const NormArgs& a, int dt, int wdt, hipStream_t stream)
{
    const int strips = layer_norm_strips(a.rows, a.cols, elem_size(dt));
    return with_types(dt, wdt, [&](auto x, auto w) {
        using T = decltype(x);
        using W = decltype(w);
        hipError_t e = hipSuccess;
        // one chunk a thread as long as 1024 threads hold the row: a thread keeps
        // two fp32 sums a column beside the row and the weight
        const int chunks = row_chunks(a.cols, sizeof(T)), waves = (int)ceil_div(chunks, 64);
        if (a.rows > 0 && a.rows <= kFewRows && chunks > 0 && waves <= 32) {
            int per_row = 1;
            while (per_row < waves && per_row < 16) per_row *= 2;
            const int row_blocks = (int)ceil_div(a.rows, 16 / per_row);
            const dim3 grid((unsigned)(row_blocks + ceil_div(a.cols, 64)));
            return waves <= 16 ? start(&layer_norm_backward_few_kernel<T, W, 1>, grid, 1024, stream, a, row_blocks, per_row)
                               : start(&layer_norm_backward_few_kernel<T, W, 2>, grid, 1024, stream, a, row_blocks, per_row);
        }
        if (a.rows > 0 && chunks > 0 && waves <= 32) {
            const int per_row = waves <= 16 ? waves : (waves + 1) / 2;
            const auto go = [&](auto kernel, int threads) { return start(kernel, dim3(strips), threads, stream, a, per_row); };
            e = waves == 1   ? go(&layer_norm_backward_kernel<T, W, true, 1>, kThreads)
                : waves <= 16 ? go(&layer_norm_backward_kernel<T, W, false, 1>, 64 * waves * (16 / waves))
                              : go(&layer_norm_backward_kernel<T, W, false, 2>, 64 * per_row);
        } else if (a.rows > 0) {
            const int strip_rows = (int)ceil_div(a.rows, strips);
            e = start(a.cols <= kThreads ? &layer_norm_dx_any_kernel<T, W, true> : &layer_norm_dx_any_kernel<T, W, false>,
                      dim3(any_grid(a.rows)), kThreads, stream, a);
            if (e == hipSuccess)
                e = start(&layer_norm_strip_any_kernel<T, W>, dim3((unsigned)ceil_div(a.cols, kThreads), strips), kThreads,
                          stream, a, strip_rows);
        }
        if (e != hipSuccess) return e;
        return start(&layer_norm_join_kernel<W>, dim3((unsigned)std::min<int64_t>(ceil_div(2 * (int64_t)a.cols, 64), kMaxRowGrid)), 1024, stream, a, strips);
    });
}

// f(the activation as a constant)
template <class F> hipError_t with_act(int act, F&& f)
{
    switch (act) {
    case ACT_SILU: return f(std::integral_constant<int, ACT_SILU>{});
    case ACT_GELU: return f(std::integral_constant<int, ACT_GELU>{});
    case ACT_GELU_TANH: return f(std::integral_constant<int, ACT_GELU_TANH>{});
    default: return f(std::integral_constant<int, ACT_RELU>{});
    }
}

hipError_t launch_gated_grad(const GatedGradArgs& a, int dt, hipStream_t stream)
{
    const dim3 grid((unsigned)((a.hidden + 63) / 64) * (unsigned)((a.rows + 63) / 64));
    return with_act(a.act, [&](auto act) {
        constexpr int ACT = decltype(act)::value;
        return start(dt == DT_F16 ? &gated_grad_kernel<DT_F16, ACT> : &gated_grad_kernel<DT_BF16, ACT>, grid, kGradThreads,
                     stream, a);
    });
}

hipError_t launch_gated_repair(const GatedGradArgs& a, hipStream_t stream)
{
    const int64_t pieces = (ceil_div(a.hidden, 64) + ceil_div(a.rows, 64)) * ceil_div(a.cols, 64);
    return with_act(a.act, [&](auto act) {
        return start(&gated_repair_kernel<decltype(act)::value>, dim3((unsigned)std::min<int64_t>(pieces, 2 * kNumCUs)), kThreads,
                     stream, a);
    });
}

hipError_t launch_quantize_rows(const void* x, int64_t x_stride, signed char* q, float* scale, int rows,
                                int cols, int dt, hipStream_t stream)
{
    const QuantArgs a{x, q, scale, x_stride, rows, cols};
    const RowShape s = row_shape(cols, elem_size(dt));
    return with_types(dt, dt, [&](auto x0, auto w) {
        using T = decltype(x0);
        if constexpr (std::is_same_v<T, decltype(w)>) {
            if (!s.g)
                return start(cols <= kThreads ? &quantize_rows_any_kernel<T, true> : &quantize_rows_any_kernel<T, false>,
                             dim3(any_grid(rows)), kThreads, stream, a);
            return with_shape(s, [&](auto g, auto v) {
                constexpr int G = decltype(g)::value;
                const int grid = even_grid(rows, kGroups<G>, row_groups(rows, cols, sizeof(T), kGroupThreads<G>));
                return start(&quantize_rows_kernel<T, G, decltype(v)::value>, dim3(grid), kGroupThreads<G>, stream, a);
            });
        }
        return hipErrorInvalidValue;
    });
}

}  // namespace gemm_relu_hip
