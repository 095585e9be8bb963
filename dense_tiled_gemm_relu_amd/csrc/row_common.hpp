// What the row kernels share: sums over a wave and over the threads of a row, rows
// held in registers, columns of rows of any length, and the choice of their grids.
#pragma once

#include <type_traits>

#include "api_common.hpp"
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

// ---- sums and maxima over a wave, the same value in every lane: register
// exchanges inside rows of 16 lanes, then between them (a shuffle through LDS
// costs about a hundred cycles a step)
template <int CTRL> __device__ __forceinline__ unsigned dpp(unsigned v)
{
    return (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}
struct Sum {
    static __device__ __forceinline__ float of(float a, float b) { return a + b; }
};
struct Max {
    static __device__ __forceinline__ unsigned of(unsigned a, unsigned b) { return a > b ? a : b; }
};
// ... over the 16 lanes of a row
__device__ __forceinline__ float row16_sum(float v)
{
    v += __builtin_bit_cast(float, dpp<0xB1>(__builtin_bit_cast(unsigned, v)));
    v += __builtin_bit_cast(float, dpp<0x4E>(__builtin_bit_cast(unsigned, v)));
    v += __builtin_bit_cast(float, dpp<0x141>(__builtin_bit_cast(unsigned, v)));
    return v + __builtin_bit_cast(float, dpp<0x140>(__builtin_bit_cast(unsigned, v)));
}
template <class F, class T> __device__ __forceinline__ T wave_all(T v)
{
    auto bits = [](T x) { return __builtin_bit_cast(unsigned, x); };
    auto val = [](unsigned x) { return __builtin_bit_cast(T, x); };
    v = F::of(v, val(dpp<0xB1>(bits(v))));        // lane ^ 1
    v = F::of(v, val(dpp<0x4E>(bits(v))));        // lane ^ 2
    v = F::of(v, val(dpp<0x141>(bits(v))));       // the other four of 8
    v = F::of(v, val(dpp<0x140>(bits(v))));       // the other eight of 16
    const auto p = __builtin_amdgcn_permlane16_swap(bits(v), bits(v), false, false);
    v = F::of(val(p[0]), val(p[1]));
    const auto q = __builtin_amdgcn_permlane32_swap(bits(v), bits(v), false, false);
    return F::of(val(q[0]), val(q[1]));
}
// ... over the G threads that share a row.  lds holds G / 64 values; the caller
// alternates between two of them, so one barrier a sum is enough: whoever writes
// a buffer again has passed the barrier of the other one, behind every read.
template <int G, class F, class T> __device__ __forceinline__ T group_all(T v, T* lds)
{
    v = wave_all<F>(v);
    if constexpr (G > 64) {
        const int wave = (int)(threadIdx.x >> 6);
        if ((threadIdx.x & 63) == 0) lds[wave] = v;
        __syncthreads();
        v = lds[0];
#pragma unroll
        for (int k = 1; k < G / 64; ++k) v = F::of(v, lds[k]);
    }
    return v;
}

// ---- a row held in registers by G threads, V chunks of 16 bytes each
// Rows need only the alignment of an element (16-byte loads at any address).  A
// row whose length is no multiple of a chunk ends in a chunk moved back inside
// it; the elements it shares with its neighbour are left out of sums, and are
// written twice with the same value.  Only the last of a thread's chunks can be
// moved or missing: rows have more than (V - 1) G chunks.
template <class T> struct Chunk {
    static constexpr int N = 16 / sizeof(T);
    typedef T Vec __attribute__((ext_vector_type(N)));
};
template <class T, int N> struct VecN {
    typedef T Vec __attribute__((ext_vector_type(N)));
};
template <class V, class T> __device__ __forceinline__ V load_vec(const T* p)
{
    V v;
    __builtin_memcpy(&v, p, sizeof v);
    return v;
}

// Keeps a vector packed across this point: without it the compiler holds the fp32
// values it has unpacked, two registers for one, and spills.
template <class V> __device__ __forceinline__ void stay_packed(V& v)
{
    u32x4_t* words = reinterpret_cast<u32x4_t*>(&v);
#pragma unroll
    for (unsigned k = 0; k < sizeof(V) / 16; ++k) asm volatile("" : "+v"(words[k]));
}

template <class T, int V> struct RowMap {
    static constexpr int N = Chunk<T>::N;
    int start[V], skip;      // first column of each chunk; elements of the last one that the neighbour owns
    bool last;               // whether the last chunk exists
    // thread t of the g that share the row
    __device__ __forceinline__ RowMap(int cols, int t, int g)
    {
#pragma unroll
        for (int v = 0; v < V; ++v) start[v] = (v * g + t) * N;
        const int j = start[V - 1];
        last = j < cols;
        start[V - 1] = min(j, cols - N);
        skip = j - start[V - 1];
    }
    __device__ __forceinline__ bool has(int v) const { return v < V - 1 || last; }
    // whether element e of chunk v belongs to this thread
    __device__ __forceinline__ bool owns(int v, int e) const { return v < V - 1 || e >= skip; }
};

// Rows r, r + step, ... of a group; G = 64: four groups a workgroup.
template <int G> __device__ __forceinline__ int group_index()
{
    return G == 64 ? (int)(blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6)) : (int)blockIdx.x;
}
template <int G> constexpr int kGroupThreads = G == 64 ? kThreads : G;
template <int G> constexpr int kGroups = kGroupThreads<G> / G;

// ---- rows shorter than a chunk, or longer than 1024 threads hold: one workgroup
// a row, read once per use (a long row's second and third reads come from L2)

// use(j, load(j)) for every column j of a thread, the loads of a batch in flight
// together.  64-bit columns: the last one's successors may pass 2^31.  SHORT: at most
// one column a thread (the same kernels without their loops, whose registers would
// cost such rows a third: 100000 x 5 bf16 85 us against 66).
constexpr int kBatch = 16;
template <bool SHORT, class L, class U, class E>
__device__ __forceinline__ void each_column(int cols, L&& load, U&& use, E&& end_of_batch)
{
    if constexpr (SHORT) {
        if ((int)threadIdx.x < cols) use((int64_t)threadIdx.x, load((int64_t)threadIdx.x));
        end_of_batch();
        return;
    }
    int64_t j = threadIdx.x;
    for (; j + (kBatch - 1) * kThreads < cols; j += kBatch * kThreads) {
        decltype(load(j)) v[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) v[u] = load(j + u * kThreads);
#pragma unroll
        for (int u = 0; u < kBatch; ++u) use(j + u * kThreads, v[u]);
        end_of_batch();
    }
    for (; j < cols; j += kThreads) use(j, load(j));
    end_of_batch();
}
template <bool SHORT, class L, class U> __device__ __forceinline__ void each_column(int cols, L&& load, U&& use)
{
    each_column<SHORT>(cols, load, use, [] {});
}
// Means over a row of load(j)'s SUMS values: a batch in fp32, the batches in
// binary64 (a row may have 2^31 elements, millions a thread, and an fp32 sum of so
// many stops growing).  lds holds one of two buffers, as in group_all.
template <int SUMS> struct Values {
    float v[SUMS];
};
template <int SUMS> struct RowSums {
    double v[SUMS];
};
template <bool SHORT, int SUMS, class L> __device__ __forceinline__ Values<SUMS> row_means(int cols, L&& load, RowSums<SUMS>* lds)
{
    if constexpr (SHORT) {
        Values<SUMS> one{};
        if ((int)threadIdx.x < cols) one = load((int64_t)threadIdx.x);
#pragma unroll
        for (int k = 0; k < SUMS; ++k)
            one.v[k] = group_all<kThreads, Sum>(one.v[k], reinterpret_cast<float*>(lds) + k * (kThreads / 64)) / (float)cols;
        return one;
    }
    RowSums<SUMS> all{};
    Values<SUMS> part{};
    each_column<SHORT>(
        cols, load,
        [&](int64_t, Values<SUMS> v) {
#pragma unroll
            for (int k = 0; k < SUMS; ++k) part.v[k] += v.v[k];
        },
        [&] {
#pragma unroll
            for (int k = 0; k < SUMS; ++k) all.v[k] += (double)part.v[k];
            part = Values<SUMS>{};
        });
#pragma unroll
    for (int k = 0; k < SUMS; ++k)
#pragma unroll
        for (int step = 1; step < 64; step *= 2) all.v[k] += __shfl_xor(all.v[k], step);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = all;
    __syncthreads();
    all = lds[0];
#pragma unroll
    for (int w = 1; w < kThreads / 64; ++w)
#pragma unroll
        for (int k = 0; k < SUMS; ++k) all.v[k] += lds[w].v[k];
#pragma unroll
    for (int k = 0; k < SUMS; ++k) part.v[k] = (float)(all.v[k] / cols);
    return part;
}
template <class... A> hipError_t start(void (*kernel)(A...), dim3 grid, int threads, hipStream_t stream, A... args)
{
    void* params[] = {&args...};
    return hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, dim3(threads), params, 0, stream);
}

constexpr int kMaxRowGrid = 1 << 20;     // workgroups of a kernel that takes rows that far apart
int any_grid(int rows) { return rows < kMaxRowGrid ? rows : kMaxRowGrid; }

// Threads that share a row (0: the kernels for any length) and 16-byte chunks of
// it each: up to four chunks a thread, one wave where that holds the row, so that
// short rows need no barrier.
struct RowShape {
    int g, v;
};
int row_chunks(int cols, int bytes)
{
    const int n = 16 / bytes;
    return cols < n ? 0 : (int)(((int64_t)cols + n - 1) / n);
}
RowShape row_shape(int cols, int bytes)
{
    const int chunks = row_chunks(cols, bytes);
    for (int g = 64; chunks > 0 && g <= 1024; g *= 2) {
        const int v = (int)ceil_div(chunks, g);
        if (v <= 4) return {g, v};
    }
    return {0, 0};
}
// Calls f<G, V> for a shape row_shape can give.
template <class F> hipError_t with_shape(RowShape s, F&& f)
{
#define GR_SHAPE(G, V) \
    if (s.g == G && s.v == V) return f(std::integral_constant<int, G>{}, std::integral_constant<int, V>{});
    GR_SHAPE(64, 1) GR_SHAPE(64, 2) GR_SHAPE(64, 3) GR_SHAPE(64, 4) GR_SHAPE(128, 3) GR_SHAPE(128, 4)
    GR_SHAPE(256, 3) GR_SHAPE(256, 4) GR_SHAPE(512, 3) GR_SHAPE(512, 4) GR_SHAPE(1024, 3) GR_SHAPE(1024, 4)
#undef GR_SHAPE
    return hipErrorInvalidValue;
}
template <class F> hipError_t with_types(int dt, int wdt, F&& f)
{
    if (dt == DT_F32) return f(float{}, float{});
    if (dt == DT_F16) return wdt == DT_F32 ? f(_Float16{}, float{}) : f(_Float16{}, _Float16{});
    return wdt == DT_F32 ? f(__bf16{}, float{}) : f(__bf16{}, __bf16{});
}
int elem_size(int dt) { return dt == DT_F32 ? 4 : 2; }

// Workgroups that take rows in turns: at most `most`, and as many rows each as
// the busiest has anyway, so that they end together.
// A forward kernel's limit is a full device (256 CUs of 2048 threads), so that the
// weight is read once a group; four times that where the rows come from HBM
// (above 64 MiB), whose waits more short workgroups cover better: 16384 x 8192
// bf16 93 us against 98, but 4097 x 3001 fp16 12.8 against 10.9.
int row_groups(int64_t rows, int64_t cols, int bytes, int threads)
{
    return kNumCUs * 2048 / threads * (rows * cols * bytes > (int64_t(64) << 20) ? 4 : 1);
}
int even_grid(int64_t rows, int rows_each_turn, int most)
{
    const int64_t turns = ceil_div(rows, (int64_t)rows_each_turn * most);
    return (int)ceil_div(rows, rows_each_turn * turns);
}

}  // namespace

}  // namespace gemm_relu_hip
