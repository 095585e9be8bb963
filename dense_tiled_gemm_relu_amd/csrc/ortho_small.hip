// Orthogonalisation where the shorter side is at most 128: all steps of a small matrix in one
// workgroup, one launch a step of a long one.
//
// A step's three products on the tile kernel are three launches of 5 us whatever the
// size.  Where a padded matrix has at most 32768 elements, eight waves hold X in fp32 registers (64 a lane), its float16 copy and A and B
// = b A + c A^2 without their diagonals in LDS, so a call is one launch.  Arithmetic and
// scales are those of ortho.hip, but for X, which is fp32 here.  Rows in LDS are padded by
// 16 bytes, which puts the 16 rows of a matrix operand on different banks.
//
// A step is bound by LDS: a wave's blocks share their operands' reads (2 x 4 blocks of A
// take 6 reads of 16 bytes a lane for 8 matrix instructions).  The matrix comes and goes
// through LDS in short loops: a workgroup runs such code once, and with 61 KB of unrolled
// loads and stores 128 x 256 without any step took 27 us, with the loops 11.  Five steps: 128
// x 256 bf16 53 us, 64 x 512 37, 64 x 128 16 (41, 28 and 12 with B times X's larger half
// alone); on the tile kernel 87 to 94.
//
// A long matrix's step is such a step of each part of 256 columns, between launches that
// exchange the parts' sums of A: 8 to 16 us, of which 3 the launch, 1 to 3 the sums, 1 to 2 X
// from and to memory, and the rest as above.
#include "block.hpp"
#include "row_common.hpp"

namespace gemm_relu_hip {

namespace {

constexpr int kSmallThreads = 512, kSmallWaves = kSmallThreads / 64;

// P: the padded shorter side; CB: blocks of 16 columns of X a wave has, the padded longer
// side being 128 CB, or with LONG a workgroup's part of it
template <int P, int CB, bool LONG>
__global__ void __launch_bounds__(kSmallThreads) ortho_small_kernel(OrthoArgs a, OrthoSteps c, OrthoLong part_of, int dt)
{
    using In = InTraits<DT_F16, 16>;
    using Op = typename In::Op;
    typedef _Float16 H4 __attribute__((ext_vector_type(4)));
    constexpr int Q = 16 * kSmallWaves * CB, RB = P / 16;
    constexpr int XP = Q + 8, AP = P + 8;                       // row pitches in LDS
    constexpr int GR = P / 64, GC = P / 32;                     // a wave's blocks of A and B: rows and columns
    constexpr int RP = Q + 4;                                   // of the fp32 matrix that comes in
    constexpr int HALVES = P * (XP + 2 * AP), STAGED = 2 * P * RP;
    __shared__ __attribute__((aligned(16))) _Float16 memory[HALVES > STAGED ? HALVES : STAGED];
    _Float16 *const xh = memory, *const am = xh + P * XP, *const bm = am + P * AP;
    float* const raw = reinterpret_cast<float*>(memory);
    __shared__ __attribute__((aligned(16))) float diag_a[P], diag_b[P];
    __shared__ double part[kSmallWaves];
    const int lane = (int)(threadIdx.x & 63), wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int r16 = lane & 15, g4 = lane >> 4;
    const size_t batch = LONG ? blockIdx.y : blockIdx.x;
    const int q0 = LONG ? (int)blockIdx.x * Q : 0;
    const bool tall = a.rows > a.cols;
    const int row0 = tall ? q0 : 0, col0 = tall ? 0 : q0;

    // in: |g| in binary64 (the values may be any fp32 ones) on the way, zeros around it
    double s = 0.0;
    const auto load_all = [&](auto zero) {
        using T = decltype(zero);
        const T* g = static_cast<const T*>(a.g) + batch * (size_t)a.g_batch;
        // a wave a row, 8 loads of a lane in flight
        const auto rows_of = [&](auto wide, auto high) {
            constexpr int WIDE = decltype(wide)::value, HIGH = decltype(high)::value, COLS = WIDE / 64;
            constexpr int ROWS = COLS >= 8 ? 1 : 8 / COLS;
            for (int r0 = wave; r0 < HIGH; r0 += ROWS * kSmallWaves) {
                T v[ROWS][COLS];
#pragma unroll
                for (int u = 0; u < ROWS; ++u)
#pragma unroll
                    for (int k = 0; k < COLS; ++k)
                        v[u][k] = g[(size_t)min(row0 + r0 + u * kSmallWaves, a.rows - 1) * (size_t)a.g_stride +
                                    min(col0 + 64 * k + lane, a.cols - 1)];
#pragma unroll
                for (int u = 0; u < ROWS; ++u)
#pragma unroll
                    for (int k = 0; k < COLS; ++k) {
                        const int r = r0 + u * kSmallWaves, j = 64 * k + lane;
                        const float in = row0 + r < a.rows && col0 + j < a.cols ? (float)v[u][k] : 0.0f;
                        if constexpr (!LONG) s = fma((double)in, (double)in, s);
                        raw[tall ? j * RP + r : r * RP + j] = in;
                    }
            }
        };
        if (tall)
            rows_of(std::integral_constant<int, P>{}, std::integral_constant<int, Q>{});
        else
            rows_of(std::integral_constant<int, Q>{}, std::integral_constant<int, P>{});
    };
    // element (p, q) of X, q the longer side; a lane has rows 16 i + r16, columns 4 g4 .. +3
    // of its wave's CB blocks
    f32x4_t x[RB][CB];
    const auto column = [&](int j) { return (wave * CB + j) * 16 + 4 * g4; };
    const auto start_x = [&] {
        if (dt == DT_F32)
            load_all(0.0f);
        else if (dt == DT_F16)
            load_all((_Float16)0.0f);
        else
            load_all((__bf16)0.0f);
        if constexpr (LONG) {
#pragma unroll
            for (int k = 0; k < kOrthoParts; k += 64) s += k + lane < a.parts ? a.squares[batch * kOrthoParts + k + lane] : 0.0;
        }
#pragma unroll
        for (int step = 1; step < 64; step *= 2) s += __shfl_xor(s, step);
        if (!LONG && lane == 0) part[wave] = s;
        __syncthreads();
        if constexpr (!LONG) {
            s = part[0];
#pragma unroll
            for (int k = 1; k < kSmallWaves; ++k) s += part[k];
        }
        // the scale as an fp32 number times a power of two, as in ortho_start_kernel
        const double scale = (double)kOrthoX / (sqrt(s) + (double)a.eps);
        int power;
        const float factor = (float)frexp(scale, &power);
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
            for (int j = 0; j < CB; ++j) {
                x[i][j] = *reinterpret_cast<const f32x4_t*>(raw + (16 * i + r16) * RP + column(j));
#pragma unroll
                for (int e = 0; e < 4; ++e) x[i][j][e] = ldexpf(x[i][j][e], power) * factor;
            }
        __syncthreads();                                        // read, so xh may take its place
    };
    // X as float16, or LOW kLowScale times what that loses
    const auto put_x = [&](auto low) {
        constexpr bool LOW = decltype(low)::value;
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
            for (int j = 0; j < CB; ++j) {
                H4 h;
                if constexpr (LOW) asm volatile("" : "+v"(x[i][j]));    // converted again, not kept since the step began (spills)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    h[e] = (_Float16)x[i][j][e];
                    if constexpr (LOW) h[e] = (_Float16)((x[i][j][e] - (float)h[e]) * kLowScale);
                }
                *reinterpret_cast<H4*>(&xh[(16 * i + r16) * XP + column(j)]) = h;
            }
    };
    const std::false_type high{};
    const std::true_type low{};

    // rows 16 b .. of a matrix whose rows run along k, k-step s
    const auto row_operand = [&](const _Float16* m, int pitch, int b, int s) {
        return __builtin_bit_cast(Op, *reinterpret_cast<const u32x4_t*>(m + (16 * b + r16) * pitch + 32 * s + 8 * g4));
    };
    // the wave's GR x GC blocks of m m^T
    const int gr0 = wave / 2 * GR, gc0 = wave % 2 * GC;
    f32x4_t acc[GR][GC];
    const auto square = [&](const _Float16* m, int pitch, int steps) {
#pragma unroll
        for (int i = 0; i < GR; ++i)
#pragma unroll
            for (int j = 0; j < GC; ++j) acc[i][j] = f32x4_t{};
#pragma unroll 2
        for (int s = 0; s < steps; ++s) {
            Op left[GR], right[GC];
#pragma unroll
            for (int i = 0; i < GR; ++i) left[i] = row_operand(m, pitch, gr0 + i, s);
#pragma unroll
            for (int j = 0; j < GC; ++j) right[j] = row_operand(m, pitch, gc0 + j, s);
#pragma unroll
            for (int i = 0; i < GR; ++i)
#pragma unroll
                for (int j = 0; j < GC; ++j) acc[i][j] = In::mfma(right[j], left[i], acc[i][j]);
        }
    };

    // the rest of a step from the sums of A = X X^T in acc; xh holds X
    const auto rest_of_step = [&](float ca, float cb, float cc) {
#pragma unroll
        for (int i = 0; i < GR; ++i)
#pragma unroll
            for (int j = 0; j < GC; ++j) {
                const int m = 16 * (gr0 + i) + r16, n = 16 * (gc0 + j) + 4 * g4;
                H4 h;
#pragma unroll
                for (int e = 0; e < 4; ++e) h[e] = (_Float16)(acc[i][j][e] * (kOrthoA / (kOrthoX * kOrthoX)));
                if (gr0 + i == gc0 + j) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (m == n + e) {
                            h[e] = (_Float16)0.0f;
                            diag_a[m] = acc[i][j][e] * (1.0f / (kOrthoX * kOrthoX));
                        }
                }
                *reinterpret_cast<H4*>(&am[m * AP + n]) = h;
            }
        __syncthreads();
        square(am, AP, P / 32);
#pragma unroll
        for (int i = 0; i < GR; ++i)
#pragma unroll
            for (int j = 0; j < GC; ++j) {
                const int m = 16 * (gr0 + i) + r16, n = 16 * (gc0 + j) + 4 * g4;
                const H4 o = *reinterpret_cast<const H4*>(&am[m * AP + n]);
                const f32x4_t dn = *reinterpret_cast<const f32x4_t*>(&diag_a[n]);
                const float d = diag_a[m];
                // off the diagonal b O + c (O^2 + (d_m + d_n) O), O being A without its diagonal d; on
                // it b d + c (O^2 + d^2)
                H4 h;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    h[e] = (_Float16)fmaf(acc[i][j][e], cc * (kOrthoB / (kOrthoA * kOrthoA)),
                                          (float)o[e] * fmaf(cc * (kOrthoB / kOrthoA), d + dn[e], cb * (kOrthoB / kOrthoA)));
                if (gr0 + i == gc0 + j) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (m == n + e) {
                            h[e] = (_Float16)0.0f;
                            diag_b[m] = cb * d + cc * (acc[i][j][e] * (1.0f / (kOrthoA * kOrthoA)) + d * d);
                        }
                }
                *reinterpret_cast<H4*>(&bm[m * AP + n]) = h;
            }
        __syncthreads();
        // B X, its wave's columns: X's rows run along n, so its operands are read transposed.
        // First with X's float16, then with what that loses, in the same place: the columns
        // are the wave's own here, so its own order is enough.
        f32x4_t y[RB][CB];
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
            for (int j = 0; j < CB; ++j) y[i][j] = f32x4_t{};
#pragma unroll 1
        for (int half_of_x = 0; half_of_x < 2; ++half_of_x) {
            if (half_of_x) {
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                put_x(low);
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
                for (int i = 0; i < RB; ++i)
#pragma unroll
                    for (int j = 0; j < CB; ++j) y[i][j] *= kLowScale;
            }
#pragma unroll
            for (int s = 0; s < P / 32; ++s) {
                Op right[CB];
#pragma unroll
                for (int j = 0; j < CB; ++j) {
                    i16x4_t half[2];
#pragma unroll
                    for (int t = 0; t < 2; ++t)
                        half[t] = lds_read_tr16((const GR_LDS unsigned char*)&xh[(32 * s + 8 * g4 + 4 * t + (r16 >> 2)) * XP +
                                                                                 (wave * CB + j) * 16 + 4 * (r16 & 3)]);
                    right[j] = __builtin_bit_cast(Op, __builtin_shufflevector(half[0], half[1], 0, 1, 2, 3, 4, 5, 6, 7));
                }
#pragma unroll
                for (int i = 0; i < RB; ++i) {
                    const Op left = row_operand(bm, AP, i, s);
#pragma unroll
                    for (int j = 0; j < CB; ++j) y[i][j] = In::mfma(right[j], left, y[i][j]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < RB; ++i) {
            const float d = ca + diag_b[16 * i + r16];
#pragma unroll
            for (int j = 0; j < CB; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[i][j][e] = fmaf(d, x[i][j][e], y[i][j][e] * (1.0f / (kOrthoB * kLowScale)));
        }
        __syncthreads();                                        // every wave has read xh
    };

    if constexpr (!LONG) {
        start_x();
        for (int step = 0; step < c.steps; ++step) {
            put_x(high);
            __syncthreads();
            square(xh, XP, Q / 32);
            rest_of_step(c.v[3 * step], c.v[3 * step + 1], c.v[3 * step + 2]);
        }
    } else {
        // Where a lane's values lie: its own ones of X, and those of A of each part of the
        // matrix, which it adds in order.
        f32x4_t* const own = reinterpret_cast<f32x4_t*>(part_of.x) + ((batch * gridDim.x + blockIdx.x) * (RB * CB)) * kSmallThreads + threadIdx.x;
        const auto sums_of = [&](float* p, size_t chunk) {
            return reinterpret_cast<f32x4_t*>(p) + ((batch * gridDim.x + chunk) * (GR * GC)) * kSmallThreads + threadIdx.x;
        };
        if (part_of.first) {
            start_x();
            if (!part_of.last) put_x(high);
        } else {
#pragma unroll
            for (int i = 0; i < RB; ++i)
#pragma unroll
                for (int j = 0; j < CB; ++j) x[i][j] = own[(i * CB + j) * kSmallThreads];
#pragma unroll
            for (int i = 0; i < GR; ++i)
#pragma unroll
                for (int j = 0; j < GC; ++j) acc[i][j] = f32x4_t{};
            constexpr int AHEAD = P == 64 ? 4 : 2;
            for (int k = 0; k < (int)gridDim.x; k += AHEAD) {
                f32x4_t v[AHEAD][GR * GC];
#pragma unroll
                for (int u = 0; u < AHEAD; ++u) {
                    const f32x4_t* from = sums_of(part_of.in, min(k + u, (int)gridDim.x - 1));
#pragma unroll
                    for (int b = 0; b < GR * GC; ++b) v[u][b] = from[b * kSmallThreads];
                }
#pragma unroll
                for (int u = 0; u < AHEAD; ++u)
                    if (k + u < (int)gridDim.x) {
#pragma unroll
                        for (int b = 0; b < GR * GC; ++b) acc[b / GC][b % GC] += v[u][b];
                    }
            }
            put_x(high);
            rest_of_step(part_of.ca, part_of.cb, part_of.cc);
            if (!part_of.last) put_x(high);
        }
        if (!part_of.last) {
            __syncthreads();
            square(xh, XP, Q / 32);
            f32x4_t* to = sums_of(part_of.out, blockIdx.x);
#pragma unroll
            for (int b = 0; b < GR * GC; ++b) to[b * kSmallThreads] = acc[b / GC][b % GC];
#pragma unroll
            for (int i = 0; i < RB; ++i)
#pragma unroll
                for (int j = 0; j < CB; ++j) own[(i * CB + j) * kSmallThreads] = x[i][j];
            return;
        }
    }

    // out, through LDS again
    typedef __bf16 B4 __attribute__((ext_vector_type(4)));
    __bf16* const staged = reinterpret_cast<__bf16*>(memory);
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < CB; ++j) {
            B4 four;
#pragma unroll
            for (int e = 0; e < 4; ++e) four[e] = (__bf16)(x[i][j][e] * (1.0f / kOrthoX));
            *reinterpret_cast<B4*>(&staged[(16 * i + r16) * XP + column(j)]) = four;
        }
    __syncthreads();
    __bf16* out = static_cast<__bf16*>(a.out) + batch * (size_t)a.rows * (size_t)a.cols;
    const int rows = min(a.rows - row0, tall ? Q : P), cols = min(a.cols - col0, tall ? P : Q);
    for (int r = wave; r < rows; r += kSmallWaves)
#pragma unroll 4
        for (int j = lane; j < cols; j += 64)
            out[(size_t)(row0 + r) * (size_t)a.cols + col0 + j] = tall ? staged[j * XP + r] : staged[r * XP + j];
}

}  // namespace

hipError_t launch_ortho_small(const OrthoArgs& a, const OrthoSteps& c, int dt, hipStream_t stream)
{
    const int blocks = (a.q + 127) / 128;
    const auto go = [&](auto kernel) { return start(kernel, dim3(a.batch), kSmallThreads, stream, a, c, OrthoLong{}, dt); };
    if (a.p <= 64) {
        switch (blocks) {
        case 1: return go(&ortho_small_kernel<64, 1, false>);
        case 2: return go(&ortho_small_kernel<64, 2, false>);
        case 3: return go(&ortho_small_kernel<64, 3, false>);
        case 4: return go(&ortho_small_kernel<64, 4, false>);
        default: return hipErrorInvalidValue;
        }
    }
    switch (blocks) {
    case 1: return go(&ortho_small_kernel<128, 1, false>);
    case 2: return go(&ortho_small_kernel<128, 2, false>);
    default: return hipErrorInvalidValue;
    }
}

hipError_t launch_ortho_long(const OrthoArgs& a, const OrthoSteps& c, float* x, float* sums, int dt, hipStream_t stream)
{
    hipError_t e = launch_ortho_squares(a, dt, stream);
    const int parts = ortho_parts(a.q);
    const size_t size = (size_t)a.batch * (size_t)parts * (size_t)a.P * (size_t)a.P;
    // the launch before the first step leaves X and the parts' A, each step the next's
    for (int step = -1; step < c.steps && e == hipSuccess; ++step) {
        OrthoLong part_of{x, sums + (step & 1 ? 0 : size), sums + (step & 1 ? size : 0), step < 0, step == c.steps - 1, 0.0f, 0.0f, 0.0f};
        if (step >= 0) {
            part_of.ca = c.v[3 * step];
            part_of.cb = c.v[3 * step + 1];
            part_of.cc = c.v[3 * step + 2];
        }
        e = start(a.p <= 64 ? &ortho_small_kernel<64, 2, true> : &ortho_small_kernel<128, 2, true>, dim3(parts, a.batch),
                  kSmallThreads, stream, a, OrthoSteps{}, part_of, dt);
    }
    return e;
}

}  // namespace gemm_relu_hip
