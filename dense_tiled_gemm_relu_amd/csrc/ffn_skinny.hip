// Products with few rows of x, or few outputs, B stored (N,K): gated projections, the
// product with bias, activation and residual, and the scaled 8-bit product of a decode
// step or a small batch.
//
// What bounds them is reading the weight once (M <= 64), or the latency of a
// tile's K loop where the tiles do not fill the device.  A workgroup of four
// waves takes 16 MT rows of x and 16 NT rows of the weight and cuts K between
// its waves: chunk q of CB bytes is wave q mod 4's.  Each wave copies its chunks
// of both operands into a ring of its own in LDS, so no wave waits for another
// before the end, and every CU has tens of KiB on the way; the four partial sums
// meet in LDS and are added in order.
//
// The copies go through LDS and not straight into the operand registers because
// of their lane order: consecutive lanes read consecutive 16-byte pieces of a row.
// The operand's order (16 rows, 16 bytes each) reads the L2 at 9-16 TB/s, and at
// 2.4 TB/s where rows do not start at a multiple of 4 bytes; whole row pieces
// come at 22 TB/s, and at 12-15 TB/s from any address.
//
// Measured: one token on 7168 x 4096 gated bf16 weights 22 us (5.3 TB/s; 26 on 64 x
// 64 tiles), on 8192 x 8192 8-bit weights 11.3 (5.9 TB/s; 17); 64 x 1000 x 4096 gated
// 8.9 (18.1), 128 x 1000 x 1000 8-bit 3.4 (9.3).  Above about 64 rows of a wide
// weight the tiles' fewer bytes from the L2 win: 64 x 8192 x 8192 gated 89 against 60.
// 32 x 48 and 48 x 32 are for what just misses one round of smaller ones: 77 x 3001 x
// 5003 8-bit 13.3 against 19, 100 x 3000 x 3000 7.2 against 10; elsewhere they are
// slower (64 x 4096 x 8192 10.4 against 9.2).  64 x 32 reads a wide weight once for up to 64
// rows and just fits one round where 32 x 32 takes two: with bias, activation and residual,
// weights from HBM, 64 x 8192 x 8192 35 us (47 on 32 x 32; HBM's share 26), 64 x 7168 x 4096
// 13.8 (18.4 on 64 x 64), 128 x 4096 x 4096 12.4 (18.4).
#include "api_common.hpp"
#include "ffn.hpp"

namespace gemm_relu_hip {

namespace {

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kStepBytes = 64;                 // of K per matrix instruction: 32 16-bit or 64 8-bit elements

template <int IN, int OUT, int EPI, int MT, int NT, int CB, int STAGES>
__global__ void __launch_bounds__(kThreads) skinny_kernel(KernelArgs a)
{
    using In = InTraits<IN, 16>;
    using Acc = typename In::Acc;
    using Op = typename In::Op;
    constexpr int EB = In::EB;
    constexpr bool GATED = EPI == EPI_GATED;
    constexpr int BLOCKS = MT * NT;
    constexpr int U = CB / kStepBytes;          // matrix steps per chunk
    constexpr int ROW_CH = CB / 16;             // 16-byte pieces per row of a chunk
    constexpr int COPIES = CB / 64;             // copies per 16-row block: 16 CB bytes
    constexpr int BLOCK_BYTES = 16 * CB, STAGE_BYTES = (MT + NT) * BLOCK_BYTES, RING = STAGES * STAGE_BYTES;
    constexpr int LOADS = (MT + NT) * COPIES;
    static_assert(RING >= BLOCKS * 64 * 16, "a wave's partial sums fit its ring");
    static_assert((STAGES - 1) * LOADS < 64, "vmcnt range");
    __shared__ __attribute__((aligned(1024))) unsigned char smem_raw[kWaves * RING];
    GR_LDS unsigned char* const smem = (GR_LDS unsigned char*)smem_raw;

    const int lane = (int)(threadIdx.x & 63);
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int r16 = lane & 15, g4 = lane >> 4;
    int tm, tn;
    tile_coords((int)blockIdx.x, a.tiles_m, a.tiles_n, a.panel, a.nxcd, tm, tn);
    const int m0 = tm * 16 * MT;
    // columns of the output: a gated block of 16 weight rows is 8 gate and 8 up rows
    const int cols = GATED ? a.hidden : a.N, c0 = tn * NT * (GATED ? 8 : 16);

    // row r of block b (the MT blocks of x, then the NT of the weight); rows past
    // the edge are the last one's (their results are not stored)
    auto row_at = [&](int b, int r) {
        if (b < MT) return a.A + (size_t)min(m0 + 16 * b + r, a.M - 1) * (size_t)a.lda * EB;
        const int j = b - MT, c = min(c0 + (GATED ? 8 * j + (r & 7) : 16 * j + r), cols - 1);
        return a.B + ((size_t)c + (GATED && r >= 8 ? (size_t)a.hidden : 0)) * (size_t)a.ldb * EB;
    };
    const int bytes = a.K * EB, full = bytes / CB;         // whole chunks; the rest of K is the tail
    const int n = full > wave ? (full - wave + kWaves - 1) / kWaves : 0;

    // the tail, to the wave whose turn it is: straight into operand registers.
    // Pieces past the end of K are zero, the one across it is read from 16 bytes
    // before the end (K has at least 16) with what the previous piece holds
    // cleared, in both operands alike.
    u32x4_t tail[MT + NT][U];
    auto tail_at = [&](int u) { return full * CB + u * kStepBytes + 16 * g4; };
    const bool has_tail = full * CB < bytes && full % kWaves == wave;
    if (has_tail) {
#pragma unroll
        for (int b = 0; b < MT + NT; ++b)
#pragma unroll
            for (int u = 0; u < U; ++u)
                __builtin_memcpy(&tail[b][u], row_at(b, r16) + min(tail_at(u), bytes - 16), 16);
    }

    // copy k of block b brings rows (64 / ROW_CH) k .. of it, each lane the piece
    // that belongs at its place in the swizzled block
    const unsigned char* src[LOADS];
#pragma unroll
    for (int l = 0; l < LOADS; ++l) {
        const int q = (l % COPIES) * 64 + lane, r = q / ROW_CH, c = (q % ROW_CH) ^ swz_krow<ROW_CH>(r);
        src[l] = row_at(l / COPIES, r) + wave * CB + c * 16;
    }
    const uint32_t ring = lds_addr(smem) + wave * RING;
    auto fetch = [&](int stage) {
#pragma unroll
        for (int l = 0; l < LOADS; ++l) {
            copy_to_lds(src[l], ring + stage * STAGE_BYTES + l * 1024);
            src[l] += kWaves * CB;
        }
    };

    Acc acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = Acc{};
    auto multiply = [&](auto&& operand) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            Op x[MT], w[NT];
#pragma unroll
            for (int i = 0; i < MT; ++i) x[i] = __builtin_bit_cast(Op, operand(i, u));
#pragma unroll
            for (int j = 0; j < NT; ++j) w[j] = __builtin_bit_cast(Op, operand(MT + j, u));
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j) acc[i][j] = In::mfma(w[j], x[i], acc[i][j]);
        }
    };

#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s)
        if (s < n) fetch(s);
    int stage = 0;
    for (int t = 0; t < n; ++t) {
        // the slot of stage t - 1 takes stage t + STAGES - 1: its reads are done
        if (t + STAGES - 1 < n) {
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            fetch(stage == 0 ? STAGES - 1 : stage - 1);
            __builtin_amdgcn_s_waitcnt(waitcnt_vm((STAGES - 1) * LOADS));
        } else {
            __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
        }
        asm volatile("" ::: "memory");
        const GR_LDS unsigned char* from = smem + wave * RING + stage * STAGE_BYTES;
        multiply([&](int b, int u) {
            return lds_read_b128(from + b * BLOCK_BYTES + r16 * CB + (((4 * u + g4) ^ swz_krow<ROW_CH>(r16)) << 4));
        });
        stage = stage == STAGES - 1 ? 0 : stage + 1;
    }
    if (has_tail)
        multiply([&](int b, int u) { return clear_front(tail[b][u], min(max(tail_at(u) - (bytes - 16), 0), 16)); });

    // partial sums, each wave's in its own ring
    typedef GR_LDS Acc* AccPtr;
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
            *(AccPtr)(smem + wave * RING + ((i * NT + j) * 64 + lane) * 16) = acc[i][j];
    __syncthreads();
    // lane: row m of x, weight rows 4 g4 .. 4 g4 + 3 of the block
#pragma unroll
    for (int b0 = 0; b0 < BLOCKS; b0 += kWaves) {
        const int b = b0 + wave;
        if (b >= BLOCKS) break;
        const int i = b / NT, j = b % NT, m = m0 + 16 * i + r16;
        Acc s = *(AccPtr)(smem + (b * 64 + lane) * 16);
#pragma unroll
        for (int k = 1; k < kWaves; ++k) s += *(AccPtr)(smem + k * RING + (b * 64 + lane) * 16);
        f32x4_t v;
        int c;
        bool mine = m < a.M;
        if constexpr (GATED) {
            c = c0 + 8 * j + 4 * (g4 & 1);
            if (a.GU && mine && c < cols)
                store_sums(a.GU + (size_t)m * (size_t)(2 * (int64_t)cols) + (g4 < 2 ? 0 : cols) + c, s, c, cols);
            with_activation(a.act, [&](auto kind) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float up = __shfl_xor(s[e], 32);
                    v[e] = activation<decltype(kind)::value>(s[e]) * up;
                }
            });
            mine = mine && g4 < 2;
        } else if constexpr (EPI == EPI_ACT) {
            c = c0 + 16 * j + 4 * g4;
            const f32x4_t z = s + load_bias<IN>(a, c, cols);
            if (a.GU && mine && c < cols) store_sums(a.GU + (size_t)m * (size_t)cols + c, z, c, cols);
            u32x2_t r = {0u, 0u};
            if (a.R)
                r = load_half4(reinterpret_cast<const unsigned short*>(a.R) + (size_t)min(m, a.M - 1) * (size_t)a.ldr, c, cols);
            with_activation_or_none(a.act, [&](auto kind) {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = activation<decltype(kind)::value, true>(z[e]);
            });
            if (a.R) v += to_float4<IN>(r);
        } else {
            c = c0 + 16 * j + 4 * g4;
            const float sa = a.scale_a[min(m, a.M - 1)];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = (float)s[e] * sa * a.scale_b[min(c + e, cols - 1)];
        }
        if (!mine || c >= cols) continue;
        if constexpr (OUT == DT_F32) {
            store_sums(reinterpret_cast<float*>(a.C) + (size_t)m * (size_t)cols + c, v, c, cols);
        } else {
            unsigned short* dst = reinterpret_cast<unsigned short*>(a.C) + (size_t)m * (size_t)cols + c;
            unsigned short h[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) h[e] = OutTraits<OUT>::cvt(v[e]);
            if (c + 4 <= cols) {
                __builtin_memcpy(dst, h, 8);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (c + e < cols) dst[e] = h[e];
            }
        }
    }
}

template <int IN, int OUT, int EPI, int MT, int NT, int CB, int STAGES>
hipError_t launch(const KernelArgs& args, int grid, hipStream_t stream)
{
    void* params[] = {const_cast<KernelArgs*>(&args)};
    return hipLaunchKernel(reinterpret_cast<const void*>(&skinny_kernel<IN, OUT, EPI, MT, NT, CB, STAGES>), dim3(grid),
                           dim3(kThreads), params, 0, stream);
}

template <int IN, int OUT, int EPI> LinearLaunchFn pick(int cfg)
{
    switch (cfg) {
    case LIN_K16: return &launch<IN, OUT, EPI, 1, 1, 128, 4>;
    case LIN_K32: return &launch<IN, OUT, EPI, 2, 2, 128, 4>;
    case LIN_K32X48: return &launch<IN, OUT, EPI, 2, 3, 128, 3>;
    case LIN_K48X32: return &launch<IN, OUT, EPI, 3, 2, 128, 3>;
    case LIN_K64X32:
        if constexpr (EPI == EPI_ACT) return &launch<IN, OUT, EPI, 4, 2, 128, 3>;
        return nullptr;
    default: return nullptr;
    }
}

}  // namespace

LinearLaunchFn launcher_skinny_gated(int dt, int cfg)
{
    return dt == DT_F16 ? pick<DT_F16, DT_F16, EPI_GATED>(cfg) : pick<DT_BF16, DT_BF16, EPI_GATED>(cfg);
}

LinearLaunchFn launcher_skinny_act(int dt, int cfg)
{
    return dt == DT_F16 ? pick<DT_F16, DT_F16, EPI_ACT>(cfg) : pick<DT_BF16, DT_BF16, EPI_ACT>(cfg);
}

LinearLaunchFn launcher_skinny_i8(int out_dt, int cfg)
{
    if (out_dt == DT_F16) return pick<DT_I8, DT_F16, EPI_I8>(cfg);
    if (out_dt == DT_BF16) return pick<DT_I8, DT_BF16, EPI_I8>(cfg);
    return pick<DT_I8, DT_F32, EPI_I8>(cfg);
}

}  // namespace gemm_relu_hip
