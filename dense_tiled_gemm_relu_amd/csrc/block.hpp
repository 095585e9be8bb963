// Launch interface of the kernels around the half layer, between the C-ABI unit
// (block_api.hip) and the kernel units.
#pragma once

#include "ffn.hpp"

namespace gemm_relu_hip {

// ---- column sums over strips of rows: column j of result k is scale factor_j times the sum
// over strips of partial[strip][of cols + j]
constexpr int kMaxResults = 4;
struct JoinArgs {
    const float* partial;       // strips x sums x cols
    struct Result {
        void* out;              // null: not wanted
        int of;
        const void* factor;     // of the results' type; null: 1
        float scale;
    } result[kMaxResults];
    int results, sums, cols, strips;
};
hipError_t launch_join(const JoinArgs& a, int out_dt, hipStream_t stream);

// ---- gradient of act(z) (block_rows.hip)
constexpr int kActGradThreads = 512;       // of a workgroup, which takes a 64 x 64 tile
struct ActGradArgs {
    const float* z;             // (rows, n)
    const void* dy;
    void* dz;                   // (rows, n), rows ld apart; null: not wanted
    void* dz_t;                 // (n, rows), rows ld_t apart
    float* sums;                // of dz over each 64 rows (64-row tiles x n); null: not wanted
    int64_t dy_stride;
    int ld, ld_t;
    int rows, n, act;
    float scale;                // of what dz and dz_t hold
    unsigned* flags;            // `nflags` arrival counters to clear for a K split that follows
    int nflags;
};
hipError_t launch_act_grad(const ActGradArgs& a, int dt, hipStream_t stream);

// ---- residual sum and norms (block_rows.hip)
// The sums over rows that the backward pass leaves in strips: of dy norm(s), of dy, and of
// dresidual norm(x) (norm(x): x itself without a post_weight), from which dgate and
// dpost_weight both follow; with a matrix for a gate, of dt norm(x).
constexpr int kNormSums = 3;
struct AddNormArgs {
    const void* x;
    const void* r;
    const void* gate;           // null: 1
    const void* pw;             // null: x is not normed
    const void* w;              // null: no y
    const void* b;
    void* s;
    void* y;
    float* stats;               // 4 a row: mean and 1 / deviation of x, and of s
    const void* dy;             // backward
    const void* ds;
    void* dx;
    void* dr;
    void* dgate;                // of a gate matrix; the sums over rows go to `partial`
    const void* db;             // null: not wanted
    float* partial;             // strips x kNormSums x cols
    float* row_sums;            // 2 a row: the means that dresidual takes (rows of any length)
    int64_t x_stride, r_stride, gate_stride, dy_stride, ds_stride;    // gate_stride 0: one row
    int rows, cols;
    int layer;                  // layer norm, else root mean square
    float scale, eps;
};
hipError_t launch_add_norm(const AddNormArgs& a, int dt, int wdt, hipStream_t stream);
// strips of rows the backward pass sums on their own before launch_join
int add_norm_strips(int64_t rows);
hipError_t launch_add_norm_backward(const AddNormArgs& a, int dt, int wdt, hipStream_t stream);

// ---- orthogonalisation (ortho.hip)
// X (p x q, p <= q) is padded to P x Q, multiples of 64, with zeros, which the steps
// leave zeros.  The matrix instructions take float16: X times 2^8, A = X X^T without its
// diagonal times 2^10 and B = b A + c A^2 without its diagonal times 2^8; the scales keep
// what is far below a matrix's norm inside float16's normal range (its smallest value of
// full precision, 2^-14, is 2^-22 of X's and B's norm and 2^-24 of A's), and leave room
// for norms of 2^8, 2^6 and 2^8.  (What multiplies X's low half is B over kLowScale, a multiple of
// 2^-21 of B's norm at the least: 2^-33 beside the rest.)
constexpr float kOrthoX = 256.0f, kOrthoA = 1024.0f, kOrthoB = 256.0f;
struct OrthoArgs {
    const void* g;              // batch x rows x cols
    int64_t g_stride, g_batch;  // elements from row to row, from matrix to matrix
    void* out;                  // batch x rows x cols bfloat16
    int rows, cols, batch;
    int p, q, P, Q;             // q: the longer side
    float eps;
    double* squares;            // sums of squares: `parts` a matrix, kOrthoParts apart
    int parts;
    // X times kOrthoX as float16 (xh) and kLowScale times what that loses (xl): P x Q each, one
    // matrix's 2 P Q values from the next's, so that [xl; xh] is one operand of 2 P rows
    void* xh;
    void* xl;
    unsigned* flags;            // nflags counters a matrix, to clear
    int nflags;
};
constexpr int kOrthoParts = 256;
int ortho_square_parts(int64_t rows, int64_t cols, int dt);
hipError_t launch_ortho_start(const OrthoArgs& a, int dt, hipStream_t stream);
hipError_t launch_ortho_copy(const OrthoArgs& a, hipStream_t stream);      // no steps: X as it is
// all steps of small matrices in one launch (ortho_small.hip): the shorter side at most 128
// and padded to 64 or 128, the longer padded to a multiple of 128, at most 2^15 elements
struct OrthoSteps {
    float v[3 * 64];
    int steps;
};
inline bool ortho_is_small(int64_t p, int64_t q)
{
    const int64_t P = p <= 64 ? 64 : 128;
    return p <= 128 && (q + 127) / 128 * 128 * P <= (int64_t(1) << 15);
}
// ... and one launch a step of longer ones, in parts of 256 along the longer side, where
// every workgroup adds the parts' A = X X^T and makes B of it by itself.  That costs more the
// more parts there are and the larger A is, so the tile kernel takes the longest ones, and
// batches that would be more than a round of workgroups.  Five steps in bf16, here and there:
// 64 x 1024 49 us and 97, 64 x 16384 112 and 130, 64 of 64 x 1024 80 and 150; 128 x 512 85
// and 94, 128 x 2048 109 and 105, 8 of them 124 and 133.  (Parts of 128 columns of 128 rows, before
// X's low half was an operand: 128 x 512 62 us for 72, but 64 of them 28 more, 32 of 128 x 1024 55 more.)
struct OrthoLong {
    float* x;                   // X times kOrthoX: batch x parts x what a workgroup's lanes hold
    float *in, *out;            // A's sums of each part, before the step and after
    int first, last;
    float ca, cb, cc;
};
constexpr int kOrthoPart = 256;
inline int ortho_parts(int64_t q) { return int((q + kOrthoPart - 1) / kOrthoPart); }
inline bool ortho_is_long(int64_t batch, int64_t p, int64_t q)
{
    const int64_t P = p <= 64 ? 64 : 128;
    return p <= 128 && !ortho_is_small(p, q) && ortho_parts(q) * P * P * P <= (int64_t(1) << 24) && ortho_parts(q) * batch <= 256;
}
hipError_t launch_ortho_squares(const OrthoArgs& a, int dt, hipStream_t stream);
hipError_t launch_ortho_long(const OrthoArgs& a, const OrthoSteps& c, float* x, float* sums, int dt, hipStream_t stream);
hipError_t launch_ortho_small(const OrthoArgs& a, const OrthoSteps& c, int dt, hipStream_t stream);
// one of the products for every matrix of the batch
struct OrthoProduct {
    KernelArgs k;
    uint64_t a, b, c, r, low;   // bytes from one matrix's A, B, C, R and L, low to the next's
    uint64_t diag, ws, flags;   // values from one matrix's diagonals, partial sums, counters to the next's
};
typedef hipError_t (*OrthoLaunchFn)(const OrthoProduct& p, int tiles, int batch, hipStream_t stream);
OrthoLaunchFn launcher_ortho(int epi, int cfg);

}  // namespace gemm_relu_hip
