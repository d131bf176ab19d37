// Internal interface of the matrix operators: the product (mhcm_product.cuh),
// the feed-forward block (mhcm_ffn.cu), the orthogonalised update (mhcm_orth.cu)
// and their host checks (mhcm_api.cu).
#pragma once
#include "mhcs_internal.h"

namespace mhcpb {

// Tensor map over a 16-bit matrix [rows, cols], rows `ld` elements apart (a
// multiple of 8; base 16-byte aligned): boxes of 64 columns and box_rows rows,
// 128-byte swizzle (defined in mhcpb_api.cu).
bool encode_16bit_map(CUtensorMap* m, bool bf16, const void* base, int64_t rows, int64_t cols, int64_t ld,
                      uint32_t box_rows);

namespace product {

enum Mode {
    kPlain = 0,
    kSideBySide = 1,   // two products of one A, with B of b0 and of b1 (C has N columns of each)
    kLongK = 2,        // the sum of two products, a0 b0 + a1 b1
    kGroups = 3,       // two products, a0 b0 and a1 b1
    kSymmetric = 4     // C is symmetric: tiles on and above the diagonal, written twice
};
struct Shape {
    int64_t M, N;
    int k_steps;       // of 64, per product
    int mode;
    int a_mn, b_mn;    // the operand's rows are k (else its rows are m, or n)
    int bf16;          // else FP16
    int narrow;        // the epilogue's matrices are taken element by element (see Eight)
    int twice;         // A's 64 rows are followed by 64 of what their rounding lost: both are multiplied, as rows
                       // of one MMA, and the results added at the end (M <= 64: single blocks; Epilogue::kTwice)
    float second;      // twice: what one of those rows' numbers stands for
    int stall;         // a test's: the MMA issuer waits for what nothing signals
    // set by choose()
    int m_tiles, n_tiles, tiles;
    int full;          // tiles from this one on are halves (pairs of blocks)
    int tile_n;        // columns of C per tile (of each product, side by side)
    int split;         // blocks that share a tile's sum
    int b_box;         // rows of B in one box, 0: boxes of 64
    int stages, part_row, tmem_columns;   // single blocks: see product_kernel
    uint32_t b_bytes;
};
struct Choice {
    bool pair;
    bool long_sum;     // a block's sum has more than kPieceSteps steps and is taken in pieces
    int grid;
    uint32_t smem;     // of a single block
};
Choice choose(Shape& s);

constexpr int kBox = 64;                           // columns, and mostly rows, of a box
constexpr uint32_t kBoxBytes = kBox * kBox * 2;    // 8 KiB
constexpr int kMaxStages = 8;
// The tensor cores cut what they add to an FP32 accumulator, so that a sum of one sign loses some 2^-23 of
// itself with every 16 terms (2^20 positive ones: 6.4e-3, 0.8 of that).  Sums of more steps of 64 k than this
// are taken in pieces of as many (32,768 terms: 2e-4), which are added rounded.
constexpr int kPieceSteps = 512;
constexpr uint32_t kSharedMost = 232448;           // per block; two blocks share 233,472 with 1 KiB each for the system

// A 16-bit factor of a product, and its map with boxes of 64 rows.
struct Factor {
    CUtensorMap map;
    const void* ptr;
    int64_t rows, cols, ld;
    bool bf16;
    bool encode(CUtensorMap* m, int box_rows) const {
        return encode_16bit_map(m, bf16, ptr, rows, cols, ld, (uint32_t)box_rows);
    }
    cudaError_t make(bool is_bf16, const void* p, int64_t r, int64_t c, int64_t distance) {
        ptr = p, rows = r, cols = c, ld = distance, bf16 = is_bf16;
        return encode(&map, kBox) ? cudaSuccess : cudaErrorInvalidValue;
    }
};

inline int64_t padded(int64_t n) { return (n + 7) / 8 * 8; }

}  // namespace product

namespace ffn {
struct Args {
    int64_t T, D, F;
    int type, activation;
    const void *x, *w_gate, *w_up, *w_down;
    int64_t x_stride;
    void* y;
    int64_t y_stride;
    void *gate, *up;              // [T, F]; the forward's may be null
    const void* grad_y;
    int64_t gy_stride;
    void* grad_x;                 // may be null
    int64_t gx_stride;
    void* grad_w[3];              // gate, up, down; each may be null
    int grad_type;
    bool accumulate, stall;
    void* workspace;
};
// few tokens (mhcm_token.cu): whether the sizes are taken, and the forward
bool few_tokens(int64_t T, int64_t D, int64_t F);
cudaError_t few_tokens_forward(const Args& a, cudaStream_t stream);
cudaError_t few_tokens_site(uint32_t* site);
size_t forward_workspace_bytes(int64_t T, int64_t D, int64_t F);
size_t backward_workspace_bytes(int64_t T, int64_t D, int64_t F);
cudaError_t forward(const Args& a, cudaStream_t stream);
cudaError_t backward(const Args& a, cudaStream_t stream);
cudaError_t setup();
cudaError_t checked_site(uint32_t* site);
cudaError_t device_status(uint32_t* status, bool clear);
}  // namespace ffn

namespace orth {
struct Args {
    int64_t m, n;
    int type;
    const void* g;
    int64_t g_stride;
    void* out;                    // BF16
    int64_t out_stride;
    int steps;
    float eps;
    float scale;
    void* workspace;
};
// few rows or columns (mhcm_orth_few.cu): whether the sizes are taken, and the call
bool few_rows(int64_t m, int64_t n);
cudaError_t few_rows_orthogonalize(const Args& a, cudaStream_t stream);
cudaError_t few_rows_site(uint32_t* site);
size_t workspace_bytes(int64_t m, int64_t n);
cudaError_t orthogonalize(const Args& a, cudaStream_t stream);
cudaError_t setup();
cudaError_t checked_site(uint32_t* site);
cudaError_t device_status(uint32_t* status, bool clear);
}  // namespace orth
}  // namespace mhcpb
