// The orthogonalised update (sm_103a): with X = G / (|G|_F + eps), `steps` times
//
//   A = X X^T (or X^T X, by the shorter side),  B = b A + c A^2,  X = a X + B X (or X B)
//
// (a, b, c) = (3.4445, -4.7750, 2.0315): every singular value s of X goes to
// a s + b s^3 + c s^5, which takes (0, 1] to about [0.7, 1.2] in five steps
// (Jordan et al., "Muon", 2024).  Singular vectors stay as they are.
//
// Rounding.  Products take FP16 operands: X, A and B are bounded whatever G is
// (|X| <= 1.21 in the 2-norm after any step, so |A| <= 1.47 and |B| <= 2.81), so
// powers of two put them at the top of FP16's range and 11 bits of each are kept
// down to 2^-29 of the bound.  The rounding of X must not pass from step to step,
// since a direction that G hardly has grows by a factor of a in each: X itself is
// kept in FP32, a X is formed from that, and only B X sees the FP16 copy (B's range
// is the space of X, so noise outside that space does not enter).  A and B have
// their largest elements on the diagonal, alike where X is near its end; what
// rounding takes there is kept in FP32 and put back: A^2 and b A to first order,
// B X in the factor of X.  Five steps of a 24 x 2000 Gaussian matrix are 1.2e-3 off
// the exact ones before the output's rounding, without the diagonals 2.5e-3; of one
// of rank 6, 1.0e-3.
// A and A^2 are symmetric: tiles on and above the diagonal, written twice.
//
// 12800 x 5120 in FP32: 4.2 ms; a step alone takes 206 us for A (1.63 PFLOP/s of the
// half that is formed), 97 for B and 425 for X (1.58; it also moves 0.8 GB), the norm
// and the first copy 107 (both read G: 0.6 GB in all).
#include "mhcm_orth.cuh"

namespace mhcpb {
namespace orth {

namespace {

using product::Shape;

constexpr float kScaleX = 32768.f, kScaleA = 32768.f, kScaleB = 16384.f;   // 1.21, 1.46 and 2.81 times these < 65504

constexpr int kNormBlocks = 608, kNormThreads = 256;

__device__ __forceinline__ double block_sum(double v) {
    __shared__ double warps[kNormThreads / 32];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int i = 0; i < kNormThreads / 32; ++i) v += warps[i];
    return v;
}

// The norm's kernels go over G in pieces of 1024 elements of a row, a warp each: eight neighbours per lane
// four times, or one 32 times.
template <bool EIGHT, class Each>
__device__ __forceinline__ void over_pieces(const Input& g, int site, Each each) {
    constexpr int kWidth = EIGHT ? 8 : 1, kAtOnce = EIGHT ? 4 : 8;
    using Span = std::conditional_t<EIGHT, product::Eight, product::One>;
    const int64_t across = (g.cols + 1023) / 1024, pieces = g.rows * across;
    const int64_t warps = (int64_t)gridDim.x * (kNormThreads / 32);
    for (int64_t i = (int64_t)blockIdx.x * (kNormThreads / 32) + threadIdx.x / 32; i < pieces; i += warps) {
        const int64_t row = i / across, end = min(g.cols, (i - row * across + 1) * 1024);
        for (int64_t col = (i - row * across) * 1024 + (threadIdx.x & 31) * kWidth; col < end; col += 32 * kWidth * kAtOnce) {
            product::Raw<float, Span> raw[kAtOnce];
#pragma unroll
            for (int q = 0; q < kAtOnce; ++q) {
                const Span at{row, col + 32 * kWidth * q, col + 32 * kWidth * q < end};
                if (at.is) raw[q] = g.raw(at, site);
            }
#pragma unroll
            for (int q = 0; q < kAtOnce; ++q) {
                const Span at{row, col + 32 * kWidth * q, col + 32 * kWidth * q < end};
                if (!at.is) continue;
                float v[Span::n];
                g.to(raw[q], v);
                each(at, v);
            }
        }
    }
}

template <bool EIGHT>
__global__ void __launch_bounds__(kNormThreads) squares_kernel(const Input g, double* partial) {
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    Squares s;
    over_pieces<EIGHT>(g, 0, [&](const auto&, const auto& v) {
        for (float e : v) s.add(e);
    });
    const double total = block_sum(s.sum());
    if (threadIdx.x == 0 && check::in(partial + blockIdx.x, 8, partial, kNormBlocks * 8, 1)) partial[blockIdx.x] = total;
}

// FP16 copy of G / (|G| + eps), and the factors for later; where G's rows are not made of whole vectors also
// its FP32 copy, which the first step then reads instead of G.
template <bool EIGHT>
__global__ void __launch_bounds__(kNormThreads)
    first_copy_kernel(const Input g, const double* partial, double eps, Inverse* inverse, Matrix<__half> x,
                      Matrix<float> full) {
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    double total = 0.0;
    for (int i = threadIdx.x; i < kNormBlocks; i += kNormThreads) total += partial[i];
    total = block_sum(total);
    __shared__ Inverse shared;
    if (threadIdx.x == 0) shared = inverse_of(sqrt(total) + eps);   // (FP64: by one thread)
    __syncthreads();
    const Inverse inv = shared;
    if (blockIdx.x == 0 && threadIdx.x == 0) *inverse = inv;
    over_pieces<EIGHT>(g, 2, [&](const auto& at, const auto& v) {
        using Span = std::decay_t<decltype(at)>;
        float r[Span::n];
#pragma unroll
        for (int k = 0; k < Span::n; ++k) r[k] = scaled(v[k], inv);
        if (!EIGHT) full.store(at, r, 20);
#pragma unroll
        for (int k = 0; k < Span::n; ++k) r[k] *= kScaleX;
        x.store(at, r, 3);
    });
}

// What an FP16 matrix's diagonal lost to rounding, FP32 [size], in the matrix's units.
struct Diagonal {
    float* lost;
    int64_t size;
    __device__ __forceinline__ float at(int64_t i, uint32_t site) const {
        return check::in(lost + i, 4, lost, (size_t)size * 4, site) ? lost[i] : 0.f;
    }
    // of a row whose diagonal element is among these scaled ones
    template <class Span>
    __device__ __forceinline__ void keep(const Span& at, const float (&v)[Span::n], float scale, uint32_t site) const {
#pragma unroll
        for (int i = 0; i < Span::n; ++i)
            if (at.row == at.column(i) && check::in(lost + at.row, 4, lost, (size_t)size * 4, site))
                lost[at.row] = (v[i] - __half2float(__float2half_rn(v[i]))) / scale;
    }
};

// A = C at kScaleA
struct GramEpilogue {
    static constexpr bool kDual = false, kMirror = true, kTwice = false;
    Matrix<__half> out;
    Diagonal lost;
    __device__ __forceinline__ void ahead(int, int64_t, int64_t, int) const {}
    template <class Span>
    struct Read {};
    template <class Span>
    __device__ __forceinline__ Read<Span> read(int, const Span&) const {
        return {};
    }
    template <class Span>
    __device__ __forceinline__ void write(int, const Span& at, const float (&v)[Span::n], const float (&)[Span::n],
                                          const Read<Span>&) const {
        float r[Span::n];
#pragma unroll
        for (int i = 0; i < Span::n; ++i) r[i] = v[i] * (kScaleA / (kScaleX * kScaleX));
        out.store(at, r, 4);
        lost.keep(at, r, kScaleA, 5);
    }
};

// B = b A + c A^2 at kScaleB from C, the product of the rounded A's, and what the
// diagonal lost: (A + l)^2 = A^2 + l A + A l + l^2
struct PolynomialEpilogue {
    static constexpr bool kDual = false, kMirror = true, kTwice = false;
    Matrix<__half> out;
    Matrix<const __half> gram;
    Diagonal gram_lost, lost;
    __device__ __forceinline__ void ahead(int, int64_t, int64_t, int) const {}
    template <class Span>
    struct Read {
        product::Raw<__half, Span> gram;
    };
    template <class Span>
    __device__ __forceinline__ Read<Span> read(int, const Span& at) const {
        return {gram.raw(at, 6)};
    }
    template <class Span>
    __device__ __forceinline__ void write(int, const Span& at, const float (&v)[Span::n], const float (&)[Span::n],
                                          const Read<Span>& in) const {
        float r[Span::n];
        in.gram.to(r);
        const float l = gram_lost.at(at.row, 7);
#pragma unroll
        for (int i = 0; i < Span::n; ++i) {
            const float k = gram_lost.at(at.column(i), 8);
            r[i] = fmaf(kC * kScaleB / (kScaleA * kScaleA), v[i], (kB + kC * (l + k)) * (kScaleB / kScaleA) * r[i]);
            if (at.row == at.column(i)) r[i] += kScaleB * (kB + kC * l) * l;
        }
        out.store(at, r, 9);
        lost.keep(at, r, kScaleB, 10);
    }
};

// X = (a + B's lost diagonal) X + C
struct UpdateEpilogue {
    static constexpr bool kDual = false, kMirror = false, kTwice = false;
    Input g;                    // the first step's X, times *inverse
    const Inverse* inverse;     // null after the first step
    Diagonal lost;
    bool tall;                  // X B: the diagonal goes by columns
    Matrix<float> x;            // X between the steps
    Matrix<__half> copy;        // its FP16 copy
    Matrix<__nv_bfloat16> out;  // the last step's X, times scale; null before
    float scale;
    // (X sent for ahead: 1285 x 3427 took 373 us for 368, 12800 x 5120 1% longer)
    __device__ __forceinline__ void ahead(int, int64_t, int64_t, int) const {}
    template <class Span>
    using Read = product::Raw<float, Span>;
    template <class Span>
    __device__ __forceinline__ Read<Span> read(int, const Span& at) const {
        return inverse != nullptr ? g.raw(at, 11) : x.raw(at, 12);
    }
    template <class Span>
    __device__ __forceinline__ void write(int, const Span& at, const float (&v)[Span::n], const float (&)[Span::n],
                                          const Read<Span>& in) const {
        float r[Span::n];
        if (inverse != nullptr) {
            const Inverse inv = *inverse;
            g.to(in, r);
#pragma unroll
            for (int i = 0; i < Span::n; ++i) r[i] = scaled(r[i], inv);
        } else {
            in.to(r);
        }
        const float by_row = tall || !at.is ? 0.f : lost.at(at.row, 13);
#pragma unroll
        for (int i = 0; i < Span::n; ++i) {
            const float l = tall && at.is ? lost.at(at.column(i), 14) : by_row;
            r[i] = fmaf(kA + l, r[i], v[i] * (1.f / (kScaleB * kScaleX)));
        }
        if (out.ptr != nullptr) {
#pragma unroll
            for (int i = 0; i < Span::n; ++i) r[i] *= scale;
            out.store(at, r, 15);
            return;
        }
        x.store(at, r, 16);
#pragma unroll
        for (int i = 0; i < Span::n; ++i) r[i] *= kScaleX;
        copy.store(at, r, 17);
    }
};

size_t up(size_t bytes) { return (bytes + 255) / 256 * 256; }
int steps_of(int64_t k) { return (int)((k + 63) / 64); }

struct Layout {
    size_t partial, inverse, lost[2], x, copy[2], gram, poly, bytes;
};
Layout layout(int64_t m, int64_t n) {
    const int64_t s = m < n ? m : n, np = product::padded(n), sp = product::padded(s);
    Layout l{};
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t p = at;
        at += up(bytes);
        return p;
    };
    l.partial = take(kNormBlocks * sizeof(double));
    l.inverse = take(sizeof(Inverse));
    l.lost[0] = take((size_t)sp * 4);
    l.lost[1] = take((size_t)sp * 4);
    l.x = take((size_t)(m * np) * 4);
    l.copy[0] = take((size_t)(m * np) * 2);
    l.copy[1] = take((size_t)(m * np) * 2);
    l.gram = take((size_t)(s * sp) * 2);
    l.poly = take((size_t)(s * sp) * 2);
    l.bytes = at;
    return l;
}

#define MHCM_TRY(call)                          \
    do {                                        \
        const cudaError_t e_ = (call);          \
        if (e_ != cudaSuccess) return e_;       \
    } while (0)

}  // namespace

size_t workspace_bytes(int64_t m, int64_t n) { return few_rows(m, n) ? 0 : layout(m, n).bytes; }

cudaError_t orthogonalize(const Args& a, cudaStream_t stream) {
    if (few_rows(a.m, a.n)) return few_rows_orthogonalize(a, stream);
    const int64_t m = a.m, n = a.n, s = m < n ? m : n, np = product::padded(n), sp = product::padded(s);
    const bool tall = m > n;
    const Layout l = layout(m, n);
    char* ws = static_cast<char*>(a.workspace);
    double* partial = reinterpret_cast<double*>(ws + l.partial);
    Inverse* inverse = reinterpret_cast<Inverse*>(ws + l.inverse);
    const Diagonal gram_lost{reinterpret_cast<float*>(ws + l.lost[0]), sp}, poly_lost{reinterpret_cast<float*>(ws + l.lost[1]), sp};
    const Input g{a.g, a.type, m, a.g_stride, n};
    auto half_matrix = [&](size_t at, int64_t rows, int64_t ld) {
        return Matrix<__half>{reinterpret_cast<__half*>(ws + at), ld, (size_t)(rows * ld)};
    };
    const Matrix<__half> copies[2] = {half_matrix(l.copy[0], m, np), half_matrix(l.copy[1], m, np)};
    const Matrix<__half> gram = half_matrix(l.gram, s, sp), poly = half_matrix(l.poly, s, sp);
    const Matrix<const __half> gram_in{gram.ptr, gram.ld, gram.elements};
    const Matrix<float> x{reinterpret_cast<float*>(ws + l.x), np, (size_t)(m * np)};
    const Matrix<__nv_bfloat16> out{static_cast<__nv_bfloat16*>(a.out), a.out_stride, (size_t)((m - 1) * a.out_stride + n)};
    product::Factor factor_x[2], factor_gram, factor_poly;
    MHCM_TRY(factor_x[0].make(false, copies[0].ptr, m, n, np));
    MHCM_TRY(factor_x[1].make(false, copies[1].ptr, m, n, np));
    MHCM_TRY(factor_gram.make(false, gram.ptr, s, s, sp));
    MHCM_TRY(factor_poly.make(false, poly.ptr, s, s, sp));

    const bool eight = g.by_eight();
    MHCM_TRY(ops::launch_early(eight ? squares_kernel<true> : squares_kernel<false>, dim3(kNormBlocks), dim3(kNormThreads),
                               0, stream, g, partial));
    const int64_t blocks = (m * ((n + 1023) / 1024) + kNormThreads / 32 - 1) / (kNormThreads / 32);
    MHCM_TRY(ops::launch_early(eight ? first_copy_kernel<true> : first_copy_kernel<false>,
                               dim3((unsigned)(blocks < 1216 ? blocks : 1216)), dim3(kNormThreads), 0, stream, g,
                               static_cast<const double*>(partial), static_cast<double>(a.eps), inverse, copies[0], x));
    for (int i = 0; i < a.steps; ++i) {
        const product::Factor* cur = &factor_x[i & 1];
        Shape p{};
        p.mode = product::kSymmetric;
        p.M = p.N = s, p.k_steps = steps_of(tall ? m : n), p.a_mn = p.b_mn = tall;
        MHCM_TRY(product::launch(p, GramEpilogue{gram, gram_lost}, cur, nullptr, cur, nullptr, stream));
        p.k_steps = steps_of(s), p.a_mn = p.b_mn = 0;
        const PolynomialEpilogue polynomial{poly, gram_in, gram_lost, poly_lost};
        MHCM_TRY(product::launch(p, polynomial, &factor_gram, nullptr, &factor_gram, nullptr, stream));
        p.mode = product::kPlain;
        p.M = m, p.N = n, p.k_steps = steps_of(s), p.b_mn = !tall;
        const bool last = i + 1 == a.steps;
        const UpdateEpilogue update{g, i == 0 && eight ? inverse : nullptr, poly_lost, tall, x, copies[(i + 1) & 1],
                                    last ? out : Matrix<__nv_bfloat16>{nullptr, 0, 0}, a.scale};
        p.narrow = last && !out.by_eight(n);   // (the output is the caller's)
        if (tall)
            MHCM_TRY(product::launch(p, update, cur, nullptr, &factor_poly, nullptr, stream));
        else
            MHCM_TRY(product::launch(p, update, &factor_poly, nullptr, cur, nullptr, stream));
    }
    return cudaSuccess;
}

cudaError_t setup() {
    MHCM_TRY(product::allow<GramEpilogue>());
    MHCM_TRY(product::allow<PolynomialEpilogue>());
    return product::allow<UpdateEpilogue>();
}
cudaError_t checked_site(uint32_t* site) {
    uint32_t other = 0;
    const cudaError_t e = check::read_and_clear(site), f = few_rows_site(&other);
    if (*site == 0) *site = other;
    return e != cudaSuccess ? e : f;
}
cudaError_t device_status(uint32_t* status, bool clear) { return product::read_status(status, clear); }

}  // namespace orth
}  // namespace mhcpb
