// The feed-forward block for one to four tokens (sm_103a): its time is the weights'
// way from memory (6 D F bytes), so this is a matrix-vector product that keeps HBM
// busy, on the CUDA cores: every weight is multiplied once per token, and a product
// with tensor cores would fill 127 of 128 rows with nothing.
//
// One block of 16 warps per SM; the block's rows of weights are a contiguous 152nd
// of all.  Four warps share a row's k (quarters), four such groups take two pairs of
// gate and up rows (or four rows of the second product) at a time: twelve 16-byte
// loads per thread are under way, 96 KB per SM (eight: 3% slower).  x lies in shared memory in FP32.
// One token, 5120 x 12800 BF16: 65 us for 393 MB (6.0 TB/s, 90% of the copy rate), of
// which the first launch 43 and the second 25; by the product kernel 91.
// act(g) u stays in FP32 between the two launches.
// Sums are FP32 in a fixed order: per thread, over the lanes, over the quarters.
// Rows that do not start at 16 bytes are read by the aligned 16-byte vectors that hold
// them, and x at the shift: element k lies in plane k mod 8 at k / 8, so that the lanes
// read neighbours whatever the shift is, and one copy of x serves all eight.
// 7261 x 12360: one token 116 us, two 139 (words of 4 bytes, one element shifted: 710),
// four 236, bound by reading x, 4 bytes per weight and token (by the product kernel
// with padded copies of the weights 258).
#include "mhcm_ffn.cuh"
#include "mhcm_product.cuh"

namespace mhcpb {
namespace ffn {

namespace {

using ptx::fma2;
using ptx::pair;
using ptx::sum_of;

constexpr int kBlocks = 152, kThreads = 512, kQuarters = 4, kGroups = kThreads / 32 / kQuarters;
constexpr int kRows = 4;       // weight rows of a warp at a time
constexpr int kUnroll = 3;

// The first launch (DUAL) leaves act(g) u in FP32 for the second.
template <class T, bool DUAL>
struct TokenArgs {
    using X = std::conditional_t<DUAL, T, float>;
    using Out = std::conditional_t<DUAL, float, T>;
    const T *w0, *w1;      // [R, K]; w1: the up projection (DUAL)
    int64_t R;
    int K;
    const X* x;            // [tokens, K], rows x_ld apart
    int64_t x_ld;
    int tokens;
    Out* out;              // [tokens, R], rows out_ld apart: act(g) u, or the products
    int64_t out_ld;
    T *gate, *up;          // [tokens, R] or null
    int activation;
    int after;             // x comes from the launch before, the weights do not
};

// Vectors of eight elements that hold a row of K, wherever it starts.
__host__ __device__ constexpr int row_vectors(int K) { return (K + 14) / 8; }
// Floats of one plane: a zero, the vectors', and what keeps eight planes on different banks.
__host__ __device__ constexpr int plane_floats(int K) { return (row_vectors(K) + 4) / 8 * 8 + 4; }
// Elements of x in shared memory per token.  WIDE: the first and the second four of every eight apart
// (vectors without bank conflicts).  Else eight planes.
template <bool WIDE>
__host__ __device__ constexpr int x_floats(int K) {
    return WIDE ? K : 8 * plane_floats(K);
}
template <bool WIDE>
size_t token_smem(int tokens, int K, int64_t R, bool dual) {
    const int64_t rows = (R + kBlocks - 1) / kBlocks + 1;
    return ((size_t)tokens * x_floats<WIDE>(K) + (size_t)rows * (dual ? 2 : 1) * kQuarters * tokens) * 4;
}

// Elements of other rows ahead of `row` in the 16 bytes that it starts in.
template <class T>
__device__ int ahead(const T* row) { return (int)((reinterpret_cast<uintptr_t>(row) >> 1) & 7); }

template <class T, int NT, bool DUAL, bool WIDE>
__global__ void __launch_bounds__(kThreads, 1) token_kernel(const TokenArgs<T, DUAL> a) {
    using X = typename TokenArgs<T, DUAL>::X;
    using Out = typename TokenArgs<T, DUAL>::Out;
    extern __shared__ float4 shared[];
    float* xs = reinterpret_cast<float*>(shared);
    constexpr int kOutputs = DUAL ? kRows / 2 : kRows;     // rows of the output per warp and turn
    const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) % kQuarters, group = threadIdx.x / (32 * kQuarters);
    const int K = a.K, xn = x_floats<WIDE>(K), plane = plane_floats(K);
    float* part = xs + (size_t)NT * xn;                    // [row of the block][which of two][quarter][token]
    const int64_t first = blockIdx.x * a.R / gridDim.x, end = (blockIdx.x + 1) * a.R / gridDim.x;
    const size_t weight_bytes = (size_t)a.R * K * sizeof(T);

    if (a.after)   // the block's first weights on their way while the launch before ends
        for (int64_t i = first * K * (int64_t)sizeof(T) + threadIdx.x * 128;
             i < end * K * (int64_t)sizeof(T) && i < first * K * (int64_t)sizeof(T) + 131072; i += kThreads * 128)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const char*>(a.w0) + i));
    ptx::grid_dependency_wait();

    const size_t x_bytes = ((a.tokens - 1) * a.x_ld + K) * sizeof(X);
    if constexpr (WIDE) {
        for (int i = threadIdx.x; i < NT * (K / 8); i += kThreads) {
            const int t = NT == 1 ? 0 : i / (K / 8), v = i - t * (K / 8);
            const X* p = a.x + t * a.x_ld + v * 8;
            float4 lo = make_float4(0.f, 0.f, 0.f, 0.f), hi = lo;
            if (t < a.tokens && check::in(p, 8 * sizeof(X), a.x, x_bytes, 12)) {
                if constexpr (sizeof(X) == 4) {
                    lo = reinterpret_cast<const float4*>(p)[0], hi = reinterpret_cast<const float4*>(p)[1];
                } else {
                    const uint4 u = *reinterpret_cast<const uint4*>(p);
                    const float2 e0 = product::Pair16<X>::unpack(u.x), e1 = product::Pair16<X>::unpack(u.y),
                                 e2 = product::Pair16<X>::unpack(u.z), e3 = product::Pair16<X>::unpack(u.w);
                    lo = make_float4(e0.x, e0.y, e1.x, e1.y), hi = make_float4(e2.x, e2.y, e3.x, e3.y);
                }
            }
            *reinterpret_cast<float4*>(xs + t * xn + v * 4) = lo;
            *reinterpret_cast<float4*>(xs + t * xn + K / 2 + v * 4) = hi;
        }
    } else {
        const int across = 8 * (plane - 1);                // elements 0 .. K - 1 and zeros on both sides
        for (int i = threadIdx.x; i < NT * (across + 8); i += kThreads) {
            const int t = i / (across + 8), k = i - t * (across + 8) - 8;
            const X* p = a.x + t * a.x_ld + k;
            const bool is = t < a.tokens && k >= 0 && k < K && check::in(p, sizeof(X), a.x, x_bytes, 12);
            xs[t * xn + (k & 7) * plane + 1 + (k >> 3)] = is ? (float)*p : 0.f;
        }
    }
    __syncthreads();

    const int vectors = WIDE ? K / 8 : row_vectors(K);
    const int v0 = (int)((int64_t)quarter * vectors / kQuarters), v1 = (int)((int64_t)(quarter + 1) * vectors / kQuarters);
    for (int64_t f = first + group * kOutputs; f < end; f += kGroups * kOutputs) {
        uint64_t acc[NT][kRows];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < kRows; ++r) acc[t][r] = 0;
        const T* row[kRows];
        bool valid[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const int64_t i = f + (DUAL ? r / 2 : r);
            valid[r] = i < end;
            row[r] = (DUAL && (r & 1) ? a.w1 : a.w0) + i * K;
        }
        for (int v = v0 + lane; v < v1; v += 32 * kUnroll) {
            if constexpr (WIDE) {
                uint4 u[kUnroll][kRows];
#pragma unroll
                for (int j = 0; j < kUnroll; ++j)
#pragma unroll
                    for (int r = 0; r < kRows; ++r) {
                        u[j][r] = make_uint4(0, 0, 0, 0);
                        const T* p = row[r] + (int64_t)(v + 32 * j) * 8;
                        if (valid[r] && v + 32 * j < v1 &&
                            check::in(p, 16, DUAL && (r & 1) ? a.w1 : a.w0, weight_bytes, 13))
                            u[j][r] = __ldcs(reinterpret_cast<const uint4*>(p));
                    }
#pragma unroll
                for (int j = 0; j < kUnroll; ++j) {
                    if (v + 32 * j >= v1) break;
                    uint64_t x[NT][4];
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const float4 lo = *reinterpret_cast<const float4*>(xs + t * xn + (v + 32 * j) * 4);
                        const float4 hi = *reinterpret_cast<const float4*>(xs + t * xn + K / 2 + (v + 32 * j) * 4);
                        x[t][0] = pair(lo.x, lo.y), x[t][1] = pair(lo.z, lo.w);
                        x[t][2] = pair(hi.x, hi.y), x[t][3] = pair(hi.z, hi.w);
                    }
#pragma unroll
                    for (int r = 0; r < kRows; ++r) {
                        const uint32_t w[4] = {u[j][r].x, u[j][r].y, u[j][r].z, u[j][r].w};
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const float2 e = product::Pair16<T>::unpack(w[q]);
#pragma unroll
                            for (int t = 0; t < NT; ++t) acc[t][r] = fma2(pair(e.x, e.y), x[t][q], acc[t][r]);
                        }
                    }
                }
            } else {
                // vector i of a row: elements 8 i - ahead .. 8 i - ahead + 7, of which the first and the last
                // vector have some of the rows beside it
                uint4 u[kUnroll][kRows];
#pragma unroll
                for (int j = 0; j < kUnroll; ++j)
#pragma unroll
                    for (int r = 0; r < kRows; ++r) {
                        u[j][r] = make_uint4(0, 0, 0, 0);
                        const int k = 8 * (v + 32 * j) - ahead(row[r]);
                        const T* p = row[r] + k;
                        const T* const base = DUAL && (r & 1) ? a.w1 : a.w0;
                        if (!valid[r] || v + 32 * j >= v1 || k >= K) continue;
                        if (p >= base && p + 8 <= base + a.R * K) {
                            if (check::in(p, 16, base, weight_bytes, 14)) u[j][r] = __ldcs(reinterpret_cast<const uint4*>(p));
                        } else {   // the matrix's first or last
                            uint32_t w[4] = {};
#pragma unroll
                            for (int q = 0; q < 8; ++q)
                                if (k + q >= 0 && k + q < K && check::in(p + q, 2, base, weight_bytes, 14))
                                    w[q / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[q] << (16 * (q & 1));
                            u[j][r] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    const int shift = ahead(row[r]);
                    int at[8];
#pragma unroll
                    for (int q = 0; q < 8; ++q) at[q] = ((q - shift) & 7) * plane + 1 + ((q - shift) >> 3);
#pragma unroll
                    for (int j = 0; j < kUnroll; ++j) {
                        const int i = v + 32 * j, k = 8 * i - shift;
                        if (i >= v1) break;
                        uint32_t w[4] = {u[j][r].x, u[j][r].y, u[j][r].z, u[j][r].w};
                        if (k < 0 || k + 8 > K) {
#pragma unroll
                            for (int q = 0; q < 8; ++q)
                                if (k + q < 0 || k + q >= K) w[q / 2] &= q & 1 ? 0x0000FFFFu : 0xFFFF0000u;
                        }
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const float2 e = product::Pair16<T>::unpack(w[q]);
#pragma unroll
                            for (int t = 0; t < NT; ++t) {
                                const float* x = xs + t * xn + i;
                                acc[t][r] = fma2(pair(e.x, e.y), pair(x[at[2 * q]], x[at[2 * q + 1]]), acc[t][r]);
                            }
                        }
                    }
                }
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                float v = sum_of(acc[t][r]);
#pragma unroll
                for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
                if (lane == 0 && valid[r])
                    part[(((f - first) * (DUAL ? 2 : 1) + r) * kQuarters + quarter) * NT + t] = v;
            }
    }
    // (not earlier: what the next launch prefetches would be gone again before it is used)
    ptx::grid_launch_dependents();
    __syncthreads();
    const int rows = (int)(end - first);
    for (int i = threadIdx.x; i < rows * NT; i += kThreads) {
        const int t = i / rows, r = i - t * rows;
        if (t >= a.tokens) continue;
        auto total = [&](int line) {
            float v = 0.f;
#pragma unroll
            for (int q = 0; q < kQuarters; ++q) v += part[(line * kQuarters + q) * NT + t];
            return v;
        };
        const int64_t f = first + r;
        Out* o = a.out + t * a.out_ld + f;
        const bool ok = check::in(o, sizeof(Out), a.out, ((a.tokens - 1) * a.out_ld + a.R) * sizeof(Out), 15);
        if constexpr (DUAL) {
            const float g = total(2 * r), u = total(2 * r + 1);
            if (ok) *o = activate(g, a.activation).x * u;
            if (a.gate != nullptr && check::in(a.gate + t * a.R + f, sizeof(T), a.gate, a.tokens * a.R * sizeof(T), 16)) {
                a.gate[t * a.R + f] = (T)g;
                a.up[t * a.R + f] = (T)u;
            }
        } else if (ok) {
            *o = (Out)total(r);
        }
    }
}

template <class T, int NT, bool DUAL, bool WIDE>
cudaError_t launch(const TokenArgs<T, DUAL>& a, cudaStream_t stream) {
    static std::atomic<uint64_t> done{0};
    auto* kernel = token_kernel<T, NT, DUAL, WIDE>;
    const cudaError_t e = ops::allow_shared(kernel, (int)product::kSharedMost, done);
    if (e != cudaSuccess) return e;
    // at least half of an SM's shared memory: of two blocks that fit one SM, some SMs would get both when
    // the launch before ends, and others none (the pair of launches took 85 us for 75)
    const size_t smem = token_smem<WIDE>(NT, a.K, a.R, DUAL), half = 120 * 1024;
    return ops::launch_early(kernel, dim3(kBlocks), dim3(kThreads), smem > half ? smem : half, stream, a);
}
template <class T, bool DUAL, bool WIDE>
cudaError_t by_tokens(const TokenArgs<T, DUAL>& a, cudaStream_t stream) {
    return a.tokens == 1 ? launch<T, 1, DUAL, WIDE>(a, stream)
                         : a.tokens == 2 ? launch<T, 2, DUAL, WIDE>(a, stream) : launch<T, 4, DUAL, WIDE>(a, stream);
}
template <class T, bool DUAL>
cudaError_t by_rows(const TokenArgs<T, DUAL>& a, cudaStream_t stream) {
    return a.K % 8 == 0 ? by_tokens<T, DUAL, true>(a, stream) : by_tokens<T, DUAL, false>(a, stream);
}

template <class T>
cudaError_t forward_as(const Args& a, cudaStream_t stream) {
    float* hidden = static_cast<float*>(a.workspace);
    TokenArgs<T, true> first{};
    first.w0 = static_cast<const T*>(a.w_gate);
    first.w1 = static_cast<const T*>(a.w_up);
    first.R = a.F;
    first.K = (int)a.D;
    first.x = static_cast<const T*>(a.x);
    first.x_ld = a.x_stride;
    first.tokens = (int)a.T;
    first.out = hidden;
    first.out_ld = a.F;
    first.gate = static_cast<T*>(a.gate);
    first.up = static_cast<T*>(a.up);
    first.activation = a.activation;
    const cudaError_t e = by_rows(first, stream);
    if (e != cudaSuccess) return e;
    TokenArgs<T, false> second{};
    second.w0 = static_cast<const T*>(a.w_down);
    second.R = a.D;
    second.K = (int)a.F;
    second.x = hidden;
    second.x_ld = a.F;
    second.tokens = (int)a.T;
    second.out = static_cast<T*>(a.y);
    second.out_ld = a.y_stride;
    second.after = 1;
    return by_rows(second, stream);
}

bool fits(int tokens, int64_t K, int64_t R, bool dual) {
    return (K % 8 == 0 ? token_smem<true>(tokens, (int)K, R, dual) : token_smem<false>(tokens, (int)K, R, dual)) <=
           product::kSharedMost;
}

}  // namespace

bool few_tokens(int64_t T, int64_t D, int64_t F) {
    if (T > 4) return false;
    const int tokens = T == 3 ? 4 : (int)T;
    return fits(tokens, D, F, true) && fits(tokens, F, D, false);
}
cudaError_t few_tokens_forward(const Args& a, cudaStream_t stream) {
    return a.type == MHCPB_BF16 ? forward_as<__nv_bfloat16>(a, stream) : forward_as<__half>(a, stream);
}
cudaError_t few_tokens_site(uint32_t* site) { return check::read_and_clear(site); }

}  // namespace ffn
}  // namespace mhcpb
