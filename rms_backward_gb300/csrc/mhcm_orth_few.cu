// The orthogonalised update of a matrix with a short side of at most 32 (sm_103a),
// such as the projection's weight [24, K]: there the general path is seventeen
// launches of next to no work.  Here one cluster of 16 blocks holds X in its shared
// memory, in FP32, each block a sixteenth of the long side, and takes all steps in one
// launch (which fails where the process may not use so many SMs of one GPU cluster):
//
//   A = X X^T   per block over its columns, 4 x 4 tiles per thread; the blocks' parts
//               are added in rank order by every block (distributed shared memory)
//   P = a I + b A + c A^2   by every block
//   X = P X     four columns per thread, in place
//
// FP32 throughout.  24 x 20480: 81 us (156 by the general path); a step takes 27,000
// clocks, 8,600 for A and 14,400 for P X, both at the 128 bytes per clock that shared
// memory gives an SM's registers; packed FP32 arithmetic keeps below that.
#include "mhcm_orth.cuh"

namespace mhcpb {
namespace orth {

namespace {

constexpr int kCluster = 16, kThreads = 512, kMostSlices = 32;

template <int S>
struct FewCfg {
    static constexpr int columns = S <= 24 ? 4 : 2;    // of X per thread at a time (registers)
    static constexpr int row = S + 4;                  // floats from column to column of X: no bank conflicts
    static constexpr int tiles = S / 4, pairs = tiles * (tiles + 1) / 2, values = pairs * 16;
    static constexpr int slices = kThreads / pairs < kMostSlices ? kThreads / pairs : kMostSlices;
    static constexpr int fixed = slices * values + 2 * values + 2 * S * S + 64;   // floats besides X
};
template <int S>
size_t few_smem(int64_t l) {
    return (size_t)(((l + kCluster - 1) / kCluster) * FewCfg<S>::row + FewCfg<S>::fixed) * 4;
}

template <int S>
__global__ void __launch_bounds__(kThreads, 1)
    few_rows_kernel(const Input g, int tall, int s, int64_t l, int steps, double eps, float scale, Matrix<__nv_bfloat16> out) {
    using C = FewCfg<S>;
    extern __shared__ float4 shared[];
    float* parts = reinterpret_cast<float*>(shared);   // [slices][values]
    float* sums = parts + C::slices * C::values;       // two turns of the block's part of A
    float* gram = sums + 2 * C::values;                // [S][S]
    float* poly = gram + S * S;                        // [S][S]
    double* squares = reinterpret_cast<double*>(poly + S * S);   // the block's sum, one per warp; the inverse
    float* x = poly + S * S + 64;                      // [columns][row]
    const int rank = (int)ptx::cluster_rank(), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t first = rank * l / kCluster;
    const int columns = (int)((rank + 1) * l / kCluster - first);
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();

    // X's column k is x[k * row ..], elements beyond the short side 0; eight loads per lane under way.
    // Pieces of 256 elements along G's rows, a warp each.
    constexpr int kAtOnce = 8;
    Squares sq;
    const int rows = tall ? columns : s, width = tall ? s : columns, across = (width + 255) / 256;
    for (int piece = warp; piece < rows * across; piece += kThreads / 32) {
        const int r = piece / across, c = (piece - r * across) * 256 + lane;
        product::Raw<float, product::One> raw[kAtOnce];
#pragma unroll
        for (int q = 0; q < kAtOnce; ++q)
            raw[q] = g.raw(product::One{tall ? first + r : r, (tall ? 0 : first) + c + 32 * q, c + 32 * q < width}, 18);
#pragma unroll
        for (int q = 0; q < kAtOnce; ++q) {
            if (c + 32 * q >= width) break;
            float v[1];
            g.to(raw[q], v);
            sq.add(v[0]);
            x[tall ? r * C::row + c + 32 * q : (c + 32 * q) * C::row + r] = v[0];
        }
    }
    for (int e = threadIdx.x; e < columns * (S - s); e += kThreads)
        x[e / (S - s) * C::row + s + e % (S - s)] = 0.f;
    double total = sq.sum();
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, d);
    if (lane == 0) squares[1 + warp] = total;
    __syncthreads();
    if (threadIdx.x == 0) {
        total = 0.0;
        for (int w = 0; w < kThreads / 32; ++w) total += squares[1 + w];
        squares[0] = total;
    }
    ptx::cluster_arrive();
    ptx::cluster_wait();
    Inverse* inverse = reinterpret_cast<Inverse*>(squares + 20);
    if (threadIdx.x == 0) {   // (FP64: by one thread)
        double part[kCluster];
#pragma unroll
        for (int z = 0; z < kCluster; ++z) part[z] = ptx::ld_cluster_f64(ptx::map_rank(ptx::smem_u32(squares), z));
        total = 0.0;
#pragma unroll
        for (int z = 0; z < kCluster; ++z) total += part[z];
        *inverse = inverse_of(sqrt(total) + eps);
    }
    __syncthreads();
    const Inverse inv = *inverse;
    for (int e = threadIdx.x; e < columns * (C::row / 4); e += kThreads) {   // (the columns' gaps too)
        float4 v = reinterpret_cast<float4*>(x)[e];
        v.x = scaled(v.x, inv), v.y = scaled(v.y, inv), v.z = scaled(v.z, inv), v.w = scaled(v.w, inv);
        reinterpret_cast<float4*>(x)[e] = v;
    }

    // this thread's tile of A: rows 4 ti .., columns 4 tj ..
    const int pair = threadIdx.x % C::pairs, slice = threadIdx.x / C::pairs;
    int ti = 0, tj = pair;
    while (tj >= C::tiles - ti) tj -= C::tiles - ti++;
    tj += ti;
    for (int step = 0; step < steps; ++step) {
        __syncthreads();
        if (slice < C::slices) {
            uint64_t acc[4][2] = {};
            for (int k = slice; k < columns; k += C::slices) {
                const float4 a = *reinterpret_cast<const float4*>(x + k * C::row + 4 * ti);
                const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(x + k * C::row + 4 * tj);
                const float u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint64_t two = ptx::pair(u[i], u[i]);
                    acc[i][0] = ptx::fma2(two, b.x, acc[i][0]);
                    acc[i][1] = ptx::fma2(two, b.y, acc[i][1]);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<ulonglong2*>(parts + slice * C::values + pair * 16 + 4 * i) =
                    make_ulonglong2(acc[i][0], acc[i][1]);
        }
        __syncthreads();
        float* mine = sums + (step & 1) * C::values;   // (a block may still read the last step's)
        for (int e = threadIdx.x; e < C::values; e += kThreads) {
            float v = 0.f;
#pragma unroll 4
            for (int q = 0; q < C::slices; ++q) v += parts[q * C::values + e];
            mine[e] = v;
        }
        ptx::cluster_arrive();
        ptx::cluster_wait();
        for (int e = threadIdx.x; e < C::values; e += kThreads) {
            const uint32_t at = ptx::smem_u32(mine + e);
            float v[kCluster];
#pragma unroll
            for (int z = 0; z < kCluster; ++z) v[z] = ptx::ld_cluster_f32(ptx::map_rank(at, z));
            float t = 0.f;
#pragma unroll
            for (int z = 0; z < kCluster; ++z) t += v[z];
            int i = 0, j = e / 16;
            while (j >= C::tiles - i) j -= C::tiles - i++;
            const int r = 4 * i + e % 16 / 4, c = 4 * (i + j) + e % 4;
            gram[r * S + c] = t;
            if (j != 0) gram[c * S + r] = t;
        }
        __syncthreads();
        for (int e = threadIdx.x; e < S * S; e += kThreads) {
            const int i = e / S, j = e - i * S;
            float t = 0.f;
#pragma unroll 8
            for (int k = 0; k < S; ++k) t = fmaf(gram[i * S + k], gram[k * S + j], t);
            poly[e] = fmaf(kC, t, kB * gram[e]) + (i == j ? kA : 0.f);
        }
        __syncthreads();
        // (shared memory gives a warp 128 bytes per clock, of a broadcast too: P is read once for several columns)
        constexpr int N = C::columns;
        const int stride = (columns + N - 1) / N;
        for (int k = threadIdx.x; k < stride; k += kThreads) {
            uint64_t u[S][N / 2];
#pragma unroll
            for (int j = 0; j < S; j += 4)
#pragma unroll
                for (int c = 0; c < N; c += 2) {
                    const float4 a = *reinterpret_cast<const float4*>(x + min(k + c * stride, columns - 1) * C::row + j);
                    const float4 b = *reinterpret_cast<const float4*>(x + min(k + (c + 1) * stride, columns - 1) * C::row + j);
                    u[j][c / 2] = ptx::pair(a.x, b.x), u[j + 1][c / 2] = ptx::pair(a.y, b.y);
                    u[j + 2][c / 2] = ptx::pair(a.z, b.z), u[j + 3][c / 2] = ptx::pair(a.w, b.w);
                }
#pragma unroll 1
            for (int i = 0; i < S; i += 4) {
                uint64_t p[4][N / 2] = {};
#pragma unroll
                for (int j = 0; j < S; ++j) {   // (P is symmetric)
                    const float4 m = *reinterpret_cast<const float4*>(poly + j * S + i);
                    const uint64_t two[4] = {ptx::pair(m.x, m.x), ptx::pair(m.y, m.y), ptx::pair(m.z, m.z), ptx::pair(m.w, m.w)};
#pragma unroll
                    for (int c = 0; c < N / 2; ++c)
#pragma unroll
                        for (int r = 0; r < 4; ++r) p[r][c] = ptx::fma2(two[r], u[j][c], p[r][c]);
                }
#pragma unroll
                for (int c = 0; c < N; ++c) {
                    float q[4];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float2 f = ptx::both(p[r][c / 2]);
                        q[r] = c & 1 ? f.y : f.x;
                    }
                    // (a place beyond the last column holds that one's elements, for another thread to write)
                    if (k + c * stride < columns)
                        *reinterpret_cast<float4*>(x + (k + c * stride) * C::row + i) = make_float4(q[0], q[1], q[2], q[3]);
                }
            }
        }
    }
    __syncthreads();
    if (tall)
        for (int e = threadIdx.x; e < columns * s; e += kThreads) {
            const int k = e / s, i = e - k * s;
            const float v[1] = {scale * x[k * C::row + i]};
            out.store(product::One{first + k, i, true}, v, 19);
        }
    else
        for (int i = warp; i < s; i += kThreads / 32)
            for (int k = lane; k < columns; k += 32) {
                const float v[1] = {scale * x[k * C::row + i]};
                out.store(product::One{i, first + k, true}, v, 19);
            }
    ptx::cluster_arrive();   // no block leaves while another may read its part
    ptx::cluster_wait();
}

template <int S>
cudaError_t launch(const Args& a, cudaStream_t stream) {
    const int64_t s = a.m < a.n ? a.m : a.n, l = a.m < a.n ? a.n : a.m;
    auto* kernel = few_rows_kernel<S>;
    static std::atomic<uint64_t> done{0}, wide{0};
    cudaError_t e = ops::allow_shared(kernel, (int)product::kSharedMost, done);
    if (e != cudaSuccess) return e;
    int device = 0;
    if ((e = cudaGetDevice(&device)) != cudaSuccess) return e;
    const uint64_t bit = device < 64 ? (uint64_t)1 << device : 0;
    if ((wide.load(std::memory_order_acquire) & bit) == 0) {   // more blocks than the 8 of every GPU's clusters
        if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess) return e;
        wide.fetch_or(bit, std::memory_order_release);
    }
    cudaLaunchConfig_t config{};
    cudaLaunchAttribute attr[2]{};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kCluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    config.attrs = attr;
    config.numAttrs = 2;
    config.blockDim = kThreads;
    config.gridDim = kCluster;
    config.dynamicSmemBytes = few_smem<S>(l);
    config.stream = stream;
    const Input g{a.g, a.type, a.m, a.g_stride, a.n};
    const Matrix<__nv_bfloat16> out{static_cast<__nv_bfloat16*>(a.out), a.out_stride,
                                    (size_t)((a.m - 1) * a.out_stride + a.n)};
    return cudaLaunchKernelEx(&config, kernel, g, a.m > a.n ? 1 : 0, (int)s, l, a.steps, static_cast<double>(a.eps), a.scale,
                              out);
}

}  // namespace

bool few_rows(int64_t m, int64_t n) {
    const int64_t s = m < n ? m : n, l = m < n ? n : m;
    if (s > 32) return false;
    const size_t need = s <= 8 ? few_smem<8>(l) : s <= 16 ? few_smem<16>(l) : s <= 24 ? few_smem<24>(l) : few_smem<32>(l);
    return need <= product::kSharedMost;
}
cudaError_t few_rows_orthogonalize(const Args& a, cudaStream_t stream) {
    const int64_t s = a.m < a.n ? a.m : a.n;
    return s <= 8 ? launch<8>(a, stream) : s <= 16 ? launch<16>(a, stream) : s <= 24 ? launch<24>(a, stream) : launch<32>(a, stream);
}
cudaError_t few_rows_site(uint32_t* site) { return check::read_and_clear(site); }

}  // namespace orth
}  // namespace mhcpb
