// Embedding lookup into the residual streams, and the table's gradient.
//
//   forward    x[t, s, :] = bf16(scale E[id_t, :])  for each stream s
//   backward   dE[v, :] = scale sum over tokens t with id_t = v, streams s, of dx[t, s, :]
// An id outside [0, V) (a padding id) reads as a row of zeros and has no gradient.
//
// The backward orders the tokens by (id, t) and sums each run of equal ids in
// that order, without atomics, so the same inputs give the same bits on every
// call.  Sorting: tiles of 4096 tokens in shared memory, then, above 4096
// tokens, passes that merge 16 sorted runs at a time (an element's place is
// its place in its own run plus, for each other run, the number of smaller
// elements there; (id, t) pairs are all different, so places are too).
// Summing: the ordered tokens are cut into chunks; a block sums one chunk over
// one slab of columns.  A run inside one chunk is written at once; the pieces
// of a run that crosses chunks go to the workspace and a last kernel adds them
// in order, so that one frequent token does not leave one block with most of
// the work.  Rows without tokens are zeroed by blocks of the summing kernel.
#include "mhcs_common.cuh"
#include "mhcs_internal.h"

namespace mhcpb {
namespace ops {
namespace embed {

namespace {

using bf16 = __nv_bfloat16;
constexpr int kThreads = 128;
constexpr int kSortTile = 4096;      // tokens per sorted tile: 32 KiB of shared memory
constexpr int kSortThreads = 1024;
constexpr int kFan = 16;             // runs per merge pass
constexpr int kBatch = 32;           // ordered tokens read ahead at a time
constexpr int kZeroRows = 32;        // table rows per zeroing block
constexpr int kMaxChunks = 1024;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Ordered tokens per summing chunk: 32, or more where that would make over 1024 chunks.
int64_t chunk_tokens(int64_t T) {
    const int64_t c = (T + kMaxChunks - 1) / kMaxChunks;
    return c < kBatch ? kBatch : (c + kBatch - 1) / kBatch * kBatch;
}
int64_t chunk_count(int64_t T) { return (T + chunk_tokens(T) - 1) / chunk_tokens(T); }

size_t order_bytes(int64_t T) { return ((size_t)T * 8 + 255) / 256 * 256; }

template <typename I>
__device__ __forceinline__ int64_t id_at(const Span<const I>& ids, int64_t t, int64_t V, uint32_t site) {
    if (!ids.has((size_t)t, 1, site)) return V;
    const int64_t id = (int64_t)ids.p[t];
    return id < 0 || id >= V ? V : id;
}

// ------------------------------------------------------------ forward
template <typename E, typename I, int N>
__global__ void __launch_bounds__(kThreads) lookup_kernel(int64_t V, int64_t D, int n_streams, float scale,
                                                          Span<const E> table, Span<const I> ids,
                                                          Span<bf16> x) {
    const int64_t t = blockIdx.x;
    const int64_t id = id_at(ids, t, V, 0);
    for (int64_t c = (int64_t)threadIdx.x * N; c < D; c += kThreads * N) {
        float v[N];
        if (id < V) {
            load_at<N>(table, (size_t)(id * D + c), v, 1);
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] *= scale;
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] = 0.f;
        }
        for (int s = 0; s < n_streams; ++s) store_at<N>(x, (size_t)((t * n_streams + s) * D + c), v, 2);
    }
}

// ------------------------------------------------------------ ordering
// (id, t) as one 64-bit number; ids outside the table come last, as id V
template <typename I>
__global__ void __launch_bounds__(kSortThreads) sort_tiles_kernel(int64_t T, int64_t V, Span<const I> ids,
                                                                  Span<uint64_t> order) {
    __shared__ uint64_t s[kSortTile];
    const int64_t base = (int64_t)blockIdx.x * kSortTile;
    const int n = (int)(T - base < kSortTile ? T - base : kSortTile);
    int padded = 2;
    while (padded < n) padded *= 2;
    for (int i = threadIdx.x; i < padded; i += kSortThreads)
        s[i] = i < n ? ((uint64_t)id_at(ids, base + i, V, 3) << 32) | (uint64_t)(base + i) : ~0ull;
    __syncthreads();
    // bitonic network: the elements are all different, so no stability is needed
    for (int k = 2; k <= padded; k *= 2)
        for (int j = k / 2; j > 0; j /= 2) {
            for (int p = threadIdx.x; p < padded / 2; p += kSortThreads) {
                const int a = 2 * p - (p & (j - 1)), b = a + j;
                const uint64_t va = s[a], vb = s[b];
                if ((va > vb) == ((a & k) == 0)) {
                    s[a] = vb;
                    s[b] = va;
                }
            }
            __syncthreads();
        }
    for (int i = threadIdx.x; i < n; i += kSortThreads)
        if (order.has((size_t)(base + i), 1, 4)) order.p[base + i] = s[i];
}

__device__ __forceinline__ uint64_t order_at(const Span<const uint64_t>& o, int64_t i, uint32_t site) {
    return o.has((size_t)i, 1, site) ? o.p[i] : ~0ull;
}
__device__ __forceinline__ int64_t key_at(const Span<const uint64_t>& o, int64_t i, uint32_t site) {
    return (int64_t)(order_at(o, i, site) >> 32);
}

__global__ void __launch_bounds__(256) merge_runs_kernel(int64_t T, int64_t run, Span<const uint64_t> in,
                                                         Span<uint64_t> out) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= T) return;
    const uint64_t v = order_at(in, i, 5);
    const int64_t group = i / (run * kFan) * (run * kFan);
    int64_t place = group;
    for (int r = 0; r < kFan; ++r) {
        const int64_t lo = group + r * run;
        if (lo >= T) break;
        const int64_t hi = lo + run < T ? lo + run : T;
        if (i >= lo && i < hi) {
            place += i - lo;
            continue;
        }
        int64_t a = lo, n = hi - lo;   // the number of elements below v
        while (n > 0) {
            const int64_t half = n / 2;
            if (order_at(in, a + half, 5) < v) {
                a += half + 1;
                n -= half + 1;
            } else {
                n = half;
            }
        }
        place += a - lo;
    }
    if (out.has((size_t)place, 1, 6)) out.p[place] = v;
}

// ------------------------------------------------------------ summing
// The number of ordered tokens with an id below `key`, found by a whole warp:
// each step keeps one of 32 equal parts.
__device__ __forceinline__ int64_t lower_bound_warp(const Span<const uint64_t>& o, int64_t T, int64_t key) {
    const int lane = threadIdx.x & 31;
    int64_t lo = 0, n = T;
    while (n > 0) {
        const int64_t step = (n + 31) / 32;
        const int64_t p = lo + (lane + 1) * step - 1;
        const bool below = p < lo + n && key_at(o, p, 7) < key;
        const int64_t next = lo + (int64_t)__popc(__ballot_sync(kFullMask, below)) * step;
        const int64_t left = lo + n - next;
        n = left < step - 1 ? left : step - 1;
        lo = next;
    }
    return lo;
}

struct SumArgs {
    int64_t T, V, D, chunk, chunks, slabs;
    int n_streams;
    float scale;
    bool accumulate;
    Span<const bf16> grad_x;
    Span<const uint64_t> order;
    Span<float> table;
    Span<float> pieces;   // [chunks][2][D]: of the run that began before the chunk, and of the one that goes on after it
};

template <int N>
__device__ __forceinline__ void write_row(const SumArgs& a, int64_t key, int64_t c, const float (&acc)[N],
                                          uint32_t site) {
    float v[N];
    const size_t at = (size_t)(key * a.D + c);
    if (a.accumulate) {
        load_at<N>(a.table, at, v, site);
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = fmaf(a.scale, acc[k], v[k]);
    } else {
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = a.scale * acc[k];
    }
    store_at<N>(a.table, at, v, site);
}

template <int N>
__device__ void zero_rows(const SumArgs& a, int64_t first) {
    __shared__ uint32_t present;
    const int64_t last = first + kZeroRows < a.V ? first + kZeroRows : a.V;
    if (threadIdx.x == 0) present = 0;
    __syncthreads();
    if (threadIdx.x < 32) {
        const int64_t lo = lower_bound_warp(a.order, a.T, first), hi = lower_bound_warp(a.order, a.T, last);
        uint32_t bits = 0;
        for (int64_t i = lo + threadIdx.x; i < hi; i += 32) bits |= 1u << (key_at(a.order, i, 8) - first);
        atomicOr(&present, bits);
    }
    __syncthreads();
    const uint32_t rows = present;
    const float zero[N] = {};
    for (int64_t v = first; v < last; ++v) {
        if (rows >> (v - first) & 1u) continue;
        for (int64_t c = (int64_t)threadIdx.x * N; c < a.D; c += kThreads * N)
            store_at<N>(a.table, (size_t)(v * a.D + c), zero, 9);
    }
}

// Blocks 0 .. chunks * slabs - 1 sum; the others zero kZeroRows rows each.
template <int N>
__global__ void __launch_bounds__(kThreads) sum_runs_kernel(SumArgs a) {
    if ((int64_t)blockIdx.x >= a.chunks * a.slabs) {
        zero_rows<N>(a, ((int64_t)blockIdx.x - a.chunks * a.slabs) * kZeroRows);
        return;
    }
    __shared__ uint64_t s[kBatch + 1];
    const int64_t chunk = blockIdx.x / a.slabs;
    const int64_t c = ((int64_t)(blockIdx.x % a.slabs) * kThreads + threadIdx.x) * N;
    const int64_t begin = chunk * a.chunk;
    const int64_t end = begin + a.chunk < a.T ? begin + a.chunk : a.T;
    bool began_here = begin == 0 || key_at(a.order, begin - 1, 10) != key_at(a.order, begin, 10);
    float acc[N];
#pragma unroll
    for (int k = 0; k < N; ++k) acc[k] = 0.f;
    for (int64_t b = begin; b < end; b += kBatch) {
        __syncthreads();
        if (threadIdx.x <= kBatch) s[threadIdx.x] = b + threadIdx.x < a.T ? order_at(a.order, b + threadIdx.x, 10) : ~0ull;
        __syncthreads();
        const int m = (int)(end - b < kBatch ? end - b : kBatch);
        for (int i = 0; i < m; ++i) {
            const int64_t key = (int64_t)(s[i] >> 32), t = (int64_t)(uint32_t)s[i];
            if (key >= a.V) break;   // only ids outside the table follow
            if (c < a.D)
                for (int st = 0; st < a.n_streams; ++st) {
                    float v[N];
                    load_at<N>(a.grad_x, (size_t)((t * a.n_streams + st) * a.D + c), v, 11);
#pragma unroll
                    for (int k = 0; k < N; ++k) acc[k] += v[k];
                }
            const bool ends = (int64_t)(s[i + 1] >> 32) != key;
            if (ends || b + i + 1 == end) {
                if (c < a.D) {
                    if (began_here && ends)
                        write_row<N>(a, key, c, acc, 12);
                    else
                        store_at<N>(a.pieces, (size_t)((chunk * 2 + (began_here ? 1 : 0)) * a.D + c), acc, 13);
                }
                began_here = true;
#pragma unroll
                for (int k = 0; k < N; ++k) acc[k] = 0.f;
            }
        }
    }
}

// Block (chunk, slab): if a run begins in this chunk and goes on after it,
// adds its pieces in order.
template <int N>
__global__ void __launch_bounds__(kThreads) join_runs_kernel(SumArgs a) {
    const int64_t chunk = blockIdx.x / a.slabs;
    const int64_t c = ((int64_t)(blockIdx.x % a.slabs) * kThreads + threadIdx.x) * N;
    const int64_t begin = chunk * a.chunk;
    int64_t end = begin + a.chunk < a.T ? begin + a.chunk : a.T;
    const int64_t key = key_at(a.order, end - 1, 14);
    if (key >= a.V || end >= a.T || key_at(a.order, end, 14) != key) return;
    if (begin > 0 && key_at(a.order, begin - 1, 14) == key) return;
    if (c >= a.D) return;
    float acc[N];
    load_at<N>(a.pieces, (size_t)((chunk * 2 + 1) * a.D + c), acc, 15);
    for (int64_t q = chunk + 1; q < a.chunks; ++q) {
        float v[N];
        load_at<N>(a.pieces, (size_t)(q * 2 * a.D + c), v, 15);
#pragma unroll
        for (int k = 0; k < N; ++k) acc[k] += v[k];
        end = (q + 1) * a.chunk;
        if (end >= a.T || key_at(a.order, end, 14) != key) break;
    }
    write_row<N>(a, key, c, acc, 16);
}

template <typename E, typename I>
cudaError_t lookup_typed(const Args& a, cudaStream_t stream) {
    const Span<const E> table{static_cast<const E*>(a.table), (size_t)(a.V * a.D)};
    const Span<const I> ids{static_cast<const I*>(a.ids), (size_t)a.T};
    const Span<bf16> x{static_cast<bf16*>(a.x), (size_t)(a.T * a.n_streams * a.D)};
    if (a.D % 8 == 0 && aligned16(a.table) && aligned16(a.x))
        lookup_kernel<E, I, 8><<<(unsigned)a.T, kThreads, 0, stream>>>(a.V, a.D, a.n_streams, a.scale, table, ids, x);
    else
        lookup_kernel<E, I, 1><<<(unsigned)a.T, kThreads, 0, stream>>>(a.V, a.D, a.n_streams, a.scale, table, ids, x);
    return cudaGetLastError();
}
template <typename E>
cudaError_t lookup_ids(const Args& a, cudaStream_t stream) {
    return a.id_bytes == 8 ? lookup_typed<E, int64_t>(a, stream) : lookup_typed<E, int32_t>(a, stream);
}

template <int N>
cudaError_t sum_typed(SumArgs s, cudaStream_t stream) {
    s.slabs = (s.D + kThreads * N - 1) / (kThreads * N);
    const int64_t zeroing = s.accumulate ? 0 : (s.V + kZeroRows - 1) / kZeroRows;
    sum_runs_kernel<N><<<(unsigned)(s.chunks * s.slabs + zeroing), kThreads, 0, stream>>>(s);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || s.chunks < 2) return e;
    join_runs_kernel<N><<<(unsigned)(s.chunks * s.slabs), kThreads, 0, stream>>>(s);
    return cudaGetLastError();
}

}  // namespace

size_t workspace_bytes(int64_t T, int64_t /*V*/, int64_t D) {
    if (T == 0) return 0;
    return 2 * order_bytes(T) + (size_t)chunk_count(T) * 2 * (size_t)D * sizeof(float);
}

cudaError_t forward(const Args& a, cudaStream_t stream) {
    if (a.type == 0) return lookup_ids<bf16>(a, stream);
    if (a.type == 1) return lookup_ids<__half>(a, stream);
    return lookup_ids<float>(a, stream);
}

cudaError_t backward(const Args& a, cudaStream_t stream) {
    char* ws = static_cast<char*>(a.workspace);
    uint64_t* order = reinterpret_cast<uint64_t*>(ws);
    uint64_t* other = reinterpret_cast<uint64_t*>(ws + order_bytes(a.T));
    cudaError_t e;
    if (a.T > 0) {
        const unsigned tiles = (unsigned)((a.T + kSortTile - 1) / kSortTile);
        const Span<uint64_t> out{order, (size_t)a.T};
        if (a.id_bytes == 8)
            sort_tiles_kernel<int64_t><<<tiles, kSortThreads, 0, stream>>>(
                a.T, a.V, Span<const int64_t>{static_cast<const int64_t*>(a.ids), (size_t)a.T}, out);
        else
            sort_tiles_kernel<int32_t><<<tiles, kSortThreads, 0, stream>>>(
                a.T, a.V, Span<const int32_t>{static_cast<const int32_t*>(a.ids), (size_t)a.T}, out);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        for (int64_t run = kSortTile; run < a.T; run *= kFan) {
            merge_runs_kernel<<<(unsigned)((a.T + 255) / 256), 256, 0, stream>>>(
                a.T, run, Span<const uint64_t>{order, (size_t)a.T}, Span<uint64_t>{other, (size_t)a.T});
            if ((e = cudaGetLastError()) != cudaSuccess) return e;
            uint64_t* const swap = order;
            order = other;
            other = swap;
        }
    }
    SumArgs s{};
    s.T = a.T;
    s.V = a.V;
    s.D = a.D;
    s.chunk = chunk_tokens(a.T);
    s.chunks = chunk_count(a.T);
    s.n_streams = a.n_streams;
    s.scale = a.scale;
    s.accumulate = a.accumulate;
    s.grad_x = Span<const bf16>{static_cast<const bf16*>(a.grad_x), (size_t)(a.T * a.n_streams * a.D)};
    s.order = Span<const uint64_t>{order, (size_t)a.T};
    s.table = Span<float>{a.grad_table, (size_t)(a.V * a.D)};
    s.pieces = Span<float>{reinterpret_cast<float*>(ws + 2 * order_bytes(a.T)), (size_t)(s.chunks * 2 * a.D)};
    if (a.T == 0 && a.accumulate) return cudaSuccess;
    if (a.D % 8 == 0 && aligned16(a.grad_x) && aligned16(a.grad_table)) return sum_typed<8>(s, stream);
    return sum_typed<1>(s, stream);
}

cudaError_t setup() { return cudaSuccess; }
cudaError_t checked_site(uint32_t* site) { return check::read_and_clear(site); }

}  // namespace embed
}  // namespace ops
}  // namespace mhcpb
