// Embedding lookup into the residual streams, and the table's gradient.
//
//   forward    x[t, s, :] = bf16(scale E[id_t, :])  for each stream s
//   backward   dE[v, :] = scale sum over tokens t with id_t = v, streams s, of dx[t, s, :]
// An id outside [0, V) (a padding id) reads as a row of zeros and has no gradient.
//
// The backward orders the tokens by (id, t) and sums each run of equal ids in
// that order, without atomics, so the same inputs give the same bits on every
// call.
//
// Ordering: a token's place in its tile is the number of smaller (id, t) pairs
// there, counted by comparing it with the whole tile in shared memory; the
// comparisons of one tile are spread over many blocks.  For 4096 tokens that is
// 17 M comparisons, a few microseconds on the whole GPU (a bitonic network in
// one block took 37).  Above 4096 tokens the tiles have 1024, and passes merge
// 16 sorted runs at a time: an element's place is its place in its own run
// plus, for each other run, the number of smaller elements.  (One tile against
// tiles of 1024 and a pass, T=4096, D=5120: 59 and 64 us; sixteen tiles of 4096
// and a pass against tiles of 1024 and two, T=65536, D=1024: 200 and 177.)
// Summing: the ordered tokens are cut into chunks; a block sums one chunk over
// one slab of columns.  A run inside one chunk is written at once; the pieces
// of a run that crosses chunks go to the workspace and a last kernel adds them
// in order, so that one frequent token does not leave one block with most of
// the work.  Rows without tokens are zeroed by blocks of the summing kernel.
// Bound by HBM: grad_x is read once and the table's gradient written once.
// T=4096, four streams of 5120 into V=32768 rows: 130.5 us written (95% of the
// 6.77 TB/s of a plain copy), 59 added (63%: ordering takes 8 us and joining 6,
// launches' latencies, and the sum 38).  T=16384: 170 us added (79%); T=65536,
// D=1024: 177 (57%: ordering 50).  T=1000, one stream of 1285: 12 us, three
// launches and the trips to memory that follow one another.
#include "mhcpb.h"
#include "mhcs_common.cuh"
#include "mhcs_internal.h"
#include "mhcs_ring.cuh"
#include "mhcs_words.cuh"
#include "ptx.cuh"

namespace mhcpb {
namespace ops {
namespace embed {

namespace {

using bf16 = __nv_bfloat16;
constexpr int kThreads = 128;
constexpr int kLookupThreads = 256;
constexpr int kOneTile = 4096;       // tokens ordered in one tile
constexpr int kTile = 1024;          // tokens per tile when there are more
constexpr int kRanked = 32;          // tokens a ranking block places, 8 threads each
constexpr int kFan = 16;             // runs per merge pass
constexpr int kBatch = 32;           // ordered tokens per listing of rows
constexpr int kAhead = 8;            // rows loaded ahead of the one being added
constexpr int kMaxChunks = 4096;
constexpr int kJoinBlocks = 4 * 152;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Ordered tokens per summing chunk: T / 256 between 4 and 32, so that a short
// batch too is spread over the GPU, and more where that would make over 4096.
// (32 always: T=512, D=5120 takes 27.1 us instead of 13.3, T=4096 64.8 instead
// of 59.9.  At most 16: T=65536, D=1024 184.8 instead of 177.0.)
int64_t chunk_tokens(int64_t T) {
    int64_t c = T / 256;
    c = c < 4 ? 4 : c > kBatch ? kBatch : c;
    const int64_t least = (T + kMaxChunks - 1) / kMaxChunks;
    return c >= least ? c : (least + kBatch - 1) / kBatch * kBatch;
}
int64_t chunk_count(int64_t T) { return (T + chunk_tokens(T) - 1) / chunk_tokens(T); }

// Table rows that a zeroing warp looks after: 2048 floats, between one row and
// eight.  One row: T=4096, D=5120, V=32768 takes 130 us (four: 140), but D=64,
// V=65536 34 us (eight: 19) and T=512, D=515 41 us (three: 29).
int64_t zero_rows_of(int64_t D) {
    const int64_t rows = 2048 / D;
    return rows < 1 ? 1 : rows > 8 ? 8 : rows;
}

int64_t piece_pitch(int64_t D) { return (D + 7) / 8 * 8; }
size_t order_bytes(int64_t T) { return ((size_t)T * 8 + 255) / 256 * 256; }
size_t heads_bytes(int64_t T) { return ((size_t)(1 + chunk_count(T)) * 4 + 255) / 256 * 256; }

template <typename I>
__device__ __forceinline__ int64_t id_at(const Span<const I>& ids, int64_t t, int64_t V, uint32_t site) {
    if (!ids.has((size_t)t, 1, site)) return V;
    const int64_t id = (int64_t)ids.p[t];
    return id < 0 || id >= V ? V : id;
}

// ------------------------------------------------------------ forward
// Eight columns per thread; WORDS: rows at any address (mhcs_words.cuh), D of any size.
// The streams' rows are written from registers, so a table row is read once for
// all of them.  T=16384, D=5120, four streams, V=65536: 113 us (96%), from an FP32
// table 127 (93%); T=4096: 30.2 (93%) and 34.1 (92%).
template <typename E, typename I, bool WORDS>
__global__ void __launch_bounds__(kLookupThreads) lookup_kernel(int64_t T, int64_t V, int64_t D, VectorGrid grid,
                                                                int n_streams, float scale, Span<const E> table,
                                                                Span<const I> ids, Span<bf16> x) {
    constexpr int N = 8, kParts = N / Elem<E>::kPack, H = Elem<E>::kPack / 2;
    __shared__ uint4 parts[WORDS ? kLookupThreads / 32 * kParts * kWarpSlots : 1];
    ptx::grid_dependency_wait();
    const VectorPlace place = grid.place(T);
    const int64_t t = place.token;
    const int c = place.vector * N, lane = threadIdx.x & 31;
    if (WORDS ? t >= T : !place.valid) return;   // WORDS: whole warps of one token
    const int64_t id = id_at(ids, t, V, 0);
    float2 v[N / 2];
#pragma unroll
    for (int k = 0; k < N / 2; ++k) v[k] = pair(0.f);
    uint4* const mine = parts + (WORDS ? (threadIdx.x >> 5) * (kParts * kWarpSlots) : 0);
    if (id < V) {
        const size_t at = (size_t)(id * D + c);
        if constexpr (WORDS) {
            // FP32: two parts of 32 vectors, traded so that a lane gets eight columns
            const bool edge = edge_row<E>(id, V, D);
            const size_t first = at - lane * N;
            const int width = (int)D - c + lane * N;
            if (edge) {
#pragma unroll 1
                for (int q = 0; q < kParts; ++q)
                    copy_edge(mine + q * kWarpSlots, table.p, table.count, first + q * 32 * Elem<E>::kPack,
                                  width - q * 32 * Elem<E>::kPack, 1);
            } else {
#pragma unroll
                for (int q = 0; q < kParts; ++q)
                    copy_chunks(mine + q * kWarpSlots, table, first + q * 32 * Elem<E>::kPack,
                                width - q * 32 * Elem<E>::kPack, 1);
            }
            copies_commit();
            copies_wait<0>();
            __syncwarp();
#pragma unroll
            for (int q = 0; q < kParts; ++q)
                align_chunks<E>(mine + q * kWarpSlots, misaligned(table.p + first),
                                width - (q * 32 + lane) * Elem<E>::kPack);
            __syncwarp();
        }
#pragma unroll
        for (int q = 0; q < kParts; ++q) {
            uint4 raw = make_uint4(0u, 0u, 0u, 0u);
            if constexpr (WORDS) {
                const int vector = lane * kParts + q;
                raw = mine[vector / 32 * kWarpSlots + vector % 32];
            } else {
                const size_t piece = at + q * Elem<E>::kPack;
                if (table.has(piece, Elem<E>::kPack, 1)) raw = *reinterpret_cast<const uint4*>(table.p + piece);
            }
            float2 f[H];
            unpack<E>(raw, f);
#pragma unroll
            for (int k = 0; k < H; ++k) v[q * H + k] = mul2(f[k], pair(scale));
        }
        if (WORDS) __syncwarp();
    }
    const uint4 out = pack<bf16>(v);
    for (int s = 0; s < n_streams; ++s) {
        const size_t at = (size_t)((t * n_streams + s) * D + c);
        if constexpr (WORDS) {
            store_words(mine, x, at - lane * N, (int)D - c + lane * N, out, 2);
        } else {
            if (x.has(at, N, 2)) *reinterpret_cast<uint4*>(x.p + at) = out;
        }
    }
}

// ------------------------------------------------------------ ordering
// (id, t) as one 64-bit number; ids outside the table come last, as id V
template <typename I>
__global__ void __launch_bounds__(256) rank_kernel(int64_t T, int64_t V, int tile, Span<const I> ids,
                                                   Span<uint64_t> order, uint32_t* heads) {
    __shared__ uint4 quads[kOneTile / 4];
    uint32_t* const keys = reinterpret_cast<uint32_t*>(quads);
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    if (blockIdx.x == 0 && threadIdx.x == 0) *heads = 0;   // for the summing kernel
    const int blocks_per_tile = tile / kRanked;
    const int64_t base = (int64_t)(blockIdx.x / blocks_per_tile) * tile;
    const int n = (int)(T - base < tile ? T - base : tile), padded = (n + 31) / 32 * 32;
    constexpr int kPer = 16 / sizeof(I);   // ids per 16-byte read
    const int packed = (reinterpret_cast<uintptr_t>(ids.p) & 15u) == 0 ? n / kPer * kPer : 0;
#pragma unroll 8
    for (int k = threadIdx.x * kPer; k < packed; k += 256 * kPer)
        if (ids.has((size_t)(base + k), kPer, 3)) {
            const uint4 raw = *reinterpret_cast<const uint4*>(ids.p + base + k);
            const I* const v = reinterpret_cast<const I*>(&raw);
#pragma unroll
            for (int q = 0; q < kPer; ++q) keys[k + q] = v[q] < 0 || v[q] >= V ? (uint32_t)V : (uint32_t)v[q];
        }
    for (int k = packed + threadIdx.x; k < padded; k += 256)
        keys[k] = k < n ? (uint32_t)id_at(ids, base + k, V, 3) : 0xffffffffu;
    __syncthreads();
    const int i = (int)(blockIdx.x % blocks_per_tile) * kRanked + (threadIdx.x >> 3), part = threadIdx.x & 7;
    const uint32_t key = i < n ? keys[i] : 0u;
    int before = 0;
#pragma unroll 4
    for (int q = part; q < padded / 4; q += 8) {
        const uint4 v = quads[q];
        // an equal id counts when its token comes first
        const uint32_t bound = q < i / 4 ? key + 1 : key;
        before += (v.x < bound) + (v.y < bound) + (v.z < bound) + (v.w < bound);
    }
    if ((i / 4 & 7) == part && i < n)
        for (int k = i / 4 * 4; k < i; ++k) before += keys[k] == key;   // the token's own four
    before += __shfl_xor_sync(kFullMask, before, 1);
    before += __shfl_xor_sync(kFullMask, before, 2);
    before += __shfl_xor_sync(kFullMask, before, 4);
    if (part == 0 && i < n && order.has((size_t)(base + before), 1, 4))
        order.p[base + before] = (uint64_t)key << 32 | (uint64_t)(base + i);
}

__device__ __forceinline__ uint64_t order_at(const Span<const uint64_t>& o, int64_t i, uint32_t site) {
    return o.has((size_t)i, 1, site) ? o.p[i] : ~0ull;
}
__device__ __forceinline__ int64_t key_at(const Span<const uint64_t>& o, int64_t i, uint32_t site) {
    return (int64_t)(order_at(o, i, site) >> 32);
}

// Places kMergePlaced consecutive elements in the merge of their group of 16
// runs.  Few per block, so that a short batch occupies the GPU: 512, 256, 128, 64
// take 69, 62, 54, 55 us for the whole gradient at T=16384, D=1280, one stream,
// and 79, 70, 67, 64 at T=8192, D=2560.  Runs of 8 a pass instead of 16: 163 us
// instead of 177 at T=65536, but 61 instead of 55 at T=16384 (a pass more).
//  The runs hold consecutive tokens, so an equal id counts when its run
// comes before the element's.  The block searches kSamples ids of every run in
// shared memory, then what lies between two of them in global memory (with
// 1024 samples, reading them cost more than the two halvings they save).
constexpr int kSamples = 256;         // per run; divides every run but the last
constexpr int kSamplePitch = kSamples + 1;   // the 16 runs' searches start at the same place: in 16 banks
constexpr int kMergeThreads = 512;
constexpr int kMergePlaced = 64;
constexpr int kMergeSide = 2;         // searches of a thread side by side
constexpr size_t kMergeShared = (size_t)kFan * kSamplePitch * 4 + kMergePlaced * 8;
__global__ void __launch_bounds__(kMergeThreads) merge_runs_kernel(int64_t T, int64_t run, Span<const uint64_t> in,
                                                                   Span<uint64_t> out) {
    extern __shared__ uint32_t samples[];   // [kFan][kSamplePitch], then the places
    uint64_t* const places = reinterpret_cast<uint64_t*>(samples + kFan * kSamplePitch);
    ptx::grid_launch_dependents();
    ptx::grid_dependency_wait();
    const int64_t first = (int64_t)blockIdx.x * kMergePlaced, group = first / (run * kFan) * (run * kFan);
    const int64_t stride = run / kSamples;
#pragma unroll 8
    for (int k = threadIdx.x; k < kFan * kSamples; k += kMergeThreads) {
        const int64_t at = group + k / kSamples * run + k % kSamples * stride;
        samples[k / kSamples * kSamplePitch + k % kSamples] = at < T ? (uint32_t)key_at(in, at, 5) : 0xffffffffu;
    }
    for (int k = threadIdx.x; k < kMergePlaced; k += kMergeThreads) places[k] = 0;
    __syncthreads();
    // thread: run r of elements e, e + kMergeThreads / kFan, ...
    const int r = threadIdx.x % kFan;
    const int64_t lo = group + r * run;
    const int64_t length = lo >= T ? 0 : lo + run < T ? run : T - lo;
    const int sampled = (int)((length + stride - 1) / stride);
    constexpr int kElements = kMergeThreads / kFan;
    for (int base = threadIdx.x / kFan; base < kMergePlaced; base += kElements * kMergeSide) {
        uint32_t bound[kMergeSide];
        int a[kMergeSide], n[kMergeSide];   // samples below the bound: in [a, a + n]
        int64_t below[kMergeSide];
#pragma unroll
        for (int s = 0; s < kMergeSide; ++s) {
            const int64_t i = first + base + s * kElements;
            const uint32_t key = i < T ? (uint32_t)key_at(in, i, 5) : 0u;
            bound[s] = lo + run <= i ? key + 1 : key;
            a[s] = 0;
            n[s] = sampled;
        }
#pragma unroll 1
        for (int step = kSamples; step > 0; step >>= 1)
#pragma unroll
            for (int s = 0; s < kMergeSide; ++s)
                if (n[s] > 0) {
                    const int half = n[s] >> 1;
                    const bool less = samples[r * kSamplePitch + a[s] + half] < bound[s];
                    a[s] = less ? a[s] + half + 1 : a[s];
                    n[s] = less ? n[s] - half - 1 : half;
                }
#pragma unroll
        for (int s = 0; s < kMergeSide; ++s) {
            const int64_t i = first + base + s * kElements;
            if (i >= lo && i < lo + run) {
                below[s] = i - lo;   // its own run
            } else if (a[s] == 0) {
                below[s] = 0;
            } else {
                int64_t from = (a[s] - 1) * stride + 1, left = a[s] * stride < length ? stride - 1 : length - from;
                while (left > 0) {
                    const int64_t half = left / 2;
                    if ((uint32_t)key_at(in, lo + from + half, 5) < bound[s]) {
                        from += half + 1;
                        left -= half + 1;
                    } else {
                        left = half;
                    }
                }
                below[s] = from;
            }
        }
#pragma unroll
        for (int s = 0; s < kMergeSide; ++s) {
#pragma unroll
            for (int o = kFan / 2; o > 0; o >>= 1) below[s] += __shfl_xor_sync(kFullMask, below[s], o);
            if (r == 0) places[base + s * kElements] = (uint64_t)(group + below[s]);
        }
    }
    __syncthreads();
    for (int k = threadIdx.x; k < kMergePlaced; k += kMergeThreads)
        if (first + k < T && out.has((size_t)places[k], 1, 6)) out.p[places[k]] = order_at(in, first + k, 5);
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

// A thread's columns: eight of a row.  WORDS: rows of grad_x and of the table at
// any address (mhcs_words.cuh); the workspace's rows have a pitch of whole
// vectors.
struct SumArgs {
    int64_t T, V, D, pitch, chunk, chunks, slabs, zero_rows;   // zero_rows: of a warp
    int n_streams;
    float scale;
    bool accumulate;
    Span<const bf16> grad_x;
    Span<const uint64_t> order;
    Span<float> table;
    Span<uint32_t> heads; // count, then the chunks in which a run begins that goes on after them, in any order
    Span<float> pieces;   // [chunks][2][pitch]: of the run that began before the chunk, and of the one that goes on after it
};
constexpr int N = 8;

// Eight FP32 values: one 32-byte access where the address allows it (two of 16
// bytes, 32 apart, touch every sector twice).
__device__ __forceinline__ void load_floats(const Span<float>& s, size_t at, float (&v)[N], uint32_t site) {
    if ((reinterpret_cast<uintptr_t>(s.p + at) & 31u) == 0 && s.has(at, N, site)) {
        asm volatile("ld.global.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                     : "l"(s.p + at)
                     : "memory");
    } else {
        load_at<N>(s, at, v, site);
    }
}
__device__ __forceinline__ void store_floats(const Span<float>& s, size_t at, const float (&v)[N], uint32_t site) {
    if ((reinterpret_cast<uintptr_t>(s.p + at) & 31u) == 0) {
        if (s.has(at, N, site))
            asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(s.p + at), "f"(v[0]), "f"(v[1]),
                         "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                         : "memory");
    } else {
        store_at<N>(s, at, v, site);
    }
}
// A finished row of the gradient.  When accumulating, its old values are read
// when the row is finished and added when the next one is (or at the end), so
// that the read's latency is not waited for.  All lanes of a warp call it.
// WORDS: the lanes first trade their eight columns for columns lane, lane + 32,
// ... of the warp's 256, so that each access takes consecutive words.
template <bool WORDS>
struct RowWriter {
    int64_t key = -1;
    float sum[N], old[N];
    float* trade;         // WORDS: the warp's 256 floats of shared memory

    // the thread's columns of row `row`: at() + k * kStride for k < N, those below D
    static constexpr int kStride = WORDS ? 32 : 1;
    static __device__ __forceinline__ int64_t column(int64_t c) {
        const int lane = threadIdx.x & 31;
        return WORDS ? c - lane * N + lane : c;
    }
    __device__ __forceinline__ void store(const SumArgs& a, int64_t row, int64_t c, const float (&v)[N]) {
        const size_t at = (size_t)(row * a.D + column(c));
        if constexpr (!WORDS) {
            if (c < a.D) store_floats(a.table, at, v, 12);
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k)
                if (column(c) + 32 * k < a.D && a.table.has(at + 32 * k, 1, 12)) a.table.p[at + 32 * k] = v[k];
        }
    }
    __device__ __forceinline__ void complete(const SumArgs& a, int64_t c) {
        if (key < 0) return;
#pragma unroll
        for (int k = 0; k < N; ++k) old[k] = fmaf(a.scale, sum[k], old[k]);
        store(a, key, c, old);
        key = -1;
    }
    __device__ __forceinline__ void write(const SumArgs& a, int64_t row, int64_t c, const float (&acc)[N]) {
        float v[N];
        if constexpr (WORDS) {
            const int lane = threadIdx.x & 31;
            __syncwarp();
            float4* const mine = reinterpret_cast<float4*>(trade) + 2 * lane;
            mine[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
            mine[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
            __syncwarp();
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] = trade[lane + 32 * k];
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] = acc[k];
        }
        if (!a.accumulate) {
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] *= a.scale;
            store(a, row, c, v);
            return;
        }
        complete(a, c);
        key = row;
        const size_t at = (size_t)(row * a.D + column(c));
#pragma unroll
        for (int k = 0; k < N; ++k) sum[k] = v[k];
        if constexpr (!WORDS) {
            if (c < a.D) load_floats(a.table, at, old, 12);
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k)
                old[k] = column(c) + 32 * k < a.D && a.table.has(at + 32 * k, 1, 12) ? a.table.p[at + 32 * k] : 0.f;
        }
    }
};

// A warp zeroes the absent ones of zero_rows rows.
template <bool WORDS>
__device__ void zero_rows(const SumArgs& a, int64_t first) {
    const int lane = threadIdx.x & 31;
    const int64_t last = first + a.zero_rows < a.V ? first + a.zero_rows : a.V;
    int64_t at = -1, next = -1;   // next: the first id at or above the row, at its place
    const float zero[4] = {0.f, 0.f, 0.f, 0.f}, one[1] = {0.f};
    for (int64_t v = first; v < last; ++v) {
        if (next < v) {
            at = lower_bound_warp(a.order, a.T, v);
            next = at < a.T ? key_at(a.order, at, 8) : a.V;
        }
        if (next == v) continue;
        // whole chunks, and single elements before the first and after the last
        const size_t row = (size_t)(v * a.D);
        const int m = WORDS ? (int)(reinterpret_cast<uintptr_t>(a.table.p + row) >> 2 & 3) : 0;
        const int64_t lead = m == 0 ? 0 : 4 - m < a.D ? 4 - m : a.D, body = (a.D - lead) / 4;
        if (lane < lead) store_at<1>(a.table, row + lane, one, 9);
        for (int64_t k = lane; k < body; k += 32) store_at<4>(a.table, row + lead + 4 * k, zero, 9);
        if (lane < a.D - lead - 4 * body) store_at<1>(a.table, row + lead + 4 * body + lane, one, 9);
    }
}

// Writes the sum of the run that ends at an item, or its piece in this chunk.
template <bool WORDS>
__device__ __forceinline__ void flush(const SumArgs& a, RowWriter<WORDS>& out, int64_t chunk, int64_t key, int64_t c,
                                      bool whole, bool began, float (&acc)[N]) {
    if (whole)
        out.write(a, key, c, acc);
    else if (c < a.D)
        store_floats(a.pieces, (size_t)((chunk * 2 + (began ? 1 : 0)) * a.pitch + c), acc, 13);
    if (!whole && began && c == 0) {
        const uint32_t at = 1 + atomicAdd(a.heads.p, 1u);
        if (a.heads.has(at, 1, 17)) a.heads.p[at] = (uint32_t)chunk;
    }
#pragma unroll
    for (int k = 0; k < N; ++k) acc[k] = 0.f;
}

// Blocks 0 .. chunks * slabs - 1 sum; the warps of the others zero rows of the table.
//
// The rows of a batch of ordered tokens are listed in shared memory, NS rows
// (the streams of a token, or one row when n_streams is not 4) to an item,
// with where runs end; a thread adds its columns of one item after another.
// The rows come through per-thread copies, kAhead items of one row or
// kAhead / 2 of four ahead (twice that: T=16384, D=5120 added 185 us instead of
// 176).  Four rows to an item: T=4096, D=5120 140 us, one 152.
constexpr uint32_t kRunEnds = 1u << 31, kFlush = 1u << 30, kRowMask = kFlush - 1;   // T n_streams <= 2^28
template <bool WORDS, int NS>
__global__ void __launch_bounds__(kThreads) sum_runs_kernel(SumArgs a) {
    ptx::grid_dependency_wait();
    if ((int64_t)blockIdx.x >= a.chunks * a.slabs) {
        zero_rows<WORDS>(a, (((int64_t)blockIdx.x - a.chunks * a.slabs) * (kThreads / 32) + (threadIdx.x >> 5)) * a.zero_rows);
        return;
    }
    constexpr int kItems = NS == 1 ? kAhead : kAhead / 2;
    constexpr int P = WORDS ? kThreads / 32 * kWarpSlots : kThreads;
    __shared__ uint32_t rows[kBatch * (NS == 1 ? MHCPB_MAX_STREAMS : 1)];
    __shared__ uint32_t ids[kBatch];
    __shared__ int listed;
    __shared__ uint4 ring[kItems * NS * P];
    __shared__ float trade[WORDS ? kThreads * N : 1];
    const int per_token = NS == 1 ? a.n_streams : 1;   // items
    const int64_t chunk = blockIdx.x / a.slabs;
    const int64_t c = ((int64_t)(blockIdx.x % a.slabs) * kThreads + threadIdx.x) * N;
    const int64_t begin = chunk * a.chunk;
    const int64_t end = begin + a.chunk < a.T ? begin + a.chunk : a.T;
    bool began = begin == 0 || key_at(a.order, begin - 1, 10) != key_at(a.order, begin, 10);
    const int lane = threadIdx.x & 31;
    uint4* const mine = ring + (WORDS ? (threadIdx.x >> 5) * kWarpSlots + lane : threadIdx.x);
    RowWriter<WORDS> out;
    out.trade = trade + (WORDS ? (threadIdx.x >> 5) * 32 * N : 0);
    float acc[N];
#pragma unroll
    for (int k = 0; k < N; ++k) acc[k] = 0.f;
    for (int64_t b = begin; b < end; b += kBatch) {
        __syncthreads();
        if (threadIdx.x < kBatch) {
            const int64_t at = b + threadIdx.x;
            const bool in = at < end;
            const uint64_t v = in ? order_at(a.order, at, 10) : ~0ull;
            const int64_t key = (int64_t)(v >> 32), next = at + 1 < a.T ? key_at(a.order, at + 1, 10) : -1;
            const bool counts = in && key < a.V;   // ids outside the table come last
            const bool ends = next != key;
            const int valid = __popc(__ballot_sync(kFullMask, counts));
            if (threadIdx.x == 0) listed = valid * per_token;
            ids[threadIdx.x] = (uint32_t)key;
            if (counts)
                for (int s = 0; s < per_token; ++s) {
                    uint32_t row = (uint32_t)v * (uint32_t)a.n_streams + s;
                    if (s + 1 == per_token && (ends || at + 1 == end)) row |= kFlush | (ends ? kRunEnds : 0u);
                    rows[threadIdx.x * per_token + s] = row;
                }
        }
        __syncthreads();
        const int items = listed;
        if (items == 0) break;
        const auto row_of = [&](int item) { return (size_t)(rows[item] & kRowMask) * a.D; };
        const auto fetch = [&](int item) {
            if (item < items) {
                const uint32_t row = rows[item] & kRowMask;
                const size_t at = (size_t)row * a.D + c;
                const int width = (int)(a.D - c) + lane * N;   // from the warp's first column on
                const int64_t all = a.T * a.n_streams;
                if (WORDS && (edge_row<bf16>(row, all, a.D) || edge_row<bf16>(row + NS - 1, all, a.D))) {
#pragma unroll 1
                    for (int s = 0; s < NS; ++s)
                        copy_edge(mine + (item % kItems * NS + s) * P - lane, a.grad_x.p, a.grad_x.count,
                                  at + s * a.D - lane * N, width, 11);
                } else {
#pragma unroll
                    for (int s = 0; s < NS; ++s) {
                        uint4* const slot = mine + (item % kItems * NS + s) * P;
                        if constexpr (WORDS) {
                            copy_chunks(slot - lane, a.grad_x, at + s * a.D - lane * N, width, 11);
                        } else if (c < a.D) {
                            if (a.grad_x.has(at + s * a.D, N, 11)) copy16(slot, a.grad_x.p + at + s * a.D);
                        }
                    }
                }
            }
            copies_commit();
        };
#pragma unroll
        for (int q = 0; q < kItems; ++q) fetch(q);
        int position = 0, part = 0;   // of the item: its token in the batch, its row of the token
        for (int item = 0; item < items; ++item) {
            copies_wait<kItems - 1>();
            if (WORDS) __syncwarp();
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                uint4* const slot = mine + (item % kItems * NS + s) * P;
                if constexpr (WORDS) {
                    const bf16* const p = a.grad_x.p + row_of(item) + s * a.D + (c - lane * N);
                    align_chunks<bf16>(slot - lane, misaligned(p), (int)(a.D - c));
                }
                float2 v[4];
                unpack<bf16>(slot[0], v);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    acc[2 * k] += v[k].x;
                    acc[2 * k + 1] += v[k].y;
                }
            }
            if (WORDS) __syncwarp();
            const uint32_t row = rows[item];
            fetch(item + kItems);
            if (row & kFlush) {
                flush<WORDS>(a, out, chunk, ids[position], c, began && (row & kRunEnds), began, acc);
                began = true;
            }
            if (NS > 1 || ++part == per_token) {
                part = 0;
                ++position;
            }
        }
        copies_wait<0>();
    }
    out.complete(a, c);
}

// Adds the pieces of each run that crosses chunks, over one slab of columns at
// a time: each of kJoinParts groups of threads a part of them in order, then
// the parts in order.  A few trips to memory that follow one another: 6 to 14
// us.  2, 4, 8 parts: 182, 177, 184 us for the whole at T=65536, D=1024.
constexpr int kJoinParts = 4;
template <bool WORDS>
__global__ void __launch_bounds__(kThreads * kJoinParts) join_runs_kernel(SumArgs a) {
    __shared__ float sums[kJoinParts - 1][N][kThreads];
    __shared__ float trade[WORDS ? kThreads * N : 1];
    ptx::grid_dependency_wait();
    const int lane = threadIdx.x % kThreads, part = threadIdx.x / kThreads;
    const int64_t work = (int64_t)a.heads.p[0] * a.slabs;
    for (int64_t item = blockIdx.x; item < work; item += gridDim.x) {
        const size_t head = 1 + (size_t)(item / a.slabs);
        const int64_t chunk = a.heads.has(head, 1, 17) ? a.heads.p[head] : 0;
        const int64_t c = (item % a.slabs * kThreads + lane) * N;
        const int64_t key = key_at(a.order, (chunk + 1) * a.chunk - 1, 14);
        // piece 0 is this chunk's; then one for each next chunk that begins with the id
        int64_t count = 1;
        for (int more = kThreads * kJoinParts; more == kThreads * kJoinParts; count += more) {
            const int64_t at = (chunk + count + (int)threadIdx.x) * a.chunk;
            more = __syncthreads_count(at < a.T && key_at(a.order, at, 14) == key);
        }
        float acc[N];
#pragma unroll
        for (int k = 0; k < N; ++k) acc[k] = 0.f;
        if (c < a.D)
#pragma unroll 8
            for (int64_t q = count * part / kJoinParts; q < count * (part + 1) / kJoinParts; ++q) {
                float v[N];
                load_floats(a.pieces, (size_t)(((chunk + q) * 2 + (q == 0 ? 1 : 0)) * a.pitch + c), v, 15);
#pragma unroll
                for (int k = 0; k < N; ++k) acc[k] += v[k];
            }
        if (part > 0)   // the barriers above: the sums of the item before have been read
#pragma unroll
            for (int k = 0; k < N; ++k) sums[part - 1][k][lane] = acc[k];
        __syncthreads();
        if (part > 0) continue;
#pragma unroll
        for (int p = 0; p < kJoinParts - 1; ++p)
#pragma unroll
            for (int k = 0; k < N; ++k) acc[k] += sums[p][k][lane];
        RowWriter<WORDS> out;
        out.trade = trade + (WORDS ? (lane >> 5) * 32 * N : 0);
        out.write(a, key, c, acc);
        out.complete(a, c);
    }
}

template <typename E, typename I>
cudaError_t lookup_typed(const Args& a, cudaStream_t stream) {
    const Span<const E> table{static_cast<const E*>(a.table), (size_t)(a.V * a.D)};
    const Span<const I> ids{static_cast<const I*>(a.ids), (size_t)a.T};
    const Span<bf16> x{static_cast<bf16*>(a.x), (size_t)(a.T * a.n_streams * a.D)};
    const bool packed = a.D % 8 == 0 && aligned16(a.table) && aligned16(a.x);
    const VectorGrid grid((a.D + 7) / 8, kLookupThreads, !packed);
    return launch_early(packed ? lookup_kernel<E, I, false> : lookup_kernel<E, I, true>, dim3(grid.blocks(a.T)),
                        dim3(grid.threads), 0, stream, a.T, a.V, a.D, grid, a.n_streams, a.scale, table, ids, x);
}
template <typename E>
cudaError_t lookup_ids(const Args& a, cudaStream_t stream) {
    return a.id_bytes == 8 ? lookup_typed<E, int64_t>(a, stream) : lookup_typed<E, int32_t>(a, stream);
}

template <bool WORDS>
cudaError_t sum_typed(const SumArgs& s, cudaStream_t stream) {
    const int64_t per_block = s.zero_rows * (kThreads / 32);
    const int64_t zeroing = s.accumulate ? 0 : (s.V + per_block - 1) / per_block;
    cudaError_t e = launch_early(s.n_streams == 4 ? sum_runs_kernel<WORDS, 4> : sum_runs_kernel<WORDS, 1>,
                                 dim3((unsigned)(s.chunks * s.slabs + zeroing)), dim3(kThreads), 0, stream, s);
    if (e != cudaSuccess || s.chunks < 2) return e;
    const int64_t most = s.chunks * s.slabs < kJoinBlocks ? s.chunks * s.slabs : kJoinBlocks;
    return launch_early(join_runs_kernel<WORDS>, dim3((unsigned)most), dim3(kThreads * kJoinParts), 0, stream, s);
}

}  // namespace

size_t workspace_bytes(int64_t T, int64_t /*V*/, int64_t D) {
    if (T == 0) return 0;
    return 2 * order_bytes(T) + heads_bytes(T) + (size_t)chunk_count(T) * 2 * (size_t)piece_pitch(D) * sizeof(float);
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
        const int tile = a.T <= kOneTile ? kOneTile : kTile;
        const unsigned blocks = (unsigned)((a.T + kRanked - 1) / kRanked);
        const Span<uint64_t> out{order, (size_t)a.T};
        uint32_t* const heads = reinterpret_cast<uint32_t*>(ws + 2 * order_bytes(a.T));
        if (a.id_bytes == 8)
            e = launch_early(rank_kernel<int64_t>, dim3(blocks), dim3(256), 0, stream, a.T, a.V, tile,
                             Span<const int64_t>{static_cast<const int64_t*>(a.ids), (size_t)a.T}, out, heads);
        else
            e = launch_early(rank_kernel<int32_t>, dim3(blocks), dim3(256), 0, stream, a.T, a.V, tile,
                             Span<const int32_t>{static_cast<const int32_t*>(a.ids), (size_t)a.T}, out, heads);
        if (e != cudaSuccess) return e;
        for (int64_t run = tile; run < a.T; run *= kFan) {
            e = launch_early(merge_runs_kernel, dim3((unsigned)((a.T + kMergePlaced - 1) / kMergePlaced)), dim3(kMergeThreads),
                             kMergeShared, stream, a.T, run, Span<const uint64_t>{order, (size_t)a.T},
                             Span<uint64_t>{other, (size_t)a.T});
            if (e != cudaSuccess) return e;
            uint64_t* const swap = order;
            order = other;
            other = swap;
        }
    }
    SumArgs s{};
    s.T = a.T;
    s.V = a.V;
    s.D = a.D;
    s.pitch = piece_pitch(a.D);
    s.slabs = (a.D + kThreads * N - 1) / (kThreads * N);
    s.chunk = chunk_tokens(a.T);
    s.chunks = chunk_count(a.T);
    s.zero_rows = zero_rows_of(a.D);
    s.n_streams = a.n_streams;
    s.scale = a.scale;
    s.accumulate = a.accumulate;
    s.grad_x = Span<const bf16>{static_cast<const bf16*>(a.grad_x), (size_t)(a.T * a.n_streams * a.D)};
    s.order = Span<const uint64_t>{order, (size_t)a.T};
    s.table = Span<float>{a.grad_table, (size_t)(a.V * a.D)};
    s.heads = Span<uint32_t>{reinterpret_cast<uint32_t*>(ws + 2 * order_bytes(a.T)), (size_t)(1 + s.chunks)};
    s.pieces = Span<float>{reinterpret_cast<float*>(ws + 2 * order_bytes(a.T) + heads_bytes(a.T)), (size_t)(s.chunks * 2 * s.pitch)};
    if (a.T == 0 && a.accumulate) return cudaSuccess;
    if (a.D % 8 == 0 && aligned16(a.grad_x) && aligned16(a.grad_table)) return sum_typed<false>(s, stream);
    return sum_typed<true>(s, stream);
}

cudaError_t setup() {
    return cudaFuncSetAttribute(merge_runs_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMergeShared);
}
cudaError_t checked_site(uint32_t* site) { return check::read_and_clear(site); }

}  // namespace embed
}  // namespace ops
}  // namespace mhcpb
