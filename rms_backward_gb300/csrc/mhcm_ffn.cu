// The gated feed-forward block and its gradient (sm_103a):
//
//   g = x Wg^T,  u = x Wu^T,  a = act(g) u,  y = a Wd^T
//   da = dy Wd,  dg = da u act'(g),  du = da act(g)
//   dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x,  dWd = dy^T a
//
// Each line is made of products (mhcm_product.cuh) whose epilogues do the rest:
// the forward's first product forms g and u side by side and writes a (and g and
// u where a backward follows); the backward's first forms da and writes dg, du
// and a again from the stored g and u, so a is not kept between the two.  dx is
// one sum over both halves.  a, dg and du are operands of further products and so
// are rounded to the operands' 16-bit type (up to 64 tokens with a second number for
// what that loses, see store_both); everything else is FP32 until the output is
// stored.  Rows that are not a multiple of 8 elements long are copied to rows that are
// (the tensor maps' 16-byte rule).
#include "mhcm_ffn.cuh"
#include "mhcm_product.cuh"

namespace mhcpb {
namespace ffn {

namespace {

using product::Matrix;
using product::Shape;

// Up to 64 tokens, a, dg and du are kept as two numbers of the type, the second what the first's rounding
// lost, in row 64 further: the rounding between two products costs nothing to avoid there (the time is
// the weights'), and with few elements it would not average out.  In FP16 the second number is stored 2^11
// times: as large as the first at most, and down to steps of 2^-36, where unscaled it would be lost for a
// first number below 2^-13 (BF16 has the exponents of FP32).
constexpr int64_t kLowRows = 64;
template <class T>
constexpr float kLowScale = std::is_same<T, __half>::value ? 2048.f : 1.f;
template <class T, class Span>
__device__ __forceinline__ void store_both(const Matrix<T>& m, Span at, const float (&v)[Span::n], bool both, uint32_t site) {
    m.store(at, v, site);
    if (!both) return;
    float low[Span::n];
#pragma unroll
    for (int i = 0; i < Span::n; ++i) {
        const float high = (float)(T)v[i];
        low[i] = isfinite(high) ? (v[i] - high) * kLowScale<T> : 0.f;
    }
    at.row += kLowRows;
    m.store(at, low, site);
}

template <class T, int ACT>
struct GatedEpilogue {
    static constexpr bool kDual = true, kMirror = false, kTwice = false;
    Matrix<T> hidden, gate, up;
    bool both;
    __device__ __forceinline__ void ahead(int, int64_t, int64_t, int) const {}
    template <class Span>
    struct Read {};
    template <class Span>
    __device__ __forceinline__ Read<Span> read(int, const Span&) const {
        return {};
    }
    template <class Span>
    __device__ __forceinline__ void write(int, const Span& at, const float (&g)[Span::n], const float (&u)[Span::n],
                                          const Read<Span>&) const {
        float a[Span::n];
#pragma unroll
        for (int i = 0; i < Span::n; ++i) a[i] = activate(g[i], ACT).x * u[i];
        store_both(hidden, at, a, both, 0);
        if (gate.ptr != nullptr) {
            gate.store(at, g, 1);
            up.store(at, u, 2);
        }
    }
};

template <class T, int ACT>
struct GradEpilogue {
    static constexpr bool kDual = false, kMirror = false, kTwice = false;
    Matrix<T> gate, up, grad_gate, grad_up, hidden;   // gate and up are read
    bool both;
    // (gate and up sent for ahead: 4,096 tokens took 1% longer, 1,000 the same)
    __device__ __forceinline__ void ahead(int, int64_t, int64_t, int) const {}
    template <class Span>
    struct Read {
        product::Raw<T, Span> g, u;
    };
    template <class Span>
    __device__ __forceinline__ Read<Span> read(int, const Span& at) const {
        return {gate.raw(at, 3), up.raw(at, 4)};
    }
    template <class Span>
    __device__ __forceinline__ void write(int, const Span& at, const float (&da)[Span::n], const float (&)[Span::n],
                                          const Read<Span>& in) const {
        float g[Span::n], u[Span::n], a[Span::n];
        in.g.to(g);
        in.u.to(u);
#pragma unroll
        for (int i = 0; i < Span::n; ++i) {
            const float2 f = activate(g[i], ACT);
            a[i] = f.x * u[i];
            g[i] = da[i] * u[i] * f.y;
            u[i] = da[i] * f.x;
        }
        store_both(grad_gate, at, g, both, 5);
        store_both(grad_up, at, u, both, 6);
        hidden.store(at, a, 7);
    }
};

template <class O>
struct StoreEpilogue {
    static constexpr bool kDual = false, kMirror = false, kTwice = true;
    // (not an array: an index that is not known when it is compiled puts the arguments into local memory, and
    // every access waits for that: the block's gradient of one token, 7264 x 12360, took 406 us for 316, added 985 for 451)
    Matrix<O> out;
    O* second;   // the second group's, of the same shape
    bool accumulate;
    __device__ __forceinline__ Matrix<O> of(int group) const { return {group ? second : out.ptr, out.ld, out.elements}; }
    __device__ __forceinline__ void ahead(int group, int64_t row, int64_t col, int cols) const {
        if (accumulate) of(group).ahead(row, col, cols);
    }
    template <class Span>
    struct Read {
        product::Raw<O, Span> old;
    };
    template <class Span>
    __device__ __forceinline__ Read<Span> read(int group, const Span& at) const {
        return accumulate ? Read<Span>{of(group).raw(at, 9)} : Read<Span>{};
    }
    template <class Span>
    __device__ __forceinline__ void write(int group, const Span& at, const float (&v)[Span::n], const float (&)[Span::n],
                                          const Read<Span>& in) const {
        float r[Span::n];
        in.old.to(r);   // (zeros where nothing is added to)
#pragma unroll
        for (int i = 0; i < Span::n; ++i) r[i] = accumulate ? r[i] + v[i] : v[i];
        of(group).store(at, r, 8);
    }
};

// Matrices whose rows are copied to rows `dst_ld` (a multiple of 8) apart, in one launch: words of the
// source, shifted where a row starts in the middle of one.  1000 x 1285 and three weights of 3427 x 1285:
// 29 MB read, 13 us; bound by the words' loads (a lane's are 16 bytes apart).
constexpr int kMaxCopies = 5;
struct Copy {
    const uint16_t* src;
    uint16_t* dst;
    int64_t src_ld, dst_ld, rows, cols;
    int64_t first;   // vectors of eight before this matrix
};
struct Copies {
    Copy c[kMaxCopies];
    int count;
    int64_t vectors;
};

__global__ void __launch_bounds__(256) copy_rows_kernel(const Copies all) {
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all.vectors; i += (int64_t)gridDim.x * 256) {
        int k = 0;
        while (k + 1 < all.count && i >= all.c[k + 1].first) ++k;
        const Copy& c = all.c[k];
        const uint32_t across = (uint32_t)(c.dst_ld / 8);
        const int64_t v = i - c.first, r = v / across, col = (v - r * across) * 8;
        // the words that hold these elements, from the one with the first; the matrix itself starts at one
        const int64_t e = r * c.src_ld + col;
        const int odd = (int)(e & 1), left = (int)min((int64_t)8, c.cols - col);
        const uint16_t* p = c.src + e - odd;
        const size_t bytes = (size_t)((c.rows - 1) * c.src_ld + c.cols) * 2;
        uint32_t w[5];
#pragma unroll
        for (int q = 0; q < 5; ++q) {
            const int n = left + odd - 2 * q;   // elements from this word on
            w[q] = 0;
            if (n >= 2 && check::in(p + 2 * q, 4, c.src, bytes, 10))
                w[q] = *reinterpret_cast<const uint32_t*>(p + 2 * q);
            else if (n == 1 && check::in(p + 2 * q, 2, c.src, bytes, 10))
                w[q] = p[2 * q];
        }
        uint4 out = make_uint4(w[0], w[1], w[2], w[3]);
        if (odd)
            out = make_uint4(__funnelshift_r(w[0], w[1], 16), __funnelshift_r(w[1], w[2], 16),
                             __funnelshift_r(w[2], w[3], 16), __funnelshift_r(w[3], w[4], 16));
        uint4* q = reinterpret_cast<uint4*>(c.dst + r * c.dst_ld + col);
        if (check::in(q, 16, c.dst, (size_t)(c.rows * c.dst_ld) * 2, 11)) *q = out;
    }
}

// Parts of a workspace, each at a multiple of 256 bytes.
struct Parts {
    char* base;
    size_t used = 0;
    void* take(size_t bytes) {
        void* p = base + used;
        used += (bytes + 255) / 256 * 256;
        return p;
    }
};

size_t part(int64_t rows, int64_t cols) { return ((size_t)(rows * product::padded(cols)) * 2 + 255) / 256 * 256; }

int steps_of(int64_t k) { return (int)((k + 63) / 64); }

// Rows of a matrix over the tokens that is kept with what its rounding lost.
int64_t both_rows(int64_t T) { return T <= kLowRows ? kLowRows + T : T; }

// A factor with rows that tensor maps can read: the matrix itself, or its copy in the workspace, which
// `copies` is to make.
cudaError_t make(product::Factor& f, bool bf16, const void* p, int64_t rows, int64_t cols, int64_t ld, Parts& ws,
                 Copies& copies) {
    const int64_t wide = product::padded(cols);
    if (wide == cols) return f.make(bf16, p, rows, cols, ld);
    uint16_t* to = static_cast<uint16_t*>(ws.take((size_t)(rows * wide) * 2));
    copies.c[copies.count++] = {static_cast<const uint16_t*>(p), to, ld, wide, rows, cols, copies.vectors};
    copies.vectors += rows * (wide / 8);
    return f.make(bf16, to, rows, cols, wide);
}
cudaError_t run(const Copies& copies, cudaStream_t stream) {
    if (copies.count == 0) return cudaSuccess;
    const int64_t blocks = (copies.vectors + 255) / 256, most = 152 * 8;
    return ops::launch_early(copy_rows_kernel, dim3((unsigned)(blocks < most ? blocks : most)), dim3(256), 0, stream, copies);
}

// (a workspace's matrix: cols = ld, its padding may be written)
template <class T>
Matrix<T> matrix(const void* p, int64_t rows, int64_t cols, int64_t ld) {
    return {static_cast<T*>(const_cast<void*>(p)), ld, p == nullptr ? 0 : (size_t)((rows - 1) * ld + cols)};
}

#define MHCM_TRY(call)                          \
    do {                                        \
        const cudaError_t e_ = (call);          \
        if (e_ != cudaSuccess) return e_;       \
    } while (0)

template <class T, int ACT>
cudaError_t forward_as(const Args& a, cudaStream_t stream) {
    const int64_t T_ = a.T, D = a.D, F = a.F, Fp = product::padded(F);
    const bool bf16 = a.type == MHCPB_BF16;
    Parts ws{static_cast<char*>(a.workspace)};
    const int64_t rows = both_rows(T_);
    void* hidden = ws.take((size_t)(rows * Fp) * 2);
    Copies copies{};
    product::Factor x, wg, wu, wd, h;
    MHCM_TRY(make(x, bf16, a.x, T_, D, a.x_stride, ws, copies));
    MHCM_TRY(make(wg, bf16, a.w_gate, F, D, D, ws, copies));
    MHCM_TRY(make(wu, bf16, a.w_up, F, D, D, ws, copies));
    MHCM_TRY(make(wd, bf16, a.w_down, D, F, F, ws, copies));
    MHCM_TRY(h.make(bf16, hidden, rows, F, Fp));
    MHCM_TRY(run(copies, stream));
    Shape s{};
    s.bf16 = bf16;
    s.M = T_, s.N = F, s.k_steps = steps_of(D), s.mode = product::kSideBySide;
    const GatedEpilogue<T, ACT> gated{matrix<T>(hidden, rows, Fp, Fp), matrix<T>(a.gate, T_, F, F),
                                      matrix<T>(a.up, T_, F, F), rows > T_};
    s.narrow = !gated.gate.by_eight(F);
    MHCM_TRY(product::launch(s, gated, &x, nullptr, &wg, &wu, stream));
    s.N = D, s.k_steps = steps_of(F), s.mode = product::kPlain, s.twice = rows > T_, s.second = 1.f / kLowScale<T>;
    const StoreEpilogue<T> store{matrix<T>(a.y, T_, D, a.y_stride), nullptr, false};
    s.narrow = !store.out.by_eight(D);
    return product::launch(s, store, &h, nullptr, &wd, nullptr, stream);
}

// dWd, or dWg and dWu together or one of them: C = A^T B over the tokens
template <class O>
cudaError_t weight_gradient(const Args& a, int mode, int64_t M, int64_t N, const product::Factor* a0, const product::Factor* a1,
                            const product::Factor* b, void* out0, void* out1, cudaStream_t stream) {
    Shape s{};
    s.bf16 = a.type == MHCPB_BF16;
    s.M = M, s.N = N, s.k_steps = steps_of(a.T), s.mode = mode;
    s.a_mn = s.b_mn = 1;
    const StoreEpilogue<O> store{matrix<O>(out0, M, N, N), static_cast<O*>(out1), a.accumulate != 0};
    s.narrow = !store.out.by_eight(N);
    return product::launch(s, store, a0, a1, b, b, stream);
}

template <class T, int ACT, class O>
cudaError_t backward_as(const Args& a, cudaStream_t stream) {
    const int64_t T_ = a.T, D = a.D, F = a.F, Fp = product::padded(F);
    const bool bf16 = a.type == MHCPB_BF16;
    Parts ws{static_cast<char*>(a.workspace)};
    const int64_t rows = both_rows(T_);
    void* hidden = ws.take((size_t)(T_ * Fp) * 2);
    void *grad_gate = ws.take((size_t)(rows * Fp) * 2), *grad_up = ws.take((size_t)(rows * Fp) * 2);
    Copies copies{};
    product::Factor x, dy, wg, wu, wd, h, dg, du;
    MHCM_TRY(make(dy, bf16, a.grad_y, T_, D, a.gy_stride, ws, copies));
    MHCM_TRY(make(wd, bf16, a.w_down, D, F, F, ws, copies));
    if (a.grad_w[0] || a.grad_w[1]) MHCM_TRY(make(x, bf16, a.x, T_, D, a.x_stride, ws, copies));
    if (a.grad_x) {
        MHCM_TRY(make(wg, bf16, a.w_gate, F, D, D, ws, copies));
        MHCM_TRY(make(wu, bf16, a.w_up, F, D, D, ws, copies));
    }
    MHCM_TRY(h.make(bf16, hidden, T_, F, Fp));
    MHCM_TRY(dg.make(bf16, grad_gate, T_, F, Fp));
    MHCM_TRY(du.make(bf16, grad_up, T_, F, Fp));
    MHCM_TRY(run(copies, stream));

    Shape s{};
    s.bf16 = bf16;
    s.stall = a.stall;
    s.M = T_, s.N = F, s.k_steps = steps_of(D), s.b_mn = 1;
    const GradEpilogue<T, ACT> grad{matrix<T>(a.gate, T_, F, F), matrix<T>(a.up, T_, F, F), matrix<T>(grad_gate, rows, Fp, Fp),
                               matrix<T>(grad_up, rows, Fp, Fp), matrix<T>(hidden, T_, Fp, Fp),
                                    rows > T_};
    s.narrow = !grad.gate.by_eight(F);
    MHCM_TRY(product::launch(s, grad, &dy, nullptr, &wd, nullptr, stream));
    s.stall = 0;
    if (a.grad_x) {
        s.N = D, s.k_steps = steps_of(F), s.mode = product::kLongK;
        const StoreEpilogue<T> store{matrix<T>(a.grad_x, T_, D, a.gx_stride), nullptr, false};
        s.narrow = !store.out.by_eight(D);
        product::Factor dg_both = dg, du_both = du;
        if (rows > T_) {
            s.twice = 1, s.second = 1.f / kLowScale<T>;
            MHCM_TRY(dg_both.make(bf16, grad_gate, rows, F, Fp));
            MHCM_TRY(du_both.make(bf16, grad_up, rows, F, Fp));
        }
        MHCM_TRY(product::launch(s, store, &dg_both, &du_both, &wg, &wu, stream));
    }
    if (a.grad_w[0] && a.grad_w[1]) {
        MHCM_TRY(weight_gradient<O>(a, product::kGroups, F, D, &dg, &du, &x, a.grad_w[0], a.grad_w[1], stream));
    } else if (a.grad_w[0] || a.grad_w[1]) {
        MHCM_TRY(weight_gradient<O>(a, product::kPlain, F, D, a.grad_w[0] ? &dg : &du, nullptr, &x,
                                    a.grad_w[0] ? a.grad_w[0] : a.grad_w[1], nullptr, stream));
    }
    if (a.grad_w[2]) MHCM_TRY(weight_gradient<O>(a, product::kPlain, D, F, &dy, nullptr, &h, a.grad_w[2], nullptr, stream));
    return cudaSuccess;
}

template <class T>
cudaError_t backward_of(const Args& a, cudaStream_t stream) {
    if (a.activation == MHCPB_GELU)
        return a.grad_type == MHCPB_FP32 ? backward_as<T, MHCPB_GELU, float>(a, stream) : backward_as<T, MHCPB_GELU, T>(a, stream);
    return a.grad_type == MHCPB_FP32 ? backward_as<T, MHCPB_SILU, float>(a, stream) : backward_as<T, MHCPB_SILU, T>(a, stream);
}

}  // namespace

size_t forward_workspace_bytes(int64_t T, int64_t D, int64_t F) {
    if (few_tokens(T, D, F)) return (size_t)((T * F * 4 + 255) / 256 * 256);
    size_t n = part(both_rows(T), F);
    if (D % 8) n += part(T, D) + 2 * part(F, D);
    if (F % 8) n += part(D, F);
    return n;
}

size_t backward_workspace_bytes(int64_t T, int64_t D, int64_t F) {
    size_t n = part(T, F) + 2 * part(both_rows(T), F);
    if (D % 8) n += 2 * part(T, D) + 2 * part(F, D);
    if (F % 8) n += part(D, F);
    return n;
}

cudaError_t forward(const Args& a, cudaStream_t stream) {
    if (few_tokens(a.T, a.D, a.F)) return few_tokens_forward(a, stream);
    const bool gelu = a.activation == MHCPB_GELU;
    if (a.type == MHCPB_BF16)
        return gelu ? forward_as<__nv_bfloat16, MHCPB_GELU>(a, stream) : forward_as<__nv_bfloat16, MHCPB_SILU>(a, stream);
    return gelu ? forward_as<__half, MHCPB_GELU>(a, stream) : forward_as<__half, MHCPB_SILU>(a, stream);
}

cudaError_t backward(const Args& a, cudaStream_t stream) {
    if (a.T == 0) {   // sums over no tokens
        const size_t bytes = (size_t)(a.D * a.F) * (a.grad_type == MHCPB_FP32 ? 4 : 2);
        for (void* w : a.grad_w)
            if (w != nullptr && !a.accumulate) MHCM_TRY(cudaMemsetAsync(w, 0, bytes, stream));
        return cudaSuccess;
    }
    return a.type == MHCPB_BF16 ? backward_of<__nv_bfloat16>(a, stream) : backward_of<__half>(a, stream);
}

cudaError_t setup() {
    MHCM_TRY((product::allow<GatedEpilogue<__nv_bfloat16, MHCPB_SILU>>()));
    MHCM_TRY((product::allow<GatedEpilogue<__nv_bfloat16, MHCPB_GELU>>()));
    MHCM_TRY((product::allow<GatedEpilogue<__half, MHCPB_SILU>>()));
    MHCM_TRY((product::allow<GatedEpilogue<__half, MHCPB_GELU>>()));
    MHCM_TRY((product::allow<GradEpilogue<__nv_bfloat16, MHCPB_SILU>>()));
    MHCM_TRY((product::allow<GradEpilogue<__nv_bfloat16, MHCPB_GELU>>()));
    MHCM_TRY((product::allow<GradEpilogue<__half, MHCPB_SILU>>()));
    MHCM_TRY((product::allow<GradEpilogue<__half, MHCPB_GELU>>()));
    MHCM_TRY(product::allow<StoreEpilogue<__nv_bfloat16>>());
    MHCM_TRY(product::allow<StoreEpilogue<__half>>());
    return product::allow<StoreEpilogue<float>>();
}
cudaError_t checked_site(uint32_t* site) {
    uint32_t other = 0;
    const cudaError_t e = check::read_and_clear(site), f = few_tokens_site(&other);
    if (*site == 0) *site = other;
    return e != cudaSuccess ? e : f;
}
cudaError_t device_status(uint32_t* status, bool clear) { return product::read_status(status, clear); }

}  // namespace ffn
}  // namespace mhcpb
