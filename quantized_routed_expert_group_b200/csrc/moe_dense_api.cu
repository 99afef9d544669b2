// moe_dense_api.cu -- C ABI of the dense int8 operators (include/moe.h):
// argument checks, workspace layout and launch sequences.
#include <nvtx3/nvToolsExt.h>

#include "moe_dense.cuh"

#define MOE_API extern "C" __attribute__((visibility("default")))

namespace moe {
namespace dense {

constexpr int kMaxTokens = 1 << 28;
constexpr int kMaxContraction = 131071;  // 128 * 128 * 131071 < 2^31
constexpr int kMaxLength = 0x7FFF0000;   // kernels count columns and channels in int, up to a CTA's step past the end

static bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
static size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }
static int status_of(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ECUDA; }
static size_t elem_size(int dtype) { return dtype == MOE_F32 ? 4 : 2; }
static bool known_type(int dtype) { return dtype == MOE_F32 || dtype == MOE_BF16 || dtype == MOE_F16; }
static bool known_act(int act) { return act == MOE_ACT_SILU || act == MOE_ACT_GELU; }

struct NvtxRange {
    explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange&) = delete;
    NvtxRange& operator=(const NvtxRange&) = delete;
};

// What every product checks: sizes, strides, element types.
static int check_sizes(int T, int rows, int cols, int dtype) {
    if (T < 0 || rows <= 0 || cols <= 0) return MOE_EINVAL;
    if (!known_type(dtype)) return MOE_EINVAL;
    if (T > kMaxTokens || rows > kMaxLength || cols > kMaxLength) return MOE_EUNSUPPORTED;
    return MOE_OK;
}

static int check_weight(const uint8_t* w, int64_t ldw, const float* s, int cols) {
    if (!w || !s || !aligned(s, 4) || ldw < cols) return MOE_EINVAL;
    return MOE_OK;
}

static int check_matrix(const void* p, int dtype, int64_t ld, int cols) {
    return p && aligned(p, elem_size(dtype)) && ld >= cols ? MOE_OK : MOE_EINVAL;
}

// Copies of rows of an odd length pay from 1.5 MB on: 333 x 1000 x 777 gated (1.9
// MB) 17.9 -> 11.4 us.  Below, the device saves less than the host spends on the
// launch (300 x 1000 x 500 gated, 1.3 MB: 10.7 -> 8.5 us, and 3.5 us of the host;
// only a program that replays a graph would gain), and the few tokens that stream
// the weights gain nothing.  The sizes of workspaces know the rows' length alone:
// rows of a multiple of 16 codes at other addresses or strides are never copied.
constexpr size_t kCopyBytes = 3u << 19;

static size_t forward_room(int n_mats, int T, int rows, int cols) {
    const size_t n = pad_bytes(n_mats, T, rows, cols);
    return cols % 16 && T > kFewTokens && n >= kCopyBytes ? align256(n) : 0;
}

struct BackwardLayout {
    size_t planes, scale, partials, done, room, total;
    int64_t pitch;
};

static BackwardLayout backward_layout(int n_mats, int T, int rows, int cols, int dtype) {
    BackwardLayout L;
    L.pitch = ((int64_t)rows + 127) / 128 * 128;
    L.planes = 0;
    L.scale = align256((size_t)plane_rows(planes_of(dtype), T) * n_mats * L.pitch);
    L.partials = L.scale + align256((size_t)T * sizeof(RowScale));
    const size_t parts = n_mats == 2 ? (size_t)grad_rows_parts(T) : T / 32 < kMaxDotChunks ? T / 32 : kMaxDotChunks;
    L.done = L.partials + align256(parts * 2 * rows * sizeof(float));
    L.room = L.done + (n_mats == 2 ? 0 : align256(col_dots_tiles(rows) * sizeof(int)));
    const size_t n = pad_bytes(n_mats, 0, rows, cols);  // the weights alone
    L.total = L.room + (cols % 16 && n >= kCopyBytes ? align256(n) : 0);
    return L;
}

static int forward(GemmArgs& a, bool gated, void* workspace, size_t ws_bytes, cudaStream_t s) {
    const size_t room = forward_room(a.n_mats, a.T, a.rows, a.cols);
    if (room && workspace && ws_bytes >= room && !tma_operands(a)) {
        const int st = status_of(pad_operands(a, true, workspace, s));
        if (st) return st;
    }
    return status_of(gated ? launch_gated(a, s) : launch_matmul(a, s));
}

static int backward(int n_mats, const void* dy, int dtype, int64_t lddy, const int32_t* acc, const float* xd, int T,
                    const uint8_t* const (&w)[2], const int64_t (&ldw)[2], const float* const (&sc)[2], int rows,
                    int cols, int act, void* dx, int64_t lddx, float* sum0, float* sum1, void* workspace,
                    size_t ws_bytes, cudaStream_t s) {
    if (T == 0) {
        for (float* p : {sum0, sum1})
            if (p && cudaMemsetAsync(p, 0, (size_t)rows * sizeof(float), s) != cudaSuccess) return MOE_ECUDA;
        return MOE_OK;
    }
    if (!workspace || !aligned(workspace, 256)) return MOE_EINVAL;
    const BackwardLayout L = backward_layout(n_mats, T, rows, cols, dtype);
    if (ws_bytes < L.total) return MOE_EWORKSPACE;
    char* ws = static_cast<char*>(workspace);
    GradRowsArgs r{};
    r.dy = dy;
    r.lddy = lddy;
    r.dtype = dtype;
    r.acc = acc;
    r.xd = xd;
    r.n_mats = n_mats;
    r.T = T;
    r.N = rows;
    r.act = act;
    r.planes = reinterpret_cast<int8_t*>(ws + L.planes);
    r.pitch = L.pitch;
    r.scale = reinterpret_cast<RowScale*>(ws + L.scale);
    r.partials = reinterpret_cast<float*>(ws + L.partials);
    r.done = reinterpret_cast<int*>(ws + L.done);
    GemmArgs g{};
    for (int m = 0; m < n_mats; ++m) {
        r.s[m] = sc[m];
        g.w[m] = w[m];
        g.ldw[m] = ldw[m];
    }
    int n_part = 0;
    int st = status_of(launch_grad_rows(r, &n_part, s));
    if (st) return st;
    g.n_mats = n_mats;
    g.rows = rows;
    g.cols = cols;
    g.x = r.planes;
    g.ldx = n_mats * L.pitch;
    g.T = T;
    g.mat_pitch = L.pitch;
    g.gscale = r.scale;
    g.out = dx;
    g.ldo = lddx;
    g.dtype = dtype;
    if (L.total > L.room) st = status_of(pad_operands(g, false, ws + L.room, s));
    if (!st) st = status_of(launch_grad_matmul(g, s));
    if (!st && (sum0 || sum1))
        st = status_of(n_mats == 2 ? launch_col_sums(r.partials, n_part, rows, sum0, sum1, s)
                                   : launch_col_dots(r, sum0, sum1, s));
    return st;
}

struct FfnLayout {
    size_t xq, xd, h, hq, hd, room, total;
    int64_t ldx, ldh;
};

static FfnLayout ffn_layout(int T, int hidden, int inter) {
    FfnLayout L;
    L.ldx = ((int64_t)hidden + 15) / 16 * 16;
    L.ldh = ((int64_t)inter + 15) / 16 * 16;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t o = off;
        off = align256(off + bytes);
        return o;
    };
    L.xq = take((size_t)T * L.ldx);
    L.xd = take((size_t)T * 4);
    L.h = take((size_t)T * L.ldh * 4);
    L.hq = take((size_t)T * L.ldh);
    L.hd = take((size_t)T * 4);
    // one room for both products' odd rows
    const size_t up = forward_room(2, T, inter, hidden), down = forward_room(1, T, hidden, inter);
    L.room = take(up > down ? up : down);
    L.total = off;
    return L;
}

}  // namespace dense
}  // namespace moe

using namespace moe;
using namespace moe::dense;

MOE_API int moe_quantize_act_token(const void* x, int dtype, int64_t n_rows, int cols, int64_t ldx, int8_t* q,
                                   int64_t ldq, float* d, void* stream) {
    if (n_rows < 0 || cols <= 0 || !known_type(dtype)) return MOE_EINVAL;
    if (cols > kMaxLength) return MOE_EUNSUPPORTED;
    if (n_rows == 0) return MOE_OK;
    if (check_matrix(x, dtype, ldx, cols) || !q || ldq < cols || !d || !aligned(d, 4)) return MOE_EINVAL;
    return status_of(launch_quantize_token(x, dtype, n_rows, cols, ldx, q, ldq, d, (cudaStream_t)stream));
}

MOE_API int moe_int8_matmul(const int8_t* xq, int64_t ldx, const float* xd, int T, const uint8_t* w, int64_t ldw,
                            const float* s, int rows, int cols, const float* bias, void* out, int dtype, int64_t ldo,
                            int32_t* acc, void* workspace, size_t ws_bytes, void* stream) {
    int st = check_sizes(T, rows, cols, dtype);
    if (st) return st;
    if (cols > kMaxContraction) return MOE_EUNSUPPORTED;
    st = check_weight(w, ldw, s, cols);
    if (st) return st;
    if (!aligned(bias, 4) || !aligned(acc, 4) || !aligned(workspace, 256)) return MOE_EINVAL;
    if (T == 0) return MOE_OK;
    if (!xq || ldx < cols || !xd || !aligned(xd, 4) || check_matrix(out, dtype, ldo, rows)) return MOE_EINVAL;
    const NvtxRange range("moe/int8_matmul");
    GemmArgs a{};
    a.w[0] = w;
    a.ldw[0] = ldw;
    a.s[0] = s;
    a.n_mats = 1;
    a.rows = rows;
    a.cols = cols;
    a.x = xq;
    a.ldx = ldx;
    a.T = T;
    a.xd = xd;
    a.bias = bias;
    a.out = out;
    a.ldo = ldo;
    a.dtype = dtype;
    a.acc = acc;
    return forward(a, false, workspace, ws_bytes, (cudaStream_t)stream);
}

MOE_API int moe_gated_ffn(const int8_t* xq, int64_t ldx, const float* xd, int T, const uint8_t* w_gate, int64_t ldg,
                          const float* s_gate, const uint8_t* w_up, int64_t ldu, const float* s_up, int rows,
                          int cols, int act, void* out, int dtype, int64_t ldo, int32_t* acc, void* workspace,
                          size_t ws_bytes, void* stream) {
    int st = check_sizes(T, rows, cols, dtype);
    if (st) return st;
    if (!known_act(act)) return MOE_EINVAL;
    if (cols > kMaxContraction) return MOE_EUNSUPPORTED;
    st = check_weight(w_gate, ldg, s_gate, cols);
    if (!st) st = check_weight(w_up, ldu, s_up, cols);
    if (st) return st;
    if (!aligned(acc, 4) || !aligned(workspace, 256)) return MOE_EINVAL;
    if (T == 0) return MOE_OK;
    if (!xq || ldx < cols || !xd || !aligned(xd, 4) || check_matrix(out, dtype, ldo, rows)) return MOE_EINVAL;
    const NvtxRange range("moe/gated_ffn");
    GemmArgs a{};
    a.w[0] = w_gate;
    a.w[1] = w_up;
    a.ldw[0] = ldg;
    a.ldw[1] = ldu;
    a.s[0] = s_gate;
    a.s[1] = s_up;
    a.n_mats = 2;
    a.rows = rows;
    a.cols = cols;
    a.x = xq;
    a.ldx = ldx;
    a.T = T;
    a.xd = xd;
    a.act = act;
    a.out = out;
    a.ldo = ldo;
    a.dtype = dtype;
    a.acc = acc;
    return forward(a, true, workspace, ws_bytes, (cudaStream_t)stream);
}

MOE_API size_t moe_int8_forward_workspace_bytes(int n_mats, int T, int rows, int cols) {
    if (n_mats < 1 || n_mats > kMaxMats || T < 0 || T > kMaxTokens || rows <= 0 || rows > kMaxLength || cols <= 0 ||
        cols > kMaxContraction)
        return 0;
    return forward_room(n_mats, T, rows, cols);
}

MOE_API size_t moe_int8_backward_workspace_bytes(int n_mats, int T, int rows, int cols, int dtype) {
    if (n_mats < 1 || n_mats > kMaxMats || T < 0 || T > kMaxTokens || rows <= 0 || cols <= 0 ||
        cols > kMaxLength || (int64_t)n_mats * rows > kMaxContraction || !known_type(dtype))
        return 0;
    const size_t n = backward_layout(n_mats, T, rows, cols, dtype).total;
    return n ? n : 256;
}

MOE_API int moe_int8_matmul_backward(const void* dy, int dtype, int64_t lddy, const int32_t* acc, const float* xd,
                                     int T, const uint8_t* w, int64_t ldw, const float* s, int rows, int cols,
                                     void* dx, int64_t lddx, float* ds, float* dbias, void* workspace,
                                     size_t ws_bytes, void* stream) {
    int st = check_sizes(T, rows, cols, dtype);
    if (st) return st;
    if (rows > kMaxContraction) return MOE_EUNSUPPORTED;
    st = check_weight(w, ldw, s, cols);
    if (st) return st;
    if (!aligned(acc, 4) || !aligned(xd, 4) || !aligned(ds, 4) || !aligned(dbias, 4)) return MOE_EINVAL;
    if (T > 0 && (check_matrix(dy, dtype, lddy, rows) || check_matrix(dx, dtype, lddx, cols))) return MOE_EINVAL;
    if (T > 0 && ds && (!acc || !xd)) return MOE_EINVAL;
    const NvtxRange range("moe/int8_matmul_backward");
    return backward(1, dy, dtype, lddy, ds ? acc : nullptr, ds ? xd : nullptr, T, {w, nullptr}, {ldw, 0},
                    {s, nullptr}, rows, cols, 0, dx, lddx, ds, dbias, workspace, ws_bytes, (cudaStream_t)stream);
}

MOE_API int moe_gated_ffn_backward(const void* dh, int dtype, int64_t lddh, const int32_t* acc, const float* xd,
                                   int T, const uint8_t* w_gate, int64_t ldg, const float* s_gate,
                                   const uint8_t* w_up, int64_t ldu, const float* s_up, int rows, int cols, int act,
                                   void* dx, int64_t lddx, float* ds_gate, float* ds_up, void* workspace,
                                   size_t ws_bytes, void* stream) {
    int st = check_sizes(T, rows, cols, dtype);
    if (st) return st;
    if (!known_act(act)) return MOE_EINVAL;
    if (2 * (int64_t)rows > kMaxContraction) return MOE_EUNSUPPORTED;
    st = check_weight(w_gate, ldg, s_gate, cols);
    if (!st) st = check_weight(w_up, ldu, s_up, cols);
    if (st) return st;
    if (!aligned(acc, 4) || !aligned(xd, 4) || !aligned(ds_gate, 4) || !aligned(ds_up, 4)) return MOE_EINVAL;
    if (T > 0 && (check_matrix(dh, dtype, lddh, rows) || check_matrix(dx, dtype, lddx, cols) || !acc || !xd))
        return MOE_EINVAL;
    const NvtxRange range("moe/gated_ffn_backward");
    return backward(2, dh, dtype, lddh, acc, xd, T, {w_gate, w_up}, {ldg, ldu}, {s_gate, s_up}, rows, cols, act, dx,
                    lddx, ds_gate, ds_up, workspace, ws_bytes, (cudaStream_t)stream);
}

MOE_API size_t moe_dense_ffn_workspace_bytes(int T, int hidden, int inter) {
    if (T < 0 || T > kMaxTokens || hidden <= 0 || inter <= 0 || hidden > kMaxContraction || inter > kMaxContraction)
        return 0;
    const size_t n = ffn_layout(T, hidden, inter).total;
    return n ? n : 256;
}

MOE_API int moe_dense_ffn(const void* x, int dtype, int64_t ldx, int T, int hidden, int inter,
                          const moe_experts* experts, int act, void* out, int64_t ldo, void* workspace,
                          size_t ws_bytes, void* stream) {
    int st = check_sizes(T, inter, hidden, dtype);
    if (st) return st;
    if (!known_act(act) || !experts) return MOE_EINVAL;
    if (hidden > kMaxContraction || inter > kMaxContraction) return MOE_EUNSUPPORTED;
    st = check_weight(experts->w_gate, hidden, experts->s_gate, hidden);
    if (!st) st = check_weight(experts->w_up, hidden, experts->s_up, hidden);
    if (!st) st = check_weight(experts->w_down, inter, experts->s_down, inter);
    if (st) return st;
    if (T == 0) return MOE_OK;
    if (check_matrix(x, dtype, ldx, hidden) || check_matrix(out, dtype, ldo, hidden) || !workspace ||
        !aligned(workspace, 256))
        return MOE_EINVAL;
    const FfnLayout L = ffn_layout(T, hidden, inter);
    if (ws_bytes < L.total) return MOE_EWORKSPACE;
    char* ws = static_cast<char*>(workspace);
    int8_t* xq = reinterpret_cast<int8_t*>(ws + L.xq);
    float* xd = reinterpret_cast<float*>(ws + L.xd);
    float* h = reinterpret_cast<float*>(ws + L.h);
    int8_t* hq = reinterpret_cast<int8_t*>(ws + L.hq);
    float* hd = reinterpret_cast<float*>(ws + L.hd);
    const NvtxRange range("moe/dense_ffn");
    GemmArgs a{}, b{};
    a.w[0] = experts->w_gate;
    a.w[1] = experts->w_up;
    a.s[0] = experts->s_gate;
    a.s[1] = experts->s_up;
    a.ldw[0] = a.ldw[1] = a.cols = hidden;
    a.n_mats = 2;
    a.rows = inter;
    a.ldx = ldx;
    a.T = T;
    a.act = act;
    a.out = h;
    a.ldo = L.ldh;
    a.dtype = MOE_F32;
    b.w[0] = experts->w_down;
    b.s[0] = experts->s_down;
    b.ldw[0] = b.cols = inter;
    b.n_mats = 1;
    b.rows = hidden;
    b.ldx = L.ldh;
    b.T = T;
    b.out = out;
    b.ldo = ldo;
    b.dtype = dtype;
    if (few_quantised_fits(a, x, dtype) && few_quantised_fits(b, h, MOE_F32)) {
        // a few tokens: each product quantises its own input, two launches
        st = status_of(launch_gated_quantised(a, x, dtype, (cudaStream_t)stream));
        if (!st) st = status_of(launch_matmul_quantised(b, h, (cudaStream_t)stream));
        return st;
    }
    st = moe_quantize_act_token(x, dtype, T, hidden, ldx, xq, L.ldx, xd, stream);
    if (!st)
        st = moe_gated_ffn(xq, L.ldx, xd, T, experts->w_gate, hidden, experts->s_gate, experts->w_up, hidden,
                           experts->s_up, inter, hidden, act, h, MOE_F32, L.ldh, nullptr, ws + L.room, L.total - L.room,
                           stream);
    if (!st) st = moe_quantize_act_token(h, MOE_F32, T, inter, L.ldh, hq, L.ldh, hd, stream);
    if (!st)
        st = moe_int8_matmul(hq, L.ldh, hd, T, experts->w_down, inter, experts->s_down, hidden, inter, nullptr, out,
                             dtype, ldo, nullptr, ws + L.room, L.total - L.room, stream);
    return st;
}

MOE_API int moe_dense_device_error(void* stream, int32_t* code) {
    if (!code) return MOE_EINVAL;
    if (read_device_error((cudaStream_t)stream, code) != cudaSuccess) return MOE_ECUDA;
    return *code == 0 ? MOE_OK : MOE_EDEVICE;
}
