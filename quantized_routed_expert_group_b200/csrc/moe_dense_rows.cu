// moe_dense_rows.cu -- the row kernels of the dense int8 operators: the
// per-token quantiser, and the gradient rows (the activation's derivative, the
// fixed-point planes of a row, and the column sums that are the gradients of
// the weight scales and the bias).
#include "moe_dense.cuh"
#include "moe_device.cuh"
#include "moe_ptx.cuh"

namespace moe {
namespace dense {

// The largest |v| of a CTA, as bits: as integers, magnitudes order as the
// numbers do, and infinities and NaNs come above every finite value (a
// floating maximum would drop a NaN).  `buf` alternates between calls, so one
// barrier a call is enough.
__device__ __forceinline__ uint32_t block_max_bits(uint32_t m, uint32_t* sh, int buf) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    m = __reduce_max_sync(kFull, m);
    if (lane == 0) sh[buf * 32 + warp] = m;
    __syncthreads();
    return __reduce_max_sync(kFull, lane < nw ? sh[buf * 32 + lane] : 0u);
}

// ---------------------------------------------------------------------------
// Per-token quantiser: one CTA a row.  d = amax / 127, q = round-half-away(x *
// (1/d)), the steps of the block quantiser over the whole row.
// Memory bound: the row is read once and kept in registers (rows up to
// kQuantCache * VEC * blockDim elements; longer ones are read again from L2).
// ---------------------------------------------------------------------------
constexpr int kQuantCache = 8;

template <int DT, int VEC>
__global__ void __launch_bounds__(512)
    k_quantize_token(const typename Elem<DT>::T* __restrict__ x, int64_t ldx, int cols, int8_t* __restrict__ q,
                     int64_t ldq, float* __restrict__ d) {
    using T = typename Elem<DT>::T;
    __shared__ uint32_t sh[64];
    pdl_wait();
    pdl_launch_dependents();
    const int64_t row = blockIdx.x;
    const T* xr = x + row * ldx;
    int8_t* qr = q + row * ldq;
    const int step = blockDim.x * VEC;
    Raw<T, VEC> v[kQuantCache];
    uint32_t m = 0;
    auto peak = [&](const Raw<T, VEC>& r) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) m = max(m, __float_as_uint(to_f32(r.get(i))) & 0x7FFFFFFFu);
    };
#pragma unroll
    for (int j = 0; j < kQuantCache; ++j) {
        const int c = threadIdx.x * VEC + j * step;
        if (c < cols) v[j].load(xr + c);
    }
#pragma unroll
    for (int j = 0; j < kQuantCache; ++j)
        if (threadIdx.x * VEC + j * step < cols) peak(v[j]);
    for (int c = kQuantCache * step + threadIdx.x * VEC; c < cols; c += step) {
        Raw<T, VEC> e;
        e.load(xr + c);
        peak(e);
    }
    m = block_max_bits(m, sh, 0);
    const QuantScale qs = quant_scale(m);
    const float inv = qs.inv;
    if (threadIdx.x == 0) d[row] = qs.scale;
    auto put = [&](const Raw<T, VEC>& r, int c) {
        int o[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) o[i] = round_away(__fmul_rn(to_f32(r.get(i)), inv));
        store_bytes<VEC, 0>(qr + c, o, 0u);
    };
#pragma unroll
    for (int j = 0; j < kQuantCache; ++j) {
        const int c = threadIdx.x * VEC + j * step;
        if (c < cols) put(v[j], c);
    }
    for (int c = kQuantCache * step + threadIdx.x * VEC; c < cols; c += step) {
        Raw<T, VEC> e;
        e.load(xr + c);
        put(e, c);
    }
}

template <int DT>
static cudaError_t quantize_token(const void* x, int64_t rows, int cols, int64_t ldx, int8_t* q, int64_t ldq,
                                  float* d, cudaStream_t s) {
    using T = typename Elem<DT>::T;
    constexpr int kVec = 16 / (int)sizeof(T);
    const bool vec = reinterpret_cast<uintptr_t>(x) % 16 == 0 && ldx % kVec == 0 && cols % kVec == 0 &&
                     reinterpret_cast<uintptr_t>(q) % kVec == 0 && ldq % kVec == 0;
    const int per = vec ? kVec : 1;
    // many rows: small CTAs with several loads a thread in flight, so that all
    // rows of an SM are under way together; few rows: as wide as the row
    const int groups = (cols + per - 1) / per;
    const int each = rows >= 2 * device_info().sm_count ? 6 : 1;
    int threads = (groups + 32 * each - 1) / (32 * each) * 32;
    threads = threads > 512 ? 512 : threads;
    for (int64_t r = 0; r < rows; r += 1 << 30) {  // the grid's limit
        const unsigned grid = (unsigned)(rows - r < (1 << 30) ? rows - r : (1 << 30));
        const T* xr = static_cast<const T*>(x) + r * ldx;
        cudaError_t e;
        if (vec)
            e = launch_dense(k_quantize_token<DT, kVec>, grid, threads, 0, 1, s, xr, ldx, cols, q + r * ldq, ldq, d + r);
        else
            e = launch_dense(k_quantize_token<DT, 1>, grid, threads, 0, 1, s, xr, ldx, cols, q + r * ldq, ldq, d + r);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_quantize_token(const void* x, int dtype, int64_t rows, int cols, int64_t ldx, int8_t* q,
                                  int64_t ldq, float* d, cudaStream_t s) {
    if (dtype == MOE_F32) return quantize_token<MOE_F32>(x, rows, cols, ldx, q, ldq, d, s);
    if (dtype == MOE_BF16) return quantize_token<MOE_BF16>(x, rows, cols, ldx, q, ldq, d, s);
    return quantize_token<MOE_F16>(x, rows, cols, ldx, q, ldq, d, s);
}

// ---------------------------------------------------------------------------
// Gradient rows.  A CTA takes rows blockIdx.x, + gridDim.x, ...; a thread owns
// the same columns in each of them, so it keeps their column sums in registers
// and writes one partial sum a column and CTA, which k_col_sums adds in CTA
// order (a fixed grid, no atomics: the sums do not depend on timing).
//   gated:  dg = dh u act'(g), du = dh act(g);  v = dg s_g and du s_u;
//           column sums of dg xd acc_g and du xd acc_u
//   matmul: v = dy s;  column sums of dy xd acc and dy
// Both matrices' values share the row's fixed point, so that their products
// add up in one accumulator.
// ---------------------------------------------------------------------------
struct GradRowsParams {
    const void* dy;
    int64_t lddy;
    const int32_t* acc;
    const float* xd;
    const float* s[kMaxMats];
    int T, N, act;
    int8_t* planes;
    int64_t pitch;
    RowScale* scale;
    float* partials;
    bool bulk;  // rows of dy and acc start and end on 16 bytes
};
constexpr int kRowsAhead = 3;

// What VEC columns of a row read.
template <int MATS, int DT, int VEC>
struct GradIn {
    Raw<typename Elem<DT>::T, VEC> dy;
    Raw<int32_t, VEC> acc[MATS];
    __device__ __forceinline__ void load(const GradRowsParams& p, int64_t t, int c) {
        dy.load(static_cast<const typename Elem<DT>::T*>(p.dy) + t * p.lddy + c);
        if (MATS == 2 || p.acc) {
#pragma unroll
            for (int m = 0; m < MATS; ++m) acc[m].load(p.acc + ((int64_t)m * p.T + t) * p.N + c);
        }
    }
};

// Their values and column contributions.
template <int ACT, int MATS, int DT, int VEC>
__device__ __forceinline__ void grad_cols(const GradRowsParams& p, const GradIn<MATS, DT, VEC>& in,
                                          const Raw<float, VEC> (&sc)[MATS], float xd, float (&v)[MATS][VEC],
                                          float (&sum)[2][VEC]) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        const float dy = to_f32(in.dy.get(i));
        const float s0 = sc[0].get(i);
        if constexpr (MATS == 2) {
            const float s1 = sc[MATS - 1].get(i);
            const float xg = xd * (float)in.acc[0].get(i), xu = xd * (float)in.acc[MATS - 1].get(i);
            float act, dact;
            act_value_grad<ACT>(xg * s0, act, dact);
            const float dg = dy * (xu * s1) * dact, du = dy * act;
            v[0][i] = dg * s0;
            v[MATS - 1][i] = du * s1;
            sum[0][i] += dg * xg;
            sum[1][i] += du * xu;
        } else {
            v[0][i] = dy * s0;
            if (p.acc) sum[0][i] += dy * (xd * (float)in.acc[0].get(i));
            sum[1][i] += dy;
        }
    }
}

// The digits of VEC values into the row's planes.  Adding 128 to each of the
// lower digits' places turns the signed digits into the bytes of one integer,
// off by their top bit.  Two planes' integers are read off the mantissa of a
// sum with 1.5 * 2^23 (one fused multiply-add, where the conversion has a
// quarter of its rate); three planes' are too large for that.
template <int P, int VEC>
__device__ __forceinline__ void store_planes(const GradRowsParams& p, int64_t t, int m, int c, int mats, float mult,
                                             const float (&v)[VEC]) {
    int r[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i)
        r[i] = P == 2 ? __float_as_int(fmaf(v[i], mult, 12582912.0f)) + (0x8080 - 0x4B400000)
                      : __float2int_rn(v[i] * mult) + 0x808080;
    const int64_t row = mats * p.pitch;
    int8_t* o = p.planes + t * row + m * p.pitch + c;
    store_bytes<VEC, 0>(o, r, 0x80808080u);
    store_bytes<VEC, 1>(o + p.T * row, r, 0x80808080u);
    if constexpr (P == 3) store_bytes<VEC, 2>(o + 2 * p.T * row, r, 0x80808080u);
}

// The larger magnitude; a NaN stays one (a plain maximum would drop it).
__device__ __forceinline__ float max_abs(float a, float b) {
    float r;
    asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

template <int MATS, int VEC>
__device__ __forceinline__ void peak_of(const float (&v)[MATS][VEC], float& m) {
#pragma unroll
    for (int k = 0; k < MATS; ++k)
#pragma unroll
        for (int i = 0; i < VEC; ++i) m = max_abs(m, v[k][i]);
}

// The fixed point of a row from its largest magnitude: the multiplier D / m of
// its values, after a lift by 2^64 of tiny rows, so that D / m stays finite and
// m / D a normal number.  A row with an infinity or a NaN has no fixed point: its
// scale is NaN, whatever its digits.
template <int P>
__device__ __forceinline__ float fixed_point(uint32_t m, float& lift, RowScale& scale) {
    const float mx = __uint_as_float(m);
    lift = mx < 8.673617379884035e-19f ? 1.8446744073709552e19f : 1.0f;  // 2^-60, 2^64
    const float mp = mx * lift;
    scale = RowScale{m < kInfBits ? __fdiv_rn(mp, kPlaneMax<P>) : __uint_as_float(0x7FC00000u), 1.0f / lift};
    return m < kInfBits && mp > 0.0f ? __fdiv_rn(kPlaneMax<P>, mp) : 0.0f;
}

// A thread owns NJ groups of VEC columns; the next row's loads are in flight
// while a row waits for its largest value.
template <int MATS, int DT, int VEC, int NJ>
__global__ void __launch_bounds__(VEC == 1 ? 1024 : NJ == 2 ? 768 : 512) k_grad_rows(const GradRowsParams p) {
    constexpr int P = planes_of(DT);
    __shared__ uint32_t sh[64];
    pdl_wait();
    pdl_launch_dependents();
    GradIn<MATS, DT, VEC> in[NJ];
    Raw<float, VEC> sc[NJ][MATS];
    float sum[NJ][2][VEC], xd_next = 0.0f;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) sum[j][0][i] = sum[j][1][i] = 0.0f;
    auto col = [&](int j) { return (int)(threadIdx.x + j * blockDim.x) * VEC; };
    auto fetch = [&](int64_t t) {
        if (p.xd) xd_next = p.xd[t];
#pragma unroll
        for (int j = 0; j < NJ; ++j)
            if (col(j) < p.N) in[j].load(p, t, col(j));
    };
    // rows further ahead are asked into L2 (whole rows on the 16-byte grid)
    auto ahead = [&](int64_t t) {
        if (VEC == 1 || !p.bulk || threadIdx.x != 0 || t >= p.T) return;
        using T = typename Elem<DT>::T;
        bulk_prefetch_l2(static_cast<const T*>(p.dy) + t * p.lddy, p.N * (uint32_t)sizeof(T));
        if (MATS == 2 || p.acc)
#pragma unroll
            for (int m = 0; m < MATS; ++m) bulk_prefetch_l2(p.acc + ((int64_t)m * p.T + t) * p.N, p.N * 4u);
    };
    int buf = 0;
    fetch(blockIdx.x);
    for (int i = 1; i <= kRowsAhead; ++i) ahead(blockIdx.x + (int64_t)i * gridDim.x);
#pragma unroll
    for (int j = 0; j < NJ; ++j)
        if (col(j) < p.N)
#pragma unroll
            for (int m = 0; m < MATS; ++m) sc[j][m].load(p.s[m] + col(j));
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, buf ^= 1) {
        const float xd = xd_next;
        ahead(t + (int64_t)(kRowsAhead + 1) * gridDim.x);
        float v[NJ][MATS][VEC];
        float peak = 0.0f;
        with_act(MATS == 2 ? p.act : MOE_ACT_SILU, [&](auto act) {
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                if (col(j) < p.N) {
                    grad_cols<decltype(act)::value, MATS, DT, VEC>(p, in[j], sc[j], xd, v[j], sum[j]);
                    peak_of<MATS, VEC>(v[j], peak);
                }
        });
        if (t + gridDim.x < p.T) fetch(t + gridDim.x);
        float lift;
        RowScale scale;
        const float mult = fixed_point<P>(block_max_bits(__float_as_uint(fabsf(peak)), sh, buf), lift, scale);
        if (threadIdx.x == 0) p.scale[t] = scale;
        if (lift != 1.0f) {
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int k = 0; k < MATS; ++k)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) v[j][k][i] *= lift;
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j)
            if (col(j) < p.N)
#pragma unroll
                for (int k = 0; k < MATS; ++k) store_planes<P, VEC>(p, t, k, col(j), MATS, mult, v[j][k]);
    }
    float* part = p.partials + (int64_t)blockIdx.x * 2 * p.N;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
        if (col(j) < p.N)
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int i = 0; i < VEC; ++i) part[(int64_t)k * p.N + col(j) + i] = sum[j][k][i];
}

// Rows of any length: the values are computed twice and the column sums kept
// in the CTA's partials.
template <int MATS, int DT>
__global__ void __launch_bounds__(1024) k_grad_rows_long(const GradRowsParams p) {
    constexpr int P = planes_of(DT);
    __shared__ uint32_t sh[64];
    pdl_wait();
    pdl_launch_dependents();
    float* part = p.partials + (int64_t)blockIdx.x * 2 * p.N;
    auto column = [&](int64_t t, int c, float xd, float (&v)[MATS][1], float (&sum)[2][1]) {
        GradIn<MATS, DT, 1> in;
        Raw<float, 1> sc[MATS];
        in.load(p, t, c);
        for (int k = 0; k < MATS; ++k) sc[k].load(p.s[k] + c);
        with_act(MATS == 2 ? p.act : MOE_ACT_SILU,
                 [&](auto act) { grad_cols<decltype(act)::value, MATS, DT, 1>(p, in, sc, xd, v, sum); });
    };
    int buf = 0;
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, buf ^= 1) {
        const float xd = p.xd ? p.xd[t] : 0.0f;
        float peak = 0.0f;
        for (int c = threadIdx.x; c < p.N; c += blockDim.x) {
            float v[MATS][1], sum[2][1];
            for (int k = 0; k < 2; ++k) sum[k][0] = t == blockIdx.x ? 0.0f : part[(int64_t)k * p.N + c];
            column(t, c, xd, v, sum);
            peak_of<MATS, 1>(v, peak);
            for (int k = 0; k < 2; ++k) part[(int64_t)k * p.N + c] = sum[k][0];
        }
        float lift;
        RowScale scale;
        const float mult = fixed_point<P>(block_max_bits(__float_as_uint(fabsf(peak)), sh, buf), lift, scale);
        if (threadIdx.x == 0) p.scale[t] = scale;
        for (int c = threadIdx.x; c < p.N; c += blockDim.x) {
            float v[MATS][1], sum[2][1] = {{0.0f}, {0.0f}};
            column(t, c, xd, v, sum);
            for (int k = 0; k < MATS; ++k) {
                v[k][0] *= lift;
                store_planes<P, 1>(p, t, k, c, MATS, mult, v[k]);
            }
        }
    }
}

// out[c] = sum over the CTAs' partial sums, 32 columns a CTA: each of its 8
// warps adds every 8th partial in fp64, then the warps' sums are added in order.
// It runs under the gradient's product (small CTAs, no shared memory to speak
// of), whose end it waits for last, so that whatever follows finds both done.
__global__ void __launch_bounds__(256) k_col_sums(const float* __restrict__ partials, int n_part, int N,
                                                  float* __restrict__ out0, float* __restrict__ out1) {
    __shared__ double sh[8][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane, k = blockIdx.y;
    float* out = k ? out1 : out0;
    if (out) {
        double a = 0.0;
        if (c < N) {
#pragma unroll 8
            for (int i = warp; i < n_part; i += 8) a += (double)partials[((int64_t)i * 2 + k) * N + c];
        }
        sh[warp][lane] = a;
        __syncthreads();
        if (warp == 0 && c < N) {
            for (int i = 1; i < 8; ++i) a += sh[i][lane];
            out[c] = (float)a;
        }
    }
    pdl_wait();
}

cudaError_t launch_col_sums(const float* partials, int n_part, int N, float* out0, float* out1, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((N + 31) / 32), 2);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_col_sums, partials, n_part, N, out0, out1);
}

// CTAs of the gradient row kernel: a fixed grid (the column sums' order is the
// same from call to call), at most four an SM.
int grad_rows_grid(int T) {
    const int most = 4 * device_info().sm_count;
    return T < most ? T : most;
}

template <int MATS, int DT>
static cudaError_t grad_rows(const GradRowsArgs& a, GradRowsParams p, int& grid, cudaStream_t s) {
    const size_t vb = 4 * sizeof(typename Elem<DT>::T);
    bool vec = reinterpret_cast<uintptr_t>(a.dy) % vb == 0 && a.lddy % 4 == 0 && a.N % 4 == 0 &&
               reinterpret_cast<uintptr_t>(a.acc) % 16 == 0;
    for (int m = 0; m < MATS; ++m) vec = vec && reinterpret_cast<uintptr_t>(a.s[m]) % 16 == 0;
    const int esz = (int)sizeof(typename Elem<DT>::T);
    p.bulk = vec && reinterpret_cast<uintptr_t>(a.dy) % 16 == 0 && a.lddy * esz % 16 == 0 && a.N * esz % 16 == 0;
    const int groups = vec ? a.N / 4 : a.N;
    // two groups of four columns a thread where 768 threads suffice (85
    // registers each), four up to 512 threads; single columns one or four
    const int per = vec ? (groups <= 2 * 768 ? 2 : 4) : (groups <= 512 ? 1 : 4);
    const int threads = (groups + 32 * per - 1) / (32 * per) * 32;
    if (threads > (vec ? (per == 2 ? 768 : 512) : 1024)) {
        return launch_dense(k_grad_rows_long<MATS, DT>, grid, 1024, 0, 1, s, p);
    }
    const int per_sm = threads > 384 ? 1 : threads > 256 ? 2 : threads > 192 ? 3 : 4;
    if (grid > per_sm * device_info().sm_count) grid = per_sm * device_info().sm_count;
    if (vec)
        return per == 2 ? launch_dense(k_grad_rows<MATS, DT, 4, 2>, grid, threads, 0, 1, s, p)
                        : launch_dense(k_grad_rows<MATS, DT, 4, 4>, grid, threads, 0, 1, s, p);
    return per == 1 ? launch_dense(k_grad_rows<MATS, DT, 1, 1>, grid, threads, 0, 1, s, p)
                    : launch_dense(k_grad_rows<MATS, DT, 1, 4>, grid, threads, 0, 1, s, p);
}

cudaError_t launch_grad_rows(const GradRowsArgs& a, int* n_part, cudaStream_t s) {
    GradRowsParams p{};
    p.dy = a.dy;
    p.lddy = a.lddy;
    p.acc = a.acc;
    p.xd = a.xd;
    p.s[0] = a.s[0];
    p.s[1] = a.s[1];
    p.T = a.T;
    p.N = a.N;
    p.act = a.act;
    p.planes = a.planes;
    p.pitch = a.pitch;
    p.scale = a.scale;
    p.partials = a.partials;
    int grid = grad_rows_grid(a.T);
    cudaError_t e;
    if (a.n_mats == 2)
        e = a.dtype == MOE_F32    ? grad_rows<2, MOE_F32>(a, p, grid, s)
            : a.dtype == MOE_BF16 ? grad_rows<2, MOE_BF16>(a, p, grid, s)
                                  : grad_rows<2, MOE_F16>(a, p, grid, s);
    else
        e = a.dtype == MOE_F32    ? grad_rows<1, MOE_F32>(a, p, grid, s)
            : a.dtype == MOE_BF16 ? grad_rows<1, MOE_BF16>(a, p, grid, s)
                                  : grad_rows<1, MOE_F16>(a, p, grid, s);
    *n_part = grid;
    return e;
}

}  // namespace dense
}  // namespace moe
