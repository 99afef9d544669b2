// moe_dense_rows.cu -- the row kernels of the dense int8 operators: the
// per-token quantiser, and the gradient rows (the activation's derivative, the
// fixed-point planes of a row, and the column sums that are the gradients of
// the weight scales and the bias).
#include "moe_dense.cuh"
#include "moe_device.cuh"

namespace moe {
namespace dense {

constexpr uint32_t kInfBits = 0x7F800000u;

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

// VEC consecutive elements of a row, in one load (the caller checked the alignment).
template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T* p, float (&v)[VEC]) {
    if constexpr (VEC == 1) {
        v[0] = to_f32(*p);
    } else {
        constexpr int kBytes = VEC * (int)sizeof(T);
        static_assert(kBytes == 8 || kBytes == 16, "one load");
        T e[VEC];
        if constexpr (kBytes == 16)
            *reinterpret_cast<uint4*>(e) = *reinterpret_cast<const uint4*>(p);
        else
            *reinterpret_cast<uint2*>(e) = *reinterpret_cast<const uint2*>(p);
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = to_f32(e[i]);
    }
}

// VEC int8 codes in one store.
template <int VEC>
__device__ __forceinline__ void store_codes(int8_t* p, const int (&c)[VEC]) {
    if constexpr (VEC == 1) {
        *p = (int8_t)c[0];
    } else {
        uint32_t w[VEC / 4];
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i)
            w[i] = (uint32_t)(c[4 * i] & 255) | ((uint32_t)(c[4 * i + 1] & 255) << 8) |
                   ((uint32_t)(c[4 * i + 2] & 255) << 16) | ((uint32_t)c[4 * i + 3] << 24);
        if constexpr (VEC == 4)
            *reinterpret_cast<uint32_t*>(p) = w[0];
        else
            *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    }
}

// ---------------------------------------------------------------------------
// Per-token quantiser: one CTA a row.  d = amax / 127, q = round-half-away(x *
// (1/d)), the steps of the block quantiser over the whole row.  Rows below
// 2^-112 store zeros (so d is a normal number and 1/d finite); a row with an
// infinity or a NaN stores d = NaN, so that whatever is computed from it says so.
// Memory bound: the row is read once and kept in registers (rows up to
// kCache * VEC * blockDim elements; longer ones are read again from L2).
// ---------------------------------------------------------------------------
constexpr int kQuantCache = 4;
constexpr float kTinyRow = 1.925929944387236e-34f;  // 2^-112

template <int DT, int VEC>
__global__ void __launch_bounds__(512)
    k_quantize_token(const typename Elem<DT>::T* __restrict__ x, int64_t ldx, int cols, int8_t* __restrict__ q,
                     int64_t ldq, float* __restrict__ d) {
    __shared__ uint32_t sh[64];
    const int64_t row = blockIdx.x;
    const auto* xr = x + row * ldx;
    int8_t* qr = q + row * ldq;
    const int step = blockDim.x * VEC;
    float v[kQuantCache][VEC];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < kQuantCache; ++j) {
        const int c = (threadIdx.x + j * blockDim.x) * VEC;
        if (c < cols) {
            load_vec<typename Elem<DT>::T, VEC>(xr + c, v[j]);
#pragma unroll
            for (int i = 0; i < VEC; ++i) m = max(m, __float_as_uint(v[j][i]) & 0x7FFFFFFFu);
        }
    }
    for (int c = kQuantCache * step + threadIdx.x * VEC; c < cols; c += step) {
        float e[VEC];
        load_vec<typename Elem<DT>::T, VEC>(xr + c, e);
#pragma unroll
        for (int i = 0; i < VEC; ++i) m = max(m, __float_as_uint(e[i]) & 0x7FFFFFFFu);
    }
    m = block_max_bits(m, sh, 0);
    const float amax = __uint_as_float(m);
    const bool live = m < kInfBits && amax >= kTinyRow;
    const float scale = live ? __fdiv_rn(amax, 127.0f) : 0.0f;
    const float inv = live ? __fdiv_rn(1.0f, scale) : 0.0f;
    if (threadIdx.x == 0) d[row] = m >= kInfBits ? __uint_as_float(0x7FC00000u) : scale;
    auto code = [&](float f) {
        return live ? (int)fminf(fmaxf(roundf(__fmul_rn(f, inv)), -127.0f), 127.0f) : 0;
    };
#pragma unroll
    for (int j = 0; j < kQuantCache; ++j) {
        const int c = (threadIdx.x + j * blockDim.x) * VEC;
        if (c < cols) {
            int o[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) o[i] = code(v[j][i]);
            store_codes<VEC>(qr + c, o);
        }
    }
    for (int c = kQuantCache * step + threadIdx.x * VEC; c < cols; c += step) {
        float e[VEC];
        int o[VEC];
        load_vec<typename Elem<DT>::T, VEC>(xr + c, e);
#pragma unroll
        for (int i = 0; i < VEC; ++i) o[i] = code(e[i]);
        store_codes<VEC>(qr + c, o);
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
    int threads = ((cols + per - 1) / per + 31) / 32 * 32;
    threads = threads > 512 ? 512 : threads;
    for (int64_t r = 0; r < rows; r += 1 << 30) {  // the grid's limit
        const unsigned grid = (unsigned)(rows - r < (1 << 30) ? rows - r : (1 << 30));
        const T* xr = static_cast<const T*>(x) + r * ldx;
        if (vec)
            k_quantize_token<DT, kVec><<<grid, threads, 0, s>>>(xr, ldx, cols, q + r * ldq, ldq, d + r);
        else
            k_quantize_token<DT, 1><<<grid, threads, 0, s>>>(xr, ldx, cols, q + r * ldq, ldq, d + r);
        const cudaError_t e = cudaGetLastError();
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
};

// The values and column contributions of VEC columns of row t.
template <int MATS, int DT, int VEC>
__device__ __forceinline__ void grad_cols(const GradRowsParams& p, int64_t t, int c, float xd, float (&v)[MATS][VEC],
                                          float (&sum)[2][VEC]) {
    float dy[VEC];
    load_vec<typename Elem<DT>::T, VEC>(static_cast<const typename Elem<DT>::T*>(p.dy) + t * p.lddy + c, dy);
    int a[MATS][VEC];
#pragma unroll
    for (int m = 0; m < MATS; ++m) {
        if (MATS == 1 && !p.acc) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) a[m][i] = 0;
            continue;
        }
        const int32_t* ap = p.acc + ((int64_t)m * p.T + t) * p.N + c;
        if constexpr (VEC == 4)
            *reinterpret_cast<int4*>(a[m]) = *reinterpret_cast<const int4*>(ap);
        else
            a[m][0] = *ap;
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        const float s0 = __ldg(p.s[0] + c + i);
        if constexpr (MATS == 2) {
            const float s1 = __ldg(p.s[1] + c + i);
            const float xg = xd * (float)a[0][i], xu = xd * (float)a[1][i];
            float act, dact;
            act_value_grad(p.act, xg * s0, act, dact);
            const float dg = dy[i] * (xu * s1) * dact, du = dy[i] * act;
            v[0][i] = dg * s0;
            v[1][i] = du * s1;
            sum[0][i] += dg * xg;
            sum[1][i] += du * xu;
        } else {
            v[0][i] = dy[i] * s0;
            sum[0][i] += dy[i] * (xd * (float)a[0][i]);
            sum[1][i] += dy[i];
        }
    }
}

// The digits of VEC values into the row's planes.
template <int P, int VEC>
__device__ __forceinline__ void store_planes(const GradRowsParams& p, int64_t t, int m, int c, int mats, float pre,
                                             float inv, const float (&v)[VEC]) {
    int dig[P][VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        // the clamp holds the one value that rounding may lift past the top digit
        int r = __float2int_rn(fminf(fmaxf(v[i] * pre * inv, -kPlaneMax<P>), kPlaneMax<P>));
#pragma unroll
        for (int k = 0; k < P; ++k) {
            dig[k][i] = (int)(int8_t)r;
            r = (r - dig[k][i]) >> 8;
        }
    }
#pragma unroll
    for (int k = 0; k < P; ++k)
        store_codes<VEC>(p.planes + ((int64_t)k * p.T + t) * (mats * p.pitch) + m * p.pitch + c, dig[k]);
}

// NJ > 0: a thread owns NJ groups of VEC columns, kept in registers; NJ = 0:
// any number of columns, computed twice, with the column sums in the partials.
template <int MATS, int DT, int VEC, int NJ>
__global__ void __launch_bounds__(NJ == 4 ? 512 : 256) k_grad_rows(const GradRowsParams p) {
    constexpr int P = planes_of(DT);
    __shared__ uint32_t sh[64];
    constexpr int kN = NJ > 0 ? NJ : 1;
    float v[kN][MATS][VEC];
    float sum[kN][2][VEC];
#pragma unroll
    for (int j = 0; j < kN; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) sum[j][0][i] = sum[j][1][i] = 0.0f;
    float* part = p.partials + (int64_t)blockIdx.x * 2 * p.N;
    int buf = 0;
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, buf ^= 1) {
        const float xd = p.xd ? p.xd[t] : 0.0f;
        uint32_t m = 0;
        if constexpr (NJ > 0) {
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const int c = (threadIdx.x + j * blockDim.x) * VEC;
                if (c < p.N) {
                    grad_cols<MATS, DT, VEC>(p, t, c, xd, v[j], sum[j]);
#pragma unroll
                    for (int k = 0; k < MATS; ++k)
#pragma unroll
                        for (int i = 0; i < VEC; ++i) m = max(m, __float_as_uint(v[j][k][i]) & 0x7FFFFFFFu);
                }
            }
        } else {
            for (int c = threadIdx.x * VEC; c < p.N; c += blockDim.x * VEC) {
                const bool first = t == blockIdx.x;
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) sum[0][k][i] = first ? 0.0f : part[(int64_t)k * p.N + c + i];
                grad_cols<MATS, DT, VEC>(p, t, c, xd, v[0], sum[0]);
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) part[(int64_t)k * p.N + c + i] = sum[0][k][i];
#pragma unroll
                for (int k = 0; k < MATS; ++k)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) m = max(m, __float_as_uint(v[0][k][i]) & 0x7FFFFFFFu);
            }
        }
        m = block_max_bits(m, sh, buf);
        // A row with an infinity or a NaN has no fixed point: its scale is NaN
        // and its digits zero.  Tiny rows are lifted by 2^64 first, so that
        // D / m stays finite and m / D a normal number.
        const bool finite = m < kInfBits;
        const float mx = __uint_as_float(m);
        const float pre = mx < 8.673617379884035e-19f ? 1.8446744073709552e19f : 1.0f;  // 2^-60, 2^64
        const float mp = mx * pre;
        const bool live = finite && mp > 0.0f;
        const float inv = live ? __fdiv_rn(kPlaneMax<P>, mp) : 0.0f;
        if (threadIdx.x == 0)
            p.scale[t] = RowScale{finite ? __fdiv_rn(mp, kPlaneMax<P>) : __uint_as_float(0x7FC00000u), 1.0f / pre};
        if constexpr (NJ > 0) {
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const int c = (threadIdx.x + j * blockDim.x) * VEC;
                if (c < p.N) {
#pragma unroll
                    for (int k = 0; k < MATS; ++k) {
                        if (!live)
#pragma unroll
                            for (int i = 0; i < VEC; ++i) v[j][k][i] = 0.0f;
                        store_planes<P, VEC>(p, t, k, c, MATS, pre, inv, v[j][k]);
                    }
                }
            }
        } else {
            for (int c = threadIdx.x * VEC; c < p.N; c += blockDim.x * VEC) {
                grad_cols<MATS, DT, VEC>(p, t, c, xd, v[0], sum[0]);
#pragma unroll
                for (int k = 0; k < MATS; ++k) {
                    if (!live)
#pragma unroll
                        for (int i = 0; i < VEC; ++i) v[0][k][i] = 0.0f;
                    store_planes<P, VEC>(p, t, k, c, MATS, pre, inv, v[0][k]);
                }
            }
        }
    }
    if constexpr (NJ > 0) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int c = (threadIdx.x + j * blockDim.x) * VEC;
            if (c < p.N)
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) part[(int64_t)k * p.N + c + i] = sum[j][k][i];
        }
    }
}

// out[c] = sum over the CTAs' partial sums, 32 columns a CTA: each of its 32
// warps adds every 32nd partial in fp64, then the warps' sums are added in order.
__global__ void __launch_bounds__(1024) k_col_sums(const float* __restrict__ partials, int n_part, int N,
                                                   float* __restrict__ out0, float* __restrict__ out1) {
    __shared__ double sh[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane, k = blockIdx.y;
    float* out = k ? out1 : out0;
    if (!out) return;
    double a = 0.0;
    if (c < N)
        for (int i = warp; i < n_part; i += 32) a += (double)partials[((int64_t)i * 2 + k) * N + c];
    sh[warp][lane] = a;
    __syncthreads();
    if (warp == 0 && c < N) {
        for (int i = 1; i < 32; ++i) a += sh[i][lane];
        out[c] = (float)a;
    }
}

// CTAs of the gradient row kernel: enough to fill the SMs four times over (the
// rows of one CTA wait for its barrier; the others run meanwhile).
int grad_rows_grid(int T) {
    const int most = 4 * device_info().sm_count;
    return T < most ? T : most;
}

template <int MATS, int DT, int VEC>
static cudaError_t grad_rows(const GradRowsParams& p, int grid, cudaStream_t s) {
    const int groups = (p.N + VEC - 1) / VEC;
    const int threads = groups >= 256 ? 256 : (groups + 31) / 32 * 32;
    if (groups <= 256)
        k_grad_rows<MATS, DT, VEC, 1><<<grid, threads, 0, s>>>(p);
    else if (groups <= 512)
        k_grad_rows<MATS, DT, VEC, 2><<<grid, 256, 0, s>>>(p);
    else if (groups <= 2048)
        k_grad_rows<MATS, DT, VEC, 4><<<grid, (groups + 127) / 128 * 32, 0, s>>>(p);
    else
        k_grad_rows<MATS, DT, VEC, 0><<<grid, 256, 0, s>>>(p);
    return cudaGetLastError();
}

template <int MATS, int DT>
static cudaError_t grad_rows_dt(const GradRowsArgs& a, const GradRowsParams& p, int grid, cudaStream_t s) {
    const size_t vb = 4 * sizeof(typename Elem<DT>::T);
    const bool vec = reinterpret_cast<uintptr_t>(a.dy) % vb == 0 && a.lddy % 4 == 0 && a.N % 4 == 0 &&
                     reinterpret_cast<uintptr_t>(a.acc) % 16 == 0;
    return vec ? grad_rows<MATS, DT, 4>(p, grid, s) : grad_rows<MATS, DT, 1>(p, grid, s);
}

cudaError_t launch_grad_rows(const GradRowsArgs& a, cudaStream_t s) {
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
    const int grid = grad_rows_grid(a.T);
    cudaError_t e;
    if (a.n_mats == 2)
        e = a.dtype == MOE_F32    ? grad_rows_dt<2, MOE_F32>(a, p, grid, s)
            : a.dtype == MOE_BF16 ? grad_rows_dt<2, MOE_BF16>(a, p, grid, s)
                                  : grad_rows_dt<2, MOE_F16>(a, p, grid, s);
    else
        e = a.dtype == MOE_F32    ? grad_rows_dt<1, MOE_F32>(a, p, grid, s)
            : a.dtype == MOE_BF16 ? grad_rows_dt<1, MOE_BF16>(a, p, grid, s)
                                  : grad_rows_dt<1, MOE_F16>(a, p, grid, s);
    if (e != cudaSuccess || (!a.colsum[0] && !a.colsum[1])) return e;
    k_col_sums<<<dim3((unsigned)((a.N + 31) / 32), 2), 1024, 0, s>>>(p.partials, grid, a.N, a.colsum[0], a.colsum[1]);
    return cudaGetLastError();
}

}  // namespace dense
}  // namespace moe
