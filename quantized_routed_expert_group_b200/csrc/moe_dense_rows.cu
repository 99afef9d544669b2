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

// The larger magnitude; a NaN stays one (a plain maximum would drop it).
__device__ __forceinline__ float max_abs(float a, float b) {
    float r;
    asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// ---------------------------------------------------------------------------
// Per-token quantiser: one CTA a row.  d = amax / 127, q = round-half-away(x *
// (1/d)), the steps of the block quantiser over the whole row.
// Memory bound: the row is read once and kept in registers (rows up to
// kQuantCache * VEC * blockDim elements; longer ones are read again from L2).
// 4096 x 6144: bf16 13.1 us, fp32 21.9 us, 5.8 TB/s; one row 2 us.
// ---------------------------------------------------------------------------
constexpr int kQuantCache = 4;

template <int DT, int VEC>
__global__ void __launch_bounds__(512)
    k_quantize_token(const typename Elem<DT>::T* x, int64_t ldx, int cols, int8_t* q,
                     int64_t ldq, float* d) {
    using T = typename Elem<DT>::T;
    __shared__ uint32_t sh[64];
    pdl_wait();
    pdl_launch_dependents();
    const int64_t row = blockIdx.x;
    const T* xr = x + row * ldx;
    int8_t* qr = q + row * ldq;
    const int step = blockDim.x * VEC;
    Raw<T, VEC> v[kQuantCache];
    float pk = 0.0f;
    auto peak = [&](const Raw<T, VEC>& r) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) pk = max_abs(pk, to_f32(r.get(i)));
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
    const QuantScale qs = quant_scale(block_max_bits(__float_as_uint(fabsf(pk)), sh, 0));
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
    const int each = rows >= 2 * device_info().sm_count ? kQuantCache : 1;
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
// Gradient rows of one matrix: v = dy s.  One CTA a row, like the quantiser.
// (The column sums do not need the row's fixed point: k_col_dots forms them
// under the gradient's product, which leaves the memory idle.)
//
// Gradient rows of the gated block: dg = dh u act'(g), du = dh act(g); v = dg s_g
// and du s_u; column sums of dg xd acc_g and du xd acc_u, for which the
// derivative would have to be formed again.  A CTA takes rows blockIdx.x,
// + gridDim.x, ...; a thread owns the same columns in each of them, so it keeps
// their column sums in registers and writes a partial sum a column for every
// kSumRows of its rows, which k_col_sums adds in fp64 in a fixed order (a fixed
// grid, no atomics: the sums do not depend on timing, and their error is that of
// kSumRows additions whatever T is).  Both matrices' values share the row's fixed point, so that
// their products add up in one accumulator.
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
    float* partials;  // gated: [slots][grid][2][N]
    int slots;        // gated: partial sums that a CTA writes
    int* done;  // one matrix: counters of k_col_dots, zeroed here
    bool bulk;  // rows of dy and acc start and end on 16 bytes
};
constexpr int kRowsAhead = 3;
constexpr int kSumRows = 32;  // rows of a column sum in fp32
constexpr int kMats = 2;  // gate and up

// What VEC columns of a row read.
template <int DT, int VEC>
struct GradIn {
    Raw<typename Elem<DT>::T, VEC> dy;
    Raw<int32_t, VEC> acc[kMats];
    __device__ __forceinline__ void load(const GradRowsParams& p, int64_t t, int c) {
        dy.load(static_cast<const typename Elem<DT>::T*>(p.dy) + t * p.lddy + c);
#pragma unroll
        for (int m = 0; m < kMats; ++m) acc[m].load(p.acc + ((int64_t)m * p.T + t) * p.N + c);
    }
};

// Their values and column contributions.
template <int ACT, int DT, int VEC>
__device__ __forceinline__ void grad_cols(const GradRowsParams& p, const GradIn<DT, VEC>& in,
                                          const Raw<float, VEC> (&sc)[kMats], float xd, float (&v)[kMats][VEC],
                                          float (&sum)[2][VEC]) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        const float dy = to_f32(in.dy.get(i));
        const float s0 = sc[0].get(i), s1 = sc[1].get(i);
        const float xg = xd * (float)in.acc[0].get(i), xu = xd * (float)in.acc[1].get(i);
        float act, dact;
        act_value_grad<ACT>(xg * s0, act, dact);
        const float dg = dy * (xu * s1) * dact, du = dy * act;
        v[0][i] = dg * s0;
        v[1][i] = du * s1;
        sum[0][i] += dg * xg;
        sum[1][i] += du * xu;
    }
}

// The digits of VEC values into the row's planes.  Adding 128 to each of the
// lower digits' places turns the signed digits into the bytes of one integer,
// off by their top bit (four planes: modulo 2^32).
template <int P, int VEC>
__device__ __forceinline__ void store_planes(const GradRowsParams& p, int64_t t, int m, int c, int mats, float mult,
                                             const float (&v)[VEC]) {
    int r[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i)
        r[i] = (int)((uint32_t)__float2int_rn(v[i] * mult) + (P == 3 ? 0x808080u : 0x80808080u));
    const int64_t row = mats * p.pitch;
    int8_t* o = p.planes + plane_row<P>(t) * row + m * p.pitch + c;
    store_bytes<VEC, 0>(o, r, 0x80808080u);
    store_bytes<VEC, 1>(o + kPlaneGroup * row, r, 0x80808080u);
    store_bytes<VEC, 2>(o + 2 * kPlaneGroup * row, r, 0x80808080u);
    if constexpr (P == 4) store_bytes<VEC, 3>(o + 3 * kPlaneGroup * row, r, 0x80808080u);
}

template <int VEC>
__device__ __forceinline__ void peak_of(const float (&v)[kMats][VEC], float& m) {
#pragma unroll
    for (int k = 0; k < kMats; ++k)
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

// Rows of one matrix: v = dy s, read once and kept in registers until the row's
// largest value is known.  Bound by latency and issue (52 % of the issue slots at
// 2048 x 6144 bf16, 16.3 us with the rows in HBM: 25 MB read at 19 % of the
// memory's rate; the planes stay in L2 for the product).  The fp32 form spills 80
// bytes a thread.
constexpr int kRowCache = 6;

template <int DT, int VEC>
__global__ void __launch_bounds__(512, 2) k_grad_rows(const GradRowsParams p) {
    using T = typename Elem<DT>::T;
    constexpr int P = planes_of(DT);
    __shared__ uint32_t sh[64];
    pdl_wait();
    pdl_launch_dependents();
    const int64_t t = blockIdx.x;
    if (t == 0)
        for (int i = threadIdx.x; i < (p.N + 31) / 32; i += blockDim.x) p.done[i] = 0;
    const T* dy = static_cast<const T*>(p.dy) + t * p.lddy;
    const int step = blockDim.x * VEC;
    auto value = [&](int c, float (&v)[VEC]) {
        Raw<T, VEC> d;
        Raw<float, VEC> s;
        d.load(dy + c);
        s.load(p.s[0] + c);
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = to_f32(d.get(i)) * s.get(i);
    };
    float v[kRowCache][VEC], peak = 0.0f;
#pragma unroll
    for (int j = 0; j < kRowCache; ++j) {
        const int c = threadIdx.x * VEC + j * step;
        if (c < p.N) value(c, v[j]);
    }
#pragma unroll
    for (int j = 0; j < kRowCache; ++j)
        if (threadIdx.x * VEC + j * step < p.N)
#pragma unroll
            for (int i = 0; i < VEC; ++i) peak = max_abs(peak, v[j][i]);
    for (int c = threadIdx.x * VEC + kRowCache * step; c < p.N; c += step) {
        float w[VEC];
        value(c, w);
#pragma unroll
        for (int i = 0; i < VEC; ++i) peak = max_abs(peak, w[i]);
    }
    float lift;
    RowScale scale;
    const float mult = fixed_point<P>(block_max_bits(__float_as_uint(fabsf(peak)), sh, 0), lift, scale);
    if (threadIdx.x == 0) p.scale[t] = scale;
    auto put = [&](int c, float (&w)[VEC]) {
        if (lift != 1.0f) {
#pragma unroll
            for (int i = 0; i < VEC; ++i) w[i] *= lift;
        }
        store_planes<P, VEC>(p, t, 0, c, 1, mult, w);
    };
#pragma unroll
    for (int j = 0; j < kRowCache; ++j) {
        const int c = threadIdx.x * VEC + j * step;
        if (c < p.N) put(c, v[j]);
    }
    for (int c = threadIdx.x * VEC + kRowCache * step; c < p.N; c += step) {
        float w[VEC];
        value(c, w);
        put(c, w);
    }
}

// ds[c] = sum_t dy xd acc, dbias[c] = sum_t dy.  A CTA takes 32 VEC columns of a
// chunk of the rows, a row for each of its warps at a time, four of them under
// way; its sums go to the partials, and the CTA that finishes a column tile last
// joins the chunks' in their order (so the result does not depend on which one
// that is; k_grad_rows zeroed the tiles' counters).  A warp adds kSumRows rows in
// fp32 and those sums in fp64, as are the warps' and the chunks', so that the error
// is that of 32 additions whatever T is (one fp32 sum a thread: 1e-4 at 60,000
// tokens of one sign).
// It runs under the gradient's product, which leaves the memory idle: 256
// threads and 8 KB of shared memory fit beside a pair's CTA.  It waits for that
// product's end last, so that whatever follows finds both done.
constexpr int kDotsWarps = 8;

struct ColDotsParams {
    const void* dy;
    int64_t lddy;
    const int32_t* acc;  // null: no ds
    const float* xd;
    int T, N, chunks;
    float* partials;  // [chunks][2][N]
    int* done;        // [tiles]
    float* ds;
    float* dbias;
};

template <int DT, int VEC>
__global__ void __launch_bounds__(32 * kDotsWarps, 4) k_col_dots(const ColDotsParams p) {
    using T = typename Elem<DT>::T;
    __shared__ double sh[kDotsWarps][32 * VEC];
    __shared__ int last;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tile = blockIdx.x / p.chunks, chunk = blockIdx.x % p.chunks;
    const int c = tile * 32 * VEC + lane * VEC;
    const int64_t r1 = (int64_t)p.T * (chunk + 1) / p.chunks;
    // fp64 sums of ds wait in shared memory (a slot for each thread and column),
    // those of dbias in registers: with both in registers a CTA takes 80 a thread
    // and finds no room beside a pair (157 against 108 us of the product's training
    // step, 2048 x 2048 x 6144)
    double total[VEC] = {};
#pragma unroll
    for (int i = 0; i < VEC; ++i) sh[warp][32 * i + lane] = 0.0;
    if (c < p.N) {
        const T* dy = static_cast<const T*>(p.dy) + c;
        const int32_t* acc = p.acc + c;
        float sum[2][VEC] = {};
        auto flush = [&] {
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                sh[warp][32 * i + lane] += (double)sum[0][i];
                total[i] += (double)sum[1][i];
                sum[0][i] = sum[1][i] = 0.0f;
            }
        };
        int held = 0;
        for (int64_t t = (int64_t)p.T * chunk / p.chunks + warp; t < r1; t += 4 * kDotsWarps) {
            Raw<T, VEC> d[4];
            Raw<int32_t, VEC> a[4];
            float x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t r = t + k * kDotsWarps;
                if (r < r1) {
                    d[k].load(dy + r * p.lddy);
                    if (p.acc) {
                        a[k].load(acc + r * p.N);
                        x[k] = p.xd[r];
                    }
                }
            }
            if (held == kSumRows) {
                flush();
                held = 0;
            }
            held += 4;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (t + k * kDotsWarps < r1)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        const float v = to_f32(d[k].get(i));
                        if (p.acc) sum[0][i] += v * (x[k] * (float)a[k].get(i));
                        sum[1][i] += v;
                    }
        }
        flush();
    }
    for (int m = 0; m < 2; ++m) {
        if (m) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < VEC; ++i) sh[warp][32 * i + lane] = total[i];
        }
        __syncthreads();
        const int i = threadIdx.x, col = tile * 32 * VEC + i % 32 * VEC + i / 32;
        if (i < 32 * VEC && col < p.N) {
            double a = 0.0;
            for (int w = 0; w < kDotsWarps; ++w) a += sh[w][i];
            if (p.chunks == 1) {
                if (float* out = m ? p.dbias : p.ds) out[col] = (float)a;
            } else {
                p.partials[((int64_t)chunk * 2 + m) * p.N + col] = (float)a;
            }
        }
    }
    if (p.chunks > 1) {
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) last = atomicAdd(&p.done[tile], 1) == p.chunks - 1;
        __syncthreads();
        if (last) {
            __threadfence();
            for (int i = threadIdx.x; i < 2 * 32 * VEC; i += 32 * kDotsWarps) {
                const int m = i / (32 * VEC), col = tile * 32 * VEC + i % (32 * VEC);
                float* out = m ? p.dbias : p.ds;
                if (col >= p.N || !out) continue;
                double a = 0.0;
                for (int k = 0; k < p.chunks; ++k) a += (double)__ldcg(&p.partials[((int64_t)k * 2 + m) * p.N + col]);
                out[col] = (float)a;
            }
        }
    }
    pdl_wait();
}

// Rows of both matrices: v_g = dh u act'(g) s_g and v_u = dh act(g) s_u from the
// saved sums, and the CTA's part of the scales' gradients, which are column sums
// over its rows.  A thread owns NJ groups of VEC columns; the next row's loads are
// in flight while a row waits for its largest value.  Bound by the arithmetic and
// its latency: 2048 x 2048 bf16 22 us, 42 MB from HBM at 24 % of its rate, 44 % of
// the issue slots (two CTAs an SM; three and four were slower).
template <int DT, int VEC, int NJ>
__global__ void __launch_bounds__(VEC == 1 ? 1024 : 512) k_gated_rows(const GradRowsParams p) {
    constexpr int P = planes_of(DT);
    __shared__ uint32_t sh[64];
    pdl_wait();
    pdl_launch_dependents();
    GradIn<DT, VEC> in[NJ];
    Raw<float, VEC> sc[NJ][kMats];
    float sum[NJ][2][VEC], xd_next = 0.0f;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) sum[j][0][i] = sum[j][1][i] = 0.0f;
    auto col = [&](int j) { return (int)(threadIdx.x + j * blockDim.x) * VEC; };
    float* part = p.partials + (int64_t)blockIdx.x * 2 * p.N;
    auto flush = [&] {  // the column sums so far to the next slot
#pragma unroll
        for (int j = 0; j < NJ; ++j)
            if (col(j) < p.N)
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        part[(int64_t)k * p.N + col(j) + i] = sum[j][k][i];
                        sum[j][k][i] = 0.0f;
                    }
        part += (int64_t)gridDim.x * 2 * p.N;
    };
    int held = 0, slot = 0;
    auto fetch = [&](int64_t t) {
        xd_next = p.xd[t];
#pragma unroll
        for (int j = 0; j < NJ; ++j)
            if (col(j) < p.N) in[j].load(p, t, col(j));
    };
    // rows further ahead are asked into L2 (whole rows on the 16-byte grid)
    auto ahead = [&](int64_t t) {
        if (VEC == 1 || !p.bulk || threadIdx.x != 0 || t >= p.T) return;
        using T = typename Elem<DT>::T;
        bulk_prefetch_l2(static_cast<const T*>(p.dy) + t * p.lddy, p.N * (uint32_t)sizeof(T));
#pragma unroll
        for (int m = 0; m < kMats; ++m)
            bulk_prefetch_l2(p.acc + ((int64_t)m * p.T + t) * p.N, p.N * 4u);
    };
    int buf = 0;
    fetch(blockIdx.x);
    for (int i = 1; i <= kRowsAhead; ++i) ahead(blockIdx.x + (int64_t)i * gridDim.x);
#pragma unroll
    for (int j = 0; j < NJ; ++j)
        if (col(j) < p.N)
#pragma unroll
            for (int m = 0; m < kMats; ++m) sc[j][m].load(p.s[m] + col(j));
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, buf ^= 1) {
        const float xd = xd_next;
        ahead(t + (int64_t)(kRowsAhead + 1) * gridDim.x);
        if (held == kSumRows) {
            flush();
            held = 0;
            ++slot;
        }
        ++held;
        float v[NJ][kMats][VEC];
        float peak = 0.0f;
        with_act(p.act, [&](auto act) {
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                if (col(j) < p.N) {
                    grad_cols<decltype(act)::value, DT, VEC>(p, in[j], sc[j], xd, v[j], sum[j]);
                    peak_of<VEC>(v[j], peak);
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
                for (int k = 0; k < kMats; ++k)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) v[j][k][i] *= lift;
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j)
            if (col(j) < p.N)
#pragma unroll
                for (int k = 0; k < kMats; ++k) store_planes<P, VEC>(p, t, k, col(j), kMats, mult, v[j][k]);
    }
    for (; slot < p.slots; ++slot) flush();  // (the last may be one row short of a sum: zeros)
}

// Rows of any length: the values are computed twice and the column sums kept
// in the CTA's partials.
template <int DT>
__global__ void __launch_bounds__(1024) k_gated_rows_long(const GradRowsParams p) {
    constexpr int P = planes_of(DT);
    __shared__ uint32_t sh[64];
    pdl_wait();
    pdl_launch_dependents();
    float* part = p.partials + (int64_t)blockIdx.x * 2 * p.N;
    int held = 0, slot = 0;
    auto column = [&](int64_t t, int c, float xd, float (&v)[kMats][1], float (&sum)[2][1]) {
        GradIn<DT, 1> in;
        Raw<float, 1> sc[kMats];
        in.load(p, t, c);
        for (int k = 0; k < kMats; ++k) sc[k].load(p.s[k] + c);
        with_act(p.act,
                 [&](auto act) { grad_cols<decltype(act)::value, DT, 1>(p, in, sc, xd, v, sum); });
    };
    int buf = 0;
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, buf ^= 1) {
        const float xd = p.xd[t];
        if (held == kSumRows) {
            part += (int64_t)gridDim.x * 2 * p.N;
            held = 0;
            ++slot;
        }
        float peak = 0.0f;
        for (int c = threadIdx.x; c < p.N; c += blockDim.x) {
            float v[kMats][1], sum[2][1];
            for (int k = 0; k < 2; ++k) sum[k][0] = held == 0 ? 0.0f : part[(int64_t)k * p.N + c];
            column(t, c, xd, v, sum);
            peak_of<1>(v, peak);
            for (int k = 0; k < 2; ++k) part[(int64_t)k * p.N + c] = sum[k][0];
        }
        ++held;
        float lift;
        RowScale scale;
        const float mult = fixed_point<P>(block_max_bits(__float_as_uint(fabsf(peak)), sh, buf), lift, scale);
        if (threadIdx.x == 0) p.scale[t] = scale;
        for (int c = threadIdx.x; c < p.N; c += blockDim.x) {
            float v[kMats][1], sum[2][1] = {{0.0f}, {0.0f}};
            column(t, c, xd, v, sum);
            for (int k = 0; k < kMats; ++k) {
                v[k][0] *= lift;
                store_planes<P, 1>(p, t, k, c, kMats, mult, v[k]);
            }
        }
    }
    while (++slot < p.slots) {  // (at most one row short of another sum: zeros)
        part += (int64_t)gridDim.x * 2 * p.N;
        for (int c = threadIdx.x; c < p.N; c += blockDim.x)
            for (int k = 0; k < 2; ++k) part[(int64_t)k * p.N + c] = 0.0f;
    }
}

// out[c] = sum over the partial sums, 32 columns a CTA: each of its 8
// warps adds every 8th partial in fp64, then the warps' sums are added in order.
// It runs under the gradient's product (small CTAs, no shared memory to speak
// of), whose end it waits for last, so that whatever follows finds both done.
__global__ void __launch_bounds__(256) k_col_sums(const float* partials, int n_part, int N,
                                                  float* out0, float* out1) {
    __shared__ double sh[8][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = (int)(blockIdx.x >> 1) * 32 + lane, k = blockIdx.x & 1;
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
    const unsigned tiles = (unsigned)((N + 31) / 32);
    return launch_dense(k_col_sums, 2 * tiles, 256, 0, 1, s, partials, n_part, N, out0, out1);
}

// CTAs of the gated gradient row kernel: a fixed grid (the column sums' order is
// the same from call to call), at most per_sm (one or two) an SM; and the
// partial sums that each of them writes.
static int grad_rows_grid(int T, int per_sm) {
    const int most = per_sm * device_info().sm_count;
    return T < most ? T : most;
}

static int grad_rows_slots(int T, int grid) {
    const int rows = (T + grid - 1) / grid;
    return (rows + kSumRows - 1) / kSumRows;
}

int64_t grad_rows_parts(int T) {
    int64_t most = 0;
    for (int per_sm = 1; T > 0 && per_sm <= 2; ++per_sm) {
        const int grid = grad_rows_grid(T, per_sm);
        const int64_t n = (int64_t)grid * grad_rows_slots(T, grid);
        most = n > most ? n : most;
    }
    return most;
}

template <int DT>
static cudaError_t grad_rows(const GradRowsArgs& a, GradRowsParams p, int& n_part, cudaStream_t s) {
    const size_t vb = 4 * sizeof(typename Elem<DT>::T);
    bool vec = reinterpret_cast<uintptr_t>(a.dy) % vb == 0 && a.lddy % 4 == 0 && a.N % 4 == 0 &&
               reinterpret_cast<uintptr_t>(a.acc) % 16 == 0;
    for (int m = 0; m < kMats; ++m) vec = vec && reinterpret_cast<uintptr_t>(a.s[m]) % 16 == 0;
    const int esz = (int)sizeof(typename Elem<DT>::T);
    p.bulk = vec && reinterpret_cast<uintptr_t>(a.dy) % 16 == 0 && a.lddy * esz % 16 == 0 && a.N * esz % 16 == 0;
    const int groups = vec ? a.N / 4 : a.N;
    // two groups of four columns a thread, four beyond 4096 columns; single columns
    // one or four.  Two CTAs an SM without spills beat three with them (2048
    // columns: 123.0 against 125.8 us of the training step at 2048 tokens, measured
    // with two planes).  Four groups of four columns do spill, 216 to 336 bytes a
    // thread.
    const int per = vec ? (groups <= 2 * 512 ? 2 : 4) : (groups <= 512 ? 1 : 4);
    const int threads = (groups + 32 * per - 1) / (32 * per) * 32;
    const bool any = threads > (vec ? 512 : 1024);
    const int grid = grad_rows_grid(a.T, threads > 384 && !any ? 1 : 2);
    p.slots = grad_rows_slots(a.T, grid);
    n_part = grid * p.slots;
    if (any) return launch_dense(k_gated_rows_long<DT>, grid, 1024, 0, 1, s, p);
    if (vec)
        return per == 2 ? launch_dense(k_gated_rows<DT, 4, 2>, grid, threads, 0, 1, s, p)
                        : launch_dense(k_gated_rows<DT, 4, 4>, grid, threads, 0, 1, s, p);
    return per == 1 ? launch_dense(k_gated_rows<DT, 1, 1>, grid, threads, 0, 1, s, p)
                    : launch_dense(k_gated_rows<DT, 1, 4>, grid, threads, 0, 1, s, p);
}

template <int DT>
static cudaError_t one_rows(const GradRowsArgs& a, const GradRowsParams& p, cudaStream_t s) {
    using T = typename Elem<DT>::T;
    const bool vec = reinterpret_cast<uintptr_t>(a.dy) % (4 * sizeof(T)) == 0 && a.lddy % 4 == 0 && a.N % 4 == 0 &&
                     reinterpret_cast<uintptr_t>(a.s[0]) % 16 == 0;
    const int groups = vec ? a.N / 4 : a.N;
    const int each = a.T >= 2 * device_info().sm_count ? kRowCache : 1;
    int threads = (groups + 32 * each - 1) / (32 * each) * 32;
    threads = threads > 512 ? 512 : threads;
    return vec ? launch_dense(k_grad_rows<DT, 4>, a.T, threads, 0, 1, s, p)
               : launch_dense(k_grad_rows<DT, 1>, a.T, threads, 0, 1, s, p);
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
    p.done = a.done;
    if (a.n_mats == 1)
        return a.dtype == MOE_F32    ? one_rows<MOE_F32>(a, p, s)
               : a.dtype == MOE_BF16 ? one_rows<MOE_BF16>(a, p, s)
                                     : one_rows<MOE_F16>(a, p, s);
    return a.dtype == MOE_F32    ? grad_rows<MOE_F32>(a, p, *n_part, s)
           : a.dtype == MOE_BF16 ? grad_rows<MOE_BF16>(a, p, *n_part, s)
                                 : grad_rows<MOE_F16>(a, p, *n_part, s);
}

int col_dots_tiles(int N) { return (N + 31) / 32; }

template <int DT>
static cudaError_t col_dots(const GradRowsArgs& a, float* ds, float* dbias, cudaStream_t s) {
    using T = typename Elem<DT>::T;
    const bool vec = reinterpret_cast<uintptr_t>(a.dy) % (4 * sizeof(T)) == 0 && a.lddy % 4 == 0 && a.N % 4 == 0 &&
                     reinterpret_cast<uintptr_t>(a.acc) % 16 == 0;
    ColDotsParams p{a.dy, a.lddy, ds ? a.acc : nullptr, a.xd, a.T, a.N, 1, a.partials, a.done, ds, dbias};
    const int tiles = vec ? (a.N + 127) / 128 : col_dots_tiles(a.N);
    // a CTA for each SM, but 32 rows or more for each of them
    const int most = kMaxDotChunks < a.T / 32 ? kMaxDotChunks : a.T / 32;
    p.chunks = device_info().sm_count / tiles;
    p.chunks = p.chunks > most ? most : p.chunks;
    p.chunks = p.chunks < 1 ? 1 : p.chunks;
    const unsigned grid = (unsigned)(tiles * p.chunks);
    return vec ? launch_dense(k_col_dots<DT, 4>, grid, 32 * kDotsWarps, 0, 1, s, p)
               : launch_dense(k_col_dots<DT, 1>, grid, 32 * kDotsWarps, 0, 1, s, p);
}

cudaError_t launch_col_dots(const GradRowsArgs& a, float* ds, float* dbias, cudaStream_t s) {
    return a.dtype == MOE_F32    ? col_dots<MOE_F32>(a, ds, dbias, s)
           : a.dtype == MOE_BF16 ? col_dots<MOE_BF16>(a, ds, dbias, s)
                                 : col_dots<MOE_F16>(a, ds, dbias, s);
}

// ---------------------------------------------------------------------------
// Rows of codes off the 16-byte grid to rows on it, zeros past a row's end.  Up to
// three matrices a launch, one for each blockIdx.y, in chunks of 16 bytes, EACH of
// them under way a thread (1 while the threads find room on the device at once).
// Bound by latency at a few megabytes, by memory beyond: 2000 x 2049 codes and
// 3001 x 2049, 20 MB of traffic, 5 us.
// ---------------------------------------------------------------------------
struct PadParams {
    const uint8_t* src[3];
    int64_t ld[3];
    int64_t chunks[3];  // of the matrix
    uint8_t* dst[3];
    int unit[3];
    int n, cols;
    uint32_t row_chunks;
};

template <int EACH>
__global__ void __launch_bounds__(256) k_pad_rows(const PadParams p) {
    pdl_wait();
    pdl_launch_dependents();
    // (chosen by comparisons: an index would put the parameters on the stack)
    const int m = blockIdx.y;
    const uint8_t* src = m == 0 ? p.src[0] : m == 1 ? p.src[1] : p.src[2];
    uint8_t* dst = m == 0 ? p.dst[0] : m == 1 ? p.dst[1] : p.dst[2];
    const int64_t ld = m == 0 ? p.ld[0] : m == 1 ? p.ld[1] : p.ld[2];
    const int64_t n = m == 0 ? p.chunks[0] : m == 1 ? p.chunks[1] : p.chunks[2];
    const int unit = m == 0 ? p.unit[0] : m == 1 ? p.unit[1] : p.unit[2];
    for (int64_t i0 = (int64_t)blockIdx.x * (256 * EACH) + threadIdx.x; i0 < n; i0 += (int64_t)gridDim.x * (256 * EACH)) {
        uint4 v[EACH];
#pragma unroll
        for (int e = 0; e < EACH; ++e) {
            const int64_t i = i0 + 256 * e;
            const uint32_t r = (uint32_t)i / p.row_chunks, c = (uint32_t)i - r * p.row_chunks;
            if (i < n) v[e] = load16(src + r * ld, 16 * (int64_t)c, p.cols, unit);
        }
#pragma unroll
        for (int e = 0; e < EACH; ++e)
            if (i0 + 256 * e < n) *reinterpret_cast<uint4*>(dst + 16 * (i0 + 256 * e)) = v[e];
    }
}

size_t pad_bytes(int n_mats, int T, int rows, int cols) {
    return ((size_t)n_mats * rows + T) * (size_t)pad_pitch(cols);
}

cudaError_t pad_operands(GemmArgs& a, bool tokens, void* room, cudaStream_t s) {
    PadParams p{};
    p.cols = a.cols;
    const int64_t pitch = pad_pitch(a.cols);
    p.row_chunks = (uint32_t)(pitch / 16);
    uint8_t* to = static_cast<uint8_t*>(room);
    int64_t most = 0;
    // the copy of one matrix: its address, with the pitch as its stride from then on
    auto copy = [&](const void* src, int64_t& ld, int rows) {
        const int i = p.n++;
        p.src[i] = static_cast<const uint8_t*>(src);
        p.ld[i] = ld;
        p.chunks[i] = (int64_t)rows * p.row_chunks;
        p.dst[i] = to;
        p.unit[i] = unit_of(src, ld);
        to += rows * pitch;
        most = p.chunks[i] > most ? p.chunks[i] : most;
        ld = pitch;
        return p.dst[i];
    };
    // (chunks are counted in 32 bits: larger matrices are read as they lie)
    const bool w_fits = (int64_t)a.rows * p.row_chunks <= UINT32_MAX;
    const bool x_fits = (int64_t)a.T * p.row_chunks <= UINT32_MAX;
    for (int m = 0; m < a.n_mats; ++m)
        if (w_fits && unit_of(a.w[m], a.ldw[m]) < 16) a.w[m] = copy(a.w[m], a.ldw[m], a.rows);
    if (tokens && x_fits && unit_of(a.x, a.ldx) < 16) a.x = reinterpret_cast<const int8_t*>(copy(a.x, a.ldx, a.T));
    if (!p.n) return cudaSuccess;
    const int sms = device_info().sm_count;
    const bool few = p.n * most <= 512 * (int64_t)sms;
    const int64_t per = few ? 256 : 512, want = (most + per - 1) / per, cap = 8 * sms / p.n;
    const dim3 grid((unsigned)(want < cap ? want : cap), p.n);
    return launch_dense(few ? k_pad_rows<1> : k_pad_rows<2>, grid, 256, 0, 1, s, p);
}

}  // namespace dense
}  // namespace moe
