// moe_dense_few.cu -- the dense int8 products of a few tokens: a stream of the
// weights.
//
// With up to 16 tokens the products read every weight once and little else, so
// what counts is bytes in flight and few instructions for each.  A CTA takes 16
// rows (gated: of both matrices), its warps every WARPS-th 64-byte column of
// them: a lane loads 16 bytes of two rows straight into the A fragments of two
// m16n8k32 products (the order of k inside a fragment is free as long as the
// tokens' B fragments use the same), with kUnroll columns under way.  Up to 8
// tokens cost what one does.  The warps' integer sums meet in shared memory.
// (The tcgen05 kernels need a tile of 128 rows in shared memory first; here that
// detour costs more than the products.)
//
// With QUANT the tokens come as floats: every CTA quantises all of them into
// shared memory, with the arithmetic of k_quantize_token, while its first
// weights are under way; that saves a launch and a trip through L2.
//
// Bound by the weights' way from L2 or HBM, and by the launch.  Three CTAs of 8
// warps an SM where there are rows for them (16 tokens through 2048 x 6144: 3.8
// us with the weights in L2, against 6.6 us with one; 5.0 us with the weights in
// HBM), one CTA of 16 warps otherwise (one token through 6144 x 2048: 2.8 us with
// the weights in L2, 4.1 us, 3.1 TB/s, in HBM; the gated block 6.8 and 8.1 us, 3.1
// TB/s).  The bound of three CTAs leaves the quantising form 80 registers, and it
// spills 140 bytes a thread.
#include <type_traits>

#include "moe_dense.cuh"
#include "moe_device.cuh"
#include "moe_ptx.cuh"

namespace moe {
namespace dense {

constexpr int kFewRows = 16;

struct FewParams {
    const uint8_t* w[kMaxMats];
    int64_t ldw[kMaxMats];
    const void* x;
    int64_t ldx;
    const float* xd;
    const float* s[kMaxMats];
    const float* bias;
    void* out;
    int64_t ldo;
    int32_t* acc;
    int T, rows, cols;
    int pitch;   // QUANT: bytes of a token's codes in shared memory
    int act, dtype;
    int w_unit[kMaxMats], x_unit;
    bool dependent;  // the kernel before this one does not write the weights
};

__device__ __forceinline__ void mma_16832(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
        "%3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// XT: int8_t codes, or the type of tokens to quantise.  NB: blocks of 8 tokens.
// FAST: weight rows (and codes) on the 16-byte grid and cols a multiple of 16.
template <int MODE, int NB, typename XT, bool FAST, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, WARPS == 8 ? (MODE == kMatmul ? 3 : 2) : 1)
    k_dense_few(const FewParams p) {
    constexpr int M = MODE == kGated ? 2 : 1;
    constexpr bool QUANT = sizeof(XT) > 1;
    constexpr int kUnroll = !FAST ? 2 : M == 2 || QUANT || WARPS == 8 ? 4 : 6;
    extern __shared__ __align__(16) uint8_t few_smem[];
    int* red = reinterpret_cast<int*>(few_smem);  // [WARPS][M][NB][128]
    uint32_t* peak = reinterpret_cast<uint32_t*>(few_smem + WARPS * M * NB * 512);  // QUANT: [8 NB]
    uint8_t* codes = reinterpret_cast<uint8_t*>(peak + 8 * NB);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int64_t row0 = (int64_t)blockIdx.x * kFewRows;
    const int nch = (p.cols + 63) / 64;
    const uint8_t* wr[M][2];
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) wr[m][h] = p.w[m] + min(row0 + g + 8 * h, (int64_t)p.rows - 1) * p.ldw[m];
    uint4 a[kUnroll][M][2];
    auto load_w = [&](int ch) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int c = (ch + u * WARPS) * 64 + 16 * q;
#pragma unroll
            for (int m = 0; m < M; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    a[u][m][h] = c >= p.cols ? make_uint4(0, 0, 0, 0)
                                 : FAST      ? ld_once_v4(wr[m][h] + c)
                                             : load16(wr[m][h], c, p.cols, p.w_unit[m]);
        }
    };
    if (!p.dependent) pdl_wait();
    load_w(warp);
    if (p.dependent) pdl_wait();
    pdl_launch_dependents();
    if constexpr (QUANT) {
        if (threadIdx.x < 8 * NB) peak[threadIdx.x] = 0;
        __syncthreads();
        // `per` warps a token (one warp takes every WARPS-th token where there are
        // more): its vectors loaded together and kept for the second pass
        constexpr int V = 16 / (int)sizeof(XT), kKeep = 8;
        const int per = max(1, WARPS / p.T), sub = warp % per;
        const XT* x = static_cast<const XT*>(p.x);
        Raw<XT, V> e[kKeep];
        const int c0 = V * (lane + 32 * sub), step = V * 32 * per;
        auto peak_of = [&](const Raw<XT, V>& r, uint32_t m) {
#pragma unroll
            for (int i = 0; i < V; ++i) m = max(m, __float_as_uint(to_f32(r.get(i))) & 0x7FFFFFFFu);
            return m;
        };
        auto scan = [&](int t) {
            const XT* xr = x + t * p.ldx;
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < kKeep; ++i)
                if (c0 + i * step < p.cols) e[i].load(xr + c0 + i * step);
#pragma unroll
            for (int i = 0; i < kKeep; ++i)
                if (c0 + i * step < p.cols) m = peak_of(e[i], m);
            for (int c = c0 + kKeep * step; c < p.cols; c += step) {
                Raw<XT, V> r;
                r.load(xr + c);
                m = peak_of(r, m);
            }
            return __reduce_max_sync(kFull, m);
        };
        auto put = [&](int t, uint32_t m) {
            const XT* xr = x + t * p.ldx;
            int8_t* o = reinterpret_cast<int8_t*>(codes) + t * p.pitch;
            const float inv = quant_scale(m).inv;
            auto one = [&](const Raw<XT, V>& r, int c) {
                int q8[V];
#pragma unroll
                for (int i = 0; i < V; ++i) q8[i] = round_away(__fmul_rn(to_f32(r.get(i)), inv));
                store_bytes<V, 0>(o + c, q8, 0u);
            };
#pragma unroll
            for (int i = 0; i < kKeep; ++i)
                if (c0 + i * step < p.cols) one(e[i], c0 + i * step);
            for (int c = c0 + kKeep * step; c < p.cols; c += step) {
                Raw<XT, V> r;
                r.load(xr + c);
                one(r, c);
            }
        };
        if (per == 1) {
            for (int t = warp; t < p.T; t += WARPS) {
                const uint32_t m = scan(t);
                if (lane == 0) peak[t] = m;
                put(t, m);
            }
        } else {
            const int t = warp / per;
            if (t < p.T) {
                const uint32_t m = scan(t);
                if (lane == 0) atomicMax(&peak[t], m);
            }
            __syncthreads();
            if (t < p.T) put(t, peak[t]);
        }
        __syncthreads();
    }
    int acc[M][NB][4];
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m][n][i] = 0;
    for (int ch = warp; ch < nch; ch += kUnroll * WARPS) {
        if (ch > warp) load_w(ch);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int c = (ch + u * WARPS) * 64 + 16 * q;
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                const int t = 8 * n + g;
                uint4 b = make_uint4(0, 0, 0, 0);
                if (t < p.T && c < p.cols) {
                    if constexpr (QUANT)
                        b = *reinterpret_cast<const uint4*>(codes + t * p.pitch + c);
                    else
                        b = FAST ? *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.x) + t * p.ldx + c)
                                 : load16(static_cast<const uint8_t*>(p.x) + t * p.ldx, c, p.cols, p.x_unit);
                }
#pragma unroll
                for (int m = 0; m < M; ++m) {
                    const uint4 lo = a[u][m][0], hi = a[u][m][1];
                    mma_16832(acc[m][n], lo.x, hi.x, lo.y, hi.y, b.x, b.y);
                    mma_16832(acc[m][n], lo.z, hi.z, lo.w, hi.w, b.z, b.w);
                }
            }
        }
    }
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)  // [token][row]
                red[((warp * M + m) * NB + n) * 128 + (2 * q + (i & 1)) * 16 + g + 8 * (i >> 1)] = acc[m][n][i];
    __syncthreads();
    for (int i = threadIdx.x; i < p.T * kFewRows; i += 32 * WARPS) {
        const int t = i / kFewRows;
        const int64_t row = row0 + i % kFewRows;
        if (row >= p.rows) continue;
        int v[M];
#pragma unroll
        for (int m = 0; m < M; ++m) {
            v[m] = 0;
            for (int k = 0; k < WARPS; ++k) v[m] += red[(k * M + m) * NB * 128 + i];
            if (p.acc) p.acc[((int64_t)m * p.T + t) * p.rows + row] = v[m];
        }
        const float xd = QUANT ? quant_scale(peak[t]).scale : p.xd[t];
        float y = (float)v[0] * (xd * p.s[0][row]);
        if constexpr (MODE == kGated)
            with_act(p.act, [&](auto act) {
                y = act_value<decltype(act)::value>(y) * ((float)v[M - 1] * (xd * p.s[M - 1][row]));
            });
        else if (p.bias)
            y += p.bias[row];
        store_elem(p.out, t * p.ldo + row, p.dtype, y);
    }
}

// x_type: -1 for codes, else the element type of tokens to quantise.
template <int MODE>
static cudaError_t run_few(const GemmArgs& a, const void* x, int x_type, bool dependent, cudaStream_t s) {
    FewParams p{};
    bool fast = a.cols % 16 == 0;
    for (int m = 0; m < a.n_mats; ++m) {
        p.w[m] = a.w[m];
        p.ldw[m] = a.ldw[m];
        p.s[m] = a.s[m];
        p.w_unit[m] = unit_of(a.w[m], a.ldw[m]);
        fast = fast && p.w_unit[m] == 16;
    }
    p.x = x;
    p.ldx = a.ldx;
    p.x_unit = unit_of(x, a.ldx);
    if (x_type < 0) fast = fast && p.x_unit == 16;
    p.xd = a.xd;
    p.bias = a.bias;
    p.out = a.out;
    p.ldo = a.ldo;
    p.acc = a.acc;
    p.T = a.T;
    p.rows = a.rows;
    p.cols = a.cols;
    p.act = a.act;
    p.dtype = a.dtype;
    p.dependent = dependent;
    p.pitch = (a.cols + 127) / 128 * 128 + 64;  // two tokens' 64 bytes fall on different banks
    const unsigned grid = (unsigned)((a.rows + (int64_t)kFewRows - 1) / kFewRows);
    auto go = [&](auto nb, auto type, auto is_fast, auto warps) {
        using XT = decltype(type);
        constexpr int NB = decltype(nb)::value, WARPS = decltype(warps)::value;
        auto* kernel = k_dense_few<MODE, NB, XT, decltype(is_fast)::value, WARPS>;
        static bool attr_done[64];
        cudaError_t e = allow_smem(kernel, attr_done);
        if (e != cudaSuccess) return e;
        const size_t smem = WARPS * (MODE == kGated ? 2 : 1) * NB * 512 + (x_type < 0 ? 0 : 32 * NB + (size_t)a.T * p.pitch);
        return launch_dense(kernel, grid, 32 * WARPS, smem, 1, s, p);
    };
    using std::integral_constant;
    // 16 warps a CTA where the rows give the SMs less than two CTAs each
    auto by_size = [&](auto type) {
        auto by_fast = [&](auto is_fast) {
            auto by_warps = [&](auto nb) {
                return (int64_t)grid < 2 * (int64_t)device_info().sm_count
                           ? go(nb, type, is_fast, integral_constant<int, 16>())
                           : go(nb, type, is_fast, integral_constant<int, 8>());
            };
            return a.T <= 8 ? by_warps(integral_constant<int, 1>()) : by_warps(integral_constant<int, 2>());
        };
        if constexpr (sizeof(type) > 1)
            return by_fast(integral_constant<bool, true>());
        else
            return fast ? by_fast(integral_constant<bool, true>()) : by_fast(integral_constant<bool, false>());
    };
    if (x_type < 0) return by_size(int8_t());
    if constexpr (MODE == kGated) {
        if (x_type == MOE_BF16) return by_size(__nv_bfloat16());
        if (x_type == MOE_F16) return by_size(__half());
    }
    return by_size(float());  // (the product's tokens are the gated block's fp32 results)
}

cudaError_t launch_few_matmul(const GemmArgs& a, cudaStream_t s) { return run_few<kMatmul>(a, a.x, -1, false, s); }

cudaError_t launch_few_gated(const GemmArgs& a, cudaStream_t s) { return run_few<kGated>(a, a.x, -1, false, s); }

bool few_quantised_fits(const GemmArgs& a, const void* x, int x_type) {
    bool ok = a.T <= kFewTokens && a.cols % 16 == 0 && (int64_t)a.T * a.cols <= 96 * 1024 &&
              unit_of(x, a.ldx * (x_type == MOE_F32 ? 4 : 2)) == 16;
    for (int m = 0; m < a.n_mats; ++m) ok = ok && unit_of(a.w[m], a.ldw[m]) == 16;
    return ok;
}

cudaError_t launch_gated_quantised(const GemmArgs& a, const void* x, int x_type, cudaStream_t s) {
    return run_few<kGated>(a, x, x_type, false, s);
}

cudaError_t launch_matmul_quantised(const GemmArgs& a, const float* x, cudaStream_t s) {
    return run_few<kMatmul>(a, x, MOE_F32, true, s);
}

}  // namespace dense
}  // namespace moe
