// moe_dense.cuh -- what the dense int8 operators share: element types, the
// gated block's activations and their derivatives, the fixed-point planes of a
// gradient row, and the parameters of the kernels in moe_dense_*.cu.
//
// The operators are the dense counterpart of the routed experts' integer-dot
// matmuls (GeekNews "Show HN: 느린 컴퓨터에서 GLM 5.2 실행하기", §구현된 주요 기능:
// int8 rows with per-row scales times int8 activations; the engine keeps its
// dense parts resident at int8): one scale for each token and one for each
// weight row, so the integer sum runs over the whole row and is scaled once.
#pragma once

#include <cfloat>
#include <cstdint>
#include <type_traits>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "moe_internal.h"

namespace moe {
namespace dense {

constexpr int kMaxMats = 2;

// ---------------------------------------------------------------------------
// Element types of activations, results and gradients (MOE_F32 / BF16 / F16)
// ---------------------------------------------------------------------------
template <int DT>
struct Elem;
template <>
struct Elem<MOE_F32> {
    using T = float;
};
template <>
struct Elem<MOE_BF16> {
    using T = __nv_bfloat16;
};
template <>
struct Elem<MOE_F16> {
    using T = __half;
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

template <typename OT>
__device__ __forceinline__ OT from_f32(float v) {
    if constexpr (sizeof(OT) == 4)
        return v;
    else if constexpr (std::is_same<OT, __nv_bfloat16>::value)
        return __float2bfloat16_rn(v);
    else
        return __float2half_rn(v);
}

// One result element, rounded once to its type.
__device__ __forceinline__ void store_elem(void* out, int64_t i, int dtype, float v) {
    if (dtype == MOE_F32)
        static_cast<float*>(out)[i] = v;
    else if (dtype == MOE_BF16)
        static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v);
    else
        static_cast<__half*>(out)[i] = __float2half_rn(v);
}

// ---------------------------------------------------------------------------
// act(g) = g sigmoid(z(g)): z = g (SiLU), z = 2 sqrt(2/pi)(g + 0.044715 g^3)
// (the tanh form of GELU, since (1 + tanh y)/2 = sigmoid(2 y); written so, it
// does not cancel for negative g).  With e = exp(-|z|) <= 1 nothing overflows:
// sigmoid(z) is 1/(1+e) or e/(1+e), and its derivative e/(1+e)^2.  The
// reciprocal of 1 + e, in [1, 2], is the intrinsic good to two units in the last
// place: the exactly rounded one branches, which keeps the values of a thread
// from overlapping (the gated product's epilogue took 18,000 cycles a tile with
// it).
// ---------------------------------------------------------------------------
constexpr float kGelu0 = 1.5957691216057308f;  // 2 sqrt(2/pi)
constexpr float kGelu1 = 0.044715f;

template <int ACT>
__device__ __forceinline__ float act_value(float g) {
    const float z = ACT == MOE_ACT_SILU ? g : kGelu0 * (g + kGelu1 * g * g * g);
    const float e = expf(-fabsf(z));
    const float r = __fdividef(1.0f, 1.0f + e);
    return g * (z >= 0.0f ? r : e * r);
}

template <int ACT>
__device__ __forceinline__ void act_value_grad(float g, float& a, float& da) {
    const float z = ACT == MOE_ACT_SILU ? g : kGelu0 * (g + kGelu1 * g * g * g);
    const float e = expf(-fabsf(z));
    const float r = __fdividef(1.0f, 1.0f + e);
    const float sig = z >= 0.0f ? r : e * r;
    const float dsig = e * r * r;
    a = g * sig;
    // far out the derivative of the sigmoid is zero while g or dz may be infinite
    const float gd = ACT == MOE_ACT_SILU ? g : g * (kGelu0 * (1.0f + 3.0f * kGelu1 * g * g));
    da = sig + (dsig == 0.0f ? 0.0f : gd * dsig);
}

// f(integral constant ACT) with the activation as a compile-time value, so that
// a kernel pays for the one it runs.
template <typename F>
__device__ __forceinline__ void with_act(int act, F f) {
    if (act == MOE_ACT_SILU)
        f(std::integral_constant<int, MOE_ACT_SILU>());
    else
        f(std::integral_constant<int, MOE_ACT_GELU>());
}

// ---------------------------------------------------------------------------
// The per-token quantiser's arithmetic.  From the bits of a row's largest
// magnitude: d = amax / 127 and 1/d.  Rows below 2^-112 store zeros (so d is a
// normal number and 1/d finite); a row with an infinity or a NaN stores d = NaN,
// so that whatever is computed from it says so.
// ---------------------------------------------------------------------------
constexpr uint32_t kInfBits = 0x7F800000u;
constexpr float kTinyRow = 1.925929944387236e-34f;  // 2^-112

struct QuantScale {
    float scale, inv;
};

__device__ __forceinline__ QuantScale quant_scale(uint32_t peak_bits) {
    const float amax = __uint_as_float(peak_bits);
    const bool live = peak_bits < kInfBits && amax >= kTinyRow;
    const float d = live ? __fdiv_rn(amax, 127.0f) : 0.0f;
    return QuantScale{peak_bits >= kInfBits ? __uint_as_float(0x7FC00000u) : d, live ? __fdiv_rn(1.0f, d) : 0.0f};
}

// round-half-away-from-zero of |v| < 2^23: adding half towards zero never
// carries past an integer that v + half does not reach, and the conversion cuts
// the rest.  (amax times fl(1/d) stays below 127.5, so codes need no clamp;
// 0 * inf and NaN convert to 0.)
__device__ __forceinline__ int round_away(float v) { return __float2int_rz(__fadd_rz(v, copysignf(0.5f, v))); }

// ---------------------------------------------------------------------------
// Vectors of a row's elements and codes
// ---------------------------------------------------------------------------
// VEC consecutive elements of a row, in 16- or 8-byte loads (the caller checked the alignment).
template <typename T, int VEC>
struct Raw {
    static constexpr int kWords = VEC * (int)sizeof(T) / 4;
    union {
        T e[VEC];
        uint32_t w[kWords > 0 ? kWords : 1];
    };
    __device__ __forceinline__ Raw() {}
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (VEC == 1) {
            e[0] = *p;
        } else if constexpr (kWords == 2) {
            const uint2 v = *reinterpret_cast<const uint2*>(p);
            w[0] = v.x;
            w[1] = v.y;
        } else {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i) {
                const uint4 v = reinterpret_cast<const uint4*>(p)[i];
                w[4 * i] = v.x;
                w[4 * i + 1] = v.y;
                w[4 * i + 2] = v.z;
                w[4 * i + 3] = v.w;
            }
        }
    }
    __device__ __forceinline__ T get(int i) const { return e[i]; }
};

// Byte K of four words, in order.
template <int K>
__device__ __forceinline__ uint32_t gather_byte(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    const uint32_t ab = __byte_perm(a, b, K | ((K + 4) << 4));
    const uint32_t cd = __byte_perm(c, d, K | ((K + 4) << 4));
    return __byte_perm(ab, cd, 0x5410);
}

// Byte K of VEC words, XOR-ed with flip, as codes in one store.
template <int VEC, int K>
__device__ __forceinline__ void store_bytes(int8_t* p, const int (&c)[VEC], uint32_t flip) {
    if constexpr (VEC == 1) {
        *p = (int8_t)(((uint32_t)c[0] >> (8 * K)) ^ (flip & 0xFFu));
    } else {
        uint32_t w[VEC / 4];
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i)
            w[i] = gather_byte<K>((uint32_t)c[4 * i], (uint32_t)c[4 * i + 1], (uint32_t)c[4 * i + 2],
                                  (uint32_t)c[4 * i + 3]) ^ flip;
        if constexpr (VEC == 4)
            *reinterpret_cast<uint32_t*>(p) = w[0];
        else
            *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    }
}

// ---------------------------------------------------------------------------
// Fixed-point planes of a gradient row.  A row v with m = max|v| is written as
// the integers round(v D / m) of P signed base-256 digits, D = 8355600 for P = 3
// and 2139060224 for P = 4 (a little below 127 in all digits, so that the
// product's rounding never lifts the top one), so that
//   sum_n v_n w_n = (m / D) sum_p 256^p (digit_p . w)
// runs as P int8 products against the packed weight rows as they lie, each
// exact in int32.  v D / m rounds as fp32 numbers do (the multiplier and the
// product: 2^-23 of v), and to the fixed point, by at most m / (2 D): m 2^-24
// for P = 3, m 2^-32 for P = 4.  That second part is what a row of a wide range
// can lose: its elements far below m.  16-bit gradients have three planes: N
// such roundings stay below their result's own where the row has one element
// far above the others (a softmax less its target over 128,256 rows: 2^-13 of
// sum |v w|; two planes, 16 bits, lost a fifth of dx there).  fp32 gradients have
// four, which keep an element's 24 bits down to m / 128 and leave less than an
// fp32 sum's own rounding over 131,071 of them.
// ---------------------------------------------------------------------------
constexpr int planes_of(int dtype) { return dtype == MOE_F32 ? 4 : 3; }
template <int P>
constexpr float kPlaneMax = P == 3 ? 8355600.0f : 2139060224.0f;

// The planes of 16 tokens lie together, [T / 16][P][16] rows, so that a tile's
// tokens are one box of memory whatever P is.
constexpr int kPlaneGroup = 16;
inline int64_t plane_rows(int planes, int64_t T) {
    return (T + kPlaneGroup - 1) / kPlaneGroup * kPlaneGroup * planes;
}
// Row of token t's first plane (the others follow kPlaneGroup rows apart).
template <int P>
__device__ __forceinline__ int64_t plane_row(int64_t t) {
    return t / kPlaneGroup * (P * kPlaneGroup) + t % kPlaneGroup;
}

// A row scale: value = integer * a * b (b a power of two that keeps a normal
// when the row is tiny).
struct RowScale {
    float a, b;
};

// ---------------------------------------------------------------------------
// Launches.  Every dense kernel may start while the kernel before it on the
// stream ends (programmatic dependent launch): it waits (pdl_wait) before it
// touches memory that others write, and lets its own successor start once it
// runs, so that launches and prologues of a chain overlap.  What a kernel reads
// may thus have been written during its own lifetime: none of its loads is
// marked as read-only (no __ldg, no const __restrict__), which would also let
// the compiler move it above the wait.
// ---------------------------------------------------------------------------
// 16 bytes that are read once: past L1, 256 bytes at a time into L2 (volatile:
// not to be moved above the wait).
__device__ __forceinline__ uint4 ld_once_v4(const void* p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p));
    return r;
}

template <typename... P, typename... A>
cudaError_t launch_dense(void (*kernel)(P...), dim3 grid, int threads, size_t smem, int cluster, cudaStream_t s,
                         A&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// Up to 16 bytes at any address, from the aligned words that hold them (no word
// without one of them is read): first the loads, then the bytes, zeros past `left`.
struct Words {
    uint32_t w[5];
    int shift, left;
};

__device__ __forceinline__ Words load_words(const uint8_t* src, int left) {
    Words r;
    r.shift = 8 * (int)(reinterpret_cast<uintptr_t>(src) & 3);
    r.left = left;
    const uint32_t* p = reinterpret_cast<const uint32_t*>(src - r.shift / 8);
    const int n = left > 0 ? (r.shift / 8 + left + 3) / 4 : 0;
#pragma unroll
    for (int i = 0; i < 5; ++i) r.w[i] = i < n ? p[i] : 0u;
    return r;
}

__device__ __forceinline__ uint4 join_words(const Words& r) {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int keep = r.left - 4 * i;  // bytes of this word
        o[i] = __funnelshift_r(r.w[i], r.w[i + 1], r.shift);
        o[i] = keep >= 4 ? o[i] : keep <= 0 ? 0u : o[i] & ((1u << (8 * keep)) - 1u);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// Sixteen bytes of a row from its column c on (bytes at and past `cols` read as
// zero); unit: the widest load that suits the row.
__device__ __forceinline__ uint4 load16(const uint8_t* row, int64_t c, int64_t cols, int unit) {
    const int left = (int)min((int64_t)16, max((int64_t)0, cols - c));
    if (left < 16 || unit < 4) return join_words(load_words(row + c, left));
    if (unit == 16) return *reinterpret_cast<const uint4*>(row + c);
    if (unit == 8) {
        const uint2 a = *reinterpret_cast<const uint2*>(row + c), b = *reinterpret_cast<const uint2*>(row + c + 8);
        return make_uint4(a.x, a.y, b.x, b.y);
    }
    const uint32_t* p = reinterpret_cast<const uint32_t*>(row + c);
    return make_uint4(p[0], p[1], p[2], p[3]);
}

// Bytes of the widest load that suits every row: 16, 8, 4 or 1.
inline int unit_of(const void* p, int64_t ld) {
    const uint64_t b = reinterpret_cast<uintptr_t>(p) | (uint64_t)ld;
    return b % 16 == 0 ? 16 : b % 8 == 0 ? 8 : b % 4 == 0 ? 4 : 1;
}

// The device's whole shared memory for a kernel (once a device).
template <typename K>
cudaError_t allow_smem(K kernel, bool (&done)[64]) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64 && done[dev]) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, device_info().max_smem_optin);
    if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
    return e;
}

// ---------------------------------------------------------------------------
// The products (moe_dense_gemm.cu, moe_dense_few.cu)
// ---------------------------------------------------------------------------
enum GemmMode { kMatmul = 0, kGated = 1, kGrad = 2 };

struct GemmArgs {
    // weights: n_mats matrices [rows][cols] of int8, row strides ldw
    const uint8_t* w[kMaxMats];
    int64_t ldw[kMaxMats];
    int n_mats;
    int rows, cols;
    // forward: codes [T][cols], row stride ldx.  gradient: rows of planes (see
    // plane_row) of ldx bytes, matrix m's part at byte m * mat_pitch
    const int8_t* x;
    int64_t ldx;
    int T;
    int64_t mat_pitch;
    const float* xd;         // forward: token scales
    const float* s[kMaxMats];  // forward: row scales
    const float* bias;       // matmul only, may be null
    const RowScale* gscale;  // gradient: row scales of the planes
    int act;
    void* out;
    int64_t ldo;
    int dtype;
    int32_t* acc;  // forward: integer sums [n_mats][T][rows], or null
};

cudaError_t launch_matmul(const GemmArgs& a, cudaStream_t s);
cudaError_t launch_gated(const GemmArgs& a, cudaStream_t s);
// Up to kFewTokens tokens (launch_matmul and launch_gated go there by themselves).
constexpr int kFewTokens = 16;
cudaError_t launch_few_matmul(const GemmArgs& a, cudaStream_t s);
cudaError_t launch_few_gated(const GemmArgs& a, cudaStream_t s);
// The products of a few tokens given as floats (rows of x with stride a.ldx),
// quantised inside the kernel; for operands that few_quantised_fits.  The second
// follows the first on the stream: as that does not write the weights, it reads
// them before it ends.
bool few_quantised_fits(const GemmArgs& a, const void* x, int x_type);
cudaError_t launch_gated_quantised(const GemmArgs& a, const void* x, int x_type, cudaStream_t s);
cudaError_t launch_matmul_quantised(const GemmArgs& a, const float* x, cudaStream_t s);
cudaError_t launch_grad_matmul(const GemmArgs& a, cudaStream_t s);
cudaError_t read_device_error(cudaStream_t s, int32_t* code);

// Whether TMA can take every operand: addresses and row strides on 16 bytes.
inline bool tma_operands(const GemmArgs& a) {
    bool ok = unit_of(a.x, a.ldx) == 16;
    for (int m = 0; m < a.n_mats; ++m) ok = ok && unit_of(a.w[m], a.ldw[m]) == 16;
    return ok;
}

// Copies the operands that are off the 16-byte grid to rows of pad_pitch(cols)
// bytes in `room` (pad_bytes), and points `a` at them.  A pass over odd rows
// costs their bytes twice and a launch; the products' own loads of them cost
// about four times what TMA does (2000 x 2049 x 3001: 106 us as they lie).
inline int64_t pad_pitch(int cols) { return ((int64_t)cols + 15) / 16 * 16; }
size_t pad_bytes(int n_mats, int T, int rows, int cols);
cudaError_t pad_operands(GemmArgs& a, bool tokens, void* room, cudaStream_t s);

// ---------------------------------------------------------------------------
// Row kernels (moe_dense_rows.cu)
// ---------------------------------------------------------------------------
cudaError_t launch_quantize_token(const void* x, int dtype, int64_t rows, int cols, int64_t ldx, int8_t* q,
                                  int64_t ldq, float* d, cudaStream_t s);

struct GradRowsArgs {
    const void* dy;  // [T][N]
    int64_t lddy;
    int dtype;
    const int32_t* acc;  // [n_mats][T][N]; may be null for one matrix (no scale gradient)
    const float* xd;     // [T]; null with acc
    const float* s[kMaxMats];
    int n_mats;
    int T, N;
    int act;
    int8_t* planes;  // [plane_rows(P, T)][n_mats * pitch]
    int64_t pitch;
    RowScale* scale;   // [T]
    float* partials;   // column sums: gated [grad_rows_parts][2][N]; one matrix [chunks][2][N]
    int* done;         // one matrix: counters of the column sums' tiles
};
int64_t grad_rows_parts(int T);     // gated: partial sums of a column, at most
constexpr int kMaxDotChunks = 64;  // row chunks of one matrix's column sums
int col_dots_tiles(int N);         // their counters, at most
// n_part: gated, how many partial sums of each column there are.
cudaError_t launch_grad_rows(const GradRowsArgs& a, int* n_part, cudaStream_t s);
// The column sums (each may be null), after the gradient's product on the
// stream and beside it: what they read was complete before that product began.
// gated: ds_gate and ds_up from the partials
cudaError_t launch_col_sums(const float* partials, int n_part, int N, float* out0, float* out1, cudaStream_t s);
// one matrix: ds and dbias from dy and acc
cudaError_t launch_col_dots(const GradRowsArgs& a, float* ds, float* dbias, cudaStream_t s);

}  // namespace dense
}  // namespace moe
