// moe_dense_gemm.cu -- the tensor-core products of the dense int8 operators.
//
// One kernel for three products, with the weights as the MMA's 128-row operand
// and the tokens as its columns:
//   matmul  acc[t, n] = sum_k xq[t, k] w[n, k]
//   gated   the same for two matrices at once, joined by act(g) u
//   grad    dx[t, k]  = sum_n v[t, n] w[n, k] over one or two matrices, v in
//           fixed-point planes; the weight tile is read as it lies in memory
//           (rows of w are the contraction there), so the MMA takes it in its
//           row-transposed form and nothing is ever transposed in memory
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "moe_dense.cuh"
#include "moe_device.cuh"
#include "moe_ptx.cuh"
#include "moe_tc.cuh"

namespace moe {
namespace tc {
cudaError_t encode_2d(CUtensorMap* map, const void* base, CUtensorMapDataType dtype, uint64_t cols, uint64_t rows,
                      uint64_t row_bytes, uint32_t box_cols, uint32_t box_rows, CUtensorMapSwizzle swz);
}
namespace dense {

using namespace tc;

// Code of the last fault a dense product recorded on this device (kErrTimeout).
__device__ int32_t g_dense_error;

constexpr uint64_t kWaitNs = 100000000ull;  // one pipeline wait
constexpr uint64_t kWaitAllNs = 4 * kWaitNs;  // the epilogue's wait for the whole tile
constexpr int kMaxStages = 8;
constexpr int kTileThreads = 192;  // producer warp, MMA warp, four epilogue warps
constexpr int kCtlBytes = 2048;    // barriers, the TMEM address, 128 token scales

struct TileParams {
    const uint8_t* w[kMaxMats];
    int64_t ldw[kMaxMats];
    const uint8_t* x;
    int64_t ldx;
    int64_t mat_pitch;
    const float* xd;
    const float* s[kMaxMats];
    const float* bias;
    const RowScale* gscale;
    void* out;
    int64_t ldo;
    int32_t* acc;
    int T, rows, cols;
    int out_rows;   // channels of the result (rows; cols for the gradient)
    int k_steps;    // 128-code steps of one matrix's contraction
    int steps;      // steps of the whole contraction
    int nt;         // tokens of a tile (a multiple of 16)
    int tiles_n;    // weight tiles
    int stages;
    int stage_bytes;
    int tmem_cols;
    int act, dtype;
    int direct;     // operands that TMA cannot take: plain loads by the epilogue warps
    int w_unit[kMaxMats], x_unit;  // direct: bytes of the widest aligned load
};

// Matrix descriptor of a weight tile whose 128-byte rows run along the MMA's
// M: 8-row groups (of K) 1024 bytes apart, 128-byte swizzle; one 32-code step
// of K is 32 rows, 4096 bytes.
__device__ __forceinline__ uint64_t desc_mn128_sw128(const void* tile) { return desc_k128_sw128(tile); }

template <int MODE>
__device__ __forceinline__ uint32_t idesc_tile(int n) {
    return idesc_i8(n) | (MODE == kGrad ? 1u << 15 : 0u);  // A transposed
}

// Sixteen bytes of a row from its column c on (bytes at and past `cols` read as zero).
__device__ __forceinline__ uint4 load16(const uint8_t* row, int64_t c, int64_t cols, int unit) {
    union {
        uint4 v;
        uint64_t q[2];
        uint32_t d[4];
        uint8_t b[16];
    } u;
    u.v = make_uint4(0, 0, 0, 0);
    const int64_t left = cols - c;
    if (left >= 16 && unit >= 4) {
        if (unit >= 16) {
            u.v = __ldg(reinterpret_cast<const uint4*>(row + c));
        } else if (unit == 8) {
            u.q[0] = __ldg(reinterpret_cast<const unsigned long long*>(row + c));
            u.q[1] = __ldg(reinterpret_cast<const unsigned long long*>(row + c + 8));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) u.d[i] = __ldg(reinterpret_cast<const uint32_t*>(row + c + 4 * i));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (i < left) u.b[i] = __ldg(row + c + i);
    }
    return u.v;
}

// A tile of n rows of 128 bytes at (row0, col0) of [rows][cols] into the
// 128-byte-swizzle layout, by 128 threads.
__device__ __forceinline__ void load_tile_direct(uint8_t* tile, const uint8_t* base, int64_t ld, int64_t rows,
                                                 int64_t cols, int64_t row0, int64_t col0, int n, int unit, int tid) {
    const int c = tid & 7;
    for (int r = tid >> 3; r < n; r += 16) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (row0 + r < rows) v = load16(base + (row0 + r) * ld, col0 + 16 * c, cols, unit);
        *reinterpret_cast<uint4*>(tile + sw128_chunk(r, c)) = v;
    }
}

__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ int ld_peer(const int32_t* p, uint32_t rank) {
    uint32_t a;
    int v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

// Joins a token's sums of one channel and stores the result.
template <int MODE, int P>
__device__ __forceinline__ void finish(const TileParams& p, const int (&v)[MODE == kGated ? 2 : P], int64_t t, int n,
                                       float ta, float tb, float s0, float s1, float bias) {
    if constexpr (MODE == kGrad) {
        // digits joined in fp32: each plane's sum rounds by 2^-24 of itself
        float f = (float)v[P - 1];
#pragma unroll
        for (int i = P - 2; i >= 0; --i) f = fmaf(f, 256.0f, (float)v[i]);
        store_elem(p.out, t * p.ldo + n, p.dtype, f * ta * tb);
    } else {
        if (p.acc) {
            p.acc[t * p.rows + n] = v[0];
            if constexpr (MODE == kGated) p.acc[((int64_t)p.T + t) * p.rows + n] = v[1];
        }
        const float y = (float)v[0] * (ta * s0);
        if constexpr (MODE == kGated)
            store_elem(p.out, t * p.ldo + n, p.dtype, act_value(p.act, y) * ((float)v[1] * (ta * s1)));
        else
            store_elem(p.out, t * p.ldo + n, p.dtype, y + bias);
    }
}

// One 128-channel x nt-token tile per cluster; the CTAs of a cluster split the
// contraction and add their integer sums through distributed shared memory
// (exact, so the split changes no bit).  Every wait is bounded by the global
// timer and records kErrTimeout.
template <int MODE, int P>
__global__ void __launch_bounds__(kTileThreads)
    k_dense_tile(const __grid_constant__ CUtensorMap wmap0, const __grid_constant__ CUtensorMap wmap1,
                 const __grid_constant__ CUtensorMap xmap, const TileParams p) {
    constexpr int kV = MODE == kGated ? 2 : P;         // sums of a result element
    constexpr int kA = MODE == kGated ? 2 : 1;         // weight tiles of a stage
    constexpr int kATile = kTileRows * kStageK;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ctl = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(ctl);
    uint64_t* empty = full + kMaxStages;
    uint64_t* accf = empty + kMaxStages;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(accf + 1);
    RowScale* tok = reinterpret_cast<RowScale*>(ctl + 512);  // [nt] token scales
    uint8_t* sm = ctl + kCtlBytes;

    uint32_t rank, split;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(split));
    const int tile = blockIdx.x / split;
    const int n0 = (tile % p.tiles_n) * kTileRows;
    const int64_t t0 = (int64_t)(tile / p.tiles_n) * p.nt;
    const int nv = (int)min((int64_t)p.nt, p.T - t0);  // tokens of this tile
    const int ks0 = (int)((int64_t)p.steps * rank / split), ks1 = (int)((int64_t)p.steps * (rank + 1) / split);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int btile = P * p.nt * kStageK;  // bytes of a stage's token tile

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(&full[s], p.direct ? 128 : 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(accf, 1);
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, p.tmem_cols);
        tmem_relinquish();
    }
    for (int i = threadIdx.x; i < nv; i += kTileThreads)
        tok[i] = MODE == kGrad ? p.gscale[t0 + i] : RowScale{p.xd[t0 + i], 1.0f};
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        if (lane == 0 && !p.direct) {
            // ---------------- producer ----------------
            tma_prefetch_map(&wmap0);
            if (MODE != kMatmul) tma_prefetch_map(&wmap1);
            tma_prefetch_map(&xmap);
            int s = 0, issued = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int ks = ks0; ks < ks1; ++ks) {
                if (!mbar_wait_ns(&empty[s], ph ^ 1u, kWaitNs)) {
                    ok = false;
                    break;
                }
                mbar_arrive_expect_tx(&full[s], kA * kATile + btile);
                uint8_t* st = sm + s * p.stage_bytes;
                if constexpr (MODE == kGrad) {
                    const int m = ks / p.k_steps, k = (ks - m * p.k_steps) * kStageK;
                    tma_load_2d(st, m ? &wmap1 : &wmap0, n0, k, &full[s]);
#pragma unroll
                    for (int i = 0; i < P; ++i)
                        tma_load_2d(st + kATile + i * p.nt * kStageK, &xmap, (int)(m * p.mat_pitch) + k,
                                    (int)((int64_t)i * p.T + t0), &full[s]);
                } else {
                    tma_load_2d(st, &wmap0, ks * kStageK, n0, &full[s]);
                    if constexpr (MODE == kGated) tma_load_2d(st + kATile, &wmap1, ks * kStageK, n0, &full[s]);
                    tma_load_2d(st + kA * kATile, &xmap, ks * kStageK, (int)t0, &full[s]);
                }
                ++issued;
                if (++s == p.stages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            if (!ok) {
                set_error(&g_dense_error, kErrTimeout);
                // let the copies in flight land before the CTA ends
                for (int i = max(0, issued - p.stages); i < issued; ++i)
                    mbar_wait_ns(&full[i % p.stages], (uint32_t)(i / p.stages) & 1u, kWaitNs);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------- MMA issuer ----------------
        if (lane == 0) {
            int s = 0;
            uint32_t ph = 0;
            bool ok = true;
            const uint32_t idesc = idesc_tile<MODE>(P * p.nt);
            for (int ks = ks0; ks < ks1; ++ks) {
                if (!mbar_wait_short(&full[s], ph, kWaitNs)) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                uint8_t* st = sm + s * p.stage_bytes;
                const uint64_t a0 = MODE == kGrad ? desc_mn128_sw128(st) : desc_k128_sw128(st);
                const uint64_t b0 = desc_k128_sw128(st + kA * kATile);
#pragma unroll
                for (int j = 0; j < kStageK / 32; ++j) {
                    const uint64_t aj = a0 + (MODE == kGrad ? 256 * j : 2 * j);
                    mma_i8(tmem, aj, b0 + 2 * j, idesc, ks > ks0 || j > 0);
                    if constexpr (MODE == kGated)
                        mma_i8(tmem + p.nt, aj + (kATile >> 4), b0 + 2 * j, idesc, ks > ks0 || j > 0);
                }
                mma_commit(&empty[s]);
                if (++s == p.stages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            if (!ok) set_error(&g_dense_error, kErrTimeout);
            mma_commit(accf);
        }
        __syncwarp();
    } else if (p.direct) {
        // ---------------- plain loads (operands off the 16-byte grid) ----------------
        const int tid = threadIdx.x - 64;
        int s = 0;
        uint32_t ph = 0;
        for (int ks = ks0; ks < ks1; ++ks) {
            if (!mbar_wait_ns(&empty[s], ph ^ 1u, kWaitNs)) {
                set_error(&g_dense_error, kErrTimeout);
                break;
            }
            uint8_t* st = sm + s * p.stage_bytes;
            if constexpr (MODE == kGrad) {
                const int m = ks / p.k_steps, k = (ks - m * p.k_steps) * kStageK;
                load_tile_direct(st, p.w[m], p.ldw[m], p.rows, p.cols, k, n0, kTileRows, p.w_unit[m], tid);
                for (int i = 0; i < P; ++i)
                    load_tile_direct(st + kATile + i * p.nt * kStageK, p.x + (int64_t)i * p.T * p.ldx + m * p.mat_pitch,
                                     p.ldx, p.T, p.rows, t0, k, p.nt, p.x_unit, tid);
            } else {
                for (int m = 0; m < kA; ++m)
                    load_tile_direct(st + m * kATile, p.w[m], p.ldw[m], p.rows, p.cols, n0, (int64_t)ks * kStageK,
                                     kTileRows, p.w_unit[m], tid);
                load_tile_direct(st + kA * kATile, p.x, p.ldx, p.T, p.cols, t0, (int64_t)ks * kStageK, p.nt, p.x_unit,
                                 tid);
            }
            fence_proxy_async_smem();
            mbar_arrive(&full[s]);
            if (++s == p.stages) {
                s = 0;
                ph ^= 1u;
            }
        }
        __syncwarp();
    }

    // ---------------- epilogue ----------------
    const int quad = warp & 3, ch = 32 * quad + lane;  // warps 2..5: TMEM lane quarters 2, 3, 0, 1
    const int n = n0 + ch;
    float s0 = 0.0f, s1 = 0.0f, bias = 0.0f;
    int32_t* part = reinterpret_cast<int32_t*>(sm);  // split: [column][128] sums of this CTA
    if (warp >= 2) {
        if constexpr (MODE != kGrad) {
            if (n < p.out_rows) {
                s0 = __ldg(p.s[0] + n);
                if constexpr (MODE == kGated) s1 = __ldg(p.s[1] + n);
                if (MODE == kMatmul && p.bias) bias = __ldg(p.bias + n);
            }
        }
        if (!mbar_wait_ns(accf, 0, kWaitAllNs)) set_error(&g_dense_error, kErrTimeout);
        tc_fence_after_sync();
        const uint32_t tl = tmem + ((uint32_t)(32 * quad) << 16);
        for (int c = 0; c < nv; c += 16) {
            uint32_t r[kV][16];
#pragma unroll
            for (int i = 0; i < kV; ++i) tmem_ld16(tl + i * p.nt + c, r[i]);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                if (split > 1) {
#pragma unroll
                    for (int i = 0; i < kV; ++i) part[(i * p.nt + c + j) * 128 + ch] = (int)r[i][j];
                } else if (c + j < nv && n < p.out_rows) {
                    int v[kV];
#pragma unroll
                    for (int i = 0; i < kV; ++i) v[i] = (int)r[i][j];
                    finish<MODE, P>(p, v, t0 + c + j, n, tok[c + j].a, tok[c + j].b, s0, s1, bias);
                }
            }
        }
    }
    // The accumulators are released before this CTA waits for its peers: no
    // CTA holds TMEM that another needs while it waits.
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 1) tmem_dealloc(tmem, p.tmem_cols);
    if (split > 1) {
        cluster_sync_all();
        if (warp >= 2 && n < p.out_rows) {
            const int per = (nv + (int)split - 1) / (int)split;
            const int c1 = min(nv, (int)(rank + 1) * per);
            for (int c = (int)rank * per; c < c1; ++c) {
                int v[kV];
#pragma unroll
                for (int i = 0; i < kV; ++i) v[i] = 0;
                for (uint32_t q = 0; q < split; ++q)
#pragma unroll
                    for (int i = 0; i < kV; ++i) v[i] += ld_peer(&part[(i * p.nt + c) * 128 + ch], q);
                finish<MODE, P>(p, v, t0 + c, n, tok[c].a, tok[c].b, s0, s1, bias);
            }
        }
        cluster_sync_all();  // the peers have read this CTA's sums
    }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
static int unit_of(const void* p, int64_t ld) {
    const uint64_t b = reinterpret_cast<uintptr_t>(p) | (uint64_t)ld;
    return b % 16 == 0 ? 16 : b % 8 == 0 ? 8 : b % 4 == 0 ? 4 : 1;
}

template <typename K>
static cudaError_t allow_smem(K kernel, bool (&done)[64]) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64 && done[dev]) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, device_info().max_smem_optin);
    if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
    return e;
}

template <int MODE, int P>
static cudaError_t run_tile(const GemmArgs& a, cudaStream_t s) {
    static bool attr_done[64];
    cudaError_t e = allow_smem(k_dense_tile<MODE, P>, attr_done);
    if (e != cudaSuccess) return e;
    constexpr int kA = MODE == kGated ? 2 : 1;
    TileParams p{};
    p.T = a.T;
    p.rows = a.rows;
    p.cols = a.cols;
    p.out_rows = MODE == kGrad ? a.cols : a.rows;
    p.k_steps = ((MODE == kGrad ? a.rows : a.cols) + kStageK - 1) / kStageK;
    p.steps = p.k_steps * (MODE == kGrad ? a.n_mats : 1);
    const int nt_max = P == 3 ? 64 : 128;
    p.nt = a.T <= 16 ? 16 : a.T <= 32 ? 32 : a.T <= 64 ? 64 : nt_max;
    const int cols = (MODE == kGated ? 2 : P) * p.nt;
    p.tmem_cols = cols <= 32 ? 32 : cols <= 64 ? 64 : cols <= 128 ? 128 : 256;
    p.tiles_n = (p.out_rows + kTileRows - 1) / kTileRows;
    const int64_t tiles = (int64_t)p.tiles_n * ((a.T + p.nt - 1) / p.nt);
    const int sms = device_info().sm_count;
    int split = 1;
    if (tiles < sms) {
        split = (int)(sms / tiles);
        split = split > 8 ? 8 : split;
        split = split > p.steps ? p.steps : split;
    }
    if (tiles * split > 0x7FFFFFFF) return cudaErrorInvalidValue;
    p.stage_bytes = kA * kTileRows * kStageK + P * p.nt * kStageK;
    const int per_cta = (p.steps + split - 1) / split;
    const int budget = (tiles * split <= sms ? 200 : 108) * 1024;
    p.stages = budget / p.stage_bytes;
    p.stages = p.stages > kMaxStages ? kMaxStages : p.stages;
    p.stages = p.stages > per_cta ? per_cta : p.stages;
    // Shared memory in proportion to the TMEM columns, so that the CTAs that
    // fit an SM together also find their columns there.
    int smem = p.stages * p.stage_bytes;
    if (split > 1 && smem < cols * 512) smem = cols * 512;
    smem += kCtlBytes + 1024;
    if (smem < 456 * p.tmem_cols - 1024) smem = 456 * p.tmem_cols - 1024;

    p.direct = 0;
    for (int m = 0; m < a.n_mats; ++m) {
        p.w[m] = a.w[m];
        p.ldw[m] = a.ldw[m];
        p.s[m] = a.s[m];
        p.w_unit[m] = unit_of(a.w[m], a.ldw[m]);
        if (p.w_unit[m] < 16) p.direct = 1;
    }
    p.x = reinterpret_cast<const uint8_t*>(a.x);
    p.ldx = a.ldx;
    p.x_unit = unit_of(a.x, a.ldx);
    if (p.x_unit < 16) p.direct = 1;
    p.mat_pitch = a.mat_pitch;
    p.xd = a.xd;
    p.bias = a.bias;
    p.gscale = a.gscale;
    p.out = a.out;
    p.ldo = a.ldo;
    p.acc = a.acc;
    p.act = a.act;
    p.dtype = a.dtype;

    CUtensorMap wm[kMaxMats] = {}, xm = {};
    if (!p.direct) {
        for (int m = 0; m < a.n_mats; ++m) {
            e = encode_2d(&wm[m], a.w[m], CU_TENSOR_MAP_DATA_TYPE_UINT8, a.cols, a.rows, a.ldw[m], kStageK, kTileRows,
                          CU_TENSOR_MAP_SWIZZLE_128B);
            if (e != cudaSuccess) return e;
        }
        if (a.n_mats == 1) wm[1] = wm[0];
        e = encode_2d(&xm, a.x, CU_TENSOR_MAP_DATA_TYPE_UINT8, MODE == kGrad ? a.n_mats * a.mat_pitch : a.cols,
                      (uint64_t)a.planes * a.T, a.ldx, kStageK, p.nt, CU_TENSOR_MAP_SWIZZLE_128B);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * split));
    cfg.blockDim = dim3(kTileThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = split;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_dense_tile<MODE, P>, wm[0], wm[1], xm, p);
}

cudaError_t launch_matmul(const GemmArgs& a, cudaStream_t s) { return run_tile<kMatmul, 1>(a, s); }

cudaError_t launch_gated(const GemmArgs& a, cudaStream_t s) { return run_tile<kGated, 1>(a, s); }

cudaError_t launch_grad_matmul(const GemmArgs& a, cudaStream_t s) {
    return a.planes == 2 ? run_tile<kGrad, 2>(a, s) : run_tile<kGrad, 3>(a, s);
}

cudaError_t read_device_error(cudaStream_t s, int32_t* code) {
    int32_t zero = 0, v = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_dense_error, sizeof(v), 0, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e == cudaSuccess && v) e = cudaMemcpyToSymbolAsync(g_dense_error, &zero, sizeof(zero), 0,
                                                           cudaMemcpyHostToDevice, s);
    if (e == cudaSuccess && v) e = cudaStreamSynchronize(s);
    *code = v;
    return e;
}

}  // namespace dense
}  // namespace moe
