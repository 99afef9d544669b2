// moe_dense_gemm.cu -- the tensor-core products of the dense int8 operators.
//
// Three products, each exact in int32 over its whole contraction:
//   matmul  acc[t, n] = sum_k xq[t, k] w[n, k]
//   gated   the same for two matrices at once, joined by act(g) u
//   grad    dx[t, k]  = sum_n v[t, n] w[n, k] over one or two matrices, v in
//           fixed-point planes; the weight tile is read as it lies in memory
//           (rows of w are the contraction there), so the MMA takes it in its
//           row-transposed form and nothing is ever transposed in memory
// and two kernels: k_dense_tile (a CTA a tile, or a cluster that splits the
// contraction) and k_dense_pair (persistent pairs of CTAs) for larger batches.
// Up to 16 tokens the forward products stream the weights in moe_dense_few.cu.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>
#include <type_traits>

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
constexpr int kTileThreads = 192;    // producer warp, MMA warp, four epilogue warps
constexpr int kDirectThreads = 320;  // with operands off the 16-byte grid: eight warps that load, four of them the epilogue
constexpr int kLoaders = kDirectThreads - 64;
constexpr int kCtlBytes = 2048;    // barriers, the TMEM address, 128 token scales

struct TileParams {
    const uint8_t* w[kMaxMats];
    int64_t ldw[kMaxMats];
    const uint8_t* x;
    int64_t ldx;
    int64_t mat_pitch, x_rows;
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
    int quad;       // results and sums may be stored four at a time
    int direct;     // operands that TMA cannot take: loads by the epilogue warps
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

// Asynchronous copy of up to BYTES bytes (n of them; the rest is zero-filled).
template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, int n) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(n)
                     : "memory");
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// At most `ahead` (0, 1 or 2) of this thread's groups still on their way.
__device__ __forceinline__ void cp_async_wait(int ahead) {
    if (ahead == 0)
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    else if (ahead == 1)
        asm volatile("cp.async.wait_group 1;" ::: "memory");
    else
        asm volatile("cp.async.wait_group 2;" ::: "memory");
}

template <int UNIT>
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* row, int64_t c, int left) {
#pragma unroll
    for (int i = 0; i < 16; i += UNIT) {
        const int n = min(max(left - i, 0), UNIT);
        cp_async<UNIT>(dst + i, n > 0 ? row + c + i : row, n);
    }
}

// A tile of n rows of 128 bytes at (row0, col0) of [rows][cols] into the
// 128-byte-swizzle layout, by kLoaders threads (32 rows a pass); bytes outside read
// as zero.  Rows on a 16-, 8- or 4-byte grid are copied asynchronously (the
// caller commits and waits); others are put together from aligned words, four
// passes of loads under way at a time.
__device__ __forceinline__ void load_tile_direct(uint8_t* tile, const uint8_t* base, int64_t ld, int64_t rows,
                                                 int64_t cols, int64_t row0, int64_t col0, int n, int unit, int tid) {
    const int c = tid & 7;
    const int64_t col = col0 + 16 * c;
    const int in_row = (int)min((int64_t)16, max((int64_t)0, cols - col));  // bytes of the chunk inside the row
    if (unit >= 4) {
        for (int r = tid >> 3; r < n; r += kLoaders / 8) {
            const bool ok = row0 + r < rows;
            const uint8_t* row = base + (ok ? row0 + r : 0) * ld;
            const uint32_t dst = smem_addr(tile + sw128_chunk(r, c));
            const int left = ok ? in_row : 0;
            if (unit == 16)
                copy16<16>(dst, row, col, left);
            else if (unit == 8)
                copy16<8>(dst, row, col, left);
            else
                copy16<4>(dst, row, col, left);
        }
        return;
    }
    for (int r0 = tid >> 3; r0 < n; r0 += kLoaders / 2) {
        Words w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int r = r0 + kLoaders / 8 * k;
            const bool ok = r < n && row0 + r < rows;
            w[k] = load_words(base + (ok ? row0 + r : 0) * ld + col, ok ? in_row : 0);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int r = r0 + kLoaders / 8 * k;
            if (r < n) *reinterpret_cast<uint4*>(tile + sw128_chunk(r, c)) = join_words(w[k]);
        }
    }
}

__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Four sums of the CTA `rank` of the cluster, at this CTA's address p.
__device__ __forceinline__ int4 ld_peer(const int32_t* p, uint32_t rank) {
    uint32_t a;
    int4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}

// TMEM words as the integers they are.
template <int N>
__device__ __forceinline__ uint32_t (&as_words(int (&v)[N]))[N] {
    return reinterpret_cast<uint32_t(&)[N]>(v);
}

// Accumulator column of sum i of a tile's token c (a multiple of 16; the next 15
// follow): the gradient's planes alternate every 16 tokens, the gated block's
// two projections lie nt apart.
template <int MODE, int P>
__device__ __forceinline__ int sum_col(int i, int c, int nt) {
    return MODE == kGrad ? c * P + kPlaneGroup * i : i * nt + c;
}

// Where a product's results go, for lanes that are channels.
struct ChannelOut {
    void* out;
    int64_t ldo;
    int32_t* acc;
    int64_t acc_pitch;  // gated: from the gate's sums to the up projection's
    int rows;           // row length of acc
    int act;
};

// A result from its integer sums v[.][j] (gated: gate and up; gradient: the
// planes) and scales: the token's, the channel's, the bias.
template <int MODE, int P, int ACT, int N>
__device__ __forceinline__ float join(const int (&v)[MODE == kGated ? 2 : P][N], int j, const RowScale tok, float s0,
                                      float s1, float bias) {
    if constexpr (MODE == kGrad) {
        // digits joined in fp32: each plane's sum rounds by 2^-24 of itself
        float d = (float)v[P - 1][j];
#pragma unroll
        for (int i = P - 2; i >= 0; --i) d = fmaf(d, 256.0f, (float)v[i][j]);
        return d * tok.a * tok.b;
    } else if constexpr (MODE == kGated) {
        return act_value<ACT>((float)v[0][j] * (tok.a * s0)) * ((float)v[1][j] * (tok.a * s1));
    } else {
        return (float)v[0][j] * (tok.a * s0) + bias;
    }
}

// The results of one channel n for up to N consecutive tokens t ..: `v` are the
// integer sums (gated: gate and up; gradient: planes), `ts` the tokens' scales
// (16-byte aligned).  All values are formed before the first store, so that the
// columns' arithmetic overlaps; a warp's stores run along the tokens' rows.
template <int MODE, int P, typename OT, int N>
__device__ __forceinline__ void emit_channel(const ChannelOut& o, const int (&v)[MODE == kGated ? 2 : P][N], int64_t t,
                                             int n, int valid, const RowScale* ts, float s0, float s1, float bias) {
    float f[N];
    with_act(MODE == kGated ? o.act : MOE_ACT_SILU, [&](auto act) {
        constexpr int A = decltype(act)::value;
#pragma unroll
        for (int j = 0; j < N; j += 2) {
            const float4 sc = *reinterpret_cast<const float4*>(ts + j);
            f[j] = join<MODE, P, A, N>(v, j, RowScale{sc.x, sc.y}, s0, s1, bias);
            f[j + 1] = join<MODE, P, A, N>(v, j + 1, RowScale{sc.z, sc.w}, s0, s1, bias);
        }
    });
    OT* out = static_cast<OT*>(o.out) + t * o.ldo + n;
    if (valid >= N) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            *out = from_f32<OT>(f[j]);
            out += o.ldo;
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if (j < valid) *out = from_f32<OT>(f[j]);
            out += o.ldo;
        }
    }
    if (MODE != kGrad && o.acc) {
#pragma unroll
        for (int m = 0; m < (MODE == kGated ? 2 : 1); ++m) {
            int32_t* acc = o.acc + m * o.acc_pitch + t * o.rows + n;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                if (j < valid) *acc = v[m][j];
                acc += o.rows;
            }
        }
    }
}

// One 128-channel x nt-token tile per cluster; the CTAs of a cluster split the
// contraction and add their integer sums through distributed shared memory
// (exact, so the split changes no bit).  Every wait is bounded by the global
// timer and records kErrTimeout.  Bound by latency: the ring's fill, the tile's
// epilogue and the cluster's barriers (333 x 1008 x 784: 5.8 us; with rows of 1000
// codes, loaded by threads, 8.9).
template <int MODE, int P, typename OT>
__global__ void __launch_bounds__(kDirectThreads)
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
            mbar_init(&full[s], p.direct ? kLoaders : 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(accf, 1);
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, p.tmem_cols);
        tmem_relinquish();
    }
    pdl_wait();
    pdl_launch_dependents();
    for (int i = threadIdx.x; i < p.nt; i += blockDim.x)
        tok[i] = i >= nv ? RowScale{0.0f, 0.0f} : MODE == kGrad ? p.gscale[t0 + i] : RowScale{p.xd[t0 + i], 1.0f};
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
                    tma_load_2d(st + kATile, &xmap, (int)(m * p.mat_pitch) + k, (int)t0 * P, &full[s]);
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
        // ---------------- operands off the 16-byte grid ----------------
        // Stage it's copies are left on their way while the next `ahead` are
        // issued; then they are waited for, made visible to the tensor core
        // and announced.
        const int tid = threadIdx.x - 64, n_st = ks1 - ks0;
        const int ahead = min(2, p.stages - 1);
        for (int it = 0; it < n_st + ahead; ++it) {
            if (it < n_st) {
                const int ks = ks0 + it, s = it % p.stages;
                if (!mbar_wait_ns(&empty[s], ((uint32_t)(it / p.stages) & 1u) ^ 1u, kWaitNs)) {
                    set_error(&g_dense_error, kErrTimeout);
                    break;
                }
                uint8_t* st = sm + s * p.stage_bytes;
                if constexpr (MODE == kGrad) {
                    const int m = ks / p.k_steps, k = (ks - m * p.k_steps) * kStageK;
                    load_tile_direct(st, p.w[m], p.ldw[m], p.rows, p.cols, k, n0, kTileRows, p.w_unit[m], tid);
                    load_tile_direct(st + kATile, p.x + m * p.mat_pitch, p.ldx, p.x_rows, p.rows, t0 * P, k, P * p.nt,
                                     p.x_unit, tid);
                } else {
                    for (int m = 0; m < kA; ++m)
                        load_tile_direct(st + m * kATile, p.w[m], p.ldw[m], p.rows, p.cols, n0, (int64_t)ks * kStageK,
                                         kTileRows, p.w_unit[m], tid);
                    load_tile_direct(st + kA * kATile, p.x, p.ldx, p.x_rows, p.cols, t0, (int64_t)ks * kStageK, p.nt,
                                     p.x_unit, tid);
                }
            }
            cp_async_commit();  // (an empty group after the last stage)
            if (it >= ahead) {
                cp_async_wait(ahead);
                fence_proxy_async_smem();
                mbar_arrive(&full[(it - ahead) % p.stages]);
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
    }

    // ---------------- epilogue ----------------
    const int quad = warp & 3, ch = 32 * quad + lane;  // warps 2..5: TMEM lane quarters 2, 3, 0, 1
    const int n = n0 + ch;
    float s0 = 0.0f, s1 = 0.0f, bias = 0.0f;
    int32_t* part = reinterpret_cast<int32_t*>(sm);  // split: [column][128] sums of this CTA
    const ChannelOut co{p.out, p.ldo, p.acc, (int64_t)p.T * p.rows, p.rows, p.act};
    if (warp >= 2 && warp < 6) {
        if constexpr (MODE != kGrad) {
            if (n < p.out_rows) {
                s0 = p.s[0][n];
                if constexpr (MODE == kGated) s1 = p.s[1][n];
                if (MODE == kMatmul && p.bias) bias = p.bias[n];
            }
        }
        if (!mbar_wait_ns(accf, 0, kWaitAllNs)) set_error(&g_dense_error, kErrTimeout);
        tc_fence_after_sync();
        const uint32_t tl = tmem + ((uint32_t)(32 * quad) << 16);
        for (int c = 0; c < nv; c += 16) {
            int r[kV][16];
#pragma unroll
            for (int i = 0; i < kV; ++i) tmem_ld16(tl + sum_col<MODE, P>(i, c, p.nt), as_words(r[i]));
            tmem_wait_ld();
            if (split > 1) {
#pragma unroll
                for (int j = 0; j < 16; ++j)
#pragma unroll
                    for (int i = 0; i < kV; ++i) part[(sum_col<MODE, P>(i, c, p.nt) + j) * 128 + ch] = r[i][j];
            } else if (n < p.out_rows) {
                emit_channel<MODE, P, OT, 16>(co, r, t0 + c, n, nv - c, tok + c, s0, s1, bias);
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
        // The tokens are dealt to the CTAs, a CTA's to its warps; a lane joins
        // four channels, every peer's sums of them under way together.
        const int nq = n0 + 4 * lane;
        float sq[2][4] = {}, bq[4] = {};
        if constexpr (MODE != kGrad) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (nq + k < p.out_rows) {
                    sq[0][k] = p.s[0][nq + k];
                    if constexpr (MODE == kGated) sq[1][k] = p.s[1][nq + k];
                    if (MODE == kMatmul && p.bias) bq[k] = p.bias[nq + k];
                }
        }
        for (int c = (int)rank + (int)split * warp; c < nv; c += (int)split * (int)(blockDim.x / 32)) {
            int4 w[8][kV];
#pragma unroll
            for (uint32_t q = 0; q < 8; ++q)
#pragma unroll
                for (int i = 0; i < kV; ++i)
                    w[q][i] = q < split ? ld_peer(&part[(sum_col<MODE, P>(i, c & ~15, p.nt) + (c & 15)) * 128 + 4 * lane], q) : make_int4(0, 0, 0, 0);
            int v[kV][4];
#pragma unroll
            for (int i = 0; i < kV; ++i) {
                v[i][0] = v[i][1] = v[i][2] = v[i][3] = 0;
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    v[i][0] += w[q][i].x;
                    v[i][1] += w[q][i].y;
                    v[i][2] += w[q][i].z;
                    v[i][3] += w[q][i].w;
                }
            }
            const RowScale sc = tok[c];
            const int64_t t = t0 + c;
            alignas(16) OT o[4];
            with_act(MODE == kGated ? p.act : MOE_ACT_SILU, [&](auto act) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    o[k] = from_f32<OT>(join<MODE, P, decltype(act)::value>(v, k, sc, sq[0][k], sq[1][k], bq[k]));
            });
            OT* out = static_cast<OT*>(p.out) + t * p.ldo + nq;
            if (p.quad && nq + 4 <= p.out_rows) {
                if constexpr (sizeof(OT) == 4)
                    *reinterpret_cast<uint4*>(out) = *reinterpret_cast<const uint4*>(o);
                else
                    *reinterpret_cast<uint2*>(out) = *reinterpret_cast<const uint2*>(o);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (nq + k < p.out_rows) out[k] = o[k];
            }
            if (MODE != kGrad && p.acc) {
#pragma unroll
                for (int m = 0; m < (MODE == kGated ? 2 : 1); ++m) {
                    int32_t* acc = p.acc + (m * (int64_t)p.T + t) * p.rows + nq;
                    if (p.quad && nq + 4 <= p.out_rows) {
                        *reinterpret_cast<int4*>(acc) = make_int4(v[m][0], v[m][1], v[m][2], v[m][3]);
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (nq + k < p.out_rows) acc[k] = v[m][k];
                    }
                }
            }
        }
        cluster_sync_all();  // the peers have read this CTA's sums
    }
}

// ---------------------------------------------------------------------------
// Large batches: CTA pairs, one 256-row MMA over both SMs' shared memory
// ---------------------------------------------------------------------------
// A pair of CTAs (cluster of two) works on tiles of 256 x n columns: each CTA
// holds 128 rows of the MMA's first operand and half of the second operand's
// rows, so a stage of 128 codes moves 32 KB a CTA for 128 x 256 x 128 products:
// half of what a CTA alone would load and read for them.  The CTAs are
// persistent (tiles pair, pair + pairs, ...), and the accumulator is doubled,
// so a tile's epilogue runs under the next tile's products.
//   matmul, grad: rows = 256 channels, columns = tokens (times planes): a lane
//     is a channel, and a warp's stores run along a token's row
//   gated: rows = 256 tokens, columns = 128 gate and 128 up channels (one half
//     from each CTA), so that a lane holds a token's g and u of one channel
// Bound by the tensor pipe and the power limit: 4096 x 6144 x 6144 (bf16 results)
// 97 us, 3.19 POP/s, the pipe busy in 78 % of all cycles at 1.65 GHz; gated 4096 x
// 6144 x 2048 66 us, 3.12 POP/s, 72 %; the rest is the last round's remainder and
// the last tile's epilogue.
constexpr int kPairThreads = 320;  // producer warp, MMA warp, eight epilogue warps
// (the gated kernel gives a stage's room to its epilogue's staging)
template <int MODE>
constexpr int kPairStages = MODE == kGated ? 5 : 6;
constexpr int kStageWarp = 32 * 144;  // a warp's staging: 32 rows of 128 bytes, padded
constexpr int kPairCtl = 1024 + 8 * 2 * 128 * 8;  // barriers; each epilogue warp's scales of two tiles' columns
template <int MODE>
constexpr int kPairSmem = kPairStages<MODE> * 2 * kTileBytes + kPairCtl + 1024 + (MODE == kGated ? 8 * kStageWarp : 0);
constexpr int kPairRows = 256;

// Tensor maps: a: the 256-row operand (grad: one a matrix), b: the column
// operand (gated: one a CTA), small: the same in boxes for the parts of a tile.
struct PairMaps {
    CUtensorMap a[2], b[2], small[2];
};

struct PairParams {
    const float* xd;
    const float* s[kMaxMats];
    const float* bias;
    const RowScale* gscale;
    void* out;
    int64_t ldo;
    int32_t* acc;
    int64_t mat_pitch;
    int T, rows, out_rows;
    int k_steps, steps;
    int nt;            // matmul, grad: tokens of a tile; gated: channels of a tile
    int tiles_r;       // tiles along the 256 rows
    int64_t whole;     // tiles worked on whole
    int parts;         // column parts of each tile after those
    int64_t units;     // whole tiles and parts
    int act, dtype;
    int vec;           // gated: results and sums may be stored 16 bytes at a time
};

__device__ __forceinline__ uint32_t map_rank(const void* p, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    return a;
}

// A box into this CTA's shared memory, completing on a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, "
        "%3}], [%4];" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void mma_i8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
}

// Arrive on the barrier at this offset in both CTAs when the MMAs issued so far are done.
__device__ __forceinline__ void mma_commit_pair(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_addr(bar)),
        "h"((uint16_t)3)
        : "memory");
}

__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Bounded wait on a barrier that the other CTA arrives on too.
__device__ __forceinline__ bool wait_cluster(uint64_t* bar, uint32_t parity, uint64_t budget_ns) {
    uint64_t t0 = 0;
    for (uint32_t i = 0;; ++i) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_addr(bar)), "r"(parity), "r"(64u)
            : "memory");
        if (ok) return true;
        if ((i & 255u) == 0) {
            const uint64_t t = global_timer_ns();
            if (i == 0)
                t0 = t;
            else if (t - t0 > budget_ns)
                return false;
        }
    }
}

// A unit of work: rows r0 .. r0 + 255, nt columns from c0.
struct PairUnit {
    int64_t r0, c0;
    int nt;
    bool part;
};

__device__ __forceinline__ PairUnit pair_unit(const PairParams& p, int64_t u) {
    const bool part = u >= p.whole;
    const int64_t tile = part ? p.whole + (u - p.whole) / p.parts : u;
    const int nt = part ? p.nt / p.parts : p.nt;
    const int64_t sub = part ? (u - p.whole) % p.parts : 0;
    return PairUnit{tile % p.tiles_r * kPairRows, tile / p.tiles_r * p.nt + sub * nt, nt, part};
}

// 32 consecutive 32-bit columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr)
        : "memory");
}

// 32 values of each of a warp's 32 rows (a lane holds its row's columns n ..
// n + 31) to rows t0 .. of [T][N] at n, through the warp's staging buffer: a row
// is written by 32 * sizeof(V) / 16 neighbouring lanes, 16 bytes each, where out,
// N and ld are multiples of that (vec), and by 32 lanes an element each elsewhere.
// (Each lane storing its own odd row took 97 us in place of 38 at 2000 x 2049 x
// 3001, gated.)
template <typename V, typename W>
__device__ __forceinline__ void store_rows32(V* out, int64_t ld, int64_t T, int N, int64_t t0, int n,
                                             const W (&v)[32], int vec, uint8_t* stage, int lane) {
    static_assert(sizeof(V) == sizeof(W), "the same elements");
    constexpr int kPieces = 32 * (int)sizeof(V) / 16, kPitch = 16 * kPieces + 16, kEach = 16 / (int)sizeof(V);
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
        *reinterpret_cast<uint4*>(stage + lane * kPitch + 16 * i) = reinterpret_cast<const uint4*>(v)[i];
    __syncwarp();
    if (vec) {
        const int piece = lane % kPieces;
        const bool in = n + (piece + 1) * kEach <= N;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int row = i * (32 / kPieces) + lane / kPieces;
            const uint4 w = *reinterpret_cast<const uint4*>(stage + row * kPitch + 16 * piece);
            if (in && t0 + row < T) *reinterpret_cast<uint4*>(out + (t0 + row) * ld + n + piece * kEach) = w;
        }
    } else if (n + lane < N) {
        const int nr = (int)(T - t0 < 32 ? T - t0 : 32);
        V* o = out + t0 * ld + n + lane;
#pragma unroll 8
        for (int row = 0; row < nr; ++row, o += ld)
            *o = *reinterpret_cast<const V*>(stage + row * kPitch + lane * (int)sizeof(V));
    }
    __syncwarp();
}

template <int MODE, int P, typename OT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    k_dense_pair(const __grid_constant__ PairMaps maps, const PairParams p) {
    constexpr int kStages = kPairStages<MODE>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* ctl = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(ctl);
    uint64_t* empty = full + kStages;
    uint64_t* accf = empty + kStages;  // [2]
    uint64_t* acce = accf + 2;             // [2]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acce + 2);
    uint8_t* sm = ctl + kPairCtl;
    constexpr int kStage = 2 * kTileBytes;

    uint32_t rank;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kCols = MODE == kGated ? 2 : P;  // the MMA's columns for each of a unit's
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&accf[b], 1);
            mbar_init(&acce[b], 16);  // the epilogue warps of both CTAs
        }
        fence_barrier_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)),
                     "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before_sync();
    cluster_sync_all();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    pdl_launch_dependents();

    if (warp == 0) {
        if (lane == 0) {
            // ---------------- producer (both CTAs) ----------------
            const CUtensorMap* bw = &maps.b[MODE == kGated ? rank : 0];
            const CUtensorMap* bs = &maps.small[MODE == kGated ? rank : 0];
            tma_prefetch_map(&maps.a[0]);
            if (MODE == kGrad) tma_prefetch_map(&maps.a[1]);
            tma_prefetch_map(bw);
            tma_prefetch_map(bs);
            int s = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int64_t unit = pair; ok && unit < p.units; unit += pairs) {
                const PairUnit u = pair_unit(p, unit);
                const int r0 = (int)u.r0 + 128 * rank;
                const CUtensorMap* bm = u.part ? bs : bw;
                // this CTA's half of the columns: token rows (planes: P for a token), or its own weight's
                const int c0 = (int)u.c0 * P + (MODE == kGated ? 0 : (int)rank * (P * u.nt / 2));
                const uint32_t tx = 2 * (kTileBytes + kCols * u.nt / 2 * kStageK);  // both CTAs' boxes
                for (int ks = 0; ks < p.steps; ++ks) {
                    if (!wait_cluster(&empty[s], ph ^ 1u, kWaitNs)) {
                        ok = false;
                        break;
                    }
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], tx);
                    const uint32_t bar = map_rank(&full[s], 0);
                    uint8_t* st = sm + s * kStage;
                    if constexpr (MODE == kGrad) {
                        const int m = ks / p.k_steps, k = (ks - m * p.k_steps) * kStageK;
                        tma_load_2d_pair(st, &maps.a[m], r0, k, bar);
                        tma_load_2d_pair(st + kTileBytes, bm, (int)(m * p.mat_pitch) + k, c0, bar);
                    } else {
                        tma_load_2d_pair(st, &maps.a[0], ks * kStageK, r0, bar);
                        tma_load_2d_pair(st + kTileBytes, bm, ks * kStageK, c0, bar);
                    }
                    if (++s == kStages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            if (!ok) set_error(&g_dense_error, kErrTimeout);
            // every box has been consumed before the CTA ends
            for (int i = 0; i < kStages; ++i) {
                if (!wait_cluster(&empty[s], ph ^ 1u, kWaitNs)) {
                    set_error(&g_dense_error, kErrTimeout);
                    break;
                }
                if (++s == kStages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            // ---------------- MMA issuer (the pair's first CTA) ----------------
            int s = 0;
            uint32_t ph = 0;
            bool ok = true;
            int nu = 0;
            for (int64_t unit = pair; ok && unit < p.units; unit += pairs, ++nu) {
                const int buf = nu & 1;
                const uint32_t idesc = (idesc_tile<MODE>(kCols * pair_unit(p, unit).nt) & ~(31u << 24)) |
                                       ((uint32_t)(kPairRows >> 4) << 24);
                if (nu >= 2 && !wait_cluster(&acce[buf], ((nu >> 1) - 1) & 1, kWaitNs)) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const uint32_t d = tmem + 256 * buf;
                for (int ks = 0; ks < p.steps; ++ks) {
                    if (!wait_cluster(&full[s], ph, kWaitNs)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    uint8_t* st = sm + s * kStage;
                    const uint64_t a0 = MODE == kGrad ? desc_mn128_sw128(st) : desc_k128_sw128(st);
                    const uint64_t b0 = desc_k128_sw128(st + kTileBytes);
#pragma unroll
                    for (int j = 0; j < kStageK / 32; ++j)
                        mma_i8_pair(d, a0 + (MODE == kGrad ? 256 * j : 2 * j), b0 + 2 * j, idesc, ks > 0 || j > 0);
                    mma_commit_pair(&empty[s]);
                    if (++s == kStages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                mma_commit_pair(&accf[buf]);
            }
            if (!ok) set_error(&g_dense_error, kErrTimeout);
        }
        __syncwarp();
    } else {
        // ---------------- epilogue: two warps a TMEM lane quarter, half of the columns each ----------------
        const int quad = warp & 3, row = 32 * quad + lane, half = (warp - 2) >> 2;
        // a copy for each warp: the epilogue warps never wait for one another
        RowScale* tok = reinterpret_cast<RowScale*>(ctl + 1024) + (warp - 2) * 256;
        const ChannelOut co{p.out, p.ldo, p.acc, (int64_t)p.T * p.rows, p.rows, p.act};
        int nu = 0;
        for (int64_t unit = pair; unit < p.units; unit += pairs, ++nu) {
            const int buf = nu & 1;
            const PairUnit un = pair_unit(p, unit);
            const int cols = un.nt / 2;  // this warp's columns: cols from c0 on
            const int64_t r0 = un.r0 + 128 * rank + row, c0 = un.c0 + half * cols;
            RowScale* ts = tok + 128 * buf;
            for (int i = lane; i < cols; i += 32) {
                RowScale sc{0.0f, 0.0f};
                if constexpr (MODE == kGated) {
                    if (c0 + i < p.rows) sc = RowScale{p.s[0][c0 + i], p.s[1][c0 + i]};
                } else {
                    if (c0 + i < p.T) sc = MODE == kGrad ? p.gscale[c0 + i] : RowScale{p.xd[c0 + i], 1.0f};
                }
                ts[i] = sc;
            }
            float sa = 0.0f, bias = 0.0f;
            if constexpr (MODE == kGated) {
                if (r0 < p.T) sa = p.xd[r0];
            } else if constexpr (MODE == kMatmul) {
                if (r0 < p.out_rows) {
                    sa = p.s[0][r0];
                    if (p.bias) bias = p.bias[r0];
                }
            }
            __syncwarp();
            // (a whole warp gives up together)
            if (!__all_sync(kFull, wait_cluster(&accf[buf], (uint32_t)(nu >> 1) & 1u, kWaitAllNs))) {
                set_error(&g_dense_error, kErrTimeout);
                break;
            }
            tc_fence_after_sync();
            const uint32_t tl = tmem + ((uint32_t)(32 * quad) << 16) + 256 * buf + half * cols * P;
            if constexpr (MODE == kGated) {
                // 32 channels at a time, turned in shared memory so that the stores run
                // along the tokens' rows.  A unit of 16 channels computes 16 idle ones: a
                // form of its own saved 0.9 of 11.4 us at 333 x 1000 x 777 and doubled
                // this code.
                uint8_t* stage = sm + kStages * kStage + (warp - 2) * kStageWarp;
                const int64_t t0 = r0 - lane;
                const int end = (int)min((int64_t)p.rows, c0 + cols);
                for (int c = 0; c < cols; c += 32) {
                    uint32_t g[32], u[32];
                    tmem_ld32(tl + c, g);
                    tmem_ld32(tl + un.nt + c, u);
                    tmem_wait_ld();
                    const int n = (int)c0 + c;
                    if (p.acc) {
                        store_rows32(p.acc, p.rows, p.T, end, t0, n, g, p.vec, stage, lane);
                        store_rows32(p.acc + p.T * (int64_t)p.rows, p.rows, p.T, end, t0, n, u, p.vec, stage, lane);
                    }
                    alignas(16) OT h[32];
                    with_act(p.act, [&](auto act) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            const RowScale sc = ts[c + j];
                            h[j] = from_f32<OT>(act_value<decltype(act)::value>((float)(int)g[j] * (sa * sc.a)) *
                                                ((float)(int)u[j] * (sa * sc.b)));
                        }
                    });
                    store_rows32(static_cast<OT*>(p.out), p.ldo, p.T, end, t0, n, h, p.vec, stage, lane);
                }
            } else {
                const int nv = (int)min((int64_t)cols, p.T - c0);
                for (int c = 0; c < nv; c += 16) {
                    int v[P][16];
#pragma unroll
                    for (int i = 0; i < P; ++i) tmem_ld16(tl + sum_col<MODE, P>(i, c, un.nt), as_words(v[i]));
                    tmem_wait_ld();
                    if (r0 < p.out_rows)
                        emit_channel<MODE, P, OT, 16>(co, v, c0 + c, (int)r0, nv - c, ts + c, sa, 0.0f, bias);
                }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) arrive_cluster(map_rank(&acce[buf], 0));
        }
    }
    tc_fence_before_sync();
    cluster_sync_all();  // neither CTA ends while the other's MMAs or arrivals may still reach it
    tc_fence_after_sync();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
// [two][split]: clusters of `split` CTAs that run at once, with one or two CTAs on an SM (the
// GPU's clusters do not cover all of its SMs: of 148, clusters of 8 with a CTA
// on each SM use 120).
using ClusterTable = int[2][9];

static const ClusterTable& clusters_at_once() {
    static ClusterTable table[64];
    static std::once_flag once[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) dev = 0;
    std::call_once(once[dev], [&] {
        auto* kernel = k_dense_tile<kMatmul, 1, float>;
        static bool done[64];
        const bool ok = allow_smem(kernel, done) == cudaSuccess;
        for (int t = 0; t < 2; ++t)
            for (int c = 1; c <= 8; ++c) {
                cudaLaunchConfig_t cfg = {};
                cfg.gridDim = dim3(c * 1024);
                cfg.blockDim = dim3(kTileThreads);
                cfg.dynamicSmemBytes = (t ? 112 : 200) * 1024;
                cudaLaunchAttribute at[1];
                at[0].id = cudaLaunchAttributeClusterDimension;
                at[0].val.clusterDim.x = c;
                at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
                cfg.attrs = at;
                cfg.numAttrs = 1;
                int n = 0;
                if (!ok || cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1)
                    n = (t ? 2 : 1) * (device_info().sm_count * 4 / 5 / c);
                table[dev][t][c] = n < 1 ? 1 : n;
            }
    });
    return table[dev];
}

struct TilePlan {
    int nt, split, stages, smem;
    double us;  // estimate
};

// Tokens of a tile and CTAs of a tile's contraction.  A stage takes about 0.16
// us (gated 0.3, gradient 0.24) whatever its tokens (it is the latency of what
// is under way), a tile's end by its columns, the launch and the first loads 5, and with a split the sums' way through shared memory; what
// does not fit at once runs in rounds.  With 128 tokens, 6144 codes and 2048
// channels: 64 tokens by 4 CTAs 9.3 us, 128 by 1 17.6 us, 128 by 8 11.4 us, 16
// by 4 17.1 us.
template <int MODE, int P>
static TilePlan plan_tile(int T, int tiles_n, int steps) {
    constexpr int kA = MODE == kGated ? 2 : 1, kV = MODE == kGated ? 2 : P;
    const int sms = device_info().sm_count;
    const ClusterTable& fit = clusters_at_once();
    TilePlan best{};
    double least = 1e30;
    for (int nt = 16; nt <= (MODE == kGrad ? 64 : 128); nt *= 2) {
        const int64_t tiles = (int64_t)tiles_n * ((T + nt - 1) / nt);
        const int cols = kV * nt, stage = kA * kTileRows * kStageK + P * nt * kStageK;
        const int tmem = cols <= 32 ? 32 : cols <= 64 ? 64 : cols <= 128 ? 128 : 256;
        for (int split : {1, 2, 3, 4, 6, 8}) {
            if (split > steps) break;
            const int per_cta = (steps + split - 1) / split;
            int stages = 108 * 1024 / stage;
            stages = stages > kMaxStages ? kMaxStages : stages;
            stages = stages > per_cta ? per_cta : stages;
            // Shared memory in proportion to the TMEM columns, so that the CTAs
            // that fit an SM together also find their columns there.
            int smem = stages * stage;
            if (split > 1 && smem < cols * 512) smem = cols * 512;
            smem += kCtlBytes + 1024;
            if (smem < 456 * tmem - 1024) smem = 456 * tmem - 1024;
            const int at_once = fit[smem <= 112 * 1024][split];
            const int64_t rounds = (tiles + at_once - 1) / at_once;
            const double ctas = (double)(tiles < at_once ? tiles : at_once) * split;
            const double share = ctas > sms ? ctas / sms : 1.0;  // CTAs that share an SM
            const double k = kV == 1 ? 1.0 : kV == 2 ? 1.7 : kV == 3 ? 2.4 : 3.1;
            const double end = split == 1 ? 1.5 + 0.023 * nt * k : 0.3 + (0.016 + 0.045 / split) * nt * k;
            const double stage_us = MODE == kGated ? 0.3 : MODE == kGrad ? 0.24 : 0.16;
            const double us = 5.0 + rounds * share * (per_cta * stage_us + end);
            if (us < least) {
                least = us;
                best = TilePlan{nt, split, stages, smem, us};
            }
        }
    }
    return best;
}

// Rows of the token operand.
template <int MODE, int P>
static int64_t plane_rows_of(const GemmArgs& a) {
    return MODE == kGrad ? plane_rows(P, a.T) : a.T;
}

template <int MODE, int P, typename OT>
static cudaError_t run_tile(const GemmArgs& a, const TilePlan& plan, cudaStream_t s) {
    static bool attr_done[64];
    cudaError_t e = allow_smem(k_dense_tile<MODE, P, OT>, attr_done);
    if (e != cudaSuccess) return e;
    constexpr int kA = MODE == kGated ? 2 : 1;
    TileParams p{};
    p.T = a.T;
    p.rows = a.rows;
    p.cols = a.cols;
    p.out_rows = MODE == kGrad ? a.cols : a.rows;
    p.k_steps = ((MODE == kGrad ? a.rows : a.cols) + kStageK - 1) / kStageK;
    p.steps = p.k_steps * (MODE == kGrad ? a.n_mats : 1);
    p.tiles_n = (p.out_rows + kTileRows - 1) / kTileRows;
    const int split = plan.split, smem = plan.smem;
    p.nt = plan.nt;
    p.stages = plan.stages;
    const int cols = (MODE == kGated ? 2 : P) * p.nt;
    p.tmem_cols = cols <= 32 ? 32 : cols <= 64 ? 64 : cols <= 128 ? 128 : 256;
    p.stage_bytes = kA * kTileRows * kStageK + P * p.nt * kStageK;
    const int64_t tiles = (int64_t)p.tiles_n * ((a.T + p.nt - 1) / p.nt);
    if (tiles * split > 0x7FFFFFFF) return cudaErrorInvalidValue;
    p.quad = reinterpret_cast<uintptr_t>(a.out) % (4 * sizeof(OT)) == 0 && a.ldo % 4 == 0 &&
             (!a.acc || (reinterpret_cast<uintptr_t>(a.acc) % 16 == 0 && a.rows % 4 == 0));
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
    p.x_rows = plane_rows_of<MODE, P>(a);
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
                      p.x_rows, a.ldx, kStageK, P * p.nt, CU_TENSOR_MAP_SWIZZLE_128B);
        if (e != cudaSuccess) return e;
    }
    return launch_dense(k_dense_tile<MODE, P, OT>, (unsigned)(tiles * split),
                        p.direct ? kDirectThreads : kTileThreads, smem, split, s, wm[0], wm[1], xm, p);
}

// Columns of a pair's tile (channels of the gated block, tokens elsewhere).
template <int MODE, int P>
constexpr int pair_columns = MODE == kGated ? 128 : MODE == kMatmul ? 256 : 64;

struct PairPlan {
    int tiles_r, parts;
    int64_t whole, units;
    double us;  // estimate
};

// The tiles after the last full round of the pairs are cut into column parts
// where that ends sooner: a stage takes 0.27 us of a whole tile, 0.24 of a half
// and 0.235 of a quarter (by then it is latency), the last epilogue 4, 1.5 and 1.
template <int MODE, int P>
static PairPlan plan_pair(int T, int out_rows, int steps) {
    constexpr int nt = pair_columns<MODE, P>;
    const int64_t pairs = device_info().sm_count / 2;
    PairPlan p;
    p.tiles_r = ((MODE == kGated ? T : out_rows) + kPairRows - 1) / kPairRows;
    const int64_t tiles = (int64_t)p.tiles_r * (((MODE == kGated ? out_rows : T) + nt - 1) / nt);
    p.whole = tiles / pairs * pairs;
    const int64_t rest = tiles - p.whole;
    p.parts = 1;
    double end = rest ? 0.27 * steps + 4.0 : 4.0;
    for (int q = 2; rest && q <= (MODE == kGrad ? 2 : 4); q *= 2) {
        const double cost = (double)((rest * q + pairs - 1) / pairs) * steps * (q == 2 ? 0.24 : 0.235) + (q == 2 ? 1.5 : 1.0);
        if (cost < end) {
            end = cost;
            p.parts = q;
        }
    }
    p.units = p.whole + rest * p.parts;
    p.us = 4.0 + (double)(p.whole / pairs) * steps * 0.27 + end;
    return p;
}

template <int MODE, int P, typename OT>
static cudaError_t run_pair(const GemmArgs& a, const PairPlan& plan, cudaStream_t s) {
    static bool attr_done[64];
    cudaError_t e = allow_smem(k_dense_pair<MODE, P, OT>, attr_done);
    if (e != cudaSuccess) return e;
    PairParams p{};
    p.xd = a.xd;
    p.s[0] = a.s[0];
    p.s[1] = a.s[1];
    p.bias = a.bias;
    p.gscale = a.gscale;
    p.out = a.out;
    p.ldo = a.ldo;
    p.acc = a.acc;
    p.mat_pitch = a.mat_pitch;
    p.T = a.T;
    p.rows = a.rows;
    p.out_rows = MODE == kGrad ? a.cols : a.rows;
    p.k_steps = ((MODE == kGrad ? a.rows : a.cols) + kStageK - 1) / kStageK;
    p.steps = p.k_steps * (MODE == kGrad ? a.n_mats : 1);
    p.act = a.act;
    p.dtype = a.dtype;
    const int esz = a.dtype == MOE_F32 ? 4 : 2;
    p.vec = reinterpret_cast<uintptr_t>(a.out) % 16 == 0 && a.ldo * esz % 16 == 0 && a.rows * esz % 16 == 0 &&
            (!a.acc || (reinterpret_cast<uintptr_t>(a.acc) % 16 == 0 && a.rows % 4 == 0));
    p.nt = pair_columns<MODE, P>;
    p.tiles_r = plan.tiles_r;
    p.whole = plan.whole;
    p.parts = plan.parts;
    p.units = plan.units;
    // boxes: the MMA's rows are 128 a CTA, its columns half of the pair's
    PairMaps maps;
    auto map_w = [&](CUtensorMap* m, int i, int box) {
        return encode_2d(m, a.w[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, a.cols, a.rows, a.ldw[i], kStageK, box,
                         CU_TENSOR_MAP_SWIZZLE_128B);
    };
    auto map_x = [&](CUtensorMap* m, int box) {
        return encode_2d(m, a.x, CU_TENSOR_MAP_DATA_TYPE_UINT8, MODE == kGrad ? a.n_mats * a.mat_pitch : a.cols,
                         plane_rows_of<MODE, P>(a), a.ldx, kStageK, box, CU_TENSOR_MAP_SWIZZLE_128B);
    };
    const int half = MODE == kGated ? p.nt : P * p.nt / 2;
    if constexpr (MODE == kGated) {
        e = map_x(&maps.a[0], 128);
        for (int m = 0; m < 2 && e == cudaSuccess; ++m) {
            e = map_w(&maps.b[m], m, half);
            if (e == cudaSuccess && p.parts > 1) e = map_w(&maps.small[m], m, half / p.parts);
        }
    } else {
        for (int m = 0; m < a.n_mats && e == cudaSuccess; ++m) e = map_w(&maps.a[m], m, 128);
        if (e == cudaSuccess) e = map_x(&maps.b[0], half);
        if (e == cudaSuccess && p.parts > 1) e = map_x(&maps.small[0], half / p.parts);
    }
    if (e != cudaSuccess) return e;
    if (MODE != kGrad || a.n_mats == 1) maps.a[1] = maps.a[0];
    if (MODE != kGated) maps.b[1] = maps.b[0];
    if (p.parts == 1)
        for (int m = 0; m < 2; ++m) maps.small[m] = maps.b[m];
    else if (MODE != kGated)
        maps.small[1] = maps.small[0];
    const int64_t pairs = device_info().sm_count / 2;
    const unsigned grid = 2 * (unsigned)(p.units < pairs ? p.units : pairs);
    return launch_dense(k_dense_pair<MODE, P, OT>, grid, kPairThreads, kPairSmem<MODE>, 1, s, maps, p);
}

// Single CTAs or pairs, by their estimates (within 20 % of the better one over 17
// to 4096 tokens of five layer shapes, in a whole backward pass within 30 %; below
// 64 tokens a pair's rows stay empty).
template <int MODE, int P, typename OT>
static cudaError_t run_product(const GemmArgs& a, cudaStream_t s) {
    const int out_rows = MODE == kGrad ? a.cols : a.rows;
    const int steps = ((MODE == kGrad ? a.rows : a.cols) + kStageK - 1) / kStageK * (MODE == kGrad ? a.n_mats : 1);
    const TilePlan tile = plan_tile<MODE, P>(a.T, (out_rows + kTileRows - 1) / kTileRows, steps);
    if (a.T >= 64 && tma_operands(a)) {
        const PairPlan pair = plan_pair<MODE, P>(a.T, out_rows, steps);
        if (pair.us < tile.us) return run_pair<MODE, P, OT>(a, pair, s);
    }
    return run_tile<MODE, P, OT>(a, tile, s);
}

template <int MODE>
static cudaError_t run_forward(const GemmArgs& a, cudaStream_t s) {
    if (a.T <= kFewTokens) return MODE == kGated ? launch_few_gated(a, s) : launch_few_matmul(a, s);
    return a.dtype == MOE_F32    ? run_product<MODE, 1, float>(a, s)
           : a.dtype == MOE_BF16 ? run_product<MODE, 1, __nv_bfloat16>(a, s)
                                 : run_product<MODE, 1, __half>(a, s);
}

cudaError_t launch_matmul(const GemmArgs& a, cudaStream_t s) { return run_forward<kMatmul>(a, s); }

cudaError_t launch_gated(const GemmArgs& a, cudaStream_t s) { return run_forward<kGated>(a, s); }

cudaError_t launch_grad_matmul(const GemmArgs& a, cudaStream_t s) {
    return a.dtype == MOE_F32    ? run_product<kGrad, planes_of(MOE_F32), float>(a, s)
           : a.dtype == MOE_BF16 ? run_product<kGrad, planes_of(MOE_BF16), __nv_bfloat16>(a, s)
                                 : run_product<kGrad, planes_of(MOE_F16), __half>(a, s);
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
