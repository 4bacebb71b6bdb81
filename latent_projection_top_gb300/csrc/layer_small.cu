// The layer operators' products with few rows (decode batches: each weight is
// read once from memory, and reading it is the whole cost) or few tiles.
//
//   D[r, n] = sum_k A[r, k] B[k, n]
//
// Columns of D are the tensor cores' M side (128 a tile; a gated block: 64 of
// gate and the same 64 of up), its rows their N side (16 to 128 a tile), so
// that no MMA work is spent on rows that do not exist and one weight column
// never meets more than one SM per 128 rows.  A tile's contraction is split
// over a cluster of up to eight CTAs, enough of them to have the whole chip
// read: their FP32 sums meet in distributed shared memory, each CTA adds its
// share of the tile's elements over the cluster, in rank order, lets its peers
// leave and runs the operator's epilogue (layer_math.cuh) on the sums.  No partial goes through
// global memory and no second kernel or counter is needed: at 128 rows of
// 896x896 the sums' last step took 25 of 31 us when one CTA did it for a
// tile, from partials in L2.
//
// Bound by HBM where the weights are large (8x3584x7168 12.0 us, 51.7 MB: 4.3
// TB/s over the whole launch, which is the memory's rate plus 4 us of the
// launch's start, the first copies' latency and the sums), else by those
// latencies (16x64x128 3.2 us, 64x896x896 4.8).
//
// Two CTAs fit an SM, so that a call's second product fetches its first
// weights under the first one's last sums.
//
// Warp roles (320 threads): warp 0 TMA producer, warp 1 TMEM owner and MMA
// issuer, warps 2..9 epilogue.  Every wait on a copy or an MMA is bounded, as
// in layer_gemm.cu; all threads of a cluster reach its barriers whatever
// happened before.
#include <type_traits>

#include "layer.cuh"
#include "layer_math.cuh"
#include "layer_ptx.cuh"

namespace route {
namespace {

constexpr int kThreads = 320;
constexpr int kEpiThreads = 256;
constexpr uint32_t kColBytes = kSmallTile * 64 * 2;  // 128 columns x 64 k

__host__ __device__ constexpr uint32_t stage_bytes(int bn) { return kColBytes + (uint32_t)bn * 128; }
__host__ __device__ constexpr int stages_of(int bn) { return bn == 16 ? 6 : bn == 32 ? 5 : bn == 64 ? 4 : 3; }
__host__ __device__ constexpr uint32_t smem_of(int bn) { return 1024 + stages_of(bn) * stage_bytes(bn) + 256; }
static_assert(2 * (smem_of(16) + 1024) <= 228 * 1024 && 2 * (smem_of(32) + 1024) <= 228 * 1024 &&
                  2 * (smem_of(64) + 1024) <= 228 * 1024 && 2 * (smem_of(128) + 1024) <= 228 * 1024,
              "two CTAs an SM");
static_assert(128 * kSmallTile * 4 <= stages_of(128) * stage_bytes(128), "the sums fit the stages");

__device__ __forceinline__ uint64_t smem_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
    d |= (uint64_t)((sbo >> 4) & 0x3FFFu) << 32;
    d |= 1ull << 46;  // descriptor version for tcgen05
    d |= 2ull << 61;  // 128-byte swizzle
    return d;
}

// 16 k of an operand tile, as in layer_gemm.cu.
template <bool MN>
__device__ __forceinline__ uint64_t operand_desc(uint32_t base, int kk) {
    return MN ? smem_desc(base + kk * 2048u, 8192u, 1024u) : smem_desc(base + kk * 32u, 16u, 1024u);
}

__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, const GemmArgs &a,
                                           volatile int *abort_flag) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = ptx::global_timer_ns();
    for (uint32_t it = 1;; ++it) {
        if (ptx::mbar_try_wait(bar, parity)) return true;
        if ((it & 63u) == 0u) {
            if (*abort_flag) return false;
            if (ptx::global_timer_ns() - t0 > a.timeout_ns) {
                *abort_flag = 1;
                atomicOr(a.status, kStatusTimeout);
                return false;
            }
        }
    }
}

__device__ __forceinline__ void wait_drain(uint32_t bar, uint32_t parity, const GemmArgs &a) {
    const uint64_t t0 = ptx::global_timer_ns();
    while (!ptx::mbar_try_wait(bar, parity)) {
        if (ptx::global_timer_ns() - t0 > a.timeout_ns) {
            atomicOr(a.status, kStatusTimeout);
            return;
        }
    }
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ float ld_cluster_f(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ float4 ld_shared_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ float ld_shared_f(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void st_shared_f4(uint32_t addr, float4 v) {
    asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                 : "memory");
}
__device__ __forceinline__ void st_shared_f(uint32_t addr, float v) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// Four columns' sums of the cluster's C CTAs, added in rank order into this
// one's; N of them, `next` bytes apart.  Every CTA's part is on its way before
// the first is added.
template <int N>
__device__ __forceinline__ void add_parts(uint32_t at, uint32_t next, int C) {
    float4 f[N][kSmallMaxSplits];
#pragma unroll
    for (int j = 0; j < kSmallMaxSplits; ++j)
        if (j < C) {
            const uint32_t q = ptx::map_to_rank(at, (uint32_t)j);
#pragma unroll
            for (int k = 0; k < N; ++k) f[k][j] = ld_cluster_f4(q + k * next);
        }
#pragma unroll
    for (int k = 0; k < N; ++k) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int j = 0; j < kSmallMaxSplits; ++j)
            if (j < C) v.x += f[k][j].x, v.y += f[k][j].y, v.z += f[k][j].z, v.w += f[k][j].w;
        st_shared_f4(at + k * next, v);
    }
}

// The same of one value.
__device__ __forceinline__ void add_parts(uint32_t at, int C) {
    float f[kSmallMaxSplits], v = 0.f;
#pragma unroll
    for (int j = 0; j < kSmallMaxSplits; ++j)
        if (j < C) f[j] = ld_cluster_f(ptx::map_to_rank(at, (uint32_t)j));
#pragma unroll
    for (int j = 0; j < kSmallMaxSplits; ++j)
        if (j < C) v += f[j];
    st_shared_f(at, v);
}

template <int EPI, int BN>
__global__ void __launch_bounds__(kThreads, 2)
    layer_small_kernel(const __grid_constant__ GemmMaps maps, const __grid_constant__ GemmArgs args,
                       int chained) {
    constexpr int S = stages_of(BN);
    constexpr uint32_t kStage = stage_bytes(BN);
    constexpr int kTileCols = EPI == kEpiGated ? kSmallTile / 2 : kSmallTile;
    constexpr uint32_t kTmemCols = BN < 32 ? 32 : BN;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t s_tmem_base;
    __shared__ volatile int s_abort;

    const uint32_t raw = ptx::smem_addr(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    const uint32_t bars = sbase + S * kStage;
    auto full_bar = [&](int s) { return bars + 8u * s; };
    auto empty_bar = [&](int s) { return bars + 8u * (S + s); };
    const uint32_t done_bar = bars + 8u * (2 * S);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int C = args.splits;
    const int rank = blockIdx.x % C;  // clusters are C consecutive CTAs
    int i = blockIdx.x / C;
    int pi = 0;
    while (pi + 1 < args.nprob && i >= args.p[pi + 1].item_base) ++pi;
    const GemmProblem &p = args.p[pi];
    const int form = EPI == kEpiLinear ? p.form : EPI == kEpiDGate ? kFormNN : kFormNT;
    const bool r_mn = form == kFormTT;  // rows' operand: M-contiguous (BN >= 64), else K-contiguous
    const bool c_mn = form != kFormNN;  // columns' operand: N-contiguous, else K-contiguous
    i -= p.item_base;
    const int tm = i % p.tiles_m, tn = i / p.tiles_m;
    const int kb0 = (int)((long long)p.kblocks * rank / C);
    const int total = (int)((long long)p.kblocks * (rank + 1) / C) - kb0;
    const int row0 = tm * BN, col0 = tn * kTileCols;

    // TMA producer: lane 0 of warp 0
    // columns of one row tile are read once: they leave L2 first
    const uint64_t pol_c = p.tiles_m == 1 ? ptx::policy_evict_first() : ptx::policy_evict_normal();
    const uint64_t pol_r = ptx::policy_evict_last();
    // (copies of columns that do not exist take as long as others, or longer)
    const bool second = EPI == kEpiGated || !c_mn || col0 + 64 < p.e.N;
    auto columns_of = [&](int it) {
        const int kb = kb0 + it, s = it % S, seg = kb >= p.kswitch;
        const int k0 = (seg ? kb - p.kswitch : kb) * 64;
        const uint32_t sc = sbase + s * kStage, fb = full_bar(s);
        const CUtensorMap *m = &maps.m[p.b[seg][0]];
        ptx::mbar_arrive_expect_tx(fb, p.a_bytes + (second ? kColBytes : kColBytes / 2));
        if (EPI == kEpiGated) {
            ptx::tma_load_2d(sc, m, fb, col0, k0, pol_c);
            ptx::tma_load_2d(sc + 8192u, &maps.m[p.b[seg][1]], fb, col0, k0, pol_c);
        } else if (c_mn) {
            ptx::tma_load_2d(sc, m, fb, col0, k0, pol_c);
            if (second) ptx::tma_load_2d(sc + 8192u, m, fb, col0 + 64, k0, pol_c);
        } else {
            ptx::tma_load_2d(sc, m, fb, k0, col0, pol_c);
        }
    };
    auto rows_of = [&](int it) {
        const int kb = kb0 + it, s = it % S, seg = kb >= p.kswitch;
        const int k0 = (seg ? kb - p.kswitch : kb) * 64;
        const uint32_t sr = sbase + s * kStage + kColBytes, fb = full_bar(s);
        const CUtensorMap *m = &maps.m[p.a[seg]];
        if (r_mn) {
#pragma unroll
            for (int j = 0; j < (BN < 64 ? 1 : BN / 64); ++j)
                ptx::tma_load_2d(sr + 8192u * j, m, fb, row0 + 64 * j, k0, pol_r);
        } else {
            ptx::tma_load_2d(sr, m, fb, k0, row0, pol_r);
        }
    };
    // test hook: the last copies never arrive
    const int copies = total - (args.test_stall && total > 0 ? 1 : 0);
    const int first = min(copies, S);

    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_addr(&s_tmem_base), kTmemCols);
        ptx::tmem_relinquish();
    } else if (threadIdx.x == 0) {
        s_abort = 0;
        for (int s = 0; s < S; ++s) {
            ptx::mbar_init(full_bar(s), 1);
            ptx::mbar_init(empty_bar(s), 1);
        }
        ptx::mbar_init(done_bar, 1);
        ptx::fence_barrier_init();
        // the first copies go out while TMEM is being allocated
        const int n_pre = chained && !r_mn ? first : 0;
        for (int it = 0; it < n_pre; ++it) columns_of(it);
        asm volatile("griddepcontrol.wait;" ::: "memory");
        if (args.trigger) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        for (int it = 0; it < first; ++it) {
            if (it >= n_pre) columns_of(it);
            rows_of(it);
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem_base = s_tmem_base;
    bool ok = true;

    if (warp == 0) {
        if (lane == 0) {
            int issued = first;
            for (; issued < copies; ++issued) {
                const int it = issued;
                if (!wait_phase(empty_bar(it % S), ((uint32_t)(it / S) & 1u) ^ 1u, args, &s_abort)) break;
                columns_of(it);
                rows_of(it);
            }
            // Not to leave before every copy has landed: the MMAs have released its
            // stage, or, after a wait that expired (maybe only now), it is waited for.
            bool released = true;
            for (int it = issued > S ? issued - S : 0; it < issued; ++it) {
                const uint32_t parity = (uint32_t)(it / S) & 1u;
                released = released && wait_phase(empty_bar(it % S), parity, args, &s_abort);
                if (!released) wait_drain(full_bar(it % S), parity, args);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // ---------------- MMA issuer ----------------
            // kind::f16, FP32 accumulator, M = 128 columns, N = BN rows
            const uint32_t fmt = args.fp16 ? 0u : 1u;
            const uint32_t idesc0 = (1u << 4) | (fmt << 7) | (fmt << 10) | ((uint32_t)(BN >> 3) << 17) |
                                    ((uint32_t)(kSmallTile >> 4) << 24);
            auto k_loop = [&](auto cols_mn, auto rows_mn) {
                constexpr bool C_MN = decltype(cols_mn)::value, R_MN = decltype(rows_mn)::value;
                const uint32_t idesc = idesc0 | ((C_MN ? 1u : 0u) << 15) | ((R_MN ? 1u : 0u) << 16);
                for (int it = 0; it < total; ++it) {
                    const int s = it % S;
                    if (!wait_phase(full_bar(s), (uint32_t)(it / S) & 1u, args, &s_abort)) break;
                    ptx::tc_fence_after();
                    const uint32_t sc = sbase + s * kStage, sr = sc + kColBytes;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        ptx::mma_bf16(tmem_base, operand_desc<C_MN>(sc, kk), operand_desc<R_MN>(sr, kk), idesc,
                                      (it > 0 || kk > 0) ? 1u : 0u);
                    ptx::mma_commit(empty_bar(s));
                }
            };
            if (!c_mn)
                k_loop(std::false_type{}, std::false_type{});
            else if (!r_mn)
                k_loop(std::true_type{}, std::false_type{});
            else
                k_loop(std::true_type{}, std::true_type{});
            ptx::mma_commit(done_bar);  // every MMA retired (after an abort too)
        }
    }

    // ---------------- sums over the cluster, and the epilogue ----------------
    const int e = (int)threadIdx.x - 64;  // epilogue thread
    const Epilogue ep = p.e;
    const int rows = min(BN, ep.M - row0);
    // A thread's item is G columns of a row, neighbouring threads on
    // neighbouring columns: four, or one where rows cannot be accessed four
    // values at a time.  The cluster's CTAs share a tile's items.
    const bool wide = !epi_linear(EPI) || (ep.vec & kVecOut) != 0;  // (a gated block's: padded rows)
    float *sums = reinterpret_cast<float *>(smem_raw + (sbase - raw));
    if (warp >= 2) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        ok = wait_phase(done_bar, 0u, args, &s_abort) && !s_abort;
        __syncwarp();
        ptx::tc_fence_after();
        // the stages are free: this CTA's sums go there, [row][128 columns]
        const int lq = warp & 3, cs = (warp - 2) >> 2;
#pragma unroll 1
        for (int r = cs * 16; r < rows; r += 32) {
            uint32_t v[16];
            ptx::tmem_ld_x16(tmem_base + ((uint32_t)(32 * lq) << 16) + (uint32_t)r, v);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (r + j < rows) sums[(r + j) * kSmallTile + 32 * lq + lane] = total > 0 ? __uint_as_float(v[j]) : 0.f;
        }
        ptx::tc_fence_before();
    }
    __syncwarp();
    if (C > 1)
        ptx::cluster_sync();
    else
        __syncthreads();
    // A CTA's share of the cluster's sums, added into its own copy of them: of
    // each copy only its CTA's share is written, and only others are read by
    // its peers.  Columns that do not exist are not read.
    constexpr int kGroups = kTileCols / 4;
    const int cols = min(kTileCols, ep.N - col0);
    const int items = rows * kGroups, i0 = items * rank / C, i1 = items * (rank + 1) / C;
    constexpr int kStep = kEpiThreads / kTileCols;  // rows that the threads cover at once
    const int rows0 = rows * rank / C, rows1 = rows * (rank + 1) / C;
    auto item_at = [&](int x) { return sbase + (uint32_t)((x / kGroups) * kSmallTile + x % kGroups * 4) * 4u; };
    auto value_at = [&](int r) { return sbase + (uint32_t)(r * kSmallTile + e % kTileCols) * 4u; };
    // the first item's inputs besides the sums are on their way meanwhile
    auto row_of = [&](int x) { return row0 + x / kGroups; };
    auto col_of = [&](int x) { return col0 + x % kGroups * 4; };
    EpiIn<EPI> in, next;
    if (warp >= 2 && wide && i0 + e < i1) epi_load<EPI>(ep, row_of(i0 + e), col_of(i0 + e), in);
    constexpr int kRows = 4;  // of a column that a thread takes together
    const int own0 = rows0 + e / kTileCols;
    uint32_t res[kRows];
    if constexpr (epi_linear(EPI))
        if (warp >= 2 && !wide && own0 < rows1) column_load<kRows>(ep, row0 + own0, col0 + e % kTileCols, kStep, res);
    if (C > 1) {
        if (warp >= 2 && ok && wide) {
            for (int x = i0 + e; x < i1; x += kEpiThreads) {
                if (x % kGroups * 4 >= cols) continue;
                add_parts<EPI == kEpiGated ? 2 : 1>(item_at(x), kTileCols * 4u, C);
            }
        } else if (warp >= 2 && ok && e % kTileCols < cols) {
            // a thread's rows of one column
            for (int r = own0; r < rows1; r += kStep) add_parts(value_at(r), C);
        }
        __syncwarp();
        // After the last remote read (ordered: peers may leave; the order takes 0.17
        // us, 64x896x896 4.84, so 4.66) and before the stores of results, which the
        // order would wait for too (0.5 us).
        ptx::cluster_arrive();
    }
    if (warp >= 2 && ok && wide) {
        for (int x = i0 + e; x < i1; x += kEpiThreads) {
            if (x + kEpiThreads < i1) epi_load<EPI>(ep, row_of(x + kEpiThreads), col_of(x + kEpiThreads), next);
            const float4 f = ld_shared_f4(item_at(x));
            float v[4] = {0.f + f.x, 0.f + f.y, 0.f + f.z, 0.f + f.w}, u[4] = {0.f, 0.f, 0.f, 0.f};  // no -0
            if constexpr (EPI == kEpiGated) {
                const float4 h = ld_shared_f4(item_at(x) + kTileCols * 4u);
                u[0] += h.x, u[1] += h.y, u[2] += h.z, u[3] += h.w;
            }
            epilogue<EPI>(ep, row_of(x), col_of(x), v, u, in);
            in = next;
        }
    } else if (warp >= 2 && ok) {
        if constexpr (epi_linear(EPI)) {
            for (int r = own0; r < rows1; r += kStep * kRows) {
                if (r != own0) column_load<kRows>(ep, row0 + r, col0 + e % kTileCols, kStep, res);
                float v[kRows] = {};
#pragma unroll
                for (int k = 0; k < kRows; ++k)
                    if (r + k * kStep < rows1) v[k] += ld_shared_f(value_at(r + k * kStep));
                // rows of other CTAs' shares are not this one's to write
                Epilogue own = ep;
                own.M = row0 + rows1;
                column_epilogue<EPI, kRows>(own, row0 + r, col0 + e % kTileCols, kStep, v, res);
            }
        }
    }
    if (warp == 1) {
        if (lane == 0) wait_drain(done_bar, 0u, args);
        __syncwarp();
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem_base, kTmemCols);
    }
    __syncwarp();
    if (C > 1) ptx::cluster_wait();  // no CTA leaves while another may read its sums
}

const void *kernel_of(int epi, int bn) {
#define ROUTE_SMALL(E)                                                                       \
    if (epi == E)                                                                            \
        return bn == 16   ? reinterpret_cast<const void *>(layer_small_kernel<E, 16>)        \
               : bn == 32 ? reinterpret_cast<const void *>(layer_small_kernel<E, 32>)        \
               : bn == 64 ? reinterpret_cast<const void *>(layer_small_kernel<E, 64>)        \
                          : reinterpret_cast<const void *>(layer_small_kernel<E, 128>);
    ROUTE_SMALL(kEpiLinear)
    ROUTE_SMALL(kEpiAct)
    ROUTE_SMALL(kEpiGated)
    ROUTE_SMALL(kEpiDGate)
#undef ROUTE_SMALL
    return nullptr;
}

}  // namespace

cudaError_t small_configure() {
    for (int epi = 0; epi < kEpiCount; ++epi)
        for (int bn : {16, 32, 64, 128}) {
            const cudaError_t e = cudaFuncSetAttribute(
                kernel_of(epi, bn), cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_of(bn));
            if (e != cudaSuccess) return e;
        }
    return cudaSuccess;
}

int small_smem_bytes() {
    uint32_t most = 0;
    for (int bn : {16, 32, 64, 128}) most = most < smem_of(bn) ? smem_of(bn) : most;
    return (int)most;
}

cudaError_t small_launch(int epi, int rows, const GemmMaps &maps, const GemmArgs &args,
                         bool chained, cudaStream_t stream) {
    const void *k = kernel_of(epi, rows);
    if (k == nullptr || args.items < 1 || args.splits < 1 || args.splits > kSmallMaxSplits)
        return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t c = {};
    cudaLaunchAttribute attr[2];
    c.gridDim = dim3((unsigned)(args.items * args.splits));
    c.blockDim = dim3(kThreads);
    c.dynamicSmemBytes = smem_of(rows);
    c.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)args.splits;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    c.attrs = attr;
    c.numAttrs = 2;
    int ch = chained;
    void *params[] = {const_cast<GemmMaps *>(&maps), const_cast<GemmArgs *>(&args), &ch};
    return cudaLaunchKernelExC(&c, k, params);
}

}  // namespace route
