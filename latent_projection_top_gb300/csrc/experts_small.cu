// The routed experts' products of few rows at few experts: so few tiles that two
// SMs a tile (experts_kernel.cu) would leave most of the GPU idle and read the
// weights at a few SMs' rate.
//
//   D[r, c] = sum_k A[r, k] B_e[k, c]     offsets[e] <= r < offsets[e + 1]
//
// As layer_small.cu: 128 weight columns a tile (a gated block: 64 of gate and the
// same 64 of up) on the tensor cores' M side, up to 32 rows on their N side, the
// contraction split over the CTAs of a cluster, whose FP32 sums meet in
// distributed shared memory in rank order.  A cluster has one tile or none: it
// finds its expert from the offsets, and the call has no more tiles than clusters
// (the host's rule, by the rows that there could be).
//
// Bound by latencies: 1 row at two of 64 experts, 896x448, 10.0 us for both
// products (12.3 by the pair kernel, whose 16 busy SMs take 500 cycles a k-block).
//
// Warp roles (320 threads): warp 0 TMA producer, warp 1 TMEM owner and MMA
// issuer, warps 2..9 epilogue.  Every wait on a copy or an MMA is bounded; all
// threads of a cluster reach its barriers whatever happened before.
#include "experts.cuh"
#include "layer_math.cuh"
#include "layer_ptx.cuh"

namespace route {
namespace {

constexpr int kThreads = 320;
constexpr int kEpiThreads = 256;
constexpr int kStages = 5;
constexpr uint32_t kColBytes = 128 * 64 * 2;              // 128 columns x 64 k
constexpr uint32_t kRowsBytes = kFewRows * 64 * 2;
constexpr uint32_t kStage = kColBytes + kRowsBytes;
constexpr uint32_t kSmem = 1024 + kStages * kStage + 256;
constexpr uint32_t kTmemCols = 32;
static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two CTAs an SM");
static_assert(kFewRows * 128 * 4 <= kStages * kStage, "the sums fit the stages");

__device__ __forceinline__ uint64_t smem_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
    d |= (uint64_t)((sbo >> 4) & 0x3FFFu) << 32;
    d |= 1ull << 46;  // descriptor version for tcgen05
    d |= 2ull << 61;  // 128-byte swizzle
    return d;
}

__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, const ExpertsArgs &a,
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

__device__ __forceinline__ void wait_drain(uint32_t bar, uint32_t parity, const ExpertsArgs &a) {
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

// Four columns' sums of the cluster's CTAs, added in rank order: every CTA's part
// is on its way before the first is added.
__device__ __forceinline__ void add_parts(uint32_t at, int ctas, float (&v)[4]) {
    float4 f[kFewCtas];
#pragma unroll
    for (int j = 0; j < kFewCtas; ++j)
        if (j < ctas) f[j] = ld_cluster_f4(ptx::map_to_rank(at, (uint32_t)j));
    v[0] = v[1] = v[2] = v[3] = 0.f;
#pragma unroll
    for (int j = 0; j < kFewCtas; ++j)
        if (j < ctas) v[0] += f[j].x, v[1] += f[j].y, v[2] += f[j].z, v[3] += f[j].w;
}

template <int EPI>
__global__ void __launch_bounds__(kThreads, 2)
    experts_small_kernel(const __grid_constant__ ExpertsMaps maps, const __grid_constant__ ExpertsArgs args, int ctas) {
    constexpr int kCols = EPI == kEpiGated ? 64 : 128;  // columns of D a tile
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t s_tmem_base;
    __shared__ volatile int s_abort;
    __shared__ int s_count[kThreads / 32], s_run[3];

    const uint32_t raw = ptx::smem_addr(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    const uint32_t bars = sbase + kStages * kStage;
    auto full_bar = [&](int s) { return bars + 8u * s; };
    auto empty_bar = [&](int s) { return bars + 8u * (kStages + s); };
    const uint32_t done_bar = bars + 8u * (2 * kStages);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)(blockIdx.x % (unsigned)ctas), item = (int)(blockIdx.x / (unsigned)ctas);
    const int used = item / args.tiles_n, tn = item - used * args.tiles_n;  // which expert with rows, which tile
    if (tid == 0) {
        s_abort = 0;
        s_run[1] = s_run[2] = 0;
        for (int s = 0; s < kStages; ++s) {
            ptx::mbar_init(full_bar(s), 1);
            ptx::mbar_init(empty_bar(s), 1);
        }
        ptx::mbar_init(done_bar, 1);
        ptx::fence_barrier_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_addr(&s_tmem_base), kTmemCols);
        ptx::tmem_relinquish();
    }
    if (!args.chained) asm volatile("griddepcontrol.wait;" ::: "memory");

    // the `used`-th expert that has rows
    constexpr int kEach = (kMaxExperts + kThreads - 1) / kThreads;
    int o[kEach + 1], mine = 0;
#pragma unroll
    for (int j = 0; j <= kEach; ++j) o[j] = tid * kEach + j <= args.experts ? __ldcg(args.offsets + tid * kEach + j) : 0;
    auto run = [&](int j, int &lo, int &hi) {
        lo = min(max(o[j], 0), args.rows);
        hi = tid * kEach + j < args.experts ? max(min(o[j + 1], args.rows), lo) : lo;
    };
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        int lo, hi;
        run(j, lo, hi);
        mine += hi > lo;
    }
    int incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, incl, d);
        if (lane >= d) incl += u;
    }
    if (lane == 31) s_count[warp] = incl;
    __syncthreads();
    int before = incl - mine;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) before += w < warp ? s_count[w] : 0;
    if (used >= before && used < before + mine) {
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            int lo, hi;
            run(j, lo, hi);
            if (hi > lo && before++ == used) s_run[0] = tid * kEach + j, s_run[1] = lo, s_run[2] = hi;
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem_base = s_tmem_base;
    const int e = s_run[0], row0 = s_run[1], end = min(s_run[2], s_run[1] + kFewRows);
    const int kb0 = args.kblocks * rank / ctas;
    const int total = row0 < end ? args.kblocks * (rank + 1) / ctas - kb0 : 0;
    const int col0 = tn * kCols;
    bool ok = true;

    if (warp == 0) {
        if (lane == 0) {
            // ---------------- TMA producer ----------------
            const uint64_t pol_c = ptx::policy_evict_first(), pol_r = ptx::policy_evict_last();
            auto columns_of = [&](int it) {
                const int s = it % kStages, k0 = (kb0 + it) * 64;
                const uint32_t sc = sbase + s * kStage, fb = full_bar(s);
                ptx::mbar_arrive_expect_tx(fb, kStage);
                ptx::tma_load_3d(sc, &maps.w[0], fb, col0, k0, e, pol_c);
                ptx::tma_load_3d(sc + 8192u, &maps.w[EPI == kEpiGated ? 1 : 0], fb, EPI == kEpiGated ? col0 : col0 + 64,
                                 k0, e, pol_c);
            };
            auto rows_of = [&](int it) {
                const int s = it % kStages;
                ptx::tma_load_2d(sbase + s * kStage + kColBytes, &maps.t[0][kFewRows / 16 - 1], full_bar(s),
                                 (kb0 + it) * 64, row0, pol_r);
            };
            // test hook: the last rows never arrive
            auto stalled = [&](int it) { return args.test_stall && it == total - 1; };
            const int first = min(total, kStages), ahead = args.chained ? first : 0;
            for (int it = 0; it < ahead; ++it) columns_of(it);
            if (args.chained) asm volatile("griddepcontrol.wait;" ::: "memory");
            if (args.trigger) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
            int issued = 0;
            for (; issued < total; ++issued) {
                const int it = issued;
                if (it >= kStages &&
                    !wait_phase(empty_bar(it % kStages), ((uint32_t)(it / kStages) & 1u) ^ 1u, args, &s_abort))
                    break;
                if (it >= ahead) columns_of(it);
                if (!stalled(it)) rows_of(it);
            }
            // Not to leave before every copy has landed: the MMAs have released its
            // stage, or, after a wait that expired, it is waited for.
            bool released = true;
            for (int it = issued > kStages ? issued - kStages : 0; it < issued; ++it) {
                const uint32_t parity = (uint32_t)(it / kStages) & 1u;
                released = released && wait_phase(empty_bar(it % kStages), parity, args, &s_abort);
                if (!released) wait_drain(full_bar(it % kStages), parity, args);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // ---------------- MMA issuer ----------------
            // kind::f16, FP32 accumulator, M = 128 columns, N = 32 rows; the columns are
            // contiguous in memory, the rows' contraction is
            const uint32_t fmt = args.fp16 ? 0u : 1u;
            const uint32_t idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | (1u << 15) | ((uint32_t)(kFewRows >> 3) << 17) |
                                   ((128u >> 4) << 24);
            for (int it = 0; it < total; ++it) {
                const int s = it % kStages;
                if (!wait_phase(full_bar(s), (uint32_t)(it / kStages) & 1u, args, &s_abort)) break;
                ptx::tc_fence_after();
                const uint32_t sc = sbase + s * kStage, sr = sc + kColBytes;
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    ptx::mma_bf16(tmem_base, smem_desc(sc + kk * 2048u, 8192u, 1024u),
                                  smem_desc(sr + kk * 32u, 16u, 1024u), idesc, (it > 0 || kk > 0) ? 1u : 0u);
                ptx::mma_commit(empty_bar(s));
            }
            ptx::mma_commit(done_bar);  // every MMA retired (after an abort too)
        }
    }

    // ---------------- sums over the cluster, and the epilogue ----------------
    Epilogue ep = args.e;
    ep.M = end;
    const int t = tid - 64;  // epilogue thread
    float *sums = reinterpret_cast<float *>(smem_raw + (sbase - raw));
    const int rows = end - row0;
    if (warp >= 2) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        ok = wait_phase(done_bar, 0u, args, &s_abort) && !s_abort;
        __syncwarp();
        ptx::tc_fence_after();
        // the stages are free: this CTA's sums go there, [row][128 columns]
        const int lq = warp & 3, r0 = ((warp - 2) >> 2) * 16;
        uint32_t v[16];
        ptx::tmem_ld_x16(tmem_base + ((uint32_t)(32 * lq) << 16) + (uint32_t)r0, v);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (r0 + j < rows) sums[(r0 + j) * 128 + 32 * lq + lane] = total > 0 ? __uint_as_float(v[j]) : 0.f;
        ptx::tc_fence_before();
    }
    __syncwarp();
    if (ctas > 1)
        ptx::cluster_sync();
    else
        __syncthreads();
    if (warp >= 2 && ok) {
        // four columns of a row a thread; the CTAs share the tile's items
        constexpr int kGroups = kCols / 4;
        const int items = rows * kGroups, i0 = items * rank / ctas, i1 = items * (rank + 1) / ctas;
        for (int x = i0 + t; x < i1; x += kEpiThreads) {
            const int r = x / kGroups, c = x % kGroups * 4;
            const uint32_t at = sbase + (uint32_t)(r * 128 + c) * 4u;
            float v[4], u[4] = {0.f, 0.f, 0.f, 0.f};
            EpiIn<EPI> in;
            epi_load<EPI>(ep, row0 + r, col0 + c, in);
            add_parts(at, ctas, v);
            if constexpr (EPI == kEpiGated) add_parts(at + 256u, ctas, u);
            epilogue<EPI>(ep, row0 + r, col0 + c, v, u, in);
        }
    }
    __syncwarp();
    if (ctas > 1) ptx::cluster_arrive();  // after the last remote read
    if (warp == 1) {
        if (lane == 0) wait_drain(done_bar, 0u, args);
        __syncwarp();
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem_base, kTmemCols);
    }
    __syncwarp();
    if (ctas > 1) ptx::cluster_wait();  // no CTA leaves while another may read its sums
}

const void *kernel_of(int epi) {
    return epi == kEpiGated ? reinterpret_cast<const void *>(experts_small_kernel<kEpiGated>)
                            : reinterpret_cast<const void *>(experts_small_kernel<kEpiLinear>);
}

}  // namespace

cudaError_t experts_small_configure() {
    for (int epi : {kEpiGated, kEpiLinear}) {
        const cudaError_t e =
            cudaFuncSetAttribute(kernel_of(epi), cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t experts_small_launch(int epi, int tiles, int ctas, const ExpertsMaps &maps, const ExpertsArgs &args,
                                 cudaStream_t stream) {
    if (tiles < 1 || ctas < 1 || ctas > kFewCtas || args.kswitch != args.kblocks) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t c = {};
    cudaLaunchAttribute attr[2];
    c.gridDim = dim3((unsigned)(tiles * ctas));
    c.blockDim = dim3(kThreads);
    c.dynamicSmemBytes = kSmem;
    c.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    c.attrs = attr;
    c.numAttrs = 2;
    void *params[] = {const_cast<ExpertsMaps *>(&maps), const_cast<ExpertsArgs *>(&args), &ctas};
    return cudaLaunchKernelExC(&c, kernel_of(epi), params);
}

}  // namespace route
