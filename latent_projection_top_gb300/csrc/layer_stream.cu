// The layer operators' products with few token rows (decode batches): each
// weight is read once from memory, and reading it is the whole cost.
//
//   D[n, r] = sum_k W[k, n] x[r, k]
//
// Weight columns are the tensor cores' M side (128 a tile; a gated block: 64
// of gate and the same 64 of up), token rows their N side (16 to 128), so
// that no MMA work is spent on rows that do not exist.  The (tile, k-block)
// units go to the CTAs in equal contiguous runs, one CTA per SM, whatever
// the tile count: every SM streams the same number of bytes.  A run's part
// of a tile leaves TMEM as FP32 partials; the CTA that stores a tile's last
// partials adds them all, in the order of the runs and not of arrival, and
// runs the operator's epilogue (layer_math.cuh) on the sums.  CTA g's part
// of tile t has slot g + t: runs and tiles both advance along the units, so
// that pairs (g, t) in order have consecutive slots.
//
// Warp roles (320 threads): warp 0 TMA producer, warp 1 TMEM owner and MMA
// issuer, warps 2..9 partials and epilogue.  Every wait is bounded, as in
// layer_gemm.cu.
#include "layer.cuh"
#include "layer_math.cuh"
#include "sm103_ptx.cuh"

namespace route {
namespace {

constexpr int kThreads = 320;
constexpr int kEpiThreads = 256;
constexpr uint32_t kWBytes = kStreamTile * 64 * 2;

__host__ __device__ constexpr uint32_t x_area(int bn) { return (uint32_t)bn * 128; }
__host__ __device__ constexpr uint32_t stage_bytes(int bn) { return kWBytes + x_area(bn); }
// Up to 32 rows two CTAs fit an SM, so that the next product's first weights
// arrive under this one's last partials.
__host__ __device__ constexpr int stages_of(int bn) {
    return bn == 16 ? 6 : bn == 32 ? 5 : bn == 64 ? 8 : 6;
}
__host__ __device__ constexpr uint32_t smem_of(int bn) { return 1024 + stages_of(bn) * stage_bytes(bn) + 256; }
static_assert(smem_of(64) <= 227 * 1024 && smem_of(128) <= 227 * 1024, "shared memory");
static_assert(2 * (smem_of(16) + 1024) <= 228 * 1024 && 2 * (smem_of(32) + 1024) <= 228 * 1024,
              "two CTAs an SM");

__device__ __forceinline__ uint64_t smem_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
    d |= (uint64_t)((sbo >> 4) & 0x3FFFu) << 32;
    d |= 1ull << 46;  // descriptor version for tcgen05
    d |= 2ull << 61;  // 128-byte swizzle
    return d;
}

__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, const StreamArgs &a,
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

__device__ __forceinline__ void wait_drain(uint32_t bar, uint32_t parity, const StreamArgs &a) {
    const uint64_t t0 = ptx::global_timer_ns();
    while (!ptx::mbar_try_wait(bar, parity)) {
        if (ptx::global_timer_ns() - t0 > a.timeout_ns) {
            atomicOr(a.status, kStatusTimeout);
            return;
        }
    }
}

// First unit of CTA g, and the CTA that owns unit u.
__device__ __forceinline__ int first_unit(const StreamArgs &a, int g) {
    return (int)((long long)a.tiles * a.kblocks * g / a.grid);
}
__device__ __forceinline__ int owner(const StreamArgs &a, int u) {
    int g = (int)((long long)u * a.grid / ((long long)a.tiles * a.kblocks));
    while (first_unit(a, g + 1) <= u) ++g;
    return g;
}

template <int FORM, int EPI, int BN>
__global__ void __launch_bounds__(kThreads, 1)
    layer_stream_kernel(const __grid_constant__ GemmMaps maps, const __grid_constant__ StreamArgs args) {
    constexpr bool W_MN = FORM == kFormNT;  // weights N-contiguous, else K-contiguous
    constexpr int S = stages_of(BN);
    constexpr uint32_t kStage = stage_bytes(BN);
    constexpr int kTileCols = EPI == kEpiGated ? kStreamTile / 2 : kStreamTile;
    constexpr uint32_t kTmemCols = 2 * BN < 32 ? 32 : 2 * BN;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t s_tmem_base;
    __shared__ volatile int s_abort;
    __shared__ int s_last;

    const uint32_t raw = ptx::smem_addr(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    const uint32_t bars = sbase + S * kStage;
    auto full_bar = [&](int s) { return bars + 8u * s; };
    auto empty_bar = [&](int s) { return bars + 8u * (S + s); };
    auto tfull_bar = [&](int t) { return bars + 8u * (2 * S + t); };
    auto tempty_bar = [&](int t) { return bars + 8u * (2 * S + 2 + t); };
    const uint32_t drain_bar = bars + 8u * (2 * S + 4);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int g = blockIdx.x;
    const int u0 = first_unit(args, g), u1 = first_unit(args, g + 1);
    const int K = args.kblocks;

    if (threadIdx.x == 0) {
        s_abort = 0;
        for (int s = 0; s < S; ++s) {
            ptx::mbar_init(full_bar(s), 1);
            ptx::mbar_init(empty_bar(s), 1);
        }
        for (int t = 0; t < 2; ++t) {
            ptx::mbar_init(tfull_bar(t), 1);
            ptx::mbar_init(tempty_bar(t), kEpiThreads / 32);
        }
        ptx::mbar_init(drain_bar, 1);
        ptx::fence_barrier_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_addr(&s_tmem_base), kTmemCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem_base = s_tmem_base;

    if (warp == 0) {
        if (lane == 0) {
            // ---------------- TMA producer ----------------
            const uint64_t pol_w = ptx::policy_evict_first();
            const uint64_t pol_x = ptx::policy_evict_last();
            const uint32_t tx = kWBytes + args.x_bytes;
            auto weights_of = [&](int u, int s) {
                const int t = u / K, kb = u - t * K;
                const int seg = kb >= args.kswitch;
                const int k0 = (seg ? kb - args.kswitch : kb) * 64;
                const uint32_t sw = sbase + s * kStage, fb = full_bar(s);
                if (EPI == kEpiGated) {
                    ptx::tma_load_2d(sw, &maps.m[args.w[0][0]], fb, t * kTileCols, k0, pol_w);
                    ptx::tma_load_2d(sw + 8192u, &maps.m[args.w[0][1]], fb, t * kTileCols, k0, pol_w);
                } else if (W_MN) {
                    const CUtensorMap *m = &maps.m[args.w[seg][0]];
                    ptx::tma_load_2d(sw, m, fb, t * kTileCols, k0, pol_w);
                    ptx::tma_load_2d(sw + 8192u, m, fb, t * kTileCols + 64, k0, pol_w);
                } else {
                    ptx::tma_load_2d(sw, &maps.m[args.w[seg][0]], fb, k0, t * kTileCols, pol_w);
                }
            };
            auto rows_of = [&](int u, int s) {
                const int kb = u % K;
                const int seg = kb >= args.kswitch;
                const int k0 = (seg ? kb - args.kswitch : kb) * 64;
                ptx::tma_load_2d(sbase + s * kStage + kWBytes, &maps.m[args.x[seg]], full_bar(s), k0,
                                 0, pol_x);
            };
            const int total = u1 - u0;
            const int n_pre = args.wait_first ? 0 : total < S ? total : S;
            for (int it = 0; it < n_pre; ++it) {
                ptx::mbar_arrive_expect_tx(full_bar(it), tx);
                weights_of(u0 + it, it);
            }
            asm volatile("griddepcontrol.wait;" ::: "memory");
            if (args.trigger) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
            uint32_t armed = 0u, armed_par = 0u;
            bool ok = true;
            for (int it = 0; it < total; ++it) {
                const int s = it % S;
                const uint32_t ph = (uint32_t)(it / S) & 1u;
                if (!wait_phase(empty_bar(s), ph ^ 1u, args, &s_abort)) {
                    ok = false;
                    break;
                }
                if (args.test_stall && it == total - 1) break;  // test hook: it never arrives
                if (it >= n_pre) {
                    ptx::mbar_arrive_expect_tx(full_bar(s), tx);
                    weights_of(u0 + it, s);
                }
                rows_of(u0 + it, s);
                armed |= 1u << s;
                armed_par = (armed_par & ~(1u << s)) | (ph << s);
            }
            if (!ok || s_abort) {  // let every complete copy land
                for (int s = 0; s < S; ++s)
                    if (armed & (1u << s)) wait_drain(full_bar(s), (armed_par >> s) & 1u, args);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // ---------------- MMA issuer ----------------
            // kind::f16, FP32 accumulator, M = 128 weight columns, N = BN rows
            const uint32_t fmt = args.fp16 ? 0u : 1u;
            const uint32_t idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | ((W_MN ? 1u : 0u) << 15) |
                                   ((uint32_t)(BN >> 3) << 17) | ((uint32_t)(kStreamTile >> 4) << 24);
            int it = 0, job = 0;
            bool ok = true;
            for (int u = u0; u < u1 && ok; ++job) {
                const int end = min(u1, (u / K + 1) * K);
                const int t = job & 1;
                if (!wait_phase(tempty_bar(t), (((uint32_t)job >> 1) & 1u) ^ 1u, args, &s_abort)) break;
                ptx::tc_fence_after();
                const uint32_t d_tmem = tmem_base + (uint32_t)(t * BN);
                for (const int first = u; u < end; ++u, ++it) {
                    const int s = it % S;
                    if (!wait_phase(full_bar(s), (uint32_t)(it / S) & 1u, args, &s_abort)) {
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after();
                    const uint32_t sw = sbase + s * kStage, sx = sw + kWBytes;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        const uint64_t dw = W_MN ? smem_desc(sw + kk * 2048u, 8192u, 1024u)
                                                 : smem_desc(sw + kk * 32u, 16u, 1024u);
                        ptx::mma_bf16(d_tmem, dw, smem_desc(sx + kk * 32u, 16u, 1024u), idesc,
                                      (u > first || kk > 0) ? 1u : 0u);
                    }
                    ptx::mma_commit(empty_bar(s));
                }
                if (ok) ptx::mma_commit(tfull_bar(t));
            }
            ptx::mma_commit(drain_bar);  // every MMA retired before TMEM is freed
            wait_drain(drain_bar, 0u, args);
        }
    } else {
        // ---------------- partials and epilogue (warps 2..9) ----------------
        const int lq = warp & 3;         // TMEM lanes 32 lq .. + 31 = weight columns
        const int cs = (warp - 2) >> 2;  // which 16-row chunks: even or odd
        const int e = threadIdx.x - 64;
        const int rows = args.rows;
        asm volatile("griddepcontrol.wait;" ::: "memory");
        int job = 0;
        for (int u = u0; u < u1; ++job) {
            const int tile = u / K;
            const int tb = job & 1;
            const bool ok = wait_phase(tfull_bar(tb), ((uint32_t)job >> 1) & 1u, args, &s_abort);
            // every epilogue warp leaves together, or the barriers below would hang
            if (!ptx::named_bar_and(1, kEpiThreads, ok)) break;
            ptx::tc_fence_after();
            float *part = args.part + (long long)(g + tile) * rows * kStreamTile;
#pragma unroll 1
            for (int r0 = cs * 16; r0 < BN; r0 += 32) {
                if (r0 >= rows) break;
                uint32_t v[16];
                ptx::tmem_ld_x16(tmem_base + ((uint32_t)(32 * lq) << 16) + (uint32_t)(tb * BN + r0), v);
                ptx::tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (r0 + j < rows)
                        part[(r0 + j) * kStreamTile + 32 * lq + lane] = __uint_as_float(v[j]);
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(tempty_bar(tb));
            // the CTA that brings the tile's last partials adds them
            const int g0 = owner(args, tile * K), g1 = owner(args, (tile + 1) * K - 1);
            ptx::named_bar_sync(1, kEpiThreads);
            if (e == 0) {
                __threadfence();
                s_last = atomicAdd(args.arrived + tile, 1u) == (unsigned)(g1 - g0);
                if (s_last) args.arrived[tile] = 0u;
                __threadfence();
            }
            ptx::named_bar_sync(1, kEpiThreads);
            if (s_last) {
                const float *src = args.part + (long long)(g0 + tile) * rows * kStreamTile;
                const long long step = (long long)rows * kStreamTile;
                for (int i = e; i < rows * (kTileCols / 4); i += kEpiThreads) {
                    const int r = i / (kTileCols / 4), c = (i % (kTileCols / 4)) * 4;
                    const float *q = src + r * kStreamTile + c;
                    float v[4] = {0.f, 0.f, 0.f, 0.f}, up[4] = {0.f, 0.f, 0.f, 0.f};
                    EpiIn<EPI, 4> in;
                    epi_load<EPI, 4>(args.p, r, tile * kTileCols + c, in);
#pragma unroll 4
                    for (int s = g0; s <= g1; ++s, q += step) {
                        const float4 x = __ldcg(reinterpret_cast<const float4 *>(q));
                        v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
                        if (EPI == kEpiGated) {
                            const float4 y = __ldcg(reinterpret_cast<const float4 *>(q + kTileCols));
                            up[0] += y.x, up[1] += y.y, up[2] += y.z, up[3] += y.w;
                        }
                    }
                    epilogue<EPI, 4>(args.p, r, tile * kTileCols + c, v, up, in);
                }
            }
            u = min(u1, (tile + 1) * K);
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem_base, kTmemCols);
    }
}

int bn_of(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128; }

const void *kernel_of(int form, int epi, int bn) {
#define ROUTE_STREAM(F, E)                                                                        \
    if (form == F && epi == E)                                                                    \
        return bn == 16   ? reinterpret_cast<const void *>(layer_stream_kernel<F, E, 16>)         \
               : bn == 32 ? reinterpret_cast<const void *>(layer_stream_kernel<F, E, 32>)         \
               : bn == 64 ? reinterpret_cast<const void *>(layer_stream_kernel<F, E, 64>)         \
                          : reinterpret_cast<const void *>(layer_stream_kernel<F, E, 128>);
    ROUTE_STREAM(kFormNT, kEpiLinear)
    ROUTE_STREAM(kFormNT, kEpiGated)
    ROUTE_STREAM(kFormNN, kEpiLinear)
    ROUTE_STREAM(kFormNN, kEpiDGate)
#undef ROUTE_STREAM
    return nullptr;
}

}  // namespace

cudaError_t stream_configure() {
    for (int form = 0; form < 2; ++form)
        for (int epi = 0; epi < 3; ++epi)
            for (int bn : {16, 32, 64, 128})
                if (const void *k = kernel_of(form, epi, bn)) {
                    const cudaError_t e = cudaFuncSetAttribute(
                        k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_of(bn));
                    if (e != cudaSuccess) return e;
                }
    return cudaSuccess;
}

int stream_smem_bytes() { return (int)(smem_of(64) > smem_of(128) ? smem_of(64) : smem_of(128)); }

cudaError_t stream_launch(int form, int epi, const GemmMaps &maps, const StreamArgs &args,
                          cudaStream_t stream) {
    const int bn = bn_of(args.rows);
    const void *k = kernel_of(form, epi, bn);
    if (k == nullptr || args.rows < 1 || args.rows > kStreamMaxRows || args.grid < 1 ||
        args.tiles < 1 || args.tiles > kStreamMaxTiles)
        return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t c = {};
    cudaLaunchAttribute attr[1];
    c.gridDim = dim3(args.grid);
    c.blockDim = dim3(kThreads);
    c.dynamicSmemBytes = smem_of(bn);
    c.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    c.attrs = attr;
    c.numAttrs = 1;
    void *params[] = {const_cast<GemmMaps *>(&maps), const_cast<StreamArgs *>(&args)};
    return cudaLaunchKernelExC(&c, k, params);
}

}  // namespace route
