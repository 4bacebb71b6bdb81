// Tokens sorted by expert and back: the stable counting sort of the (row,
// expert) pairs, the rows copied to their places, and the weighted sums that
// bring the experts' results back, with their gradients.
#include "experts.cuh"
#include "layer_math.cuh"

namespace route {
namespace {

constexpr int kSortThreads = 1024;
// Warps that go through the pairs: sixteen cost less to set up (in one cluster 8192
// pairs 6.1 us, thirty-two 7.9), thirty-two go through many faster (1048576 pairs
// 90 us, 97).
constexpr int kSortWarps = 16, kSortMoreWarps = 32;
constexpr int kSortMorePairs = 1 << 18;
// Slices of the experts, a cluster each, from so many pairs and experts on (65536
// pairs of 896 experts: one 11.4 us, six 6.5; eight clusters of sixteen CTAs do not
// run side by side and took twice four's time).
constexpr int kSortSlices = 6, kSortSlicePairs = 1 << 10, kSortSliceExperts = 16;
constexpr int kSortMaxCtas = 16;  // of the cluster
constexpr int kSortAhead = 8;     // groups of 32 pairs whose ids are on the way together

// ---- sort -------------------------------------------------------------------------
//
// A cluster sorts the pairs of its slice of the experts (one cluster all of
// them, where the pairs are few).  Every warp takes a run of all pairs, counts its
// pairs of each of the slice's experts in shared memory, and how many are at
// experts below it; after the counts have been summed over the warps before it,
// the CTAs before its own (distributed shared memory) and the experts before each,
// it goes through its run once more and gives each pair its place: the order within
// an expert is that of the pairs.
//
// Bound by latencies up to 30,000 pairs (128 pairs 3.1 us, 8192 4.4, 32768 5.3),
// then by the votes for equal keys and the scattered stores (65536 pairs 6.5 us,
// 1048576 40).
__global__ void __launch_bounds__(kSortThreads, 1) sort_kernel(const __grid_constant__ SortArgs a, int warps, int run,
                                                               int per_slice) {
    extern __shared__ int smem[];
    __shared__ int s_scan[kSortThreads / 32], s_lows[kSortThreads / 32], s_low;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // after the wait: only the offsets and places are still to come, which no
    // kernel reads ahead of its own
    if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int ctas = gridDim.x, slices = gridDim.y, slice = blockIdx.y, rank = blockIdx.x;
    const int e0 = slice * per_slice, E = min(per_slice, a.experts - e0);
    int *counts = smem;                          // [warps][E]
    int *total = smem + warps * E;               // [E] and the pairs below, read by the cluster
    int *base = total + E + 1;                   // [E]
    const int pairs = a.rows * a.topk;
    // a warp's run of pairs: whole groups of 32
    const long long from = (long long)(rank * warps + warp) * run;
    const int p0 = warp < warps ? (int)(from < pairs ? from : pairs) : pairs;
    const int p1 = (long long)p0 + run < pairs ? p0 + run : pairs;
    // an expert's number in the slice: negative below it and where the id is nobody's
    constexpr int kNone = -0x7FFFFFFF - 1;
    auto key_of = [&](int p) {
        if (p >= p1) return kNone;
        int id;
        if (a.ld_ids == a.topk) {
            id = a.ids[p];
        } else {
            const int r = p / a.topk;
            id = a.ids[(long long)r * a.ld_ids + (p - r * a.topk)];
        }
        const int k = (int)((unsigned)id - (unsigned)a.first);
        return id >= a.first && k < a.experts ? k - e0 : kNone;
    };
    // the first ids are on their way while the counts are cleared
    int keys[kSortAhead], low = 0;
    auto fetch = [&](int p) {
#pragma unroll
        for (int j = 0; j < kSortAhead; ++j) keys[j] = key_of(p + 32 * j + lane);
    };
    fetch(p0);
    for (int i = 4 * tid; i < warps * E; i += 4 * kSortThreads) {
        if (i + 4 <= warps * E)
            *reinterpret_cast<int4 *>(counts + i) = make_int4(0, 0, 0, 0);
        else
            for (int j = i; j < warps * E; ++j) counts[j] = 0;
    }
    __syncthreads();
    for (int p = p0; p < p1; p += 32 * kSortAhead) {
        if (p > p0) fetch(p);
#pragma unroll
        for (int j = 0; j < kSortAhead; ++j) {
            if ((unsigned)keys[j] < (unsigned)E)
                atomicAdd(&counts[warp * E + keys[j]], 1);
            else
                low += keys[j] < 0 && keys[j] != kNone;
        }
    }
    if (slices > 1) {
        low = __reduce_add_sync(0xFFFFFFFFu, low);
        if (lane == 0) s_lows[warp] = low;
    } else if (tid == 0) {
        s_low = 0;
    }
    __syncthreads();
    // counts become what the CTA's warps before hold; totals of the CTA
    const int e = tid;
    int mine = 0;
    if (e < E) {
        for (int w0 = 0; w0 < warps; w0 += 8) {  // eight loads on the way together
            int c[8];
#pragma unroll
            for (int w = 0; w < 8; ++w) c[w] = w0 + w < warps ? counts[(w0 + w) * E + e] : 0;
#pragma unroll
            for (int w = 0; w < 8; ++w) {
                if (w0 + w < warps) counts[(w0 + w) * E + e] = mine;
                mine += c[w];
            }
        }
        total[e] = mine;
    }
    if (slices > 1 && warp == kSortThreads / 32 - 1) {
        low = __reduce_add_sync(0xFFFFFFFFu, s_lows[lane]);
        if (lane == 0) total[E] = s_low = low;
    }
    int before = 0, all = mine;
    if (ctas > 1) {
        auto of_cta = [&](int i, int j) {
            int c;
            asm volatile("ld.shared::cluster.s32 %0, [%1];"
                         : "=r"(c)
                         : "r"(ptx::map_to_rank(ptx::smem_addr(total + i), (uint32_t)j))
                         : "memory");
            return c;
        };
        ptx::cluster_sync();
        if (e < E) {
            int c[kSortMaxCtas];
#pragma unroll
            for (int j = 0; j < kSortMaxCtas; ++j)
                if (j < ctas) c[j] = of_cta(e, j);
            all = 0;
#pragma unroll
            for (int j = 0; j < kSortMaxCtas; ++j)
                if (j < ctas) {
                    if (j < rank) before += c[j];
                    all += c[j];
                }
        }
        if (warp == kSortThreads / 32 - 1 && slices > 1) {  // the pairs below the slice, of all CTAs
            const int t = __reduce_add_sync(0xFFFFFFFFu, lane < ctas ? of_cta(E, lane) : 0);
            if (lane == 0) s_low = t;
        }
        __syncwarp();
        ptx::cluster_arrive();  // after the last remote read
    }
    // exclusive sums over the experts
    int scan = all;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int t = __shfl_up_sync(0xFFFFFFFFu, scan, d);
        if (lane >= d) scan += t;
    }
    if (lane == 31) s_scan[warp] = scan;
    __syncthreads();
    if (warp == 0) {
        int t = s_scan[lane];
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int u = __shfl_up_sync(0xFFFFFFFFu, t, d);
            if (lane >= d) t += u;
        }
        s_scan[lane] = t;
    }
    __syncthreads();
    scan += s_low + (warp > 0 ? s_scan[warp - 1] : 0);
    if (e < E) {
        base[e] = scan - all + before;
        if (rank == 0) {
            a.offsets[e0 + e + 1] = scan;
            if (e0 + e == 0) a.offsets[0] = 0;
        }
    }
    __syncthreads();
    const bool once = p0 + 32 * kSortAhead >= p1;  // the run's keys are still at hand
    for (int p = p0; p < p1; p += 32 * kSortAhead) {
        if (!once) fetch(p);
#pragma unroll
        for (int j = 0; j < kSortAhead; ++j) {
            const int at0 = p + 32 * j;
            if (at0 >= p1) break;
            const bool here = (unsigned)keys[j] < (unsigned)E;
            const int k = here ? keys[j] : -1;
            const unsigned same = __match_any_sync(0xFFFFFFFFu, k);
            const int at = here ? base[k] + counts[warp * E + k] + __popc(same & ((1u << lane) - 1u)) : -1;
            __syncwarp();
            if (here && (same >> lane) == 1u) counts[warp * E + k] += __popc(same);  // the last of them
            __syncwarp();
            // nobody's pairs are the first slice's to mark
            if (at0 + lane < p1 && (here || (slice == 0 && keys[j] == kNone))) {
                a.place[at0 + lane] = at;
                if (here && a.source != nullptr) a.source[at] = at0 + lane;
            }
        }
    }
    if (ctas > 1) ptx::cluster_wait();  // nobody leaves while another may read its totals
}

// ---- moves ------------------------------------------------------------------------

// The values of one 16-byte piece (W of a type), or of one element.
template <int TY, bool VEC>
struct Piece {
    static constexpr int kN = VEC ? 16 / layer_esize(TY) : 1;
    uint32_t w[VEC ? 4 : 1];
    __device__ __forceinline__ void load(const void *p, long long i) {
        if constexpr (VEC) {
            const uint4 t = *reinterpret_cast<const uint4 *>(static_cast<const char *>(p) + i * layer_esize(TY));
            w[0] = t.x, w[1] = t.y, w[2] = t.z, w[3] = t.w;
        } else if constexpr (TY == kFp32) {
            w[0] = static_cast<const uint32_t *>(p)[i];
        } else {
            w[0] = static_cast<const uint16_t *>(p)[i];
        }
    }
    __device__ __forceinline__ void store(void *p, long long i) const {
        if constexpr (VEC) {
            *reinterpret_cast<uint4 *>(static_cast<char *>(p) + i * layer_esize(TY)) = make_uint4(w[0], w[1], w[2], w[3]);
        } else if constexpr (TY == kFp32) {
            static_cast<uint32_t *>(p)[i] = w[0];
        } else {
            static_cast<uint16_t *>(p)[i] = (uint16_t)w[0];
        }
    }
    __device__ __forceinline__ void values(float (&v)[kN]) const {
        if constexpr (TY == kFp32) {
#pragma unroll
            for (int e = 0; e < kN; ++e) v[e] = __uint_as_float(w[e]);
        } else if constexpr (VEC) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 f = unpack16(w[e], TY);
                v[2 * e] = f.x, v[2 * e + 1] = f.y;
            }
        } else {
            v[0] = unpack16(w[0], TY).x;
        }
    }
    __device__ __forceinline__ void set(const float (&v)[kN]) {
        if constexpr (TY == kFp32) {
#pragma unroll
            for (int e = 0; e < kN; ++e) w[e] = __float_as_uint(v[e]);
        } else if constexpr (VEC) {
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = pack16(v[2 * e], v[2 * e + 1], TY);
        } else {
            w[0] = pack16(v[0], 0.f, TY) & 0xFFFFu;
        }
    }
};

// A row's places that are there, in the row's order.
struct Places {
    int n;
    int at[kMaxTopk];
    float w[kMaxTopk];
    int j[kMaxTopk];
};
__device__ __forceinline__ void find_places(const MoveArgs &a, int r, Places &s) {
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        const long long i = (long long)r * a.topk + lane;
        const int p = lane < a.topk ? a.place[i] : -1;
        const bool there = p >= 0 && p < a.pairs;
        const unsigned all = __ballot_sync(0xFFFFFFFFu, there);
        if (there) {
            const int k = __popc(all & ((1u << lane) - 1u));
            s.at[k] = p;
            s.w[k] = a.weights != nullptr ? a.weights[i] : 1.f;
            s.j[k] = lane;
        }
        if (lane == 0) s.n = __popc(all);
        if (a.dweights != nullptr && lane < a.topk && !there) a.dweights[i] = 0.f;
    }
    __syncthreads();
}

// A block a row: out[place] = x[row], each row read once.  Bound by HBM: 4096 rows
// of 3584 BF16 to 16 places 74 us (499 MB, 6.7 TB/s).
template <int ES, bool VEC>
__global__ void __launch_bounds__(256) gather_kernel(const __grid_constant__ MoveArgs a) {
    using P = Piece<ES == 4 ? kFp32 : kBf16, VEC>;
    __shared__ Places s;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int r = blockIdx.x;
    find_places(a, r, s);
    const int n = s.n, pieces = a.dim / P::kN;
    for (int i = blockIdx.y * blockDim.x + threadIdx.x; i < pieces && n > 0; i += gridDim.y * blockDim.x) {
        P p;
        p.load(a.a, r * a.ld_a + (long long)i * P::kN);
        for (int k = 0; k < n; ++k) p.store(a.out, s.at[k] * a.ld_out + (long long)i * P::kN);
    }
}

// A block a row: out[row] = residual[row] + sum_j w_j b[place_j], in the order
// of j.  Bound by HBM: 4096 rows of 3584 BF16 from 16 places, with a residual, 82
// us (529 MB, 6.5 TB/s), as the gather's gradient 74 (6.7).
constexpr int kAhead = 8;  // experts' rows on the way together
template <int TY, bool VEC>
__global__ void __launch_bounds__(256) combine_kernel(const __grid_constant__ MoveArgs a) {
    using P = Piece<TY, VEC>;
    __shared__ Places s;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int r = blockIdx.x;
    find_places(a, r, s);
    const int n = s.n, pieces = a.dim / P::kN;
    // single values: four a thread at a time, so that as much is on the way
    constexpr int kPieces = VEC ? 1 : 4, kRows = VEC ? kAhead : 4;
    for (int i0 = blockIdx.y * kPieces * blockDim.x + threadIdx.x; i0 < pieces; i0 += gridDim.y * kPieces * blockDim.x) {
        float sum[kPieces][P::kN] = {};
        P res[kPieces];
        auto each = [&](auto &&f) {
#pragma unroll
            for (int q = 0; q < kPieces; ++q) {
                const int i = i0 + q * (int)blockDim.x;
                if (kPieces == 1 || i < pieces) f(q, (long long)i * P::kN);
            }
        };
        if (a.a != nullptr) each([&](int q, long long c) { res[q].load(a.a, r * a.ld_a + c); });
        for (int k0 = 0; k0 < n; k0 += kRows) {
            P p[kPieces][kRows];
#pragma unroll
            for (int k = 0; k < kRows; ++k)
                if (k0 + k < n) each([&](int q, long long c) { p[q][k].load(a.b, s.at[k0 + k] * a.ld_b + c); });
#pragma unroll
            for (int k = 0; k < kRows; ++k)
                if (k0 + k < n) {
                    const float w = s.w[k0 + k];
                    each([&](int q, long long) {
                        float v[P::kN];
                        p[q][k].values(v);
#pragma unroll
                        for (int e = 0; e < P::kN; ++e)
                            sum[q][e] = a.weights != nullptr ? fmaf(w, v[e], sum[q][e]) : sum[q][e] + v[e];
                    });
                }
        }
        each([&](int q, long long c) {
            if (a.a != nullptr) {
                float v[P::kN];
                res[q].values(v);
#pragma unroll
                for (int e = 0; e < P::kN; ++e) sum[q][e] += v[e];
            }
            P o;
            o.set(sum[q]);
            o.store(a.out, r * a.ld_out + c);
        });
    }
}

// A block a row, `share` warps an expert's row at a time (all of the block's
// where there are few): out[place_j] = w_j dout[row], dweights_j = <dout[row],
// b[place_j]>.  Bound by HBM: 4096 rows of 3584 BF16 at 16 places 153 us (970 MB,
// 6.3 TB/s); rows off 16 bytes by accesses of one value (4096x1001 at 4 places 31).
constexpr int kBackWarps = 8;
template <int TY, bool VEC>
__global__ void __launch_bounds__(32 * kBackWarps) combine_backward_kernel(const __grid_constant__ MoveArgs a) {
    using P = Piece<TY, VEC>;
    // on the way together (16 bytes, 4096x3584: one 178 us, two 169, four 153)
    constexpr int kPieces = VEC ? 4 : 8;
    __shared__ Places s;
    __shared__ float s_dot[kMaxTopk][kBackWarps];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int r = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    find_places(a, r, s);
    const int n = s.n, pieces = a.dim / P::kN;
    const int share = n <= 1 ? 8 : n <= 2 ? 4 : n <= 4 ? 2 : 1;
    const int part = warp & (share - 1);
    for (int k = warp / share; k < n; k += kBackWarps / share) {
        const float w = s.w[k];
        const long long ia = r * a.ld_a, ib = s.at[k] * a.ld_b, io = s.at[k] * a.ld_out;
        float dot[P::kN] = {};
        for (int i = part * 32 + lane; i < pieces; i += share * 32 * kPieces) {
            P g[kPieces], y[kPieces];
#pragma unroll
            for (int q = 0; q < kPieces; ++q) {
                const int at = i + q * share * 32;
                if (at >= pieces) break;
                g[q].load(a.a, ia + (long long)at * P::kN);
                if (a.dweights != nullptr) y[q].load(a.b, ib + (long long)at * P::kN);
            }
#pragma unroll
            for (int q = 0; q < kPieces; ++q) {
                const int at = i + q * share * 32;
                if (at >= pieces) break;
                float gv[P::kN], v[P::kN];
                g[q].values(gv);
                if (a.dweights != nullptr) {
                    y[q].values(v);
#pragma unroll
                    for (int e = 0; e < P::kN; ++e) dot[e] = fmaf(gv[e], v[e], dot[e]);
                }
                if (a.out != nullptr) {
#pragma unroll
                    for (int e = 0; e < P::kN; ++e) v[e] = w * gv[e];
                    P o;
                    o.set(v);
                    o.store(a.out, io + (long long)at * P::kN);
                }
            }
        }
        float t = 0.f;
#pragma unroll
        for (int e = 0; e < P::kN; ++e) t += dot[e];
#pragma unroll
        for (int d = 16; d > 0; d /= 2) t += __shfl_xor_sync(0xFFFFFFFFu, t, d);
        if (lane == 0) s_dot[k][part] = t;
    }
    if (a.dweights == nullptr) return;
    __syncthreads();
    if (threadIdx.x < n) {
        float t = 0.f;
        for (int j = 0; j < share; ++j) t += s_dot[threadIdx.x][j];
        a.dweights[(long long)r * a.topk + s.j[threadIdx.x]] = t;
    }
}

// Rows that may be accessed 16 bytes at a time.
bool vectors(const MoveArgs &a) {
    const int es = layer_esize(a.type);
    auto rows_on = [&](const void *p, long long ld) {
        return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * es % 16 == 0);
    };
    return a.dim * es % 16 == 0 && rows_on(a.a, a.ld_a) && rows_on(a.b, a.ld_b) && rows_on(a.out, a.ld_out);
}

// Blocks of a row: one, or, where the rows are few, one for every piece a thread
// (1 row of 3584 from 16 places 4.9 us with one).
unsigned blocks_of_row(const MoveArgs &a, bool vec, int sms) {
    const int pieces = vec ? a.dim * layer_esize(a.type) / 16 : a.dim, blocks = (pieces + 255) / 256;
    return (long long)a.rows * blocks <= 4ll * sms ? (unsigned)blocks : 1u;
}

cudaError_t launch(const void *k, dim3 grid, unsigned block, size_t smem, unsigned cluster, void **params,
                   cudaStream_t stream) {
    cudaLaunchConfig_t c = {};
    cudaLaunchAttribute attr[2];
    c.gridDim = grid;
    c.blockDim = dim3(block);
    c.dynamicSmemBytes = smem;
    c.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    c.attrs = attr;
    c.numAttrs = 2;
    return cudaLaunchKernelExC(&c, k, params);
}

size_t sort_smem(int warps, int experts) { return (((size_t)warps + 2) * experts + 1) * sizeof(int); }

#define ROUTE_MOVE(K, A, V)                                                              \
    ((A).type == kFp32   ? reinterpret_cast<const void *>(K<kFp32, V>)                   \
     : (A).type == kFp16 ? reinterpret_cast<const void *>(K<kFp16, V>)                   \
                         : reinterpret_cast<const void *>(K<kBf16, V>))

}  // namespace

cudaError_t sort_configure() {
    const cudaError_t e = cudaFuncSetAttribute(sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)sort_smem(kSortMoreWarps, kMaxExperts));
    // sixteen CTAs a cluster
    return e != cudaSuccess ? e : cudaFuncSetAttribute(sort_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
}

SortShape sort_shape() {
    for (int ctas : {kSortMaxCtas, 8}) {
        cudaLaunchConfig_t c = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)ctas;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        c.gridDim = dim3((unsigned)ctas);
        c.blockDim = dim3(kSortThreads);
        c.dynamicSmemBytes = sort_smem(kSortMoreWarps, kMaxExperts);
        c.attrs = attr;
        c.numAttrs = 1;
        int clusters = 0;
        if (cudaOccupancyMaxActiveClusters(&clusters, sort_kernel, &c) != cudaSuccess) cudaGetLastError(), clusters = 0;
        if (clusters > 0) return {ctas, clusters < kSortSlices ? clusters : kSortSlices};
    }
    return {8, 1};
}

cudaError_t sort_launch(const SortArgs &args, SortShape most_of, cudaStream_t stream) {
    const long long pairs = (long long)args.rows * args.topk;
    const long long groups = (pairs + 31) / 32;
    const int most = pairs < kSortMorePairs ? kSortWarps : kSortMoreWarps;
    int warps = groups < most ? (int)(groups < 1 ? 1 : groups) : most;
    unsigned ctas = 1;
    while (ctas < (unsigned)most_of.ctas && groups > 2ll * ctas * most) ctas *= 2;
    const int slices = pairs >= kSortSlicePairs && args.experts >= kSortSliceExperts ? most_of.slices : 1;
    int per_slice = (args.experts + slices - 1) / slices;
    const long long runs = (long long)ctas * warps;
    int run = (int)(((pairs + runs - 1) / runs + 31) & ~31ll);
    void *params[] = {const_cast<SortArgs *>(&args), &warps, &run, &per_slice};
    // (slices that are rounded up may leave the last without experts)
    return launch(reinterpret_cast<const void *>(sort_kernel),
                  dim3(ctas, (unsigned)((args.experts + per_slice - 1) / per_slice)), kSortThreads,
                  sort_smem(warps, per_slice), ctas, params, stream);
}

cudaError_t gather_launch(const MoveArgs &args, int sms, cudaStream_t stream) {
    const bool vec = vectors(args);
    const void *k = layer_esize(args.type) == 4 ? (vec ? reinterpret_cast<const void *>(gather_kernel<4, true>)
                                                       : reinterpret_cast<const void *>(gather_kernel<4, false>))
                                                : (vec ? reinterpret_cast<const void *>(gather_kernel<2, true>)
                                                       : reinterpret_cast<const void *>(gather_kernel<2, false>));
    void *params[] = {const_cast<MoveArgs *>(&args)};
    return launch(k, dim3((unsigned)args.rows, blocks_of_row(args, vec, sms)), 256, 0, 1, params, stream);
}

cudaError_t combine_launch(const MoveArgs &args, int sms, cudaStream_t stream) {
    const bool vec = vectors(args);
    const void *k = vec ? ROUTE_MOVE(combine_kernel, args, true) : ROUTE_MOVE(combine_kernel, args, false);
    void *params[] = {const_cast<MoveArgs *>(&args)};
    return launch(k, dim3((unsigned)args.rows, blocks_of_row(args, vec, sms)), 256, 0, 1, params, stream);
}

cudaError_t combine_backward_launch(const MoveArgs &args, cudaStream_t stream) {
    const void *k = vectors(args) ? ROUTE_MOVE(combine_backward_kernel, args, true)
                                  : ROUTE_MOVE(combine_backward_kernel, args, false);
    void *params[] = {const_cast<MoveArgs *>(&args)};
    return launch(k, dim3((unsigned)args.rows), 32 * kBackWarps, 0, 1, params, stream);
}

}  // namespace route
