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
    extern __shared__ __align__(16) int smem[];  // the counts are cleared 16 bytes at a time
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

// What lies between a matrix's first value and its last.
struct Span {
    const char *lo, *hi;
    __device__ __forceinline__ Span(const void *p, long long rows, long long ld, int dim, int es)
        : lo(static_cast<const char *>(p)), hi(lo + ((rows - 1) * ld + dim) * es) {}
};

// 16 bytes' values of a row, for one of its `threads` threads.  VEC: every row of
// every matrix lies on 16 bytes.  Else 16-bit values are taken out of the two
// aligned 16 bytes that they lie in, of which what belongs to others is not used,
// and the pieces of a row are those that lie aligned where they are written
// (4096x1001 BF16, 4 places: combine with a residual 16.3 us and its gradient 24, a
// value at a time 23.5 and 31; 4096x2047 from 16 places 74 and 102); and FP32 values
// are a row's threads apart, so that a warp's accesses are whole stretches of it
// (2049x1001 from 4 places 11.1 us, in shifted pieces 14.2; combine's gradient
// 4096x1001 30 and 40).
template <int TY, bool VEC>
struct Piece {
    static constexpr int kSize = layer_esize(TY), kN = 16 / kSize;
    static constexpr bool kApart = !VEC && TY == kFp32, kShifted = !VEC && TY != kFp32;
    uint32_t w[kShifted ? 8 : 4];
    unsigned off = 0;  // where in w they begin, bytes

    // Where a row's pieces are: the i-th is from value i kN - skip on, `apart` apart.
    struct Way {
        int skip, count, apart;
        // a row that is written at p (or read, where it is not written); thread t of `threads`
        __device__ __forceinline__ Way(const void *p, int dim, int t, int threads) {
            skip = kApart ? (kN - 1) * t : kShifted ? (int)(reinterpret_cast<uintptr_t>(p) & 15u) / kSize : 0;
            count = kApart ? (dim + kN * threads - 1) / (kN * threads) * threads : (dim + skip + kN - 1) / kN;
            apart = kApart ? threads : 1;
        }
        __device__ __forceinline__ int at(int i) const { return i * kN - skip; }
    };

    // The values of `row` from the c-th on.
    __device__ __forceinline__ void load(const char *row, int c, int dim, const Way &way, const Span &in) {
        const char *p = row + (long long)c * kSize;
        if constexpr (VEC) {
            const uint4 t = *reinterpret_cast<const uint4 *>(p);
            w[0] = t.x, w[1] = t.y, w[2] = t.z, w[3] = t.w;
        } else if constexpr (kApart) {
#pragma unroll
            for (int e = 0; e < kN; ++e)
                w[e] = c + e * way.apart < dim ? reinterpret_cast<const uint32_t *>(p)[e * way.apart] : 0u;
        } else {
            off = (unsigned)(reinterpret_cast<uintptr_t>(p) & 15u);
            const char *q = p - off, *q1 = off != 0u ? q + 16 : q;
            if (q >= in.lo && q1 + 16 <= in.hi) {
                const uint4 t = *reinterpret_cast<const uint4 *>(q), u = *reinterpret_cast<const uint4 *>(q1);
                w[0] = t.x, w[1] = t.y, w[2] = t.z, w[3] = t.w;
                w[4] = u.x, w[5] = u.y, w[6] = u.z, w[7] = u.w;
            } else {  // the matrix's first and last
                off = 0u;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    w[e] = 0u;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const char *at = p + 4 * e + 2 * h;
                        if (at >= in.lo && at < in.hi)
                            w[e] |= (uint32_t)*reinterpret_cast<const uint16_t *>(at) << (16 * h);
                    }
                }
            }
        }
    }
    __device__ __forceinline__ void words(uint32_t (&o)[4]) const {
        if constexpr (!kShifted) {
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = w[e];
        } else {
            uint32_t t[7], u[5];
#pragma unroll
            for (int e = 0; e < 7; ++e) t[e] = off & 4u ? w[e + 1] : w[e];
#pragma unroll
            for (int e = 0; e < 5; ++e) u[e] = off & 8u ? t[e + 2] : t[e];
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = __funnelshift_r(u[e], u[e + 1], 8u * (off & 3u));
        }
    }
    __device__ __forceinline__ void values(float (&v)[kN]) const {
        uint32_t o[4];
        words(o);
        if constexpr (TY == kFp32) {
#pragma unroll
            for (int e = 0; e < kN; ++e) v[e] = __uint_as_float(o[e]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 f = unpack16(o[e], TY);
                v[2 * e] = f.x, v[2 * e + 1] = f.y;
            }
        }
    }
    // Whether the row has the e-th value of its piece from the c-th on.
    static __device__ __forceinline__ bool has(int c, int e, int dim, const Way &way) {
        return VEC || (c + e * way.apart >= 0 && c + e * way.apart < dim);
    }
    // The values of `row` from the c-th on, those of them that it has.
    static __device__ __forceinline__ void store(char *row, int c, int dim, const Way &way, const uint32_t (&o)[4]) {
        char *p = row + (long long)c * kSize;
        if (!kApart && (VEC || (c >= 0 && c + kN <= dim))) {
            *reinterpret_cast<uint4 *>(p) = make_uint4(o[0], o[1], o[2], o[3]);
        } else {
#pragma unroll
            for (int e = 0; e < kN; ++e) {
                if (!has(c, e, dim, way)) continue;
                if constexpr (kSize == 4)
                    reinterpret_cast<uint32_t *>(p)[e * way.apart] = o[e];
                else
                    reinterpret_cast<uint16_t *>(p)[e] = (uint16_t)(o[e / 2] >> (16 * (e % 2)));
            }
        }
    }
    static __device__ __forceinline__ void store(char *row, int c, int dim, const Way &way, const float (&v)[kN]) {
        uint32_t o[4];
        if constexpr (TY == kFp32) {
#pragma unroll
            for (int e = 0; e < kN; ++e) o[e] = __float_as_uint(v[e]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = pack16(v[2 * e], v[2 * e + 1], TY);
        }
        store(row, c, dim, way, o);
    }
};

template <int TY>
__device__ __forceinline__ const char *row_of(const void *p, long long ld, long long r) {
    return static_cast<const char *>(p) + r * ld * layer_esize(TY);
}
template <int TY>
__device__ __forceinline__ char *row_of(void *p, long long ld, long long r) {
    return static_cast<char *>(p) + r * ld * layer_esize(TY);
}

// A row's places that are there, in the row's order.
struct Places {
    int n;
    int at[kMaxTopk];
    float w[kMaxTopk];
};

// Row r's places, found by the row's first 32 threads (none of a row that is not
// there); for all of the block.
__device__ __forceinline__ void find_places(const MoveArgs &a, int r, Places &s) {
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        const long long i = (long long)r * a.topk + lane;
        const bool mine = lane < a.topk && r < a.rows;
        const int p = mine ? a.place[i] : -1;
        const bool there = p >= 0 && p < a.pairs;
        const unsigned all = __ballot_sync(0xFFFFFFFFu, there);
        if (there) {
            const int k = __popc(all & ((1u << lane) - 1u));
            s.at[k] = p;
            s.w[k] = a.weights != nullptr ? a.weights[i] : 1.f;
        }
        if (lane == 0) s.n = __popc(all);
    }
    __syncthreads();
}

// Rows of gather and combine: a row's threads, a piece each, up to 256; rows of a
// block of 128 threads (a block of one warp a row: half the warps that an SM
// holds); and blocks of a row: one, or, where the rows are few, as many as its
// pieces take (1 row of 3584 from 16 places 4.9 us with one).
constexpr int kRowThreads = 256, kBlockThreads = 128, kMostRows = kBlockThreads / 32;
struct RowShape {
    dim3 grid, block;
    RowShape(const MoveArgs &a, int sms) {
        const int pieces = (a.dim * layer_esize(a.type) + 15) / 16;
        const unsigned threads = pieces < kRowThreads ? (unsigned)(pieces + 31) / 32 * 32 : kRowThreads;
        const unsigned rows = threads < kBlockThreads ? kBlockThreads / threads : 1u;
        block = dim3(threads, rows);
        const unsigned blocks = (unsigned)(pieces + kRowThreads - 1) / kRowThreads;
        grid = dim3(((unsigned)a.rows + rows - 1) / rows, (long long)a.rows * blocks > 4ll * sms ? 1u : blocks);
    }
};

// out[place] = x[row], each row read once.  Bound by HBM: 4096 rows of 3584 BF16 to
// 16 places 74 us (499 MB, 6.7 TB/s).  Short rows are bound by how many are on
// their way, so a row has no more threads than pieces (with the sort, 4096x128 to 16
// places 10.4 us; a block of 256 threads a row 14.3).
template <int ES>
__global__ void __launch_bounds__(256) gather_kernel(const __grid_constant__ MoveArgs a) {
    constexpr int TY = ES == 4 ? kFp32 : kBf16;
    using P = Piece<TY, true>;
    __shared__ Places places[kMostRows];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int r = blockIdx.x * blockDim.y + threadIdx.y;
    Places &s = places[threadIdx.y];
    const int first = blockIdx.y * blockDim.x + threadIdx.x, step = gridDim.y * blockDim.x;
    const Span in(a.a, a.rows, a.ld_a, a.dim, ES);
    const char *x = row_of<TY>(a.a, a.ld_a, r);
    const typename P::Way way(a.out, a.dim, (int)threadIdx.x, (int)blockDim.x);
    P p;
    if (first < way.count && r < a.rows) p.load(x, way.at(first), a.dim, way, in);  // beside the places
    find_places(a, r, s);
    const int n = s.n;
    for (int i = first; i < way.count && n > 0; i += step) {
        if (i != first) p.load(x, way.at(i), a.dim, way, in);
        uint32_t o[4];
        p.words(o);
        for (int k = 0; k < n; ++k) P::store(row_of<TY>(a.out, a.ld_out, s.at[k]), way.at(i), a.dim, way, o);
    }
}

// The pair of (row, place) that `threads` threads (a power of two) of a block have.
struct Pair {
    int part;  // which of them this thread is
    unsigned at, row;
    int place;  // -1: there is none
    bool mine;  // the pair is there, with or without a place
    __device__ __forceinline__ Pair(const MoveArgs &a, int threads)
        : part((int)threadIdx.x & (threads - 1)),
          at(blockIdx.x * (blockDim.x / (unsigned)threads) + threadIdx.x / (unsigned)threads),
          row(at / (unsigned)a.topk), place(-1), mine(row < (unsigned)a.rows) {
        if (mine) place = a.place[at];
        if (place >= a.pairs) place = -1;
    }
};

// gather_kernel for rows off 16 bytes: each place has its own alignment, and so its
// own pieces.
template <int ES>
__global__ void __launch_bounds__(256) gather_any_kernel(const __grid_constant__ MoveArgs a, int threads) {
    constexpr int TY = ES == 4 ? kFp32 : kBf16;
    using P = Piece<TY, false>;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Pair pair(a, threads);
    if (pair.place < 0) return;
    const Span in(a.a, a.rows, a.ld_a, a.dim, ES);
    const char *x = row_of<TY>(a.a, a.ld_a, pair.row);
    char *out = row_of<TY>(a.out, a.ld_out, pair.place);
    const typename P::Way way(out, a.dim, pair.part, threads);
    for (int i = pair.part; i < way.count; i += threads) {
        P p;
        p.load(x, way.at(i), a.dim, way, in);
        uint32_t o[4];
        p.words(o);
        P::store(out, way.at(i), a.dim, way, o);
    }
}

// Blocks an SM of combine_kernel: as many rows on their way as the registers of
// AHEAD places' pieces leave room for (4096x3584 from 16 places: 64 registers 82 us,
// 69 87).  Those of two places, of eight, and of rows off 16 bytes spill 12 to 68
// bytes for it; a block less spills nothing and is mostly slower (4096 rows, BF16: 2048
// from 2 places 13.4 us, 14.1; 3584 from 16 83.6, 88.3; 2047 from 16 77, 89; but FP32,
// 512 from 2, 7.8 and 7.5).
constexpr int combine_blocks(bool vec, int ahead) {
    return ahead <= 2 ? 7 : ahead <= 4 && vec ? 5 : 4;
}

// out[row] = residual[row] + sum_j w_j b[place_j], in the order of j, AHEAD of the
// experts' rows on the way together: fewer where a row has few places (4096x2048
// from 2 places 11.9 us, with eight ahead 18.4).  Bound by HBM: 4096 rows of 3584 BF16
// from 16 places, with a residual, 84 us (529 MB, 6.3 TB/s), as the gather's gradient
// 75 (6.6); short rows as gather's (4096x512 from 8 places 6.4 us, a block of 256
// threads a row 12.5).
template <int TY, bool VEC, int AHEAD>
__global__ void __launch_bounds__(256, combine_blocks(VEC, AHEAD))
    combine_kernel(const __grid_constant__ MoveArgs a) {
    using P = Piece<TY, VEC>;
    __shared__ Places places[kMostRows];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int r = blockIdx.x * blockDim.y + threadIdx.y;
    Places &s = places[threadIdx.y];
    find_places(a, r, s);
    if (r >= a.rows) return;
    char *out = row_of<TY>(a.out, a.ld_out, r);
    const int n = s.n;
    const typename P::Way way(out, a.dim, (int)threadIdx.x, (int)blockDim.x);
    const Span in(a.b, a.pairs, a.ld_b, a.dim, P::kSize), res_in(a.a, a.rows, a.ld_a, a.dim, P::kSize);
    for (int i = blockIdx.y * blockDim.x + threadIdx.x; i < way.count; i += gridDim.y * blockDim.x) {
        const int c = way.at(i);
        float sum[P::kN] = {};
        P res;
        if (a.a != nullptr) res.load(row_of<TY>(a.a, a.ld_a, r), c, a.dim, way, res_in);
        for (int k0 = 0; k0 < n; k0 += AHEAD) {
            P p[AHEAD];
#pragma unroll
            for (int k = 0; k < AHEAD; ++k)
                if (k0 + k < n) p[k].load(row_of<TY>(a.b, a.ld_b, s.at[k0 + k]), c, a.dim, way, in);
#pragma unroll
            for (int k = 0; k < AHEAD; ++k)
                if (k0 + k < n) {
                    const float w = s.w[k0 + k];
                    float v[P::kN];
                    p[k].values(v);
#pragma unroll
                    for (int e = 0; e < P::kN; ++e)
                        sum[e] = a.weights != nullptr ? fmaf(w, v[e], sum[e]) : sum[e] + v[e];
                }
        }
        if (a.a != nullptr) {
            float v[P::kN];
            res.values(v);
#pragma unroll
            for (int e = 0; e < P::kN; ++e) sum[e] += v[e];
        }
        P::store(out, c, a.dim, way, sum);
    }
}

// `threads` threads a pair, none of which waits for another pair's: out[place_j] =
// w_j dout[row], dweights_j = <dout[row], b[place_j]>.  Bound by HBM: 4096 rows of
// 3584 BF16 at 16 places 148 us (970 MB, 6.5 TB/s; a block a row 153).  Two pieces of
// each matrix on the way and 48 registers (one piece 175, four and 72 registers
// 159; 4096x1000 at 4 places 16.1 us, 20.0 and 18.4; a block a row 28.8).  Of 16-bit
// rows off 16 bytes 40 bytes are spilled (four blocks an SM, no spills: 4096x2047 at 16
// places 160 us, so 158; 4096x1001 at 4 23.7 and 25.4).
template <int TY, bool VEC>
__global__ void __launch_bounds__(256, 5) combine_backward_kernel(const __grid_constant__ MoveArgs a, int threads) {
    using P = Piece<TY, VEC>;
    constexpr int kPieces = P::kShifted ? 1 : 2;  // on the way together (a shifted piece is two loads)
    __shared__ float s_dot[8];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Pair pair(a, threads);
    float dot[P::kN] = {};
    if (pair.place >= 0) {
        const float w = a.weights != nullptr ? a.weights[pair.at] : 1.f;
        const Span g_in(a.a, a.rows, a.ld_a, a.dim, P::kSize), y_in(a.b, a.pairs, a.ld_b, a.dim, P::kSize);
        const char *g_row = row_of<TY>(a.a, a.ld_a, pair.row), *y_row = row_of<TY>(a.b, a.ld_b, pair.place);
        char *out = row_of<TY>(a.out, a.ld_out, pair.place);
        const typename P::Way way(a.out != nullptr ? out : y_row, a.dim, pair.part, threads);
        for (int i = pair.part; i < way.count; i += threads * kPieces) {
            P g[kPieces], y[kPieces];
#pragma unroll
            for (int q = 0; q < kPieces; ++q) {
                const int at = i + q * threads;
                if (at >= way.count) break;
                g[q].load(g_row, way.at(at), a.dim, way, g_in);
                if (a.dweights != nullptr) y[q].load(y_row, way.at(at), a.dim, way, y_in);
            }
#pragma unroll
            for (int q = 0; q < kPieces; ++q) {
                const int at = i + q * threads;
                if (at >= way.count) break;
                const int c = way.at(at);
                float gv[P::kN], v[P::kN];
                g[q].values(gv);
                if (a.dweights != nullptr) {
                    y[q].values(v);
                    // (values apart that the row does not have are zeros)
                    const bool whole = !P::kShifted || (c >= 0 && c + P::kN <= a.dim);
#pragma unroll
                    for (int e = 0; e < P::kN; ++e)
                        if (whole || P::has(c, e, a.dim, way)) dot[e] = fmaf(gv[e], v[e], dot[e]);
                }
                if (a.out != nullptr) {
#pragma unroll
                    for (int e = 0; e < P::kN; ++e) v[e] = w * gv[e];
                    P::store(out, c, a.dim, way, v);
                }
            }
        }
    }
    if (a.dweights == nullptr) return;
    float t = 0.f;
#pragma unroll
    for (int e = 0; e < P::kN; ++e) t += dot[e];
    for (int d = (threads < 32 ? threads : 32) / 2; d > 0; d /= 2) t += __shfl_xor_sync(0xFFFFFFFFu, t, d);
    if (threads > 32) {
        if (lane == 0) s_dot[warp] = t;
        __syncthreads();
        if (pair.part != 0) return;
        t = 0.f;
        for (int j = 0; j < threads / 32; ++j) t += s_dot[warp + j];
    }
    if (pair.part == 0 && pair.mine) a.dweights[pair.at] = pair.place >= 0 ? t : 0.f;
}

// Rows that may be accessed 16 bytes at a time.
bool vectors(const MoveArgs &a) {
    const int es = layer_esize(a.type);
    auto rows_on = [&](const void *p, long long ld) {
        return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * es % 16 == 0);
    };
    return a.dim * es % 16 == 0 && rows_on(a.a, a.ld_a) && rows_on(a.b, a.ld_b) && rows_on(a.out, a.ld_out);
}

cudaError_t launch(const void *k, dim3 grid, dim3 block, size_t smem, unsigned cluster, void **params,
                   cudaStream_t stream) {
    cudaLaunchConfig_t c = {};
    cudaLaunchAttribute attr[2];
    c.gridDim = grid;
    c.blockDim = block;
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

// Threads of a pair (a power of two), and the grid for blocks of 256: up to a warp,
// but four pieces each (4096x256 at 16 places 16.2 us, a piece each 30; 512 at 8
// 16.0 and 19.1); more than a warp where the pairs are few.
int pair_threads(const MoveArgs &a, int sms, dim3 &grid) {
    const int pieces = (a.dim * layer_esize(a.type) + 15) / 16;
    const long long pairs = (long long)a.rows * a.topk;
    int threads = 8;
    while (threads < 256 && threads < pieces &&
           (pairs * threads < 1024ll * sms || (threads < 32 && 8 * threads <= pieces)))
        threads *= 2;
    const int per_block = 256 / threads;
    grid = dim3((unsigned)((pairs + per_block - 1) / per_block));
    return threads;
}

cudaError_t gather_launch(const MoveArgs &args, int sms, cudaStream_t stream) {
    const bool four = layer_esize(args.type) == 4;
    dim3 grid;
    int threads = pair_threads(args, sms, grid);
    void *params[] = {const_cast<MoveArgs *>(&args), &threads};
    if (!vectors(args))
        return launch(four ? reinterpret_cast<const void *>(gather_any_kernel<4>)
                           : reinterpret_cast<const void *>(gather_any_kernel<2>),
                      grid, 256, 0, 1, params, stream);
    const RowShape shape(args, sms);
    return launch(four ? reinterpret_cast<const void *>(gather_kernel<4>)
                       : reinterpret_cast<const void *>(gather_kernel<2>),
                  shape.grid, shape.block, 0, 1, params, stream);
}

cudaError_t combine_launch(const MoveArgs &args, int sms, cudaStream_t stream) {
    const bool vec = vectors(args);
#define ROUTE_COMBINE(T)                                                                             \
    (!vec             ? reinterpret_cast<const void *>(combine_kernel<T, false, 4>) \
     : args.topk <= 2 ? reinterpret_cast<const void *>(combine_kernel<T, true, 2>)                   \
     : args.topk <= 4 ? reinterpret_cast<const void *>(combine_kernel<T, true, 4>)                   \
                      : reinterpret_cast<const void *>(combine_kernel<T, true, 8>))
    const void *k = args.type == kFp32   ? ROUTE_COMBINE(kFp32)
                    : args.type == kFp16 ? ROUTE_COMBINE(kFp16)
                                         : ROUTE_COMBINE(kBf16);
#undef ROUTE_COMBINE
    void *params[] = {const_cast<MoveArgs *>(&args)};
    const RowShape shape(args, sms);
    return launch(k, shape.grid, shape.block, 0, 1, params, stream);
}

cudaError_t combine_backward_launch(const MoveArgs &args, int sms, cudaStream_t stream) {
    const bool vec = vectors(args);
    const void *k = vec ? ROUTE_MOVE(combine_backward_kernel, args, true)
                        : ROUTE_MOVE(combine_backward_kernel, args, false);
    dim3 grid;
    int threads = pair_threads(args, sms, grid);
    void *params[] = {const_cast<MoveArgs *>(&args), &threads};
    return launch(k, grid, 256, 0, 1, params, stream);
}

}  // namespace route
