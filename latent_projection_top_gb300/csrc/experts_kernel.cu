// The routed experts' matrix products on the sm_103a tensor cores, two SMs per
// tile: every expert's weights meet the run of sorted rows that is its own.
//
//   D[r, c] = sum_k A[r, k] B_e[k, c]     offsets[e] <= r < offsets[e + 1]
//   dW_e[m, n] = sum_r A[r, m] B[r, n]    over the same rows
//
// 16-bit operands, FP32 sums, and what the operator makes of them before they
// are written (layer_math.cuh: epilogue).  How many rows an expert has is known
// on the device only: a launch is as many CTA pairs as the GPU holds, and each
// finds its tiles from the offsets.
//
// Rows kernel: columns of D (the weights') are the tensor cores' M side, 256 a
// tile and 128 a CTA, rows their N side, as many as there are up to 256 in
// steps of 32: an expert with two rows costs the reading of its weights, one
// with a thousand runs at the tensor cores' rate, and no rule chooses between
// them.  Longer runs are cut into parts (make_table).  Bound by HBM where experts
// have few rows (8 to 22 rows of 3584x2048 at 8 to 16 experts 62-112 us, 352-705 MB
// of weights, 5.4-6.5 TB/s by how the tiles divide over the pairs), by the tensor
// cores where they have many (12600 to 22900 rows at 16 experts of 3584x2048 398-603
// us, 1,370-1,690 TFLOP/s, by the power limit and how the parts divide), in between by
// whole rounds of tiles over the pairs, and by 3 us of a launch's start (0.7 of it the
// table) and 3 of the last epilogue.
//
// Gradient kernel: rows of dW are the M side, its columns the N side, 256 x 256
// a tile.  The last block of an expert's rows holds rows of the next one: what of
// them the tensor cores would read, 16 rows at a time, is overwritten with zeros in
// shared memory, in both operands (a product with zero would keep an infinity or
// a NaN).  Bound by what it writes where experts have few rows (256 experts of
// 1024x512 with 63 rows each, 805 MB: 158 us, 5.1 TB/s), by the tensor cores else.
//
// Warp roles, waits and their limits as in layer_gemm.cu.
#include "experts.cuh"
#include "layer_math.cuh"
#include "layer_ptx.cuh"

namespace route {
namespace {

constexpr uint32_t kSmemLimit = 227 * 1024;
constexpr uint32_t kWaitHintNs = 20000;

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

template <class Args>
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, const Args &a, volatile int *abort_flag) {
    if (ptx::mbar_try_wait_hint(bar, parity, kWaitHintNs)) return true;
    const uint64_t t0 = ptx::global_timer_ns();
    for (;;) {
        if (ptx::mbar_try_wait_hint(bar, parity, kWaitHintNs)) return true;
        if (*abort_flag) return false;
        if (ptx::global_timer_ns() - t0 > a.timeout_ns) {
            *abort_flag = 1;
            atomicOr(a.status, kStatusTimeout);
            return false;
        }
    }
}

// The same by all lanes of a warp, with one answer.  The MMA issuer's loop is the
// whole warp's and one lane issues: what it works out is then the same in all
// lanes, as the MMAs need their operands (a k-block's four MMAs took a thread
// alone 250 cycles to issue, the warp 65; the producer's copies gain nothing).
template <class Args>
__device__ __forceinline__ bool wait_phase_warp(uint32_t bar, uint32_t parity, const Args &a, volatile int *abort_flag) {
    if (__all_sync(0xFFFFFFFFu, ptx::mbar_try_wait_hint(bar, parity, kWaitHintNs))) return true;
    return __all_sync(0xFFFFFFFFu, wait_phase(bar, parity, a, abort_flag));
}
__device__ __forceinline__ int same(int v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }

// Bounded wait used only while tearing down.
template <class Args>
__device__ __forceinline__ void wait_drain(uint32_t bar, uint32_t parity, const Args &a) {
    const uint64_t t0 = ptx::global_timer_ns();
    while (!ptx::mbar_try_wait_hint(bar, parity, kWaitHintNs)) {
        if (ptx::global_timer_ns() - t0 > a.timeout_ns) {
            atomicOr(a.status, kStatusTimeout);
            return;
        }
    }
}

// The rows of expert e: within 0 .. rows whatever the offsets say.
struct Run {
    int lo, hi;
};
__device__ __forceinline__ Run run_of(int from, int to, int rows) {
    Run r;
    r.lo = min(max(from, 0), rows);
    r.hi = max(min(to, rows), r.lo);
    return r;
}

// ---- rows -------------------------------------------------------------------------

constexpr int kEpiGroups = 4;                               // of four epilogue warps
constexpr int kRowsThreads = 64 + 128 * kEpiGroups;
constexpr int kRowsStages = 10;                             // at most
constexpr uint32_t kWBytes = 128 * 64 * 2;                  // a CTA's weight columns of a k-block
constexpr uint32_t kRowBytes = 64 * 2;                      // one row of it
constexpr int kTurnRows = 16;                               // rows an epilogue group turns around at once
constexpr uint32_t kTurnBytes = kTurnRows * 128 * 4;
constexpr uint32_t kRowsBars = 256;
constexpr int kPartTable = 2048;                            // parts that are looked up
constexpr uint32_t kRowsTable = kPartTable * 8 + 2 * (kMaxExperts + 4) * 4;
// What is left is the stages': as many as fit of the size that the largest
// part needs (five with 256 rows, nine with 32), so that short parts, which are
// bound by memory, have more on the way.
constexpr uint32_t kRowsRing = (kSmemLimit - 1024 - kEpiGroups * kTurnBytes - kRowsBars - kRowsTable) & ~1023u;
constexpr uint32_t kRowsSmem = 1024 + kRowsRing + kEpiGroups * kTurnBytes + kRowsBars + kRowsTable;
static_assert(kRowsSmem <= kSmemLimit && kRowsRing >= 5 * (kWBytes + kExpertRows / 2 * kRowBytes), "shared memory");

// A tile: expert, rows row0 .. end, column tile, columns of the MMA (rows
// rounded up to 32).
struct Tile {
    int e, row0, end, tn, n;
};
// In shared memory: the first kPartTable parts (their first row; expert and, from
// bit 16 on, rows), parts of the experts before each ([experts]: all of them), and
// the offsets.
struct Table {
    int2 *part;
    int *first, *offsets;
    int shift;  // parts have up to 1 << shift rows
};
// The rows of each of an expert's parts but the last: equal, in steps of 32 (8192
// rows of 3584x2048: 444 us, the last one what is left: 452).  No part is empty,
// because a step is no more than the most.
__device__ __forceinline__ int part_step(int rows, int parts) {
    return parts > 1 ? ((rows + parts - 1) / parts + 31) & ~31 : rows;
}

// A pair's tiles, one after another: i = part * tiles_n + tn goes up by `pairs`
// without a division, and a part is one access (a division and a binary search a
// tile took each role 0.4 us).
struct RowsWalk {
    int part, tn, dpart, dtn;
    __device__ __forceinline__ RowsWalk(const ExpertsArgs &a, unsigned pair) {
        dpart = a.pairs / a.tiles_n, dtn = a.pairs - dpart * a.tiles_n;
        part = (int)pair / a.tiles_n, tn = (int)pair - part * a.tiles_n;
    }
    __device__ __forceinline__ void next(const ExpertsArgs &a) {
        part += dpart, tn += dtn;
        if (tn >= a.tiles_n) tn -= a.tiles_n, ++part;
    }
    __device__ __forceinline__ Tile tile(const ExpertsArgs &a, const Table &t) const {
        Tile x;
        x.tn = tn;
        if (part < kPartTable) {
            const int2 p = t.part[part];
            x.row0 = p.x, x.e = p.y & 0xFFFF, x.end = p.x + (p.y >> 16);
        } else {
            int lo = 0, hi = a.experts;  // first[lo] <= part < first[hi]
            while (hi - lo > 1) {
                const int m = (lo + hi) >> 1;
                if (t.first[m] <= part)
                    lo = m;
                else
                    hi = m;
            }
            x.e = lo;
            const Run r = run_of(t.offsets[lo], t.offsets[lo + 1], a.rows);
            const int step = part_step(r.hi - r.lo, (r.hi - r.lo + (1 << t.shift) - 1) >> t.shift);
            x.row0 = r.lo + (part - t.first[lo]) * step;
            x.end = min(r.hi, x.row0 + step);
        }
        x.n = (x.end - x.row0 + 31) & ~31;
        return x;
    }
};

// The time of a launch whose parts have up to `n` rows, in ns: a k-block of a
// tile takes 342 at 256 rows and 290 at 128 (a tile of half the rows is not half as
// long), its epilogue `epi_ns` for 64 rows and 400 for itself; the last one is in
// nobody's shadow.  Taking a k-block's time for that of its copies, and an epilogue's
// without the 400, cut launches of many rows too small: 19456 rows of 512x1024 104
// us, so 81; 11733 of 648x1528 at five experts 85 and 64.
__device__ __forceinline__ float launch_ns(const ExpertsArgs &a, int parts, int n, float epi_ns) {
    const float rounds = ceilf((float)parts * a.tiles_a_pair);
    const float blocks = (float)a.kblocks * (237.f + 0.41f * n), epi = (float)((n + 63) >> 6) * epi_ns;
    return rounds * fmaxf(blocks, epi + 400.f) + epi;
}

// All threads: the table of parts.  Returns the number of them; `most`: the
// rows of the largest part, rounded up to 32.
//
// Parts have up to 256 rows, or, where that leaves too few tiles for the pairs,
// up to 128, 64 or 32: more tiles read the same weights, from L2, and each
// pair's share and last epilogue are shorter.
__device__ __forceinline__ int make_table(const ExpertsArgs &a, Table &t, float epi_ns, int *scan, int &most) {
    constexpr int kEach = 2, kSizes = 4, kLargest = 8, kWarps = kRowsThreads / 32;
    static_assert(1 << kLargest == kExpertRows, "parts");
    static_assert(kEach * kRowsThreads >= kMaxExperts && kWarps <= 32, "a thread's experts, a lane a warp");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int o[kEach + 1], rows[kEach], lo[kEach], most_rows = 0;
    // from L2: a chained kernel reads them ahead of its wait
#pragma unroll
    for (int j = 0; j <= kEach; ++j) {
        const int e = tid * kEach + j;
        o[j] = e <= a.experts ? __ldcg(a.offsets + e) : 0;
    }
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        const int e = tid * kEach + j;
        if (e <= a.experts) t.offsets[e] = o[j];
        const Run r = run_of(o[j], o[j + 1], a.rows);
        lo[j] = r.lo;
        rows[j] = e < a.experts ? r.hi - r.lo : 0;
        most_rows = max(most_rows, rows[j]);
    }
    auto parts_of = [&](int rows, int shift) { return (rows + (1 << shift) - 1) >> shift; };
    // parts for each size of them, and the most rows of an expert
#pragma unroll
    for (int c = 0; c < kSizes; ++c) {
        int sum = 0;
#pragma unroll
        for (int j = 0; j < kEach; ++j) sum += parts_of(rows[j], kLargest - c);
        sum = __reduce_add_sync(0xFFFFFFFFu, sum);
        if (lane == 0) scan[c * kWarps + warp] = sum;
    }
    most_rows = __reduce_max_sync(0xFFFFFFFFu, most_rows);
    if (lane == 0) scan[kSizes * kWarps + warp] = most_rows;
    __syncthreads();
    auto of_warp = [&](int i) { return lane < kWarps ? scan[i * kWarps + lane] : 0; };
    most_rows = __reduce_max_sync(0xFFFFFFFFu, of_warp(kSizes));
    float best = 0.f;
    t.shift = kLargest;
    most = max(32, min(kExpertRows, (most_rows + 31) & ~31));
    if (most_rows > 32) {
#pragma unroll
        for (int c = 0; c < kSizes; ++c) {
            const int parts = __reduce_add_sync(0xFFFFFFFFu, of_warp(c));
            const int n = min(1 << (kLargest - c), (most_rows + 31) & ~31);
            const float ns = launch_ns(a, parts, n, epi_ns);
            if (c == 0 || ns < best) best = ns, t.shift = kLargest - c, most = n;
        }
    }
    int before = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? of_warp(kLargest - t.shift) : 0);
    int parts[kEach], sum = 0;
#pragma unroll
    for (int j = 0; j < kEach; ++j) parts[j] = parts_of(rows[j], t.shift), sum += parts[j];
    int incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, incl, d);
        if (lane >= d) incl += u;
    }
    before += incl - sum;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        const int e = tid * kEach + j;
        if (e < a.experts) t.first[e] = before;
        const int step = part_step(rows[j], parts[j]);
        auto put = [&](int e, int lo, int rows, int step, int at, int k) {
            if (at + k < kPartTable) t.part[at + k] = make_int2(lo + k * step, e | min(step, rows - k * step) << 16);
        };
        // few parts by the expert's thread, many by its warp
        constexpr int kFew = 8;
        if (parts[j] <= kFew)
            for (int k = 0; k < parts[j]; ++k) put(e, lo[j], rows[j], step, before, k);
        for (unsigned many = __ballot_sync(0xFFFFFFFFu, parts[j] > kFew); many != 0u; many &= many - 1u) {
            const int from = __ffs(many) - 1;
            const int e1 = __shfl_sync(0xFFFFFFFFu, e, from), lo1 = __shfl_sync(0xFFFFFFFFu, lo[j], from),
                      rows1 = __shfl_sync(0xFFFFFFFFu, rows[j], from), step1 = __shfl_sync(0xFFFFFFFFu, step, from),
                      at1 = __shfl_sync(0xFFFFFFFFu, before, from), parts1 = __shfl_sync(0xFFFFFFFFu, parts[j], from);
            for (int k = lane; k < parts1 && at1 + k < kPartTable; k += 32) put(e1, lo1, rows1, step1, at1, k);
        }
        before += parts[j];
        if (e == a.experts - 1) t.first[a.experts] = before;
    }
    __syncthreads();
    return t.first[a.experts];
}

// EPI: what the epilogue makes of the sums; W_MN: the weights' columns are
// contiguous in memory (forward), else the contraction is (gradients).
template <int EPI, bool W_MN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kRowsThreads, 1)
    experts_rows_kernel(const __grid_constant__ ExpertsMaps maps, const __grid_constant__ ExpertsArgs args) {
    constexpr int kCtaCols = EPI == kEpiGated ? 64 : 128;  // columns of D a CTA
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t s_tmem_base;
    __shared__ volatile int s_abort;
    __shared__ int s_scan[5 * kRowsThreads / 32];

    const uint32_t raw = ptx::smem_addr(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    const uint32_t turn = sbase + kRowsRing;
    const uint32_t bars = turn + kEpiGroups * kTurnBytes;
    int2 *const part_table = reinterpret_cast<int2 *>(smem_raw + (bars + kRowsBars - raw));
    int *const words = reinterpret_cast<int *>(part_table + kPartTable);
    Table table = {part_table, words, words + kMaxExperts + 4, 0};
    auto full_bar = [&](int s) { return bars + 8u * s; };  // leader's are used
    auto empty_bar = [&](int s) { return bars + 8u * (kRowsStages + s); };
    auto tfull_bar = [&](int t) { return bars + 8u * (2 * kRowsStages + t); };
    auto tempty_bar = [&](int t) { return bars + 8u * (2 * kRowsStages + 2 + t); };  // leader's
    const uint32_t drain_bar = bars + 8u * (2 * kRowsStages + 4);

    const uint32_t rank = ptx::cluster_ctarank();
    const bool leader = rank == 0u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned pair = blockIdx.x >> 1;
    if (threadIdx.x == 0) {
        s_abort = 0;
        for (int s = 0; s < kRowsStages; ++s) {
            ptx::mbar_init(full_bar(s), 1);
            ptx::mbar_init(empty_bar(s), 1);
        }
        for (int t = 0; t < 2; ++t) {
            ptx::mbar_init(tfull_bar(t), 1);
            ptx::mbar_init(tempty_bar(t), 8 * kEpiGroups);  // each epilogue warp of both CTAs
        }
        ptx::mbar_init(drain_bar, 1);
        ptx::fence_barrier_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc_pair(ptx::smem_addr(&s_tmem_base), 512);
        ptx::tmem_relinquish_pair();
    }
    ptx::tc_fence_before();
    ptx::cluster_arrive();  // this CTA's barriers initialised and TMEM allocated
    const RowsWalk begin(args, pair);
    if (!args.chained) asm volatile("griddepcontrol.wait;" ::: "memory");
    int most;
    constexpr float kEpiNs = EPI == kEpiLinear ? 800.f : EPI == kEpiGated ? 1200.f : 1500.f;
    const int parts = make_table(args, table, kEpiNs, s_scan, most);
    const uint32_t stage = kWBytes + (uint32_t)(most / 2) * kRowBytes;
    const int S = min(kRowsStages, (int)(kRowsRing / stage));
    ptx::cluster_wait();
    ptx::tc_fence_after();
    const uint32_t tmem_base = s_tmem_base;

    if (warp == 0) {
        if (lane == 0) {
            // ---------------- TMA producer (both CTAs) ----------------
            const uint64_t pol = ptx::policy_evict_normal(), pol_t = ptx::policy_evict_last();
            uint32_t armed = 0u, armed_par = 0u;
            bool ok = true;
            int it = 0, s = 0;  // k-blocks so far, and the stage and
            uint32_t ph = 0u;   // parity of the next one
            auto weights = [&](const Tile &x, int kb, int s, uint32_t ph) {
                const int half = x.n / 2, c0 = (x.tn * 2 + (int)rank) * kCtaCols;
                const uint32_t fb = ptx::map_to_rank(full_bar(s), 0u), sw = sbase + s * stage;
                if (leader) {
                    ptx::mbar_arrive_expect_tx(full_bar(s), 2u * (args.w_bytes + (uint32_t)half * kRowBytes));
                    armed |= 1u << s;
                    armed_par = (armed_par & ~(1u << s)) | (ph << s);
                }
                const int seg = kb >= args.kswitch, k0 = (seg ? kb - args.kswitch : kb) * 64;
                if (EPI == kEpiGated) {
                    ptx::tma_load_3d_pair(sw, &maps.w[0], fb, c0, k0, x.e, pol);
                    ptx::tma_load_3d_pair(sw + 8192u, &maps.w[1], fb, c0, k0, x.e, pol);
                } else if (W_MN) {
                    ptx::tma_load_3d_pair(sw, &maps.w[0], fb, c0, k0, x.e, pol);
                    ptx::tma_load_3d_pair(sw + 8192u, &maps.w[0], fb, c0 + 64, k0, x.e, pol);
                } else {
                    ptx::tma_load_3d_pair(sw, &maps.w[seg], fb, k0, c0, x.e, pol);
                }
            };
            // of the first tile the weights of the first stages, ahead of the wait
            RowsWalk walk = begin;
            const int ahead = args.chained && walk.part < parts ? min(S, args.kblocks) : 0;
            if (ahead > 0) {
                const Tile x = walk.tile(args, table);
                for (int kb = 0; kb < ahead; ++kb) weights(x, kb, kb, 0u);
            }
            if (args.chained) asm volatile("griddepcontrol.wait;" ::: "memory");
            // after the wait: what follows may read this call's weights at once
            if (args.trigger) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
            for (; ok && walk.part < parts; walk.next(args)) {
                const Tile x = walk.tile(args, table);
                const int half = x.n / 2, r0 = x.row0 + (int)rank * half;
                const CUtensorMap *mt = &maps.t[0][half / 16 - 1];
                for (int kb = 0; kb < args.kblocks; ++kb, ++it) {
                    if (it >= ahead) {
                        if (!(ok = wait_phase(empty_bar(s), ph ^ 1u, args, &s_abort))) break;
                        weights(x, kb, s, ph);
                    }
                    const int seg = kb >= args.kswitch, k0 = (seg ? kb - args.kswitch : kb) * 64;
                    // test hook: the last rows never arrive
                    if (!(args.test_stall && kb == args.kblocks - 1 && leader))
                        ptx::tma_load_2d_pair(sbase + s * stage + kWBytes, mt + seg * kTokenBoxes,
                                              ptx::map_to_rank(full_bar(s), 0u), k0, r0, pol_t);
                    if (++s == S) s = 0, ph ^= 1u;
                }
            }
            // The leader's MMAs release the last stages in both CTAs.
            for (int j = it < S ? it : S; ok && j > 0; --j) {
                // j k-blocks before the next one
                const int back = s - j, at = back < 0 ? back + S : back;
                ok = wait_phase(empty_bar(at), back < 0 ? ph ^ 1u : ph, args, &s_abort);
            }
            // After an abort the leader lets every copy it armed land.
            if (leader && !ok) {
                for (int j = 0; j < S; ++j)
                    if (armed & (1u << j)) wait_drain(full_bar(j), (armed_par >> j) & 1u, args);
            }
        }
    } else if (warp == 1) {
        if (leader) {
            // ---------------- MMA issuer (leader CTA) ----------------
            const bool issue = ptx::elect_one();
            const int stages = same(S), all = same(parts);
            const uint32_t stage_step = (uint32_t)same((int)stage) >> 4, d_base = (uint32_t)same((int)tmem_base);
            const uint32_t fmt = args.fp16 ? 0u : 1u;
            const uint32_t idesc0 = (1u << 4) | (fmt << 7) | (fmt << 10) | ((W_MN ? 1u : 0u) << 15) | ((256u >> 4) << 24);
            int s = 0, job = 0, done = 0;
            uint32_t ph = 0u;
            bool ok = true;
            // descriptors of stage 0; the others' differ in the address, the low half's
            const uint64_t a_desc = operand_desc<W_MN>(sbase, 0), b_desc = operand_desc<false>(sbase + kWBytes, 0);
            const uint32_t a0 = (uint32_t)a_desc, a_hi = (uint32_t)(a_desc >> 32), b_hi = (uint32_t)(b_desc >> 32);
            const uint32_t b_off = (uint32_t)b_desc - a0;
            constexpr uint32_t kAStep = (W_MN ? 2048u : 32u) >> 4;
            for (RowsWalk walk = begin; ok && walk.part < all; walk.next(args), ++job) {
                const uint32_t idesc = idesc0 | ((uint32_t)(same(walk.tile(args, table).n) >> 3) << 17);
                const int t = job & 1;
                if (!wait_phase_warp(tempty_bar(t), (((uint32_t)job >> 1) & 1u) ^ 1u, args, &s_abort)) break;
                ptx::tc_fence_after();
                const uint32_t d_tmem = d_base + (uint32_t)(t * 256);
                for (int kb = 0; kb < args.kblocks; ++kb) {
                    if (!(ok = wait_phase_warp(full_bar(s), ph, args, &s_abort))) break;
                    ptx::tc_fence_after();
                    const uint32_t a_lo = a0 + (uint32_t)s * stage_step, b_lo = a_lo + b_off;
                    if (issue) {
                        ptx::mma_bf16_pair(d_tmem, a_lo, a_hi, b_lo, b_hi, idesc, kb > 0 ? 1u : 0u);
#pragma unroll
                        for (int kk = 1; kk < 4; ++kk)
                            ptx::mma_bf16_pair(d_tmem, a_lo + (uint32_t)kk * kAStep, a_hi, b_lo + (uint32_t)kk * 2u,
                                               b_hi, idesc, 1u);
                        ptx::mma_commit_pair(empty_bar(s), 0x3);  // frees stage s in both CTAs
                    }
                    __syncwarp();
                    if (++s == stages) s = 0, ph ^= 1u;
                }
                if (ok && issue) ptx::mma_commit_pair(tfull_bar(t), 0x3);
                if (ok) ++done;
            }
            if (issue) {
                ptx::mma_commit_pair(drain_bar, 0x3);  // every MMA retired before TMEM is freed
                wait_drain(drain_bar, 0u, args);
                // the peer's arrivals for the last tiles have landed
                for (int t = 0; t < 2; ++t) {
                    const int tiles = (done + 1 - t) / 2;
                    if (tiles > 0) wait_drain(tempty_bar(t), (uint32_t)(tiles - 1) & 1u, args);
                }
            }
            __syncwarp();
        }
    } else {
        // ---------------- epilogue (both CTAs) ----------------
        // Columns of D are the TMEM lanes.  Four warps, a group, hold the CTA's 128
        // of them and turn 16 rows around in shared memory, so that neighbouring
        // threads have neighbouring columns; the groups take every fourth 16 rows.
        const int lq = warp & 3, group = (warp - 2) >> 2;
        const int tid = lq * 32 + lane;  // in the group
        if (args.chained) asm volatile("griddepcontrol.wait;" ::: "memory");
        const uint32_t lanes = tmem_base + ((uint32_t)(32 * lq) << 16);
        const uint32_t buf = turn + (uint32_t)group * kTurnBytes;
        constexpr int kGroups = kCtaCols / 4, kStep = 128 / kGroups, kR = kTurnRows / kStep;
        // rows worked on together: of d gate's, all four at a time did not fit the
        // registers, and inputs that are spilled are waited for (256 experts of 1024x512
        // with 63 rows: d gate 78 us, so 63)
        constexpr int kBatch = EPI == kEpiDGate ? 2 : kR, kBatches = kR / kBatch;
        const int tr = tid / kGroups, tc = tid % kGroups * 4;
        int job = 0;
        Epilogue p = args.e;
        for (RowsWalk walk = begin; walk.part < parts; walk.next(args), ++job) {
            const Tile x = walk.tile(args, table);
            const int t = job & 1;
            p.M = x.end;
            const int c = (x.tn * 2 + (int)rank) * kCtaCols + tc;
            // what is read besides goes out before the tile's sums are complete
            GroupIn<EPI, kBatch> in[kBatches];
            const int r0 = x.row0 + tr;
            auto inputs = [&](int b) {
#pragma unroll
                for (int q = 0; q < kBatches; ++q)
                    group_load<EPI, kBatch>(p, r0 + b + q * kBatch * kStep, c, kStep, in[q]);
            };
            inputs(group * kTurnRows);
            // one warp of a group polls, the others sleep at the barrier
            const bool ok = lq != 2 || wait_phase(tfull_bar(t), ((uint32_t)job >> 1) & 1u, args, &s_abort);
            if (!ptx::named_bar_and(1 + group, 128, ok)) break;
            ptx::tc_fence_after();
            const uint32_t acc = lanes + (uint32_t)(t * 256);
            for (int b = group * kTurnRows; b < x.n; b += kEpiGroups * kTurnRows) {
                if (b >= kEpiGroups * kTurnRows) inputs(b);
                uint32_t v[kTurnRows];
                ptx::tmem_ld_x16(acc + (uint32_t)b, v);
                ptx::tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < kTurnRows; ++j)
                    asm volatile("st.shared.b32 [%0], %1;" ::"r"(buf + (uint32_t)(j * 128 + tid) * 4u), "r"(v[j])
                                 : "memory");
                ptx::named_bar_sync(1 + group, 128);
                float d[kBatches][4 * kBatch], u[kBatches][EPI == kEpiGated ? 4 * kBatch : 1];
#pragma unroll
                for (int j = 0; j < kR; ++j) {
                    float *dj = d[j / kBatch] + 4 * (j % kBatch);
                    const uint32_t at = buf + (uint32_t)((tr + j * kStep) * 128 + tc) * 4u;
                    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                                 : "=f"(dj[0]), "=f"(dj[1]), "=f"(dj[2]), "=f"(dj[3])
                                 : "r"(at)
                                 : "memory");
                    if constexpr (EPI == kEpiGated) {
                        float *uj = u[j / kBatch] + 4 * (j % kBatch);
                        asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                                     : "=f"(uj[0]), "=f"(uj[1]), "=f"(uj[2]), "=f"(uj[3])
                                     : "r"(at + 256u)
                                     : "memory");
                    }
                }
                ptx::named_bar_sync(1 + group, 128);  // the rows have left shared memory
#pragma unroll
                for (int q = 0; q < kBatches; ++q)
                    group_epilogue<EPI, kBatch>(p, r0 + b + q * kBatch * kStep, c, kStep, d[q], u[q], in[q]);
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) {  // everything has left TMEM
                if (leader)
                    ptx::mbar_arrive(tempty_bar(t));
                else
                    ptx::mbar_arrive_remote_relaxed(ptx::map_to_rank(tempty_bar(t), 0u));
            }
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        // the leader's MMAs write this CTA's TMEM: the peer waits for them too
        if (lane == 0 && !leader) wait_drain(drain_bar, 0u, args);
        __syncwarp();
        ptx::tc_fence_after();
        ptx::tmem_dealloc_pair(tmem_base, 512);
    }
    ptx::cluster_sync_relaxed();  // neither CTA leaves while the other may reach its shared memory
}

// ---- weights' gradients -----------------------------------------------------------

constexpr int kGradStages = 5;
// Warps that write the zeros, one a stage (which so sees each phase of its tail
// barrier): an arrival with its order at the pair's other CTA takes 2000 cycles
// and more, which several tails then share (one warp: 256 experts of 1024x512 with
// 63 rows 184 us).
constexpr int kZeroWarps = kGradStages;
constexpr int kGradEpi = 2 + kZeroWarps;               // the first epilogue warp, of 16
constexpr int kGradThreads = 32 * kGradEpi + 512;
constexpr uint32_t kGradStage = 4 * 8192;  // a CTA's 128 rows of A and 128 columns of B of 64 rows of the batch
constexpr uint32_t kGradTurn = 32 * 64 * 2;  // a warp's 32 rows of 64 columns, 16 bits each
constexpr uint32_t kGradSmem = 1024 + kGradStages * kGradStage + 16 * kGradTurn + 256;
static_assert(kGradSmem <= kSmemLimit, "shared memory");

struct GradTile {
    int e, p, m0, n0, lo, hi;
};
// A pair's tiles, one after another, an expert's together; the next one's
// offsets are on their way while a tile is worked on.
struct GradWalk {
    int e, r, de, dr, o0, o1;
    __device__ __forceinline__ GradWalk(const GradArgs &a, unsigned pair) {
        de = a.pairs / a.per_expert, dr = a.pairs - de * a.per_expert;
        e = (int)pair / a.per_expert, r = (int)pair - e * a.per_expert;
        fetch(a);
    }
    __device__ __forceinline__ void fetch(const GradArgs &a) {
        if (e < a.experts) o0 = a.offsets[e], o1 = a.offsets[e + 1];
    }
    __device__ __forceinline__ bool more(const GradArgs &a) const { return e < a.experts; }
    __device__ __forceinline__ GradTile take(const GradArgs &a) {
        GradTile x;
        x.e = e;
        const Run run = run_of(o0, o1, a.rows);
        x.lo = run.lo, x.hi = run.hi;
        int base = 0, tiles_n = a.p[0].tiles_n;
        x.p = 0;
#pragma unroll
        for (int j = 1; j < kMaxGrads; ++j)
            if (j < a.nprob && r >= a.p[j].base) x.p = j, base = a.p[j].base, tiles_n = a.p[j].tiles_n;
        const unsigned q = (unsigned)(r - base), tm = q / (unsigned)tiles_n;
        x.m0 = (int)tm * 256, x.n0 = (int)(q - tm * (unsigned)tiles_n) * 256;
        e += de, r += dr;
        if (r >= a.per_expert) r -= a.per_expert, ++e;
        fetch(a);
        return x;
    }
};

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGradThreads, 1)
    experts_grad_kernel(const __grid_constant__ GradMaps maps, const __grid_constant__ GradArgs args) {
    constexpr int S = kGradStages;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t s_tmem_base;
    __shared__ volatile int s_abort;

    const uint32_t raw = ptx::smem_addr(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    const uint32_t turn = sbase + S * kGradStage;
    const uint32_t bars = turn + 16 * kGradTurn;
    auto full_bar = [&](int s) { return bars + 8u * s; };  // leader's are used
    auto empty_bar = [&](int s) { return bars + 8u * (S + s); };
    auto tfull_bar = [&](int t) { return bars + 8u * (2 * S + t); };
    auto tempty_bar = [&](int t) { return bars + 8u * (2 * S + 2 + t); };  // leader's
    const uint32_t drain_bar = bars + 8u * (2 * S + 4);
    // a run's last rows have landed in this CTA; one for each stage, since several
    // short runs' are on their way at once
    auto tail_bar = [&](int s) { return bars + 8u * (2 * S + 5 + s); };

    const uint32_t rank = ptx::cluster_ctarank();
    const bool leader = rank == 0u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned pair = blockIdx.x >> 1;
    if (threadIdx.x == 0) {
        s_abort = 0;
        for (int s = 0; s < S; ++s) {
            ptx::mbar_init(full_bar(s), 2);  // one arrival of each CTA
            ptx::mbar_init(empty_bar(s), 1);
            ptx::mbar_init(tail_bar(s), 1);
        }
        for (int t = 0; t < 2; ++t) {
            ptx::mbar_init(tfull_bar(t), 1);
            ptx::mbar_init(tempty_bar(t), 32);  // each epilogue warp of both CTAs
        }
        ptx::mbar_init(drain_bar, 1);
        ptx::fence_barrier_init();
    }
    if (warp == 1) {
        ptx::tmem_alloc_pair(ptx::smem_addr(&s_tmem_base), 512);
        ptx::tmem_relinquish_pair();
    }
    ptx::tc_fence_before();
    ptx::cluster_sync();
    ptx::tc_fence_after();
    const uint32_t tmem_base = s_tmem_base;
    if (!args.beside) asm volatile("griddepcontrol.wait;" ::: "memory");

    if (warp == 0) {
        if (lane == 0) {
            // ---------------- TMA producer (both CTAs) ----------------
            const uint64_t pol = ptx::policy_evict_last();
            uint32_t armed = 0u, armed_par = 0u;  // copies counted on this CTA's full barriers
            uint32_t tails = 0u, tail_par = 0u;   // and on its tail barriers: the next phase's parity
            bool ok = true;
            int it = 0;
            for (GradWalk walk(args, pair); ok && walk.more(args);) {
                const GradTile x = walk.take(args);
                const int m0 = x.m0 + (int)rank * 128, n0 = x.n0 + (int)rank * 128;
                for (int r = x.lo; r < x.hi; r += 64, ++it) {
                    const int s = it % S;
                    const uint32_t ph = (uint32_t)(it / S) & 1u;
                    if (!(ok = wait_phase(empty_bar(s), ph ^ 1u, args, &s_abort))) break;
                    // the tensor cores take 16 rows at a time: past those nothing is read
                    const bool tail = r + 64 > x.hi && (x.hi - r) % 16 != 0;
                    const bool stall = args.test_stall && r + 64 >= x.hi && leader;  // test hook: it never arrives
                    const uint32_t sa = sbase + s * kGradStage, sb = sa + 16384u;
                    const CUtensorMap *ma = &maps.a[x.p], *mb = &maps.b[x.p];
                    if (tail) {
                        // counted here: the zeros' warp goes on from there
                        const uint32_t tb = tail_bar(s);
                        ptx::mbar_arrive_expect_tx(tb, kGradStage);
                        tails |= 1u << s, armed &= ~(1u << s);
                        tail_par ^= 1u << s;
                        if (stall) continue;
                        ptx::tma_load_2d(sa, ma, tb, m0, r, pol);
                        ptx::tma_load_2d(sa + 8192u, ma, tb, m0 + 64, r, pol);
                        ptx::tma_load_2d(sb, mb, tb, n0, r, pol);
                        ptx::tma_load_2d(sb + 8192u, mb, tb, n0 + 64, r, pol);
                        continue;
                    }
                    const uint32_t fb = ptx::map_to_rank(full_bar(s), 0u);
                    tails &= ~(1u << s);
                    if (leader) {
                        ptx::mbar_arrive_expect_tx(full_bar(s), 2 * kGradStage);
                        armed |= 1u << s;
                        armed_par = (armed_par & ~(1u << s)) | (ph << s);
                    } else {
                        ptx::mbar_arrive_remote_relaxed(fb);
                    }
                    if (stall) continue;
                    ptx::tma_load_2d_pair(sa, ma, fb, m0, r, pol);
                    ptx::tma_load_2d_pair(sa + 8192u, ma, fb, m0 + 64, r, pol);
                    ptx::tma_load_2d_pair(sb, mb, fb, n0, r, pol);
                    ptx::tma_load_2d_pair(sb + 8192u, mb, fb, n0 + 64, r, pol);
                }
            }
            for (int j = it > S ? it - S : 0; ok && j < it; ++j)
                ok = wait_phase(empty_bar(j % S), (uint32_t)(j / S) & 1u, args, &s_abort);
            // After an abort every copy that was issued lands first.
            if (!ok) {
                for (int s = 0; s < S; ++s) {
                    if (armed & (1u << s)) wait_drain(full_bar(s), (armed_par >> s) & 1u, args);
                    if (tails & (1u << s)) wait_drain(tail_bar(s), ((tail_par >> s) & 1u) ^ 1u, args);
                }
            }
        }
    } else if (warp == 1) {
        if (leader) {
            // ---------------- MMA issuer (leader CTA) ----------------
            const bool issue = ptx::elect_one();
            const uint32_t d_base = (uint32_t)same((int)tmem_base);
            const uint32_t fmt = args.fp16 ? 0u : 1u;
            const uint32_t idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | (1u << 15) | (1u << 16) |
                                   ((256u >> 3) << 17) | ((256u >> 4) << 24);
            const uint64_t desc = operand_desc<true>(sbase, 0);  // of A in stage 0
            const uint32_t a0 = (uint32_t)desc, hi = (uint32_t)(desc >> 32);
            int s = 0, job = 0, done = 0;
            uint32_t ph = 0u;
            bool ok = true;
            for (GradWalk walk(args, pair); ok && walk.more(args);) {
                const GradTile x = walk.take(args);
                const int rows = same(x.hi - x.lo);
                if (rows <= 0) continue;  // zeros: the epilogue's alone
                const int t = job & 1;
                if (!wait_phase_warp(tempty_bar(t), (((uint32_t)job >> 1) & 1u) ^ 1u, args, &s_abort)) break;
                ptx::tc_fence_after();
                const uint32_t d_tmem = d_base + (uint32_t)(t * 256);
                for (int r = 0; r < rows; r += 64) {
                    if (!(ok = wait_phase_warp(full_bar(s), ph, args, &s_abort))) break;
                    ptx::tc_fence_after();
                    const uint32_t a_lo = a0 + (uint32_t)s * (kGradStage >> 4), b_lo = a_lo + (16384u >> 4);
                    if (issue) {
                        ptx::mma_bf16_pair(d_tmem, a_lo, hi, b_lo, hi, idesc, r > 0 ? 1u : 0u);
#pragma unroll
                        for (uint32_t kk = 1; kk < 4; ++kk)
                            if (r + 16 * (int)kk < rows)
                                ptx::mma_bf16_pair(d_tmem, a_lo + kk * 128u, hi, b_lo + kk * 128u, hi, idesc, 1u);
                        ptx::mma_commit_pair(empty_bar(s), 0x3);
                    }
                    __syncwarp();
                    if (++s == S) s = 0, ph ^= 1u;
                }
                if (ok && issue) ptx::mma_commit_pair(tfull_bar(t), 0x3);
                if (ok) ++done;
                ++job;
            }
            if (issue) {
                ptx::mma_commit_pair(drain_bar, 0x3);
                wait_drain(drain_bar, 0u, args);
                for (int t = 0; t < 2; ++t) {
                    const int tiles = (done + 1 - t) / 2;
                    if (tiles > 0) wait_drain(tempty_bar(t), (uint32_t)(tiles - 1) & 1u, args);
                }
            }
            __syncwarp();
        }
    } else if (warp < kGradEpi) {
        // ---------------- zeros behind a run's last row (both CTAs) ----------------
        int it = 0;
        uint32_t tail_par = 0u;
        bool ok = true;
        for (GradWalk walk(args, pair); ok && walk.more(args);) {
            const GradTile x = walk.take(args);
            const int blocks = (x.hi - x.lo + 63) / 64, left = (x.hi - x.lo) & 63;
            it += blocks;
            if (left % 16 == 0) continue;
            const int s = (it - 1) % S;
            if (s != warp - 2) continue;
            if (!(ok = wait_phase_warp(tail_bar(s), tail_par, args, &s_abort))) break;
            tail_par ^= 1u;
            // row r of the batch is 128 bytes of each of the four boxes
            const uint32_t at = sbase + s * kGradStage + (uint32_t)left * 128u;
            const int pieces = (16 - left % 16) * 8;
#pragma unroll
            for (int b = 0; b < 4; ++b)
                for (int j = lane; j < pieces; j += 32)
                    asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(at + 8192u * b + 16u * j), "r"(0)
                                 : "memory");
            ptx::fence_proxy_async_smem();  // before the tensor cores' reads
            __syncwarp();
            if (lane == 0) {
                if (leader)
                    ptx::mbar_arrive(full_bar(s));
                else
                    ptx::mbar_arrive_remote(ptx::map_to_rank(full_bar(s), 0u));
            }
        }
    } else {
        // ---------------- epilogue (both CTAs) ----------------
        const int lq = warp & 3;              // TMEM lanes 32 lq .. + 31 = rows of D
        const int cs = (warp - kGradEpi) >> 2;  // which 64 of the tile's columns
        const uint32_t lanes = tmem_base + ((uint32_t)(32 * lq) << 16);
        const uint32_t mine = turn + (uint32_t)(warp - kGradEpi) * kGradTurn;
        // the 128-byte swizzle of the results' boxes: 16 bytes (unit x) of a row sit at unit x ^ (row & 7)
        auto slot = [&](int x) { return mine + (uint32_t)(lane * 128 + ((x ^ (lane & 7)) << 4)); };
        int job = 0;
        for (GradWalk walk(args, pair); walk.more(args);) {
            const GradTile x = walk.take(args);
            const int r0 = x.m0 + (int)rank * 128 + 32 * lq, c0 = x.n0 + cs * 64;
            const bool some = x.lo < x.hi;
            const int t = job & 1;
            if (some) {
                if (!__all_sync(0xFFFFFFFFu, wait_phase(tfull_bar(t), ((uint32_t)job >> 1) & 1u, args, &s_abort))) break;
                ++job;
                ptx::tc_fence_after();
            }
            const uint32_t acc = lanes + (uint32_t)(t * 256 + cs * 64);
            if (lane == 0) ptx::bulk_wait_group_read<0>();  // the last tile's rows have left shared memory
            __syncwarp();
#pragma unroll
            for (int g = 0; g < 64; g += 32) {
                uint32_t w[16] = {};
                if (some) {
                    uint32_t v[32];
                    ptx::tmem_ld_x16(acc + (uint32_t)g, reinterpret_cast<uint32_t(&)[16]>(v[0]));
                    ptx::tmem_ld_x16(acc + (uint32_t)g + 16u, reinterpret_cast<uint32_t(&)[16]>(v[16]));
                    ptx::tmem_ld_wait();
                    float f[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(v[e]);
                    pack_values<32>(args.fp16 != 0, f, w);
                }
#pragma unroll
                for (int h = 0; h < 4; ++h)
                    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(slot(g / 8 + h)), "r"(w[4 * h]),
                                 "r"(w[4 * h + 1]), "r"(w[4 * h + 2]), "r"(w[4 * h + 3])
                                 : "memory");
            }
            if (some) ptx::tc_fence_before();
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                if (some) {
                    if (leader)
                        ptx::mbar_arrive(tempty_bar(t));
                    else
                        ptx::mbar_arrive_remote_relaxed(ptx::map_to_rank(tempty_bar(t), 0u));
                }
                if (r0 < args.p[x.p].M && c0 < args.p[x.p].N) ptx::tma_store_3d(&maps.d[x.p], mine, c0, r0, x.e);
                ptx::bulk_commit_group();
            }
        }
        if (lane == 0) ptx::bulk_wait_group_all();
    }

    // what follows this kernel follows the one before it too
    if (args.beside) asm volatile("griddepcontrol.wait;" ::: "memory");
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        if (lane == 0 && !leader) wait_drain(drain_bar, 0u, args);
        __syncwarp();
        ptx::tc_fence_after();
        ptx::tmem_dealloc_pair(tmem_base, 512);
    }
    ptx::cluster_sync_relaxed();
}

const void *kernel_of(int epi, bool n_contiguous) {
    if (epi == kEpiGated && n_contiguous) return reinterpret_cast<const void *>(experts_rows_kernel<kEpiGated, true>);
    if (epi == kEpiLinear && n_contiguous) return reinterpret_cast<const void *>(experts_rows_kernel<kEpiLinear, true>);
    if (epi == kEpiLinear) return reinterpret_cast<const void *>(experts_rows_kernel<kEpiLinear, false>);
    if (epi == kEpiDGate && !n_contiguous) return reinterpret_cast<const void *>(experts_rows_kernel<kEpiDGate, false>);
    return nullptr;
}

cudaError_t launch(const void *k, unsigned grid, unsigned block, size_t smem, void **params, cudaStream_t stream) {
    cudaLaunchConfig_t c = {};
    cudaLaunchAttribute attr[1];
    c.gridDim = dim3(grid);
    c.blockDim = dim3(block);
    c.dynamicSmemBytes = smem;
    c.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    c.attrs = attr;
    c.numAttrs = 1;
    return cudaLaunchKernelExC(&c, k, params);
}

}  // namespace

cudaError_t experts_configure() {
    for (int epi : {kEpiGated, kEpiLinear, kEpiDGate})
        for (bool n : {true, false})
            if (const void *k = kernel_of(epi, n)) {
                const cudaError_t e =
                    cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRowsSmem);
                if (e != cudaSuccess) return e;
            }
    return cudaFuncSetAttribute(experts_grad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kGradSmem);
}

int experts_smem_bytes() { return (int)(kRowsSmem > kGradSmem ? kRowsSmem : kGradSmem); }

cudaError_t experts_launch(int epi, bool n_contiguous, const ExpertsMaps &maps, const ExpertsArgs &args,
                           cudaStream_t stream) {
    const void *k = kernel_of(epi, n_contiguous);
    if (k == nullptr || args.pairs < 1) return cudaErrorInvalidConfiguration;
    void *params[] = {const_cast<ExpertsMaps *>(&maps), const_cast<ExpertsArgs *>(&args)};
    return launch(k, 2u * (unsigned)args.pairs, kRowsThreads, kRowsSmem, params, stream);
}

cudaError_t experts_grad_launch(const GradMaps &maps, const GradArgs &args, cudaStream_t stream) {
    if (args.pairs < 1 || args.per_expert < 1) return cudaErrorInvalidConfiguration;
    void *params[] = {const_cast<GradMaps *>(&maps), const_cast<GradArgs *>(&args)};
    return launch(reinterpret_cast<const void *>(experts_grad_kernel), 2u * (unsigned)args.pairs, kGradThreads,
                  kGradSmem, params, stream);
}

}  // namespace route
