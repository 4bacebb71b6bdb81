// The layer operators' matrix products on the sm_103a tensor cores, two SMs
// per tile.
//
//   D[m, n] = sum_k A[m, k] B[k, n]      16-bit operands, FP32 sums
//
// and, from the FP32 sums and without writing them to memory first, what the
// operator makes of them (layer_math.cuh: epilogue): bias, activation and
// residual; a gated block's act(gate) * up; its backward pass's d gate, d up.
// The contraction runs over either dimension of either operand, so the
// forward product, the input's and the weights' gradients read every tensor
// where and as it is stored (GemmForm).  A launch may take several products,
// so that a backward pass's fill the chip together.
//
// A tile is 256 rows of D by BN columns (a gated product: BN / 2 columns of
// gate and the same of up, the pair's first CTA loading the gate weights and
// its second the up weights), computed by a cluster of two CTAs with
// tcgen05.mma.cta_group::2: each CTA stages 128 rows of A and its half of
// the tile's B columns per 64-deep k-block and holds its 128 rows x BN
// columns of D in its TMEM.  Two accumulators alternate, so that one tile is
// drained while the next is computed.
//
// Rows of D are the TMEM lanes.  An epilogue warp takes columns of its 32 rows
// out of TMEM into shared memory and back with neighbouring threads on
// neighbouring columns (Access: how many, and on which side of shared memory
// the operator's epilogue is).  Its "TMEM is read"
// to the other CTA is a relaxed arrival: ordered after the warp's stores of
// results, as an arrival is by default, it waited for them to reach the L2
// (2050x64x3584 11.5 us, so 10.4; gelu with z kept 20.5, so 19.3).  For the
// same reason the last meeting of the pair is relaxed (0.4 us a launch): it
// orders no access, so each CTA first waits for every arrival on its barriers
// from the other.
//
// Split K: with few tiles, `splits` CTA pairs share a tile's contraction and
// store FP32 partials; gemm_finish_kernel adds them in split order and runs
// the same epilogue.  Results never depend on the order of arrival.
//
// Large products are bound by the tensor cores: 4096x3584x7168 takes 112 us in
// a burst (1,880 TFLOP/s), 126 in a long run, at the power limit (1,670).  With
// short contractions the epilogue binds: 2.1 us a 256 x 256 tile without an
// activation, and the stores of what it writes (4096x64x7168 15.6 us, 3.8
// TB/s).  With few tiles it is whole rounds of them over the pairs, and 5 us
// of a launch's start and end.
//
// Warp roles (576 or 320 threads, persistent, one CTA per SM, pairs = clusters):
//   warp 0      TMA producer (both CTAs); completion counts on the leader's
//               barrier, which the leader arms for both CTAs' bytes
//   warp 1      TMEM owner (both CTAs); the leader's lane 0 issues the MMAs
//   the others  epilogue: warp w reads TMEM lanes 32 (w % 4) .. + 31 and its
//               share of the tile's columns
//
// Every wait is bounded: after timeout_ns a waiting thread sets the device
// status word and the CTA's abort flag, in-flight copies and MMAs are
// drained, TMEM is freed and both CTAs return.
#include "layer.cuh"
#include "layer_math.cuh"
#include "layer_ptx.cuh"

namespace route {
namespace {

constexpr int kHalf = 128;                        // each CTA's rows of D
constexpr uint32_t kABytes = kHalf * 64 * 2;      // 128 rows x 64 k
// Epilogue warps, the columns of D that one turns around at once, and its
// buffer for them (a gated block: of gate and of up, with half the warps).
__host__ __device__ constexpr int epi_warps(int epi) { return epi == kEpiGated ? 8 : 16; }
__host__ __device__ constexpr int gemm_threads(int epi) { return 64 + 32 * epi_warps(epi); }
constexpr int kG = 32;
constexpr uint32_t kHalfTurn = 32 * kG * 4;
__host__ __device__ constexpr uint32_t turn_bytes(int epi) { return epi == kEpiGated ? 2 * kHalfTurn : kHalfTurn; }
constexpr uint32_t kTurns = 16 * kHalfTurn;  // all warps' buffers
constexpr uint32_t kSmemLimit = 227 * 1024;

__host__ __device__ constexpr uint32_t b_bytes(int bn) { return (uint32_t)bn / 2 * 64 * 2; }
__host__ __device__ constexpr uint32_t stage_bytes(int bn) { return kABytes + b_bytes(bn); }
__host__ __device__ constexpr int stages_of(int bn) { return bn == 256 ? 5 : 6; }
__host__ __device__ constexpr uint32_t smem_of(int bn) { return 1024 + stages_of(bn) * stage_bytes(bn) + kTurns + 256; }
static_assert(smem_of(256) <= kSmemLimit && smem_of(128) <= kSmemLimit, "shared memory");

// How long a poll of a barrier may be held in hardware.
constexpr uint32_t kWaitHintNs = 20000;

__device__ __forceinline__ uint64_t smem_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
    uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
    d |= (uint64_t)((sbo >> 4) & 0x3FFFu) << 32;
    d |= 1ull << 46;  // descriptor version for tcgen05
    d |= 2ull << 61;  // 128-byte swizzle
    return d;
}

// Descriptor of 16 k of an operand tile.  K-contiguous: 128-byte swizzled
// rows of 64 k, 8-row groups 1024 B apart; 16 k are 32 B.  M/N-contiguous:
// boxes of 64 columns x 64 k, 8192 B apart, 8-k groups 1024 B apart; 16 k
// are 2048 B.
template <bool MN>
__device__ __forceinline__ uint64_t operand_desc(uint32_t base, int kk) {
    return MN ? smem_desc(base + kk * 2048u, 8192u, 1024u) : smem_desc(base + kk * 32u, 16u, 1024u);
}

__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity, const GemmArgs &a,
                                           volatile int *abort_flag) {
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

// Bounded wait used only while tearing down.
__device__ __forceinline__ void wait_drain(uint32_t bar, uint32_t parity, const GemmArgs &a) {
    const uint64_t t0 = ptx::global_timer_ns();
    while (!ptx::mbar_try_wait_hint(bar, parity, kWaitHintNs)) {
        if (ptx::global_timer_ns() - t0 > a.timeout_ns) {
            atomicOr(a.status, kStatusTimeout);
            return;
        }
    }
}

// A work item: the tile's problem, its row and column tile, its split and
// its k-blocks.  Tiles go in bands of `band` column tiles over every row
// tile, so that the pairs at work at one time share rows of A and columns of
// B; the splits of a tile are neighbours.
struct Item {
    int p, tm, tn, split, kb0, kb1;
};
__device__ __forceinline__ Item item_of(const GemmArgs &a, int i) {
    Item w;
    w.p = 0;
    while (w.p + 1 < a.nprob && i >= a.p[w.p + 1].item_base) ++w.p;
    const GemmProblem &p = a.p[w.p];
    unsigned u = (unsigned)(i - p.item_base);
    const unsigned splits = (unsigned)p.splits, kblocks = (unsigned)p.kblocks;
    w.split = 0, w.kb0 = 0, w.kb1 = (int)kblocks;
    if (splits > 1) {
        const unsigned t = u / splits;
        w.split = (int)(u - t * splits);
        u = t;
        w.kb0 = (int)(kblocks * (unsigned)w.split / splits);
        w.kb1 = (int)(kblocks * (unsigned)(w.split + 1) / splits);
    }
    const unsigned per_band = (unsigned)(p.band * p.tiles_m);
    const unsigned b = u / per_band, r = u - b * per_band, c0 = b * (unsigned)p.band;
    const unsigned left = (unsigned)p.tiles_n - c0, bw = left < (unsigned)p.band ? left : (unsigned)p.band;
    const unsigned tm = r / bw;
    w.tm = (int)tm;
    w.tn = (int)(c0 + r - tm * bw);
    return w;
}

// A pair's items, one after another.
struct Walk {
    int c, j, i;
    __device__ __forceinline__ explicit Walk(int pair) : c(0), j(0), i(pair) {}
    __device__ __forceinline__ bool next(const GemmArgs &a, int pair, int &item) {
        if (!a.listed) {
            item = i;
            i += a.pairs;
            return item < a.items;
        }
        while (c < a.nprob && j >= a.count[c][pair]) ++c, j = 0;
        if (c == a.nprob) return false;
        item = a.p[c].item_base + a.first[c][pair] + j++;
        return true;
    }
};

// What one thread of the producer warp and the MMA thread keep over all items.
// Their loops over a tile's k-blocks are made for a form each and the form is
// looked at once an item: with the form looked at (and the descriptors put
// together from it) in every k-block, the two threads took 0.41 us a k-block
// where the MMAs take 0.34 (4096x3584x7168 139 against 115 us).
template <int BN>
struct Stages {
    const GemmArgs &args;
    volatile int *abort_flag;
    uint32_t sbase, bars;
    int it = 0;
    static constexpr int S = stages_of(BN);
    __device__ __forceinline__ uint32_t full_bar(int s) const { return bars + 8u * s; }  // leader's are used
    __device__ __forceinline__ uint32_t empty_bar(int s) const { return bars + 8u * (S + s); }
};

struct Load {
    const CUtensorMap *a0, *b0, *a1, *b1;
    int m0, n0, kb0, kb1, kswitch;
    uint32_t tx;
};

template <bool A_MN, bool B_MN, int BN>
__device__ __forceinline__ bool load_tile(Stages<BN> &st, const Load &l, bool leader, uint64_t pol,
                                          uint32_t &armed, uint32_t &armed_par) {
    constexpr int S = Stages<BN>::S;
    for (int kb = l.kb0; kb < l.kb1; ++kb, ++st.it) {
        const int s = st.it % S;
        const uint32_t ph = (uint32_t)(st.it / S) & 1u;
        if (!wait_phase(st.empty_bar(s), ph ^ 1u, st.args, st.abort_flag)) return false;
        const uint32_t fb = ptx::map_to_rank(st.full_bar(s), 0u);
        if (leader) {
            ptx::mbar_arrive_expect_tx(st.full_bar(s), l.tx);
            armed |= 1u << s;
            armed_par = (armed_par & ~(1u << s)) | (ph << s);
        }
        if (st.args.test_stall && kb == l.kb1 - 1 && leader) continue;  // test hook: it never arrives
        const bool second = kb >= l.kswitch;
        const int k0 = (second ? kb - l.kswitch : kb) * 64;
        const CUtensorMap *ma = second ? l.a1 : l.a0, *mb = second ? l.b1 : l.b0;
        const uint32_t sa = st.sbase + s * stage_bytes(BN), sb = sa + kABytes;
        if (A_MN) {
            ptx::tma_load_2d_pair(sa, ma, fb, l.m0, k0, pol);
            ptx::tma_load_2d_pair(sa + 8192u, ma, fb, l.m0 + 64, k0, pol);
        } else {
            ptx::tma_load_2d_pair(sa, ma, fb, k0, l.m0, pol);
        }
        if (B_MN) {
#pragma unroll
            for (int j = 0; j < BN / 128; ++j)
                ptx::tma_load_2d_pair(sb + 8192u * j, mb, fb, l.n0 + 64 * j, k0, pol);
        } else {
            ptx::tma_load_2d_pair(sb, mb, fb, k0, l.n0, pol);
        }
    }
    return true;
}

template <bool A_MN, bool B_MN, int BN>
__device__ __forceinline__ bool mma_tile(Stages<BN> &st, int kblocks, uint32_t d_tmem, uint32_t fmt) {
    constexpr int S = Stages<BN>::S;
    // kind::f16, FP32 accumulator, M = 256 over the pair, N = BN
    const uint32_t idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | ((A_MN ? 1u : 0u) << 15) |
                           ((B_MN ? 1u : 0u) << 16) | ((uint32_t)(BN >> 3) << 17) |
                           ((uint32_t)(kGemmBM >> 4) << 24);
    for (int kb = 0; kb < kblocks; ++kb, ++st.it) {
        const int s = st.it % S;
        if (!wait_phase(st.full_bar(s), (uint32_t)(st.it / S) & 1u, st.args, st.abort_flag)) return false;
        ptx::tc_fence_after();
        const uint32_t sa = st.sbase + s * stage_bytes(BN), sb = sa + kABytes;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
            ptx::mma_bf16_pair(d_tmem, operand_desc<A_MN>(sa, kk), operand_desc<B_MN>(sb, kk), idesc,
                               (kb > 0 || kk > 0) ? 1u : 0u);
        ptx::mma_commit_pair(st.empty_bar(s), 0x3);  // frees stage s in both CTAs
    }
    return true;
}

// How rows of the result are accessed, a kernel each for the registers: one
// column a thread (rows of odd widths); four FP32 sums a thread, where FP32
// values are read or kept beside the result; or, where there is 16-bit data
// only besides the sums, finished and packed by the thread that took a row's
// columns out of TMEM, so that half the bytes go through shared memory, in one
// pass, and a row leaves in whole 128-byte lines (4096x64x7168 15.6 us, by
// fours 23.3; 64x3584x7168's backward pass 32.8, by fours 39.4).  Packed rows
// of odd widths leave by 4-byte words (4096x64x7167 32.0, by columns 55.1;
// rows that take fours are better off with them, 4096x64x7164 26.0 and 29.7).
enum Access { kColumns = 0, kFours = 1, kPacked = 2, kPackedResidual = 3, kPackedAny = 4 };
template <int FORM, int EPI, int BN, int ACCESS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(gemm_threads(EPI), 1)
    layer_gemm_kernel(const __grid_constant__ GemmMaps maps, const __grid_constant__ GemmArgs args) {
    constexpr int S = stages_of(BN);
    constexpr uint32_t kStage = stage_bytes(BN);
    constexpr int kTileCols = EPI == kEpiGated ? BN / 2 : BN;  // columns of D a tile
    constexpr int kBCols = BN / 2;                             // B columns each CTA loads
    constexpr int kEpiWarps = epi_warps(EPI);
    constexpr bool kPack = ACCESS == kPacked || ACCESS == kPackedResidual || ACCESS == kPackedAny;
    constexpr int kWarpCols = kTileCols / (kEpiWarps / 4);     // columns of D an epilogue warp drains
    static_assert(kWarpCols % kG == 0 && kG % 16 == 0, "whole groups");
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t s_tmem_base;
    __shared__ volatile int s_abort;

    const uint32_t raw = ptx::smem_addr(smem_raw);
    const uint32_t sbase = (raw + 1023u) & ~1023u;
    const uint32_t turn = sbase + S * kStage;
    const uint32_t bars = turn + kTurns;
    auto full_bar = [&](int s) { return bars + 8u * s; };             // leader's are used
    auto empty_bar = [&](int s) { return bars + 8u * (S + s); };
    auto tfull_bar = [&](int t) { return bars + 8u * (2 * S + t); };
    auto tempty_bar = [&](int t) { return bars + 8u * (2 * S + 2 + t); };  // leader's
    const uint32_t drain_bar = bars + 8u * (2 * S + 4);

    const uint32_t rank = ptx::cluster_ctarank();
    const bool leader = rank == 0u;
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int pair = blockIdx.x >> 1;
    if (threadIdx.x == 0) {
        s_abort = 0;
        for (int s = 0; s < S; ++s) {
            ptx::mbar_init(full_bar(s), 1);
            ptx::mbar_init(empty_bar(s), 1);
        }
        for (int t = 0; t < 2; ++t) {
            ptx::mbar_init(tfull_bar(t), 1);
            ptx::mbar_init(tempty_bar(t), 2 * kEpiWarps);  // each epilogue warp of both CTAs
        }
        ptx::mbar_init(drain_bar, 1);
        ptx::fence_barrier_init();
        ptx::prefetch_tensormap(&maps.m[args.p[0].a[0]]);
        ptx::prefetch_tensormap(&maps.m[args.p[0].b[0][rank]]);
    }
    if (warp == 1) {
        ptx::tmem_alloc_pair(ptx::smem_addr(&s_tmem_base), 2 * BN);
        ptx::tmem_relinquish_pair();
    }
    ptx::tc_fence_before();
    ptx::cluster_sync();  // both CTAs' barriers initialised and TMEM allocated
    ptx::tc_fence_after();
    const uint32_t tmem_base = s_tmem_base;

    if (warp == 0) {
        if (lane == 0) {
            // ---------------- TMA producer (both CTAs) ----------------
            // operands stay in L2 before results: 2-3% less under the power cap
            // (4096x3584x7168 128.0 against 131.7 us, 8192x3584x3584 128.1
            // against 131.3) than the default; operands first out: 4-5% more
            const uint64_t pol = ptx::policy_evict_last();
            asm volatile("griddepcontrol.wait;" ::: "memory");
            // after the wait: what follows may read this call's weights at once
            if (args.trigger) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
            Stages<BN> st{args, &s_abort, sbase, bars};
            uint32_t armed = 0u, armed_par = 0u;
            bool ok = true;
            Walk walk(pair);
            for (int i; ok && walk.next(args, pair, i);) {
                const Item w = item_of(args, i);
                const GemmProblem &p = args.p[w.p];
                const Load l = {&maps.m[p.a[0]],
                                &maps.m[p.b[0][rank]],
                                &maps.m[p.a[1]],
                                &maps.m[p.b[1][rank]],
                                w.tm * kGemmBM + (int)rank * kHalf,
                                w.tn * kTileCols + (EPI == kEpiGated ? 0 : (int)rank * kBCols),
                                w.kb0,
                                w.kb1,
                                p.kswitch,
                                2u * (p.a_bytes + b_bytes(BN))};
                if (FORM == kFormNT)
                    ok = load_tile<false, true>(st, l, leader, pol, armed, armed_par);
                else if (FORM == kFormNN || p.form == kFormNN)
                    ok = load_tile<false, false>(st, l, leader, pol, armed, armed_par);
                else
                    ok = load_tile<true, true>(st, l, leader, pol, armed, armed_par);
            }
            // The leader's MMAs release the last stages in both CTAs, and nobody
            // waits for that to load another: it has arrived before they leave.
            for (int it = st.it > S ? st.it - S : 0; ok && it < st.it; ++it)
                ok = wait_phase(empty_bar(it % S), (uint32_t)(it / S) & 1u, args, &s_abort);
            // After an abort the leader lets every copy it armed land (the
            // peer's copies complete on the same barriers).
            if (leader && !ok) {
                for (int s = 0; s < S; ++s)
                    if (armed & (1u << s)) wait_drain(full_bar(s), (armed_par >> s) & 1u, args);
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && leader) {
            // ---------------- MMA issuer (leader CTA) ----------------
            const uint32_t fmt = args.fp16 ? 0u : 1u;
            Stages<BN> st{args, &s_abort, sbase, bars};
            int job = 0, done = 0;  // tiles begun, and handed to the epilogue
            bool ok = true;
            Walk walk(pair);
            for (int i; ok && walk.next(args, pair, i); ++job) {
                const Item w = item_of(args, i);
                const int t = job & 1;
                if (!wait_phase(tempty_bar(t), (((uint32_t)job >> 1) & 1u) ^ 1u, args, &s_abort)) break;
                ptx::tc_fence_after();
                const uint32_t d_tmem = tmem_base + (uint32_t)(t * BN);
                const int n = w.kb1 - w.kb0;
                if (FORM == kFormNT)
                    ok = mma_tile<false, true>(st, n, d_tmem, fmt);
                else if (FORM == kFormNN || args.p[w.p].form == kFormNN)
                    ok = mma_tile<false, false>(st, n, d_tmem, fmt);
                else
                    ok = mma_tile<true, true>(st, n, d_tmem, fmt);
                if (ok) ptx::mma_commit_pair(tfull_bar(t), 0x3), ++done;
            }
            ptx::mma_commit_pair(drain_bar, 0x3);  // every MMA retired before TMEM is freed
            wait_drain(drain_bar, 0u, args);
            // The peer's arrivals for the last tiles have landed before this CTA's
            // shared memory is another's: no later tile waits for them.
            for (int t = 0; t < 2; ++t) {
                const int tiles = (done + 1 - t) / 2;  // with accumulator t
                if (tiles > 0) wait_drain(tempty_bar(t), (uint32_t)(tiles - 1) & 1u, args);
            }
        }
    } else {
        // ---------------- epilogue (both CTAs) ----------------
        const int lq = warp & 3;         // TMEM lanes 32 lq .. + 31 = rows of D
        const int cs = (warp - 2) >> 2;  // which share of the tile's columns
        const uint32_t lanes = tmem_base + ((uint32_t)(32 * lq) << 16);
        const uint32_t mine = turn + (uint32_t)(warp - 2) * turn_bytes(EPI);
        asm volatile("griddepcontrol.wait;" ::: "memory");
        int job = 0;
        Epilogue p = args.p[0].e;
        int of = 0;  // whose
        Walk walk(pair);
        for (int i; walk.next(args, pair, i); ++job) {
            const Item w = item_of(args, i);
            if (w.p != of) p = args.p[w.p].e, of = w.p;
            const int t = job & 1;
            const int r0 = w.tm * kGemmBM + (int)rank * kHalf + 32 * lq;
            const int c0 = w.tn * kTileCols + cs * kWarpCols;
            // A thread's share of a group is four columns of kSteps rows, kStep
            // apart, worked on kBatch rows at a time: all of them without an
            // activation, else 4, because code for 64 activations in a row does
            // not stay in the instruction cache (gelu 2048x64x3584 28 us).
            constexpr int kLanesRow = kG / 4, kStep = 32 / kLanesRow, kSteps = 32 / kStep;
            constexpr int kBatch = EPI == kEpiDGate ? 2 : 4, kGroupBatches = kSteps / kBatch;
            constexpr bool kAhead = EPI != kEpiGated;  // inputs a batch ahead
            constexpr int kBatches = kWarpCols / kG * kGroupBatches;
            static_assert(kSteps % kBatch == 0, "whole batches");
            const bool whole = args.p[w.p].splits == 1;
            auto row_of = [&](int b) { return b % kGroupBatches * (kBatch * kStep) + lane / kLanesRow; };
            auto col_of = [&](int b) { return c0 + b / kGroupBatches * kG + lane % kLanesRow * 4; };
            GroupIn<EPI, kBatch> in, next;
            // Packed: a row of the warp's columns is kUnits units of 16 bytes; those of
            // the rows of a 128-byte line are interleaved.  A thread's share of them
            // on the way from and to memory: unit px of every kStepRows-th row.
            constexpr int kUnits = kWarpCols / 8, kLineRows = 8 / kUnits, kStepRows = 32 / kUnits;
            auto slot = [&](int row, int x) {
                return mine + (uint32_t)(row * kUnits * 16 + ((x ^ ((row / kLineRows) & (kUnits - 1))) << 4));
            };
            const int px = lane % kUnits, pr = lane / kUnits, pc = c0 + 8 * px;
            // what is read besides goes out before the tile's sums are complete
            if constexpr (kPack) {
                __syncwarp();  // the last tile's rows have left shared memory
                if (ACCESS == kPackedResidual && whole && pc < p.N) {
                    const uint16_t *q = static_cast<const uint16_t *>(p.residual) + (long long)(r0 + pr) * p.ld_res + pc;
#pragma unroll
                    for (int j = 0; j < 32; j += kStepRows, q += kStepRows * p.ld_res) {
                        if (r0 + pr + j >= p.M) break;
                        const uint4 w = *reinterpret_cast<const uint4 *>(q);
                        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(slot(pr + j, px)), "r"(w.x),
                                     "r"(w.y), "r"(w.z), "r"(w.w)
                                     : "memory");
                    }
                }
                if (ACCESS == kPackedResidual) __syncwarp();
            }
            if (ACCESS == kFours && whole) group_load<EPI, kBatch>(p, r0 + row_of(0), col_of(0), kStep, in);
            // one warp polls, the others sleep at the barrier
            const bool ok = warp != 2 || wait_phase(tfull_bar(t), ((uint32_t)job >> 1) & 1u, args, &s_abort);
            if (!ptx::named_bar_and(1, 32 * kEpiWarps, ok)) break;
            ptx::tc_fence_after();
            const uint32_t acc = lanes + (uint32_t)(t * BN + cs * kWarpCols);
            // Four columns (16 bytes, unit x) of a row sit at unit x ^ (row & 7):
            // rows a line apart, and columns of a row, are both free of conflicts.
            auto unit = [&](int row, int x) {
                return mine + (uint32_t)(row * kG * 4 + ((x ^ (row & 7)) << 4));
            };
            auto put = [&](uint32_t tmem, uint32_t half) {  // this thread's row of kG columns
#pragma unroll
                for (int h = 0; h < kG / 16; ++h) {
                    uint32_t v[16];
                    ptx::tmem_ld_x16(tmem + 16u * h, v);
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(unit(lane, 4 * h + x) + half),
                                     "r"(v[4 * x]), "r"(v[4 * x + 1]), "r"(v[4 * x + 2]), "r"(v[4 * x + 3])
                                     : "memory");
                }
            };
            auto get = [&](int row, uint32_t half, float (&v)[4 * kBatch]) {
#pragma unroll
                for (int j = 0; j < kBatch; ++j)
                    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                                 : "=f"(v[4 * j]), "=f"(v[4 * j + 1]), "=f"(v[4 * j + 2]), "=f"(v[4 * j + 3])
                                 : "r"(unit(row + j * kStep, lane % kLanesRow) + half)
                                 : "memory");
            };
            auto read_out = [&] {  // everything has left TMEM
                ptx::tc_fence_before();
                __syncwarp();
                if (lane != 0) return;
                if (leader)
                    ptx::mbar_arrive(tempty_bar(t));
                else
                    ptx::mbar_arrive_remote_relaxed(ptx::map_to_rank(tempty_bar(t), 0u));
            };
            if (kPack && whole) {
                if constexpr (kPack) {
                    constexpr int kTake = EPI == kEpiLinear ? 32 : 16;  // columns at a time
                    const bool half = p.out_type == kFp16;
#pragma unroll(EPI == kEpiLinear ? kWarpCols / kTake : 1)
                    for (int g = 0; g < kWarpCols; g += kTake) {
                        uint32_t raw[kTake], raw2[EPI == kEpiGated ? kTake : 1];
#pragma unroll
                        for (int h = 0; h < kTake; h += 16)
                            ptx::tmem_ld_x16(acc + (uint32_t)(g + h), reinterpret_cast<uint32_t(&)[16]>(raw[h]));
                        if constexpr (EPI == kEpiGated) ptx::tmem_ld_x16(acc + (uint32_t)(kTileCols + g), raw2);
                        ptx::tmem_ld_wait();
                        float v[kTake];
#pragma unroll
                        for (int e = 0; e < kTake; ++e) v[e] = __uint_as_float(raw[e]);
                        if constexpr (epi_linear(EPI))
                            if (p.bias != nullptr) packed_bias<kTake>(p, c0 + g, half, v);
                        if constexpr (EPI != kEpiLinear) act_values<kTake>(p.act, v);
                        if constexpr (ACCESS == kPackedResidual)
#pragma unroll
                            for (int h = 0; h < kTake / 8; ++h) {
                                uint32_t w[4];
                                asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                                             : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                                             : "r"(slot(lane, g / 8 + h))
                                             : "memory");
                                add_values(half, w, v + 8 * h);
                            }
                        if constexpr (EPI == kEpiGated)
#pragma unroll
                            for (int e = 0; e < kTake; ++e) v[e] *= __uint_as_float(raw2[e]);
                        uint32_t w[kTake / 2];
                        pack_values<kTake>(half, v, w);
#pragma unroll
                        for (int h = 0; h < kTake / 8; ++h)
                            asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(slot(lane, g / 8 + h)),
                                         "r"(w[4 * h]), "r"(w[4 * h + 1]), "r"(w[4 * h + 2]), "r"(w[4 * h + 3])
                                         : "memory");
                    }
                    read_out();
                    if constexpr (ACCESS == kPackedAny) {
                        // Rows that start at any element: a thread has a word (two columns)
                        // of the row, and where the row starts at an odd element stores the
                        // second with the next thread's first.
                        constexpr int kWords = kWarpCols / 2;
                        const int x = lane % kWords, n = p.N - c0;
                        int r = lane / kWords;
                        uint16_t *q = static_cast<uint16_t *>(p.out) + (long long)(r0 + r) * p.ld_out + c0;
#pragma unroll 8
                        for (int j = 0; j < 32; j += 32 / kWords, r += 32 / kWords, q += 32 / kWords * p.ld_out) {
                            uint32_t w;
                            asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(slot(r, x / 4) + x % 4 * 4) : "memory");
                            const uint32_t next = __shfl_down_sync(0xFFFFFFFFu, w, 1, kWords);
                            if (r0 + r >= p.M) continue;
                            const int odd = (int)(reinterpret_cast<uintptr_t>(q) >> 1) & 1, c = 2 * x + odd;
                            const uint32_t v = odd ? __byte_perm(w, next, 0x5432) : w;
                            if (c + 1 < n && !(odd && x == kWords - 1))
                                *reinterpret_cast<uint32_t *>(q + c) = v;
                            else if (c < n)
                                q[c] = (uint16_t)v;
                            if (odd && x == 0 && n > 0) q[0] = (uint16_t)w;
                        }
                    } else if (pc < p.N) {
                        uint16_t *q = static_cast<uint16_t *>(p.out) + (long long)(r0 + pr) * p.ld_out + pc;
#pragma unroll
                        for (int j = 0; j < 32; j += kStepRows, q += kStepRows * p.ld_out) {
                            uint4 w;
                            asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                                         : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                                         : "r"(slot(pr + j, px))
                                         : "memory");
                            if (r0 + pr + j < p.M) *reinterpret_cast<uint4 *>(q) = w;
                        }
                    }
                }
                continue;
            }
            if (ACCESS == kColumns && whole) {
                if constexpr (ACCESS == kColumns) {
                    constexpr int kRows = 8;
#pragma unroll 1
                    for (int g = 0; g < kWarpCols / kG; ++g) {
                        __syncwarp();  // the last group has been read
                        put(acc + (uint32_t)(g * kG), 0u);
                        __syncwarp();
                        if (g + 1 == kWarpCols / kG) read_out();
                        const int c = c0 + g * kG + lane;
#pragma unroll 1
                        for (int r = 0; r < 32; r += kRows) {
                            uint32_t in[kRows];
                            column_load<kRows>(p, r0 + r, c, 1, in);
                            float v[kRows];
#pragma unroll
                            for (int j = 0; j < kRows; ++j) {
                                const uint32_t at = unit(r + j, lane >> 2) + (lane & 3) * 4u;
                                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v[j]) : "r"(at) : "memory");
                            }
                            column_epilogue<EPI, kRows>(p, r0 + r, c, 1, v, in);
                        }
                    }
                }
                continue;
            }
#pragma unroll 1
            for (int b = 0; b < kBatches; ++b) {
                if (b % kGroupBatches == 0) {
                    const uint32_t from = acc + (uint32_t)(b / kGroupBatches * kG);
                    __syncwarp();  // the last group has been read
                    put(from, 0u);
                    if (EPI == kEpiGated) put(from + kTileCols, kHalfTurn);
                    __syncwarp();
                    if (b + kGroupBatches == kBatches) read_out();
                }
                if (ACCESS == kFours && kAhead && whole && b + 1 < kBatches)
                    group_load<EPI, kBatch>(p, r0 + row_of(b + 1), col_of(b + 1), kStep, next);
                float v[4 * kBatch], u[EPI == kEpiGated ? 4 * kBatch : 1];
                get(row_of(b), 0u, v);
                if constexpr (EPI == kEpiGated) get(row_of(b), kHalfTurn, u);
                const int r = r0 + row_of(b), c = col_of(b);
                if (ACCESS == kFours && whole) {
                    group_epilogue<EPI, kBatch>(p, r, c, kStep, v, u, in);
                } else if (c < p.N) {  // partials: rows padded to whole groups
                    float *part = p.part + (long long)w.split * p.M * p.ld_part;
                    group_keep<kBatch>(part, p.ld_part, r, p.M, c, kStep, v);
                    if constexpr (EPI == kEpiGated)
                        group_keep<kBatch>(part + p.ld_part / 2, p.ld_part, r, p.M, c, kStep, u);
                }
                if constexpr (kAhead) in = next;
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
        ptx::tmem_dealloc_pair(tmem_base, 2 * BN);
    }
    ptx::cluster_sync_relaxed();  // neither CTA leaves while the other may reach its shared memory
}

// Sums of the split partials, four columns a thread, or, where there are many
// splits (and so few results), eight threads for four columns, each adding
// every eighth split: all loads are on their way at once (backward 6846x192x64
// 15.7 us, four columns a thread 17.6; 4x115x6912 13.8 and 16.0).  The partials
// were just written and sit in L2.
template <int EPI, int LANES>
__global__ void __launch_bounds__(256) gemm_finish_kernel(const __grid_constant__ FinishArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (threadIdx.x == 0 && a.trigger) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int groups = (a.e.N + 3) >> 2;
    const long long all = (long long)groups * a.e.M;
    long long i = ((long long)blockIdx.x * blockDim.x + threadIdx.x) / LANES;
    const int lane = threadIdx.x % LANES;
    const bool mine = i < all;
    if (LANES == 1 && !mine) return;
    i = mine ? i : all - 1;  // every thread takes part in the sums below
    const int r = (int)(i / groups), c = (int)(i % groups) * 4;
    const long long step = (long long)a.e.M * a.e.ld_part;
    const float *src = a.e.part + (long long)r * a.e.ld_part + c + lane * step;
    float v[4] = {0.f, 0.f, 0.f, 0.f}, u[4] = {0.f, 0.f, 0.f, 0.f};
    EpiIn<EPI> in;
    if (lane == 0) epi_load<EPI>(a.e, r, c, in);
#pragma unroll 4
    for (int s = lane; s < a.splits; s += LANES, src += LANES * step) {
        const float4 x = *reinterpret_cast<const float4 *>(src);
        v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
        if (EPI == kEpiGated) {
            const float4 y = *reinterpret_cast<const float4 *>(src + a.e.ld_part / 2);
            u[0] += y.x, u[1] += y.y, u[2] += y.z, u[3] += y.w;
        }
    }
#pragma unroll
    for (int d = LANES / 2; d > 0; d /= 2)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[e] += __shfl_down_sync(0xFFFFFFFFu, v[e], d, LANES);
            if (EPI == kEpiGated) u[e] += __shfl_down_sync(0xFFFFFFFFu, u[e], d, LANES);
        }
    if (mine && lane == 0) epilogue<EPI>(a.e, r, c, v, u, in);
}

cudaError_t launch_chained(const void *fn, dim3 grid, dim3 block, size_t smem, void **params,
                           cudaStream_t stream) {
    cudaLaunchConfig_t c = {};
    cudaLaunchAttribute attr[1];
    c.gridDim = grid;
    c.blockDim = block;
    c.dynamicSmemBytes = smem;
    c.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    c.attrs = attr;
    c.numAttrs = 1;
    return cudaLaunchKernelExC(&c, fn, params);
}

const void *kernel_of(int form, int epi, int bn, Access access) {
#define ROUTE_GEMM(F, E, A)                                                                    \
    if (form == F && epi == E && access == A)                                                  \
        return bn == 256 ? reinterpret_cast<const void *>(layer_gemm_kernel<F, E, 256, A>)     \
                         : reinterpret_cast<const void *>(layer_gemm_kernel<F, E, 128, A>);
#define ROUTE_GEMM4(F, E) \
    ROUTE_GEMM(F, E, kColumns) ROUTE_GEMM(F, E, kFours) ROUTE_GEMM(F, E, kPacked) ROUTE_GEMM(F, E, kPackedAny)
    ROUTE_GEMM4(kFormNT, kEpiLinear)
    ROUTE_GEMM4(kFormNT, kEpiAct)
    ROUTE_GEMM(kFormNT, kEpiLinear, kPackedResidual)
    ROUTE_GEMM(kFormNT, kEpiAct, kPackedResidual)
    ROUTE_GEMM4(kFormMixed, kEpiLinear)
    // h, d gate and d up have padded rows: fours at least
    ROUTE_GEMM(kFormNT, kEpiGated, kFours)
    ROUTE_GEMM(kFormNT, kEpiGated, kPacked)
    ROUTE_GEMM(kFormNN, kEpiDGate, kFours)
#undef ROUTE_GEMM4
#undef ROUTE_GEMM
    return nullptr;
}

}  // namespace

cudaError_t gemm_configure() {
    for (int form : {kFormNT, kFormNN, kFormMixed})
        for (int epi = 0; epi < kEpiCount; ++epi)
            for (int bn : {256, 128})
                for (Access access : {kColumns, kFours, kPacked, kPackedResidual, kPackedAny})
                    if (const void *k = kernel_of(form, epi, bn, access)) {
                        const cudaError_t e = cudaFuncSetAttribute(
                            k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_of(bn));
                        if (e != cudaSuccess) return e;
                    }
    return cudaSuccess;
}

int gemm_smem_bytes() { return (int)(smem_of(256) > smem_of(128) ? smem_of(256) : smem_of(128)); }

cudaError_t gemm_launch(int form, int epi, int bn, const GemmMaps &maps, const GemmArgs &args,
                        cudaStream_t stream) {
    // A residual is read packed only where a tile's products take longer than
    // that, since no buffer is left to read it a tile ahead (residuals from memory:
    // 4096x64x3584 25.5 us, by fours 21.1; 4096x1024x3584, 16 k-blocks, 28.5 and
    // 27.5; 4096x1472x3584, 23 of them, 31.1 and 32.8; in L2 packed is as fast or
    // faster at all of these, and with one tile a pair: 700x512x2048 6.5 and 7.6).
    constexpr int kResidualBlocks = 24;
    bool fours = true, any = epi != kEpiDGate, packed = any, residual = false;
    for (int i = 0; i < args.nprob; ++i) {
        const Epilogue &e = args.p[i].e;
        fours = fours && (e.vec & kVecOut);
        any = any && (e.vec & kVecAny) && e.saved == nullptr && e.residual == nullptr;
        packed = packed && (e.vec & kVecPacked) && e.N % 8 == 0 && e.saved == nullptr;
        residual = residual || e.residual != nullptr;
        if (e.residual != nullptr && args.p[i].kblocks < kResidualBlocks) packed = false;
    }
    const Access access = packed  ? (residual ? kPackedResidual : kPacked)
                          : fours ? kFours
                          : any   ? kPackedAny
                                  : kColumns;
    const void *k = kernel_of(form, epi, bn, access);
    if (k == nullptr || args.pairs <= 0 || args.items <= 0) return cudaErrorInvalidConfiguration;
    void *params[] = {const_cast<GemmMaps *>(&maps), const_cast<GemmArgs *>(&args)};
    return launch_chained(k, dim3(2 * args.pairs), dim3(gemm_threads(epi)), smem_of(bn), params, stream);
}

cudaError_t gemm_finish_launch(int epi, const FinishArgs &args, cudaStream_t stream) {
    const int lanes = args.splits >= 8 ? 8 : 1;
#define ROUTE_FINISH(E)                                                                 \
    (lanes == 8 ? reinterpret_cast<const void *>(gemm_finish_kernel<E, 8>)              \
                : reinterpret_cast<const void *>(gemm_finish_kernel<E, 1>))
    const void *k = epi == kEpiLinear  ? ROUTE_FINISH(kEpiLinear)
                    : epi == kEpiGated ? ROUTE_FINISH(kEpiGated)
                    : epi == kEpiAct   ? ROUTE_FINISH(kEpiAct)
                                       : ROUTE_FINISH(kEpiDGate);
#undef ROUTE_FINISH
    const long long threads = (long long)((args.e.N + 3) / 4) * args.e.M * lanes;
    void *params[] = {const_cast<FinishArgs *>(&args)};
    return launch_chained(k, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, params, stream);
}

}  // namespace route
