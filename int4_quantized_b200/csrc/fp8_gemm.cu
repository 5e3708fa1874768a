// fp8_gemm.cu -- the product of e4m3 codes with a scale per block of 128, dense and by experts.
//
// y[m][n] = sum over blocks b of 128 k: xs[m][b] * ws[n / 128][b] * sum over k in b of x[m][k] w[n][k]
// (with experts: rows offsets[e] .. offsets[e + 1] - 1 of x take the weights and scales of
// expert e). The inner sums run on the tensor cores (tcgen05 kind::f8f6f4, exact products,
// fp32 sums in tensor memory); each block's sum is then multiplied by its two scales and
// added in fp32 registers ("promotion"), and y is rounded once.
//
// Few rows (fp8_stream): A = 128 weight rows, B = 16 to 64 rows of x, so that the weights,
// which are nearly all the bytes, fill the tensor core's long side; D = 128 lanes (weight
// rows) x NT columns (rows of x). K is split over a thread-block cluster where the tiles
// alone would leave SMs without work; the CTAs then exchange their partial sums through
// distributed shared memory and add them in a fixed order.
//   warp 0      TMA producer: 128 x 128 weights and NT x 128 codes of x a block of k
//   warp 1      tensor memory, MMA issue (4 instructions of 32 k a block)
//   warp 2      the rows' scales of each block, by 4-byte asynchronous copies
//   warps 4-..  promotion and stores; lane = weight row, so stores of y are contiguous
//
// Many rows (fp8_wide): one CTA makes a tile of 128 rows of x x 256 or 128 weight rows, or a
// pair of CTAs (cta_group::2) one of 256 x 256. In a pair each CTA loads its own rows of x and
// half of the weights, so that a block of k costs an SM 32 KB from L2 instead of 48 (which
// single CTAs take at 60 bytes a clock); the smaller tiles leave fewer rows empty and fill the
// machine sooner. Here D's lanes are rows of x, so that the
// scale of a thread's whole row of D is one number a block of k. A block's time is the
// epilogue's: with two buffers of all columns, an MMA, its epilogue and the signals between
// them share the time of two blocks (8192 x 4096 x 14336, as first built: no epilogue work 378
// us, reads of tensor memory only 423, all 466; without waiting for it 318). Tried and slower:
// two half buffers a block (499 us for 477), 16 epilogue warps (570 for 466), the next columns
// read while the last are added (registers spill: 514 for 445), spinning waits (474 for 460).
//   warp 0      TMA producer (of a pair both; all bytes are counted on the first CTA's barriers)
//   warp 1      tensor memory; MMA issue (in the first CTA, for both)
//   warps 4-11  promotion and stores: 32 rows x half of the columns a warp, kept in registers; the
//               first four warps give theirs up to them (setmaxnreg)
// Every wait is bounded (about one second); one that gives up sets Q4_STATUS_TIMEOUT in the
// status word and its role ends. A lane reads the timer by itself, so the lanes of a warp may not
// agree; where the warp has instructions to execute as a whole (tensor memory, cluster barriers)
// they vote before any leaves the loop. (8192 x 4096 x 14336: 437 us with the vote, 436 without; the
// same with the wait skipped, and no lane leaving, once one has run out: 458 to 480.) Before a block
// goes it still waits, with the same bound, for its copies and MMAs in flight, and for the other
// CTAs of its cluster.
#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "fp8_plan.h"
#include "kernels.h"
#include "once.cuh"
#include "overlap.cuh"
#include "tcgen05.cuh"

namespace q4 {

namespace {

constexpr int kBK = 128;             // k per block: one 128-byte swizzle row of codes
constexpr int kWRows = 128;          // weight rows per tile
constexpr int kWBytes = kWRows * kBK;
constexpr int kMaxExperts = 1024;

struct Fp8Args {
    const float *xs;         // [R][kb]
    const float *ws;         // [E][nb][kb]
    const int32_t *offsets;  // [E + 1] on the device, or null: one expert, rows 0 .. R - 1
    void *y;
    uint32_t *status;
    int64_t N;
    int32_t R, E;
    int32_t nb, kb;          // blocks of 128 along N and K
    int32_t split;           // CTAs of a cluster that share one tile's K
    int32_t stages;          // ring depth (fp8_stream)
    int32_t bulk;            // whether the TMA can store y (fp8_wide): rows of whole 16-byte units
    int32_t box;             // rows of x a copy brings (fp8_wide): 128, fewer where x has fewer
};

// The experts' rows and tiles, worked out once a block: expert e has the rows rows0[e] ..
// rows0[e + 1] - 1 and first[e] row tiles come before its own (first[E] in all). Offsets are
// taken as a running maximum held inside 0 .. R, so that whatever stands there, the experts'
// rows follow one another inside x and y. Called by the whole block; ends without a barrier.
Q4_DEVINL void count_tiles(const Fp8Args &a, int tile_rows, int32_t *first, int32_t *rows0) {
    if (threadIdx.x >= 32) return;
    const int lane = threadIdx.x;
    int32_t carry = 0, high = 0;
    for (int b = 0; b <= a.E; b += 32) {
        const int e = b + lane;
        int32_t m = a.offsets ? (e <= a.E ? a.offsets[e] : 0) : (e == 0 ? 0 : a.R);
        m = max(high, min(m, a.R));
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t v = __shfl_up_sync(0xffffffffu, m, o);
            if (lane >= o) m = max(m, v);
        }
        // expert e - 1 ends where expert e begins
        const int32_t before = __shfl_up_sync(0xffffffffu, m, 1);
        const int32_t n = (m - (lane ? before : high) + tile_rows - 1) / tile_rows;
        int32_t x = n;  // lane 0 of the first chunk has no expert before it: rows 0 .. offsets[0] - 1 are nobody's
        if (e == 0) x = 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t v = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += v;
        }
        if (e <= a.E) {
            rows0[e] = m;
            first[e] = carry + x;
        }
        carry += __shfl_sync(0xffffffffu, x, 31);
        high = __shfl_sync(0xffffffffu, m, 31);
    }
}

struct Tile {
    int e, nb;       // expert, column tile
    int row0, rows;  // rows of x
};
// Tile j of first[E] * cols (cols: column tiles of a matrix): by expert, then column tile, then
// row tile, so that the row tiles that share weights come one after the other and find them
// in L2.
Q4_DEVINL Tile tile_at(const Fp8Args &a, int tile_rows, int cols, const int32_t *first, const int32_t *rows0, int64_t j) {
    // the expert: the last e with first[e] * cols <= j
    int lo = 0, hi = a.E;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((int64_t)first[mid] * cols <= j) lo = mid;
        else hi = mid;
    }
    // several experts without rows share a first tile: the last of them is the one with rows
    const int n = first[lo + 1] - first[lo];
    const int64_t i = j - (int64_t)first[lo] * cols;
    Tile t;
    t.e = lo;
    t.nb = (int)(i / n);
    t.row0 = rows0[lo] + (int)(i - (int64_t)t.nb * n) * tile_rows;
    t.rows = min(tile_rows, rows0[lo + 1] - t.row0);
    return t;
}

// A place in a ring of n slots and the parity of its round, kept without divisions.
struct Slot {
    int i = 0;
    uint32_t round = 0;
    Q4_DEVINL void next(int n) {
        if (++i == n) {
            i = 0;
            round ^= 1;
        }
    }
};

template <typename Y>
Q4_DEVINL Y round_to(float v) {
    if constexpr (std::is_same<Y, float>::value) return v;
    else if constexpr (std::is_same<Y, __half>::value) return __float2half_rn(v);
    else return __float2bfloat16_rn(v);
}

Q4_DEVINL uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
    return r;
}
Q4_DEVINL uint32_t map_rank(uint32_t smem_addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr), "r"(rank));
    return r;
}
Q4_DEVINL void st_cluster2(uint32_t addr, float a, float b) {
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(a), "f"(b) : "memory");
}
Q4_DEVINL void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// An arrival that publishes no memory of its own: the buffers of tensor memory it frees are
// ordered by the tcgen05 fences. (With release at cluster scope each arrival waited for the
// thread's outstanding loads: 31 % of the epilogue warps' time.)
Q4_DEVINL void arrive_peer(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
Q4_DEVINL void fence_cluster() { asm volatile("fence.acq_rel.cluster;" ::: "memory"); }
Q4_DEVINL void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
Q4_DEVINL void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
Q4_DEVINL void prefetch_map(const void *tmap) { asm volatile("prefetch.tensormap [%0];" ::"l"(tmap) : "memory"); }
Q4_DEVINL void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ---- few rows ---------------------------------------------------------------------------
template <int NT>
struct Stream {
    static constexpr int kXBytes = NT * kBK;
    static constexpr int kStage = kWBytes + kXBytes;
    static constexpr int kBufs = kStreamBufs;            // tensor-memory buffers of NT columns
    static constexpr int kCols = kBufs * NT;             // 128 to 512 columns
    // one warp an SM quarter adds up to 32 columns a block of k before the next block's sums
    // are there; wider tiles take two (with one, 128 columns took 0.9 us a block, the loads and
    // waits one after the other)
    static constexpr int kEpiWarps = NT <= 32 ? 4 : 8;
    static constexpr int kOwn = NT * 4 / kEpiWarps;      // columns a warp keeps
    static constexpr int kThreads = 128 + 32 * kEpiWarps;
    static constexpr uint32_t kIdesc = (1u << 4) | ((uint32_t)(NT >> 3) << 17) | ((uint32_t)(kWRows >> 4) << 24);
};

template <int NT, typename Y>
__global__ void __launch_bounds__(Stream<NT>::kThreads, 1)
fp8_stream(const Fp8Args a, const __grid_constant__ CUtensorMap tmx, const __grid_constant__ CUtensorMap tmw) {
    using S = Stream<NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t *p = ring + (size_t)a.stages * S::kStage;
    float *parts = reinterpret_cast<float *>(p);  // [split][NT / split / 2][128][2]
    if (a.split > 1) p += kWRows * NT * 4;
    float *xsc = reinterpret_cast<float *>(p);  // [kBufs][NT]
    uint64_t *full = reinterpret_cast<uint64_t *>(p + S::kBufs * NT * 4);
    uint64_t *empty = full + a.stages;
    uint64_t *dfull = empty + a.stages;
    uint64_t *dempty = dfull + S::kBufs;
    uint64_t *sfull = dempty + S::kBufs;
    uint64_t *done = sfull + S::kBufs;
    uint64_t *joined = done + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(joined + 1);
    int32_t *first = reinterpret_cast<int32_t *>(tmem_slot + 4);
    int32_t *rows0 = first + a.E + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        prefetch_map(&tmw);
        prefetch_map(&tmx);
    }
    if (threadIdx.x == 32) {
        for (int i = 0; i < a.stages; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
        }
        for (int i = 0; i < S::kBufs; ++i) {
            mbar_init(dfull + i, 1);
            mbar_init(dempty + i, S::kEpiWarps);
            mbar_init(sfull + i, 32);
        }
        mbar_init(done, 1);
        mbar_init(joined, S::kEpiWarps * a.split);
        fence_barrier_init();
    }
    if (warp == 1) {
        __syncwarp();
        tmem_alloc(tmem_slot, S::kCols);
        tmem_relinquish();
    }
    begin_overlapped();  // nothing above touches global memory
    count_tiles(a, NT, first, rows0);
    tc_fence_before();
    __syncthreads();
    // every CTA's barriers must stand before another arrives on them: waited for before the exchange
    if (a.split > 1) cluster_arrive();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    const int rank = a.split > 1 ? (int)cluster_rank() : 0;
    const int64_t tiles = (int64_t)first[a.E] * a.nb;
    // a split tile is its cluster's only one: the exchange buffer is used once
    const int64_t step = a.split > 1 ? tiles : gridDim.x, tile0 = blockIdx.x / a.split;
    bool met = false;  // this thread has waited for the cluster
    const int k0 = (int)((int64_t)a.kb * rank / a.split), k1 = (int)((int64_t)a.kb * (rank + 1) / a.split);
    bool timed_out = false;

    if (warp == 0) {
        if (lane == 0) {
            Slot s;
            int filled = 0;
            for (int64_t j = tile0; j < tiles && !timed_out; j += step) {
                const Tile t = tile_at(a, NT, a.nb, first, rows0, j);
                const int wrow = (int)(t.e * a.N + (int64_t)t.nb * kWRows);
                for (int kb = k0; kb < k1; ++kb) {
                    // a slot that was never filled counts as freed in the round before
                    timed_out = !mbar_wait(empty + s.i, s.round ^ 1);
                    if (timed_out) break;
                    uint8_t *st = ring + (size_t)s.i * S::kStage;
                    mbar_arrive_expect_tx(full + s.i, S::kStage);
                    tma_load_2d(st, &tmw, full + s.i, kb * kBK, wrow);
                    tma_load_2d(st + kWBytes, &tmx, full + s.i, kb * kBK, t.row0);
                    s.next(a.stages);
                    filled = min(filled + 1, a.stages);
                }
            }
            // no copy may land after the block has gone: the slots' last rounds
            for (int i = 0; i < filled; ++i)
                timed_out |= !mbar_wait(full + i, i < s.i ? s.round : s.round ^ 1);
        }
    } else if (warp == 1) {
        // the whole warp keeps step and one lane issues: operands stay uniform across the warp
        Slot s, d;
        const uint64_t base = sw128_desc(ring);
        const uint32_t dt = __shfl_sync(0xffffffffu, tmem, 0);
        for (int64_t j = tile0; j < tiles && !timed_out; j += step) {
            for (int kb = k0; kb < k1; ++kb) {
                timed_out = !mbar_wait(dempty + d.i, d.round ^ 1);
                if (!timed_out) timed_out = !mbar_wait(full + s.i, s.round);
                timed_out = __any_sync(0xffffffffu, timed_out);
                if (timed_out) break;
                tc_fence_after();
                const uint64_t wd = base + (uint32_t)(s.i * (S::kStage >> 4)), xd = wd + (kWBytes >> 4);
                if (elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < kBK / 32; ++kk)
                        umma_f8(dt + (uint32_t)(d.i * NT), wd + 2 * kk, xd + 2 * kk, S::kIdesc, kk > 0 ? 1u : 0u);
                    umma_commit(empty + s.i);
                    umma_commit(dfull + d.i);
                }
                __syncwarp();
                s.next(a.stages);
                d.next(S::kBufs);
            }
        }
        if (elect_one()) umma_commit(done);
        __syncwarp();
        timed_out |= !mbar_wait(done, 0);
    } else if (warp == 2) {  // each lane copies and arrives by itself, and may leave so
        Slot d;
        for (int64_t j = tile0; j < tiles && !timed_out; j += step) {
            const Tile t = tile_at(a, NT, a.nb, first, rows0, j);
            for (int kb = k0; kb < k1; ++kb) {
                timed_out = !mbar_wait(dempty + d.i, d.round ^ 1);
                if (timed_out) break;
#pragma unroll
                for (int c = 0; c < NT; c += 32) {
                    const int col = c + lane;
                    if (col < NT)
                        cp_async4(xsc + d.i * NT + col,
                                  a.xs + (int64_t)(t.row0 + min(col, t.rows - 1)) * a.kb + kb);
                }
                cp_async_arrive(sfull + d.i);
                d.next(S::kBufs);
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp >= 4) {
        constexpr int OWN = S::kOwn;
        const int q = warp & 3, rl = 32 * q + lane, c0 = ((warp - 4) >> 2) * OWN;
        const uint32_t lane_base = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)c0;
        Y *const y = static_cast<Y *>(a.y);
        Slot d;
        for (int64_t j = tile0; j < tiles && !timed_out; j += step) {
            const Tile t = tile_at(a, NT, a.nb, first, rows0, j);
            const float *wsc = a.ws + ((int64_t)t.e * a.nb + t.nb) * a.kb;
            const int64_t n = (int64_t)t.nb * kWRows + rl;
            uint64_t acc[OWN / 2];
#pragma unroll
            for (int i = 0; i < OWN / 2; ++i) acc[i] = 0ull;
            float w_next = k0 < k1 ? wsc[k0] : 0.f;
            for (int kb = k0; kb < k1; ++kb) {
                const float wv = w_next;
                if (kb + 1 < k1) w_next = wsc[kb + 1];
                if (!__all_sync(0xffffffffu, mbar_wait(sfull + d.i, d.round) && mbar_wait(dfull + d.i, d.round))) {
                    timed_out = true;
                    break;
                }
                tc_fence_after();
                constexpr int CH = OWN < 32 ? OWN : 32;
#pragma unroll
                for (int c = 0; c < OWN; c += CH) {
                    uint32_t v[CH];
                    if constexpr (CH == 32) tmem_ld32(lane_base + (uint32_t)(d.i * NT + c), v);
                    else tmem_ld16(lane_base + (uint32_t)(d.i * NT + c), v);
                    // the columns' scales while the sums are on their way
                    float s[CH];
#pragma unroll
                    for (int i = 0; i < CH / 4; ++i) {
                        const float4 f = reinterpret_cast<const float4 *>(xsc + d.i * NT + c0 + c)[i];
                        s[4 * i] = f.x * wv, s[4 * i + 1] = f.y * wv, s[4 * i + 2] = f.z * wv, s[4 * i + 3] = f.w * wv;
                    }
                    tmem_wait_ld();
                    if (c + CH == OWN) {  // all read: the buffer and its scales are free
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(dempty + d.i);
                    }
#pragma unroll
                    for (int i = 0; i < CH / 2; ++i)
                        fma2_acc(acc[c / 2 + i], ((uint64_t)__float_as_uint(s[2 * i + 1]) << 32) | __float_as_uint(s[2 * i]),
                                 v[2 * i], v[2 * i + 1]);
                }
                d.next(S::kBufs);
            }
            auto value = [&](int c) {
                return __uint_as_float((c & 1) ? (uint32_t)(acc[c >> 1] >> 32) : (uint32_t)acc[c >> 1]);
            };
            if (a.split == 1) {
                if (n < a.N && !timed_out) {
#pragma unroll
                    for (int c = 0; c < OWN; ++c)
                        if (c0 + c < t.rows) y[(int64_t)(t.row0 + c0 + c) * a.N + n] = round_to<Y>(value(c));
                }
            } else {
                // Columns are added and stored by CTA column / (NT / split); slot r of its buffer
                // holds CTA r's part, two columns of a row side by side (each CTA has two or more)
                // and the rows of such a pair one after the other: no bank is written twice.
                const int shift = __ffs(NT / a.split) - 1, cols = 1 << shift;
                cluster_wait();
                met = true;
#pragma unroll
                for (int c = 0; c < OWN; c += 2) {
                    const int to = (c0 + c) >> shift, in = (c0 + c) & (cols - 1);
                    st_cluster2(map_rank(smem_u32(parts + ((((rank << shift) + in) << 6) + rl) * 2), (uint32_t)to), value(c),
                                value(c + 1));
                }
                fence_cluster();
                __syncwarp();
                if (lane < a.split) arrive_cluster(map_rank(smem_u32(joined), (uint32_t)lane));
                timed_out |= !mbar_wait(joined, 0);
                fence_cluster();
                if (n < a.N && !timed_out) {
                    for (int in = (warp - 4) >> 2; in < cols; in += S::kEpiWarps / 4) {
                        const int c = (rank << shift) + in;
                        if (c >= t.rows) break;
                        float sum = 0.f;
                        for (int r = 0; r < a.split; ++r) sum += parts[((((r << shift) + (in & ~1)) << 6) + rl) * 2 + (in & 1)];
                        y[(int64_t)(t.row0 + c) * a.N + n] = round_to<Y>(sum);
                    }
                }
            }
        }
    }
    if (timed_out && a.status) atomicOr(a.status, Q4_STATUS_TIMEOUT);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (a.split > 1) {
        if (!met) cluster_wait();
        // A CTA whose parts have all come cannot be written to any more. One that gave up on
        // them stays until the others have gone or given up too.
        if (__syncthreads_or(timed_out)) cluster_sync_all();
    }
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, S::kCols);
}

// ---- many rows ----------------------------------------------------------------------------
constexpr int kWideThreads = 384;  // TMA, MMA, two without a role, eight epilogue warps
// The block launches with 168 registers a thread; the first warpgroup keeps 72, the two
// epilogue warpgroups (128 fp32 sums a thread) take 216: 128 * 72 + 256 * 216 is exactly the
// 384 * 168 that the block holds, so every increase is served.
constexpr int kWideRegs = 168, kWideLow = 72, kWideHigh = 216;
static_assert(128 * kWideLow + 256 * kWideHigh == kWideThreads * kWideRegs, "register split");

// Shared memory in which an epilogue warp turns 32 rows x 64 bytes of y, 4 bytes a row apart
// from the banks of the last.
constexpr int kTurnRow = 68, kTurnBytes = 32 * kTurnRow;

// Whether full rows of y leave through shared memory and the TMA, so that the epilogue warps go
// on while they are stored (8192 x 4096 x 14336: 484 us, 472 so; 32768 rows of 64 experts: 146
// and 141). Single CTAs would pay for it with the depth of their ring (16 tokens x 2 of 8 experts
// of 14336 x 4096: 87 and 90), fp32 would not fit.
template <bool PAIR, typename Y>
constexpr bool kAsyncStore = PAIR && sizeof(Y) == 2;

// A tile of BN weight rows, made by one CTA or a pair.
template <bool PAIR, int BN, bool ASYNC>
struct Wide {
    static constexpr int kCtas = PAIR ? 2 : 1;
    static constexpr int kRows = 128 * kCtas;    // rows of x a tile
    static constexpr int kOwnCols = BN / kCtas;  // weight rows that a CTA loads
    static constexpr int kXBytes = 128 * kBK;
    static constexpr int kStage = kXBytes + kOwnCols * kBK;
    // shared memory of an epilogue warp for y: 32 rows x BN / 2 columns of 2 bytes, or the turning
    static constexpr int kOut = ASYNC ? 32 * BN : kTurnBytes;
    static constexpr int kStages = (ASYNC ? 131072 : 196608) / kStage;  // 4 or 6 of 32 KB, 4 of 48
    static constexpr int kBufs = 512 / BN;       // all 512 columns of tensor memory
    static constexpr uint32_t kIdesc = (1u << 4) | ((uint32_t)(BN >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);
    static size_t smem(int E) {
        return 1024 + (size_t)kStages * kStage + 8 * kOut + (2 * kStages + 2 * kBufs + 1) * 8 + 16 +
               (size_t)(2 * E + 2) * 4;
    }
};

template <bool PAIR>
Q4_DEVINL void umma_f8_of(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t acc) {
    if constexpr (PAIR) umma_f8_pair(d, ad, bd, idesc, acc);
    else umma_f8(d, ad, bd, idesc, acc);
}
template <bool PAIR>
Q4_DEVINL void umma_commit_of(uint64_t *bar) {
    if constexpr (PAIR) umma_commit_pair(bar);
    else umma_commit(bar);
}

// 32 bytes in one store: a whole sector, although neighbouring lanes write different rows.
Q4_DEVINL void st_v8(void *p, const uint32_t (&v)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
template <typename Y>
Q4_DEVINL uint32_t two(float lo, float hi) {
    if constexpr (std::is_same<Y, __half>::value) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

// A tile out of shared memory, and the waits for such stores of this thread: until what they read
// may be written again, and until they are done. (The copies end by themselves; no flag is
// waited for.)
Q4_DEVINL void tma_store_2d(const void *tmap, const void *src, int c0, int c1) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(tmap),
                 "r"(smem_u32(src)), "r"(c0), "r"(c1)
                 : "memory");
}
Q4_DEVINL void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
Q4_DEVINL void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
Q4_DEVINL void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

template <bool PAIR, int BN, typename Y>
__global__ void __launch_bounds__(kWideThreads, 1)
fp8_wide(const Fp8Args a, const __grid_constant__ CUtensorMap tmx, const __grid_constant__ CUtensorMap tmw,
         const __grid_constant__ CUtensorMap tmy) {
    constexpr bool ASYNC = kAsyncStore<PAIR, Y>;
    using W = Wide<PAIR, BN, ASYNC>;
    constexpr int HALF = BN / 2;  // columns an epilogue warp keeps
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t *turn = ring + W::kStages * W::kStage;
    uint64_t *full = reinterpret_cast<uint64_t *>(turn + 8 * W::kOut);
    uint64_t *empty = full + W::kStages;
    uint64_t *dfull = empty + W::kStages;
    uint64_t *dempty = dfull + W::kBufs;
    uint64_t *done = dempty + W::kBufs;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
    int32_t *first = reinterpret_cast<int32_t *>(tmem_slot + 4);
    int32_t *rows0 = first + a.E + 1;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = PAIR ? (int)cluster_rank() : 0;
    if (threadIdx.x == 0) {
        prefetch_map(&tmw);
        prefetch_map(&tmx);
    }
    if (threadIdx.x == 32) {
        for (int i = 0; i < W::kStages; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
        }
        for (int i = 0; i < W::kBufs; ++i) {
            mbar_init(dfull + i, 1);
            mbar_init(dempty + i, 8 * W::kCtas);  // the epilogue warps (of both CTAs)
        }
        mbar_init(done, 1);
        fence_barrier_init();
    }
    if (warp == 1) {
        __syncwarp();
        if constexpr (PAIR) {
            tmem_alloc2(tmem_slot, 512);
            tmem_relinquish2();
        } else {
            tmem_alloc(tmem_slot, 512);
            tmem_relinquish();
        }
    }
    begin_overlapped();  // nothing above touches global memory
    count_tiles(a, W::kRows, first, rows0);
    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int cols = (int)((a.N + BN - 1) / BN);
    const int64_t tiles = (int64_t)first[a.E] * cols, step = gridDim.x / W::kCtas, tile0 = blockIdx.x / W::kCtas;
    bool timed_out = false;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kWideLow));
        if (warp == 0) {
            if (lane == 0) {
                Slot s;
                int filled = 0;
                const uint32_t bytes = (uint32_t)(W::kCtas * (W::kStage - (128 - a.box) * kBK));
                for (int64_t j = tile0; j < tiles && !timed_out; j += step) {
                    const Tile t = tile_at(a, W::kRows, cols, first, rows0, j);
                    const int wrow = (int)(t.e * a.N + (int64_t)t.nb * BN + rank * W::kOwnCols);
                    const int xrow = t.row0 + rank * 128;
                    for (int kb = 0; kb < a.kb; ++kb) {
                        timed_out = !mbar_wait(empty + s.i, s.round ^ 1);
                        if (timed_out) break;
                        uint8_t *st = ring + s.i * W::kStage;
                        // of a pair, the first CTA's barrier counts the bytes of both
                        if (rank == 0) mbar_arrive_expect_tx(full + s.i, bytes);
                        if constexpr (PAIR) {
                            const uint32_t bar = map_rank(smem_u32(full + s.i), 0);
                            tma_load_2d_pair(st, &tmx, bar, kb * kBK, xrow);
                            tma_load_2d_pair(st + W::kXBytes, &tmw, bar, kb * kBK, wrow);
                        } else {
                            tma_load_2d(st, &tmx, full + s.i, kb * kBK, xrow);
                            tma_load_2d(st + W::kXBytes, &tmw, full + s.i, kb * kBK, wrow);
                        }
                        s.next(W::kStages);
                        filled = min(filled + 1, W::kStages);
                    }
                }
                // no copy may land after the block has gone, and no arrival from the other block of a
                // pair: the slots' last rounds, of a pair those in which the MMA has freed them (the
                // copies lie before that; those of the second block are counted in the first alone)
                bool ended = true;
                for (int i = 0; i < filled && ended; ++i)
                    ended = mbar_wait((PAIR ? empty : full) + i, i < s.i ? s.round : s.round ^ 1);
                timed_out |= !ended;
            }
        } else if (warp == 1 && rank == 0) {
            // the whole warp keeps step and one lane issues: operands stay uniform across the warp
            Slot s, d;
            const uint64_t base = sw128_desc(ring);
            const uint32_t dt = __shfl_sync(0xffffffffu, tmem, 0);
            for (int64_t j = tile0; j < tiles && !timed_out; j += step) {
                for (int kb = 0; kb < a.kb; ++kb) {
                    timed_out = !mbar_wait(dempty + d.i, d.round ^ 1);
                    if (!timed_out) timed_out = !mbar_wait(full + s.i, s.round);
                    timed_out = __any_sync(0xffffffffu, timed_out);
                    if (timed_out) break;
                    tc_fence_after();
                    const uint64_t xd = base + (uint32_t)(s.i * (W::kStage >> 4)), wd = xd + (W::kXBytes >> 4);
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < kBK / 32; ++kk)
                            umma_f8_of<PAIR>(dt + (uint32_t)(d.i * BN), xd + 2 * kk, wd + 2 * kk, W::kIdesc,
                                             kk > 0 ? 1u : 0u);
                        umma_commit_of<PAIR>(empty + s.i);
                        umma_commit_of<PAIR>(dfull + d.i);
                    }
                    __syncwarp();
                    s.next(W::kStages);
                    d.next(W::kBufs);
                }
            }
            if (elect_one()) umma_commit_of<PAIR>(done);
            __syncwarp();
            timed_out |= !mbar_wait(done, 0);
        } else if (warp == 1) {
            timed_out = !mbar_wait(done, 0);  // the MMAs' last arrival in this block
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kWideHigh));
        const int q = warp & 3, half = (warp - 4) >> 2;
        const uint32_t lane_base = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(half * HALF);
        Y *const y = static_cast<Y *>(a.y);
        constexpr int PER = 32 / (int)sizeof(Y);  // values a 32-byte store
        const bool vec = a.N % PER == 0 && (uintptr_t)a.y % 32 == 0;
        Slot d;
        for (int64_t j = tile0; j < tiles && !timed_out; j += step) {
            const Tile t = tile_at(a, W::kRows, cols, first, rows0, j);
            const int rl = rank * 128 + 32 * q + lane;  // row inside the tile
            const bool live = rl < t.rows;
            const int64_t n0 = (int64_t)t.nb * BN + half * HALF;
            const float *xsc = a.xs + (int64_t)(t.row0 + min(rl, t.rows - 1)) * a.kb;
            const float *wsc = a.ws + ((int64_t)t.e * a.nb + min((int)(n0 / 128), a.nb - 1)) * a.kb;
            uint64_t acc[HALF / 2];
#pragma unroll
            for (int i = 0; i < HALF / 2; ++i) acc[i] = 0ull;
            float x_next = xsc[0], w_next = wsc[0];
            for (int kb = 0; kb < a.kb; ++kb) {
                const float sc = x_next * w_next;
                const uint64_t s2 = ((uint64_t)__float_as_uint(sc) << 32) | __float_as_uint(sc);
                if (kb + 1 < a.kb) x_next = xsc[kb + 1], w_next = wsc[kb + 1];
                if (!__all_sync(0xffffffffu, mbar_wait(dfull + d.i, d.round))) {
                    timed_out = true;
                    break;
                }
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < HALF; c += 32) {
                    uint32_t v0[16], v1[16];
                    tmem_ld16(lane_base + (uint32_t)(d.i * BN + c), v0);
                    tmem_ld16(lane_base + (uint32_t)(d.i * BN + c + 16), v1);
                    tmem_wait_ld();
                    if (c + 32 == HALF) {  // all read: the buffer is free
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            if constexpr (PAIR) arrive_peer(map_rank(smem_u32(dempty + d.i), 0));
                            else mbar_arrive(dempty + d.i);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        fma2_acc(acc[c / 2 + i], s2, v0[2 * i], v0[2 * i + 1]);
                        fma2_acc(acc[c / 2 + 8 + i], s2, v1[2 * i], v1[2 * i + 1]);
                    }
                }
                d.next(W::kBufs);
            }
            if (timed_out) continue;
            auto value = [&](int c) {
                return __uint_as_float((c & 1) ? (uint32_t)(acc[c >> 1] >> 32) : (uint32_t)acc[c >> 1]);
            };
            auto word = [&](int c) {  // the 4 bytes of y from column c on
                if constexpr (sizeof(Y) == 4) return __float_as_uint(value(c));
                else return two<Y>(value(c), value(c + 1));
            };
            constexpr int IN4 = 4 / (int)sizeof(Y);  // columns in 4 bytes
            uint8_t *mine = turn + (warp - 4) * W::kOut;
            const int first_row = rl - lane;
            if (ASYNC && a.bulk && first_row + 32 <= t.rows) {
                if (lane == 0) bulk_wait_read();  // the last tile's rows have left
                __syncwarp();
                // 64 columns after 64, rows of 128 bytes in the 128-byte swizzle
#pragma unroll
                for (int c = 0; c < HALF; c += 8) {
                    uint8_t *at = mine + (c / 64) * 4096 + lane * 128 + (((c / 8) & 7) ^ (lane & 7)) * 16;
                    *reinterpret_cast<uint4 *>(at) =
                        make_uint4(word(c), word(c + IN4), word(c + 2 * IN4), word(c + 3 * IN4));
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) {
#pragma unroll
                    for (int c = 0; c < HALF; c += 64)
                        if (n0 + c < a.N) tma_store_2d(&tmy, mine + (c / 64) * 4096, (int)n0 + c, t.row0 + first_row);
                    bulk_commit();
                }
            } else if (vec) {
                Y *yr = y + (int64_t)(t.row0 + rl) * a.N + n0;
#pragma unroll
                for (int c = 0; c < HALF; c += PER) {
                    uint32_t v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = word(c + i * IN4);
                    if (live && n0 + c < a.N) st_v8(yr + c, v);
                }
            } else {
                // Rows of y that are not whole 32-byte stores: single elements, but a warp's 32 (or,
                // of fp32, 16 of two rows) side by side, not in 32 rows (4099 x 7801 x 880 in fp16:
                // 348 us so, 58 this way)
                constexpr int CH = 64 / (int)sizeof(Y);
                const int col = lane % CH, up = lane / CH;
                if constexpr (ASYNC) {
                    if (lane == 0) bulk_wait_read();
                    __syncwarp();
                }
#pragma unroll
                for (int c = 0; c < HALF; c += CH) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        *reinterpret_cast<uint32_t *>(mine + lane * kTurnRow + 4 * i) = word(c + i * IN4);
                    __syncwarp();
                    const int rows = min(32, t.rows - first_row);
                    if (n0 + c + col < a.N) {
                        Y *yc = y + (int64_t)(t.row0 + first_row) * a.N + n0 + c + col;
#pragma unroll 8
                        for (int r = up; r < rows; r += 32 / CH)
                            yc[(int64_t)r * a.N] = *reinterpret_cast<const Y *>(mine + r * kTurnRow + col * sizeof(Y));
                    }
                    __syncwarp();
                }
            }
        }
        if (ASYNC && lane == 0) bulk_wait();  // y is written
    }
    if (timed_out && a.status) atomicOr(a.status, Q4_STATUS_TIMEOUT);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync_all();  // neither CTA goes while the other may still reach into it
    tc_fence_after();
    if (warp == 1) {
        if constexpr (PAIR) tmem_dealloc2(tmem, 512);
        else tmem_dealloc(tmem, 512);
    }
}

// ---- host ---------------------------------------------------------------------------------
bool encode_codes_map(CUtensorMap *tm, const uint8_t *codes, int64_t rows, int64_t K, int box_rows) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)K};
    const cuuint32_t box[2] = {(cuuint32_t)kBK, (cuuint32_t)box_rows};
    const cuuint32_t es[2] = {1, 1};
    return enc(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(codes), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// y [rows][N] of 2-byte values, stored by 32 rows x 64 columns.
bool encode_rows_map(CUtensorMap *tm, void *y, int64_t rows, int64_t N) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)N, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)N * 2};
    const cuuint32_t box[2] = {64, 32};
    const cuuint32_t es[2] = {1, 1};
    return enc(tm, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, y, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

// Row tiles of `rows` rows: at most (which experts have rows is known on the device only).
int64_t row_tiles(const Fp8Args &a, int rows) {
    return a.offsets ? std::min((int64_t)a.R, (int64_t)a.E + a.R / rows) : (a.R + rows - 1) / rows;
}

template <int NT, typename Y>
cudaError_t launch_stream(Fp8Args a, const uint8_t *x, const uint8_t *w, int64_t K, int sms, cudaStream_t st) {
    using S = Stream<NT>;
    const int64_t tiles = row_tiles(a, NT) * a.nb;
    const StreamPlan plan = stream_plan(NT, tiles, a.kb, a.E, sms);
    a.split = plan.split;
    a.stages = plan.stages;
    CUtensorMap tmx, tmw;
    if (!encode_codes_map(&tmx, x, a.R, K, NT) || !encode_codes_map(&tmw, w, (int64_t)a.E * a.N, K, kWRows))
        return cudaErrorInvalidValue;
    auto kern = fp8_stream<NT, Y>;
    static std::atomic<uint64_t> ready{0};
    const cudaError_t e = once_per_device(ready, [&]() {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemMax);
    });
    if (e != cudaSuccess) return e;
    const unsigned grid = (unsigned)(a.split > 1 ? tiles * a.split : std::min<int64_t>(tiles, sms));
    return launch_overlapped(kern, grid, S::kThreads, plan.smem, st, (unsigned)a.split, a, tmx, tmw);
}

template <bool PAIR, int BN, typename Y>
cudaError_t launch_wide(Fp8Args a, const uint8_t *x, const uint8_t *w, int64_t K, int sms, cudaStream_t st) {
    using W = Wide<PAIR, BN, kAsyncStore<PAIR, Y>>;
    const int64_t tiles = row_tiles(a, W::kRows) * ((a.N + BN - 1) / BN);
    // What a smaller box leaves of the x tile in shared memory is any codes: rows of D that are
    // not stored
    a.box = (int)std::min<int64_t>(128, (a.R + 7) / 8 * 8);
    CUtensorMap tmx, tmw, tmy;
    if (!encode_codes_map(&tmx, x, a.R, K, a.box) || !encode_codes_map(&tmw, w, (int64_t)a.E * a.N, K, W::kOwnCols))
        return cudaErrorInvalidValue;
    a.bulk = kAsyncStore<PAIR, Y> && a.N % 8 == 0 && (uintptr_t)a.y % 16 == 0;
    if (!a.bulk) tmy = tmx;  // not used
    else if (!encode_rows_map(&tmy, a.y, a.R, a.N)) return cudaErrorInvalidValue;
    auto kern = fp8_wide<PAIR, BN, Y>;
    static std::atomic<uint64_t> ready{0};
    const cudaError_t e = once_per_device(ready, [&]() -> cudaError_t {
        // the register split assumes the block launches at exactly kWideRegs a thread; any other
        // allocation could leave an increase waiting: refuse to launch
        cudaFuncAttributes fa;
        const cudaError_t ge = cudaFuncGetAttributes(&fa, kern);
        if (ge != cudaSuccess) return ge;
        if (fa.numRegs != kWideRegs) return cudaErrorInvalidConfiguration;
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemMax);
    });
    if (e != cudaSuccess) return e;
    const unsigned grid = (unsigned)(W::kCtas * std::min<int64_t>(tiles, sms / W::kCtas));
    return launch_overlapped(kern, grid, kWideThreads, W::smem(a.E), st, (unsigned)W::kCtas, a, tmx, tmw, tmy);
}

template <typename Y>
cudaError_t launch_fp8(const Fp8Args &a, const uint8_t *x, const uint8_t *w, int64_t K, int sms, cudaStream_t st) {
    if (a.offsets) {
        // A few rows: fp8_stream, which splits K (weights from HBM, 4 rows: 8 experts of 4096 x 14336
        // 38.2 us, fp8_wide 50.5; 64 of 1408 x 2048: 9.1 and 11.8; but 8 rows: 76.3 and 55.7, 10.5
        // and 12.4; 16 rows: 79.4 and 75.9, 16.9 and 13.9; 64 rows: 80.1 and 76.4, 27.7 and 26.0)
        if (a.R < 8) return launch_stream<16, Y>(a, x, w, K, sms, st);
    } else {
        // Few rows: fp8_stream where its tiles leave SMs to split K over (11008 x 4096, 16 rows:
        // 16.0 us, fp8_wide 18.5; 4096 x 11008, 128 rows: 26.0 and 33.9; but 4096 x 4096, 200
        // rows: 18.0 and 16.8), and up to 64 rows where its rounds are no longer than fp8_wide's
        // (28672 x 8192, two against one twice as wide: 51 and 45)
        const int64_t tiles = (a.R + 63) / 64 * a.nb;
        if (tiles * 2 <= sms ||
            (a.R <= 64 && (tiles + sms - 1) / sms < 2 * (((a.N + 255) / 256 + sms - 1) / sms))) {
            if (a.R <= 16) return launch_stream<16, Y>(a, x, w, K, sms, st);
            if (a.R <= 32) return launch_stream<32, Y>(a, x, w, K, sms, st);
            return launch_stream<64, Y>(a, x, w, K, sms, st);
        }
    }
    switch (wide_shape(a.offsets != nullptr, a.E, a.N, a.R, sms)) {
        case kWidePair: return launch_wide<true, 256, Y>(a, x, w, K, sms, st);
        case kWideNarrow: return launch_wide<false, 128, Y>(a, x, w, K, sms, st);
        default: return launch_wide<false, 256, Y>(a, x, w, K, sms, st);
    }
}

int device_sms() {
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms > 0 ? sms : 148;
}

q4_status fp8_product(const uint8_t *x, const float *xs, int64_t R, const int32_t *offsets, int64_t E, const uint8_t *w,
                      const float *ws, int64_t N, int64_t K, void *y, q4_dtype yt, uint32_t *status, void *stream) {
    if (yt != Q4_F32 && yt != Q4_BF16 && yt != Q4_F16) return Q4_ERR_ARG;
    if (R < 0 || N < 0 || K < 1 || E < 0) return Q4_ERR_ARG;
    // 32-bit row numbers; rows of codes are whole 16-byte units (TMA)
    if (R > (1 << 30) || N > (1 << 30) || K > (1 << 30) || E > kMaxExperts || K % 16 != 0) return Q4_ERR_UNSUPPORTED;
    if (E * N > INT32_MAX) return Q4_ERR_UNSUPPORTED;
    if (R == 0 || N == 0 || E == 0) return Q4_OK;
    if (!x || !xs || !w || !ws || !y) return Q4_ERR_ARG;
    if ((uintptr_t)x % 16 || (uintptr_t)w % 16) return Q4_ERR_UNSUPPORTED;
    Fp8Args a{xs, ws, offsets, y, status, N, (int32_t)R, (int32_t)E, (int32_t)((N + 127) / 128),
              (int32_t)((K + 127) / 128), 1, 0, 0, 0};
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int sms = device_sms();
    const cudaError_t e = yt == Q4_F32    ? launch_fp8<float>(a, x, w, K, sms, st)
                          : yt == Q4_BF16 ? launch_fp8<__nv_bfloat16>(a, x, w, K, sms, st)
                                          : launch_fp8<__half>(a, x, w, K, sms, st);
    return cuda_error(e, "fp8_gemm launch");
}

}  // namespace
}  // namespace q4

extern "C" {

q4_status q4_fp8_gemm(const uint8_t *x, const float *xs, int64_t M, const uint8_t *w, const float *ws, int64_t N,
                      int64_t K, void *y, q4_dtype yt, uint32_t *status_word, void *stream) {
    return q4::fp8_product(x, xs, M, nullptr, 1, w, ws, N, K, y, yt, status_word, stream);
}

q4_status q4_fp8_gemm_grouped(const uint8_t *x, const float *xs, int64_t R, const int32_t *offsets, int64_t E,
                              const uint8_t *w, const float *ws, int64_t N, int64_t K, void *y, q4_dtype yt,
                              uint32_t *status_word, void *stream) {
    if (!offsets && R > 0 && N > 0 && E > 0) return Q4_ERR_ARG;
    return q4::fp8_product(x, xs, R, offsets, E, w, ws, N, K, y, yt, status_word, stream);
}

}  // extern "C"
