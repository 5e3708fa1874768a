// moe.cu -- tokens sorted by expert and back, with weights applied, and the gradients.
//
// Slot s = t * k + j is choice j of token t. Sorting is a stable counting sort of the slots
// by expert: pos[s] is the slot's place, tokens[p] = t the token at place p, and expert e
// holds the places offsets[e] .. offsets[e + 1] - 1. A slot whose id is outside 0 .. E - 1
// has no place (pos = -1); the places behind the last expert's are empty (tokens = -1) and
// no call writes their rows.
//
//   moe_sort_kernel   one cluster of up to 8 CTAs: every warp counts a run of slots into a
//                     histogram of its own, the CTAs read each other's totals through
//                     distributed shared memory, and the warps walk their runs again and
//                     hand out the places in slot order (a lane's rank among equal ids of its
//                     32 slots comes from one vote a bit). One launch, no workspace, and only
//                     counts are added atomically: the result is the stable order on every run.
//   moe_gather_kernel one warp copies up to 2 KB of each of two rows, or several short rows.
//   moe_combine_kernel out[t] = sum over j of w[t, j] ys[pos[t, j]], in fp32, j ascending,
//                     rounded once; without weights it is the gradient of the gather.
//   moe_combine_bwd   four warps or one for each token: dout[t] is read once for all its
//                     slots, dys[pos] = w dout is written and dw = <dout, ys[pos]> summed.
// All but the sort are bound by the rows they read and write; each lane has up to 8 accesses
// of 16 bytes on their way.
// No pointer is __restrict__: inputs may come from a kernel that still runs when these start
// (launch_overlapped), so no load may be taken for invariant and moved over the wait.
#include <cooperative_groups.h>

#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "once.cuh"
#include "overlap.cuh"

namespace q4 {

namespace {

namespace cg = cooperative_groups;

constexpr int kSortWarps = 32;  // at most, in one CTA
constexpr int kSortCtas = 8;
constexpr int kSortBatch = 8;   // chunks of 32 ids a warp has on their way
constexpr int64_t kMaxExperts = 1024;  // 32 warps x 1024 counters of 4 bytes: 128 KB of shared memory

// The expert of each lane's slot in kSortBatch chunks from s on; -1 behind end and for ids
// outside 0 .. E - 1.
template <typename T>
Q4_DEVINL void load_ids(const T *ids, int64_t s, int64_t end, int E, int (&e)[kSortBatch]) {
    T raw[kSortBatch];
#pragma unroll
    for (int i = 0; i < kSortBatch; ++i) {
        const int64_t at = s + 32 * i + (threadIdx.x & 31);
        raw[i] = (T)-1;
        if (at < end) raw[i] = ids[at];
    }
#pragma unroll
    for (int i = 0; i < kSortBatch; ++i) e[i] = raw[i] >= 0 && raw[i] < (T)E ? (int)raw[i] : -1;
}

// The lanes whose e (0 .. 2^bits - 1) equals this lane's, by one vote a bit (__match_any_sync
// took about 90 cycles a warp and SM: 65536 ids of 256 experts 24 us).
Q4_DEVINL uint32_t same_lanes(int e, int bits) {
    uint32_t same = 0xffffffffu;
    for (int b = 0; b < bits; ++b) {
        const bool one = (e >> b) & 1;
        const uint32_t v = __ballot_sync(0xffffffffu, one);
        same &= one ? v : ~v;
    }
    return same;
}

template <typename T>
__global__ void __launch_bounds__(32 * kSortWarps) moe_sort_kernel(const T *ids, int64_t R, int k, int E,
                                                                   int32_t *tokens,
                                                                   int32_t *pos,
                                                                   int32_t *offsets) {
    begin_overlapped();
    extern __shared__ int32_t sm[];
    const int W = blockDim.x >> 5;
    int32_t *hist = sm;            // [W][E]: counts, then each warp's next place after the warps before it
    int32_t *tot = sm + W * E;     // [E] this CTA's counts, read by the others
    int32_t *base = tot + E;       // [E] the first place of this CTA's slots of each expert
    int32_t *all = base + E;       // [E + 1] counts, then the experts' first places
    cg::cluster_group cl = cg::this_cluster();
    const int C = (int)cl.num_blocks(), c = (int)cl.block_rank();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t below = (1u << lane) - 1;
    // runs of whole 32-slot chunks, one a warp
    const int64_t run = ((R + (int64_t)C * W * 32 - 1) / ((int64_t)C * W * 32)) * 32;
    const int64_t s0 = min(R, (int64_t)(c * W + warp) * run), s1 = min(R, s0 + run);

    int e[kSortBatch];
    load_ids(ids, s0, s1, E, e);
    for (int i = threadIdx.x; i < W * E; i += blockDim.x) hist[i] = 0;
    __syncthreads();
    int32_t *mine = hist + warp * E;
    for (int64_t s = s0; s < s1; s += 32 * kSortBatch) {
        if (s > s0) load_ids(ids, s, s1, E, e);
#pragma unroll
        for (int i = 0; i < kSortBatch; ++i) {
            if (e[i] >= 0) atomicAdd(&mine[e[i]], 1);  // a count: its order does not matter
        }
    }
    __syncthreads();
    for (int x = threadIdx.x; x < E; x += blockDim.x) {
        int32_t sum = 0;
#pragma unroll 8
        for (int w = 0; w < W; ++w) {
            const int32_t n = hist[w * E + x];
            hist[w * E + x] = sum;
            sum += n;
        }
        tot[x] = sum;
    }
    if (C > 1) cl.sync();
    else __syncthreads();
    // all CTAs' counts of each expert, and those of the CTAs before this one
    for (int x = threadIdx.x; x < E; x += blockDim.x) {
        int32_t before = 0, n = 0;
        if (C > 1) {
            int32_t r[kSortCtas];
#pragma unroll
            for (int i = 0; i < kSortCtas; ++i) r[i] = i < C ? cl.map_shared_rank(tot, i)[x] : 0;
#pragma unroll
            for (int i = 0; i < kSortCtas; ++i) {
                before += i < c ? r[i] : 0;
                n += r[i];
            }
        } else {
            n = tot[x];
        }
        base[x] = before;
        all[x] = n;
    }
    if (C > 1) cl.sync();  // no CTA reads another's totals from here on
    else __syncthreads();
    if (warp == 0) {  // exclusive sums over the experts
        int32_t carry = 0;
        for (int b = 0; b < E; b += 32) {
            const int32_t n = b + lane < E ? all[b + lane] : 0;
            int32_t x = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int32_t y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            if (b + lane < E) {
                all[b + lane] = carry + x - n;
                base[b + lane] += carry + x - n;
            }
            carry += __shfl_sync(0xffffffffu, x, 31);
        }
        if (lane == 0) all[E] = carry;
    }
    __syncthreads();
    if (c == 0)
        for (int x = threadIdx.x; x <= E; x += blockDim.x) offsets[x] = all[x];
    const int bits = 32 - __clz(E);  // ids 0 .. E - 1, and E for no expert
    const bool once = run <= 32 * kSortBatch;  // the ids are still in registers
    for (int64_t s = s0; s < s1; s += 32 * kSortBatch) {
        if (!once) load_ids(ids, s, s1, E, e);
#pragma unroll
        for (int i = 0; i < kSortBatch; ++i) {
            const int64_t slot = s + 32 * i + lane;
            if (s + 32 * i >= s1) break;
            const uint32_t same = same_lanes(e[i] >= 0 ? e[i] : E, bits);
            const int32_t at = e[i] >= 0 ? mine[e[i]] : 0;
            __syncwarp();
            if (e[i] >= 0 && (same & below) == 0) mine[e[i]] = at + __popc(same);
            __syncwarp();
            if (slot < s1) {
                const int32_t p = e[i] >= 0 ? base[e[i]] + at + __popc(same & below) : -1;
                pos[slot] = p;
                if (e[i] >= 0) tokens[p] = (int32_t)((uint32_t)slot / (uint32_t)k);
            }
        }
    }
    for (int64_t p = all[E] + (int64_t)c * blockDim.x + threadIdx.x; p < R; p += (int64_t)C * blockDim.x) tokens[p] = -1;
}

// ---- rows ---------------------------------------------------------------------------------
// Rows of T in accesses of B bytes: 16 where rows are whole such parts at 16-byte addresses,
// else 4 or an element. (Aligned 16-byte accesses shifted to unaligned rows took longer than
// single elements: 8192 tokens x 4 of 4097 bf16 values, combine 215 us and 131.)
template <typename T, int B>
struct Row {
    using V = typename std::conditional<B == 16, uint4, typename std::conditional<B == 4, uint32_t, uint16_t>::type>::type;
    static constexpr int N = B / (int)sizeof(T);
};
template <typename T, int B>
Q4_DEVINL void unpack(const typename Row<T, B>::V &r, float (&f)[Row<T, B>::N]) {
    const T *e = reinterpret_cast<const T *>(&r);
#pragma unroll
    for (int i = 0; i < Row<T, B>::N; ++i) {
        if constexpr (std::is_same<T, float>::value) f[i] = e[i];
        else if constexpr (std::is_same<T, __half>::value) f[i] = __half2float(e[i]);
        else f[i] = __bfloat162float(e[i]);
    }
}
template <typename T, int B>
Q4_DEVINL typename Row<T, B>::V pack(const float (&f)[Row<T, B>::N]) {
    typename Row<T, B>::V r;
    T *e = reinterpret_cast<T *>(&r);
#pragma unroll
    for (int i = 0; i < Row<T, B>::N; ++i) {
        if constexpr (std::is_same<T, float>::value) e[i] = f[i];
        else if constexpr (std::is_same<T, __half>::value) e[i] = __float2half_rn(f[i]);
        else e[i] = __float2bfloat16_rn(f[i]);
    }
    return r;
}

// Accesses a lane has on its way: the narrower, the more.
template <int B>
constexpr int kInFlight = B == 16 ? 8 : 16;
constexpr int kGatherInFlight = 8;  // (16 of an element: 8192 x 4 of 4097 bf16 values 182 us, 8: 114)

// Rows written once: they go first when L2 is full, so that x, which each expert reads again,
// stays (8192 tokens x 8 of 4096 bf16 values: 132 us without, 122 with, before the chunks'
// order; the writes alone take 74). Narrower accesses leave a sector to the next store, so theirs stay too.
template <typename V>
Q4_DEVINL void store_once(V *p, V v) {
    if constexpr (sizeof(V) == 16) __stcs(p, v);
    else *p = v;
}

// A warp copies P parts of 32 accesses from each of kInFlight / P rows.
template <typename V, int P>
__global__ void __launch_bounds__(256) moe_gather_kernel(const V *x, int64_t T,
                                                         const int32_t *tokens, int64_t R, int64_t per_row,
                                                         V *xs) {
    begin_overlapped();
    constexpr int ROWS = kGatherInFlight / P;
    const uint32_t unit = blockIdx.x * 8 + (threadIdx.x >> 5);
    // all rows' first chunk, then all rows' second: what the experts read again of x in that time is
    // one chunk of its rows, which L2 holds (8192 tokens x 8 of 4096 bf16 values, 67 MB of x: row
    // after row 121 us, chunks of 4 KB 107, of 2 KB 96)
    const uint32_t groups = (uint32_t)((R + ROWS - 1) / ROWS);
    const uint32_t ch = unit / groups, g = unit - ch * groups;
    const int64_t v0 = (int64_t)ch * (32 * P) + (threadIdx.x & 31);
    int64_t t[ROWS];
    V r[ROWS][P];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int64_t p = (int64_t)g * ROWS + i;
        t[i] = p < R ? (int64_t)tokens[p] : -1;
        if (t[i] >= T) t[i] = -1;
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
#pragma unroll
        for (int j = 0; j < P; ++j)
            if (t[i] >= 0 && v0 + 32 * j < per_row) r[i][j] = x[t[i] * per_row + v0 + 32 * j];
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
#pragma unroll
        for (int j = 0; j < P; ++j)
            if (t[i] >= 0 && v0 + 32 * j < per_row)
                store_once(xs + ((int64_t)g * ROWS + i) * per_row + v0 + 32 * j, r[i][j]);
}

// A warp sums P parts of 32 accesses of a row, S slots at a time.
template <typename T, int B, int S, int P>
__global__ void __launch_bounds__(256) moe_combine_kernel(const typename Row<T, B>::V *ys, int64_t R,
                                                          const int32_t *pos,
                                                          const float *weights, int64_t tokens, int k,
                                                          int64_t per_row, uint32_t chunks,
                                                          typename Row<T, B>::V *out) {
    using V = typename Row<T, B>::V;
    constexpr int N = Row<T, B>::N;
    begin_overlapped();
    const uint32_t unit = blockIdx.x * 8 + (threadIdx.x >> 5);
    const uint32_t t = unit / chunks, ch = unit - t * chunks;
    if (t >= tokens) return;
    const int64_t v0 = (int64_t)ch * (32 * P) + (threadIdx.x & 31);
    const int64_t s0 = (int64_t)t * k;
    float acc[P][N];
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
        for (int n = 0; n < N; ++n) acc[i][n] = 0.f;
    for (int j0 = 0; j0 < k; j0 += S) {
        V r[S][P];
        float w[S];
        bool on[S];
#pragma unroll
        for (int j = 0; j < S; ++j) {
            const int32_t p = j0 + j < k ? pos[s0 + j0 + j] : -1;
            on[j] = p >= 0 && p < R;
            w[j] = on[j] && weights ? weights[s0 + j0 + j] : 1.f;
#pragma unroll
            for (int i = 0; i < P; ++i)
                if (on[j] && v0 + 32 * i < per_row) r[j][i] = ys[(int64_t)p * per_row + v0 + 32 * i];
        }
#pragma unroll
        for (int j = 0; j < S; ++j) {
            if (!on[j]) continue;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                float f[N];
                unpack<T, B>(r[j][i], f);
#pragma unroll
                for (int n = 0; n < N; ++n) acc[i][n] = fmaf(w[j], f[n], acc[i][n]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < P; ++i)
        if (v0 + 32 * i < per_row) out[(int64_t)t * per_row + v0 + 32 * i] = pack<T, B>(acc[i]);
}

// W warps take one token, S slots at a time and P accesses of each; 4 / W tokens a CTA.
template <typename T, int B, int W, int S, int P>
__global__ void __launch_bounds__(128) moe_combine_bwd(const typename Row<T, B>::V *dout,
                                                       const typename Row<T, B>::V *ys, int64_t R,
                                                       const int32_t *pos,
                                                       const float *weights, int64_t tokens, int k,
                                                       int64_t per_row, typename Row<T, B>::V *dys,
                                                       float *dweights) {
    using V = typename Row<T, B>::V;
    constexpr int N = Row<T, B>::N;
    begin_overlapped();
    __shared__ float part[4][S];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * (4 / W) + warp / W, s0 = t * k;
    const int at = W > 1 ? (int)threadIdx.x : lane;  // the lane's place among the token's
    const bool live = t < tokens;  // the same for all of a token's warps
    for (int j0 = 0; j0 < k; j0 += S) {
        int32_t p[S];
        float w[S], dot[S];
#pragma unroll
        for (int j = 0; j < S; ++j) {
            p[j] = live && j0 + j < k ? pos[s0 + j0 + j] : -1;
            if (p[j] >= R) p[j] = -1;
            w[j] = p[j] >= 0 ? weights[s0 + j0 + j] : 0.f;
            dot[j] = 0.f;
        }
        for (int64_t v0 = at; live && v0 < per_row; v0 += 32 * W * P) {
            V r[S][P], g0[P];
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int64_t v = v0 + 32 * W * i;
                if (v < per_row) {
                    g0[i] = dout[t * per_row + v];
#pragma unroll
                    for (int j = 0; j < S; ++j)
                        if (p[j] >= 0) r[j][i] = ys[(int64_t)p[j] * per_row + v];
                }
            }
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int64_t v = v0 + 32 * W * i;
                if (v >= per_row) break;
                float g[N];
                unpack<T, B>(g0[i], g);
#pragma unroll
                for (int j = 0; j < S; ++j) {
                    if (p[j] < 0) continue;
                    float f[N], d[N];
                    unpack<T, B>(r[j][i], f);
#pragma unroll
                    for (int n = 0; n < N; ++n) {
                        dot[j] = fmaf(g[n], f[n], dot[j]);
                        d[n] = w[j] * g[n];
                    }
                    dys[(int64_t)p[j] * per_row + v] = pack<T, B>(d);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < S; ++j) {
#pragma unroll
            for (int o = 16; o; o >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
            if (lane == 0) part[warp][j] = dot[j];
        }
        if (W > 1) __syncthreads();
        else __syncwarp();
        if (at < S && j0 + at < k && live) {
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < W; ++i) sum += part[W > 1 ? i : warp][at];
            dweights[s0 + j0 + at] = sum;
        }
        if (W > 1) __syncthreads();
        else __syncwarp();
    }
}

inline bool dtype_ok(q4_dtype t) { return t == Q4_F32 || t == Q4_BF16 || t == Q4_F16; }

// Warps of a launch over rows x chunks, eight a CTA; 0 where the grid cannot hold them.
inline unsigned row_grid(int64_t rows, int64_t chunks) {
    if (chunks > INT32_MAX / (rows > 0 ? rows : 1)) return 0;
    return (unsigned)((rows * chunks + 7) / 8);
}

// Each warp's histogram, and the three arrays of the block (one with a place more).
constexpr size_t sort_smem(int64_t warps, int64_t E) { return (size_t)(warps * E + 3 * E + 1) * 4; }

template <typename T>
cudaError_t sort_launch(const void *ids, int64_t R, int k, int E, int32_t *tokens, int32_t *pos, int32_t *offsets,
                        cudaStream_t st) {
    // one CTA while its warps have two chunks of 32 slots or fewer: eight take longer to meet
    const unsigned ctas = R <= 2 * 32 * kSortWarps ? 1 : kSortCtas;
    // and no more warps than chunks: every warp's histogram costs its clearing and its sum
    const int64_t chunks = (R + 31) / 32;
    const int warps = chunks >= kSortWarps ? kSortWarps : chunks < 4 ? 4 : (int)chunks;
    const size_t smem = sort_smem(warps, E);
    auto kern = moe_sort_kernel<T>;
    static std::atomic<uint64_t> ready{0};
    const cudaError_t e = once_per_device(ready, [&]() {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)sort_smem(kSortWarps, kMaxExperts));
    });
    if (e != cudaSuccess) return e;
    return launch_overlapped(kern, ctas, 32 * warps, smem, st, ctas, static_cast<const T *>(ids), R, k, E, tokens, pos,
                             offsets);
}

// Parts of 32 accesses that a warp takes of a row of per_row accesses: at most `most`, a power of 2.
inline int row_parts(int64_t per_row, int most) {
    int p = 1;
    while (p < most && 32 * (int64_t)p < per_row) p *= 2;
    return p;
}

// Bytes of an access to rows of D elements of `size` bytes at these addresses.
inline int access_bytes(int64_t D, int size, const void *a, const void *b, const void *c = nullptr) {
    const uintptr_t all = (uintptr_t)a | (uintptr_t)b | (uintptr_t)c | (uintptr_t)(D * size);
    return all % 16 == 0 ? 16 : all % 4 == 0 ? 4 : size;
}

template <typename V>
cudaError_t gather_launch(const void *x, int64_t T, const int32_t *tokens, int64_t R, int64_t bytes, void *xs,
                          cudaStream_t st, bool *fits) {
    constexpr int F = kGatherInFlight;
    const int64_t per_row = bytes / (int64_t)sizeof(V);
    const int P = row_parts(per_row, F / 2);
    const int64_t chunks = (per_row + 32 * P - 1) / (32 * P), groups = (R + F / P - 1) / (F / P);
    const unsigned grid = row_grid(groups, chunks);
    *fits = grid != 0;
    if (!grid) return cudaSuccess;
#define Q4_GATHER(P_)                                                                                             \
    return launch_overlapped(moe_gather_kernel<V, P_>, grid, 256, 0, st, 1, static_cast<const V *>(x), T, tokens, R, \
                             per_row, static_cast<V *>(xs))
    if (P == 1) Q4_GATHER(1);
    else if (P == 2) Q4_GATHER(2);
    else Q4_GATHER(4);
#undef Q4_GATHER
}

template <typename T, int B>
cudaError_t combine_rows(const void *ys, int64_t R, const int32_t *pos, const float *weights, int64_t tokens, int k,
                         int64_t D, void *out, cudaStream_t st, bool *fits) {
    using V = typename Row<T, B>::V;
    constexpr int M = kInFlight<B> / 8;
    const int64_t per_row = D / Row<T, B>::N;
    // slots times parts of a row: as many accesses on their way where the row is long enough
    const int P = row_parts(per_row, M * (k == 1 ? 8 : k == 2 ? 4 : 2));
    const int64_t chunks = (per_row + 32 * P - 1) / (32 * P);
    const unsigned grid = row_grid(tokens, chunks);
    *fits = grid != 0;
    if (!grid) return cudaSuccess;
#define Q4_COMBINE(S_, P_)                                                                                       \
    return launch_overlapped(moe_combine_kernel<T, B, S_, P_>, grid, 256, 0, st, 1, static_cast<const V *>(ys), R, \
                             pos, weights, tokens, k, per_row, (uint32_t)chunks, static_cast<V *>(out))
    if (P == 16) Q4_COMBINE(1, 16);
    else if (P == 8 && k == 1) Q4_COMBINE(1, 8);
    else if (P == 8) Q4_COMBINE(2, 8);
    else if (P == 4 && k <= 2) Q4_COMBINE(2, 4);
    else if (P == 4) Q4_COMBINE(4, 4);
    else if (P == 2) Q4_COMBINE(4, 2);
    else Q4_COMBINE(8, 1);
#undef Q4_COMBINE
}

template <typename T>
cudaError_t combine_launch(const void *ys, int64_t R, const int32_t *pos, const float *weights, int64_t tokens, int k,
                           int64_t D, void *out, cudaStream_t st, bool *fits) {
    const int B = access_bytes(D, sizeof(T), ys, out);
    if (B == 16) return combine_rows<T, 16>(ys, R, pos, weights, tokens, k, D, out, st, fits);
    if (B == 4) return combine_rows<T, 4>(ys, R, pos, weights, tokens, k, D, out, st, fits);
    return combine_rows<T, sizeof(T)>(ys, R, pos, weights, tokens, k, D, out, st, fits);
}

template <typename T, int B>
cudaError_t bwd_rows(const void *dout, const void *ys, int64_t R, const int32_t *pos, const float *weights,
                     int64_t tokens, int k, int64_t D, void *dys, float *dweights, cudaStream_t st) {
    using V = typename Row<T, B>::V;
    const int64_t per_row = D / Row<T, B>::N;
#define Q4_BWD(W_, S_, P_)                                                                                            \
    return launch_overlapped(moe_combine_bwd<T, B, W_, S_, P_>, (unsigned)((tokens + 4 / W_ - 1) / (4 / W_)), 128, 0,  \
                             st, 1, static_cast<const V *>(dout), static_cast<const V *>(ys), R, pos, weights, tokens, \
                             k, per_row, static_cast<V *>(dys), dweights)
    // rows below 128 accesses leave three of four warps idle: one warp a token there
    // (65536 tokens x 8 of 256 bf16 values: 290 us with four, 129 with one)
    constexpr int M = B == 16 ? 1 : 4;
    if (per_row >= 128) {
        if (k <= 2) Q4_BWD(4, 2, 4 * M);
        else Q4_BWD(4, 8, M);
    } else {
        if (k <= 2) Q4_BWD(1, 2, 2);
        else Q4_BWD(1, 8, 1);
    }
#undef Q4_BWD
}

template <typename T>
cudaError_t bwd_launch(const void *dout, const void *ys, int64_t R, const int32_t *pos, const float *weights,
                       int64_t tokens, int k, int64_t D, void *dys, float *dweights, cudaStream_t st) {
    const int B = access_bytes(D, sizeof(T), dout, ys, dys);
    if (B == 16) return bwd_rows<T, 16>(dout, ys, R, pos, weights, tokens, k, D, dys, dweights, st);
    if (B == 4) return bwd_rows<T, 4>(dout, ys, R, pos, weights, tokens, k, D, dys, dweights, st);
    return bwd_rows<T, sizeof(T)>(dout, ys, R, pos, weights, tokens, k, D, dys, dweights, st);
}

// Shapes that every call below shares: slots and rows in 32 bits.
q4_status check_rows(int64_t tokens, int64_t k, int64_t D, int64_t R) {
    if (tokens < 0 || k < 1 || D < 1 || R < 0) return Q4_ERR_ARG;
    if (k > INT32_MAX || D > ((int64_t)1 << 30) || R > INT32_MAX || tokens > INT32_MAX / k) return Q4_ERR_UNSUPPORTED;
    return Q4_OK;
}

}  // namespace
}  // namespace q4

extern "C" {

q4_status q4_moe_sort(const void *ids, int ids_bits, int64_t T, int64_t k, int64_t E, int32_t *tokens, int32_t *pos,
                      int32_t *offsets, void *stream) {
    if (ids_bits != 32 && ids_bits != 64) return Q4_ERR_ARG;
    if (E < 1) return Q4_ERR_ARG;
    const q4_status s = q4::check_rows(T, k, 1, 0);
    if (s != Q4_OK) return s;
    if (E > q4::kMaxExperts) return Q4_ERR_UNSUPPORTED;
    if (!offsets || (T > 0 && (!ids || !tokens || !pos))) return Q4_ERR_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = ids_bits == 32
                              ? q4::sort_launch<int32_t>(ids, T * k, (int)k, (int)E, tokens, pos, offsets, st)
                              : q4::sort_launch<int64_t>(ids, T * k, (int)k, (int)E, tokens, pos, offsets, st);
    return q4::cuda_error(e, "moe_sort launch");
}

q4_status q4_moe_gather(const void *x, q4_dtype xt, int64_t T, int64_t D, const int32_t *tokens, int64_t R, void *xs,
                        void *stream) {
    if (!q4::dtype_ok(xt)) return Q4_ERR_ARG;
    const q4_status s = q4::check_rows(T, 1, D, R);
    if (s != Q4_OK) return s;
    if (R == 0 || T == 0) return Q4_OK;
    if (!x || !tokens || !xs) return Q4_ERR_ARG;
    const int size = xt == Q4_F32 ? 4 : 2, B = q4::access_bytes(D, size, x, xs);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    bool fits = true;
    const cudaError_t e = B == 16  ? q4::gather_launch<uint4>(x, T, tokens, R, D * size, xs, st, &fits)
                          : B == 4 ? q4::gather_launch<uint32_t>(x, T, tokens, R, D * size, xs, st, &fits)
                                   : q4::gather_launch<uint16_t>(x, T, tokens, R, D * size, xs, st, &fits);
    if (!fits) return Q4_ERR_UNSUPPORTED;
    return q4::cuda_error(e, "moe_gather launch");
}

q4_status q4_moe_combine(const void *ys, q4_dtype yt, int64_t R, int64_t D, const int32_t *pos, const float *weights,
                         int64_t T, int64_t k, void *out, void *stream) {
    if (!q4::dtype_ok(yt)) return Q4_ERR_ARG;
    const q4_status s = q4::check_rows(T, k, D, R);
    if (s != Q4_OK) return s;
    if (T == 0) return Q4_OK;
    if (!pos || !out || (R > 0 && !ys)) return Q4_ERR_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    bool fits = true;
    const cudaError_t e =
        yt == Q4_F32    ? q4::combine_launch<float>(ys, R, pos, weights, T, (int)k, D, out, st, &fits)
        : yt == Q4_BF16 ? q4::combine_launch<__nv_bfloat16>(ys, R, pos, weights, T, (int)k, D, out, st, &fits)
                        : q4::combine_launch<__half>(ys, R, pos, weights, T, (int)k, D, out, st, &fits);
    if (!fits) return Q4_ERR_UNSUPPORTED;
    return q4::cuda_error(e, "moe_combine launch");
}

q4_status q4_moe_combine_backward(const void *dout, const void *ys, q4_dtype yt, int64_t R, int64_t D,
                                  const int32_t *pos, const float *weights, int64_t T, int64_t k, void *dys,
                                  float *dweights, void *stream) {
    if (!q4::dtype_ok(yt)) return Q4_ERR_ARG;
    const q4_status s = q4::check_rows(T, k, D, R);
    if (s != Q4_OK) return s;
    if (T == 0) return Q4_OK;
    if (!dout || !pos || !weights || !dweights || (R > 0 && (!ys || !dys))) return Q4_ERR_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e =
        yt == Q4_F32    ? q4::bwd_launch<float>(dout, ys, R, pos, weights, T, (int)k, D, dys, dweights, st)
        : yt == Q4_BF16 ? q4::bwd_launch<__nv_bfloat16>(dout, ys, R, pos, weights, T, (int)k, D, dys, dweights, st)
                        : q4::bwd_launch<__half>(dout, ys, R, pos, weights, T, (int)k, D, dys, dweights, st);
    return q4::cuda_error(e, "moe_combine_backward launch");
}

}  // extern "C"
