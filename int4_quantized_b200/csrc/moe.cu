// moe.cu -- tokens sorted by expert and back, with weights applied, and the gradients.
//
// Slot s = t * k + j is choice j of token t. Sorting is a stable counting sort of the slots
// by expert: pos[s] is the slot's place, tokens[p] = t the token at place p, and expert e
// holds the places offsets[e] .. offsets[e + 1] - 1. A slot whose id is outside 0 .. E - 1
// has no place (pos = -1); the places behind the last expert's are empty (tokens = -1) and
// no call writes their rows.
//
//   moe_sort_kernel   one cluster of up to 8 CTAs: every warp counts a run of slots into a
//                     histogram of its own (__match_any groups equal ids, so one lane adds
//                     for all of them), the CTAs read each other's totals through
//                     distributed shared memory, and the warps walk their runs again and
//                     hand out the places in slot order. One launch, no workspace, no
//                     atomics: the result is the stable order, the same on every run.
//   moe_gather_kernel one warp copies up to 4 KB of a row.
//   moe_combine_kernel out[t] = sum over j of w[t, j] ys[pos[t, j]], in fp32, j ascending,
//                     rounded once; without weights it is the gradient of the gather.
//   moe_combine_bwd   one CTA a token: reads dout[t] once for all its slots, writes
//                     dys[pos] = w dout and dw = <dout, ys[pos]>.
// All but the sort are bound by the rows they read and write.
#include <cooperative_groups.h>

#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace q4 {

namespace {

namespace cg = cooperative_groups;

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortCtas = 8;
constexpr int64_t kMaxExperts = 1024;  // 32 warps x 1024 counters of 4 bytes: 128 KB of shared memory

template <typename T>
Q4_DEVINL int expert_of(const T *ids, int64_t s, int64_t end, int E) {
    if (s >= end) return -1;
    const T e = ids[s];
    return e >= 0 && e < (T)E ? (int)e : -1;
}

template <typename T>
__global__ void __launch_bounds__(kSortThreads) moe_sort_kernel(const T *__restrict__ ids, int64_t R, int k, int E,
                                                                int32_t *__restrict__ tokens,
                                                                int32_t *__restrict__ pos,
                                                                int32_t *__restrict__ offsets) {
    extern __shared__ int32_t sm[];
    int32_t *hist = sm;                      // [warps][E]: counts, then the next place of each (warp, expert)
    int32_t *tot = sm + kSortWarps * E;      // [E] this CTA's counts, read by the others
    int32_t *start = tot + E;                // [E + 1] the experts' first places
    cg::cluster_group cl = cg::this_cluster();
    const int C = (int)cl.num_blocks(), c = (int)cl.block_rank();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t below = (1u << lane) - 1;
    // runs of whole 32-slot chunks, one a warp
    const int64_t run = ((R + (int64_t)C * kSortWarps * 32 - 1) / ((int64_t)C * kSortWarps * 32)) * 32;
    const int64_t s0 = min(R, (int64_t)(c * kSortWarps + warp) * run), s1 = min(R, s0 + run);

    for (int i = threadIdx.x; i < kSortWarps * E; i += kSortThreads) hist[i] = 0;
    __syncthreads();
    int32_t *mine = hist + warp * E;
    {
        int next = expert_of(ids, s0 + lane, s1, E);
        for (int64_t s = s0; s < s1; s += 32) {
            const int e = next;
            next = expert_of(ids, s + 32 + lane, s1, E);
            const uint32_t same = __match_any_sync(0xffffffffu, e);
            if (e >= 0 && (same & below) == 0) mine[e] += __popc(same);
            __syncwarp();
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kSortThreads) {
        int32_t sum = 0;
        for (int w = 0; w < kSortWarps; ++w) {
            const int32_t n = hist[w * E + e];
            hist[w * E + e] = sum;
            sum += n;
        }
        tot[e] = sum;
    }
    cl.sync();
    // all CTAs' counts of each expert, and those of the CTAs before this one
    for (int e = threadIdx.x; e < E; e += kSortThreads) {
        int32_t before = 0, all = 0;
        for (int r = 0; r < C; ++r) {
            const int32_t n = cl.map_shared_rank(tot, r)[e];
            before += r < c ? n : 0;
            all += n;
        }
        start[e] = all;
        for (int w = 0; w < kSortWarps; ++w) hist[w * E + e] += before;
    }
    cl.sync();  // no CTA reads another's totals from here on
    if (warp == 0) {  // exclusive sums over the experts
        int32_t carry = 0;
        for (int b = 0; b < E; b += 32) {
            const int32_t n = b + lane < E ? start[b + lane] : 0;
            int32_t x = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int32_t y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            __syncwarp();
            if (b + lane < E) start[b + lane] = carry + x - n;
            carry += __shfl_sync(0xffffffffu, x, 31);
        }
        if (lane == 0) start[E] = carry;
    }
    __syncthreads();
    if (c == 0)
        for (int e = threadIdx.x; e <= E; e += kSortThreads) offsets[e] = start[e];
    {
        int next = expert_of(ids, s0 + lane, s1, E);
        for (int64_t s = s0; s < s1; s += 32) {
            const int e = next;
            next = expert_of(ids, s + 32 + lane, s1, E);
            const uint32_t same = __match_any_sync(0xffffffffu, e);
            const int32_t at = e >= 0 ? mine[e] : 0;
            __syncwarp();
            if (e >= 0 && (same & below) == 0) mine[e] = at + __popc(same);
            __syncwarp();
            if (s + lane < s1) {
                const int32_t p = e >= 0 ? start[e] + at + __popc(same & below) : -1;
                pos[s + lane] = p;
                if (e >= 0) tokens[p] = (int32_t)((uint32_t)(s + lane) / (uint32_t)k);
            }
        }
    }
    for (int64_t p = start[E] + (int64_t)c * kSortThreads + threadIdx.x; p < R; p += (int64_t)C * kSortThreads)
        tokens[p] = -1;
}

// ---- rows ---------------------------------------------------------------------------------
// VEC: 16 bytes an access; else one element of T.
template <typename T, bool VEC>
struct Row {
    using V = typename std::conditional<VEC, uint4, T>::type;
    static constexpr int N = VEC ? 16 / (int)sizeof(T) : 1;
};
template <typename T, bool VEC>
Q4_DEVINL void unpack(const typename Row<T, VEC>::V &r, float (&f)[Row<T, VEC>::N]) {
    constexpr int N = Row<T, VEC>::N;
    const T *e = reinterpret_cast<const T *>(&r);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if constexpr (std::is_same<T, float>::value) f[i] = e[i];
        else if constexpr (std::is_same<T, __half>::value) f[i] = __half2float(e[i]);
        else f[i] = __bfloat162float(e[i]);
    }
}
template <typename T, bool VEC>
Q4_DEVINL typename Row<T, VEC>::V pack(const float (&f)[Row<T, VEC>::N]) {
    constexpr int N = Row<T, VEC>::N;
    typename Row<T, VEC>::V r;
    T *e = reinterpret_cast<T *>(&r);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if constexpr (std::is_same<T, float>::value) e[i] = f[i];
        else if constexpr (std::is_same<T, __half>::value) e[i] = __float2half_rn(f[i]);
        else e[i] = __float2bfloat16_rn(f[i]);
    }
    return r;
}

constexpr int kGatherVecs = 8;  // accesses a lane: 4 KB a warp in 16-byte accesses

template <typename V>
__global__ void __launch_bounds__(256) moe_gather_kernel(const V *__restrict__ x, int64_t T,
                                                         const int32_t *__restrict__ tokens, int64_t R, int64_t per_row,
                                                         uint32_t chunks, V *__restrict__ xs) {
    const uint32_t unit = blockIdx.x * 8 + (threadIdx.x >> 5);
    const uint32_t p = unit / chunks, ch = unit - p * chunks;
    if (p >= R) return;
    const int64_t t = tokens[p];
    if (t < 0 || t >= T) return;
    const int64_t v0 = (int64_t)ch * (32 * kGatherVecs) + (threadIdx.x & 31);
    const V *src = x + t * per_row;
    V *dst = xs + (int64_t)p * per_row;
    V r[kGatherVecs];
#pragma unroll
    for (int i = 0; i < kGatherVecs; ++i)
        if (v0 + 32 * i < per_row) r[i] = src[v0 + 32 * i];
#pragma unroll
    for (int i = 0; i < kGatherVecs; ++i)
        if (v0 + 32 * i < per_row) dst[v0 + 32 * i] = r[i];
}

constexpr int kCombineSlots = 4;  // row loads in flight a lane

template <typename T, bool VEC>
__global__ void __launch_bounds__(256) moe_combine_kernel(const typename Row<T, VEC>::V *__restrict__ ys, int64_t R,
                                                          const int32_t *__restrict__ pos,
                                                          const float *__restrict__ weights, int64_t tokens, int k,
                                                          int64_t per_row, uint32_t chunks,
                                                          typename Row<T, VEC>::V *__restrict__ out) {
    using V = typename Row<T, VEC>::V;
    constexpr int N = Row<T, VEC>::N;
    const uint32_t unit = blockIdx.x * 8 + (threadIdx.x >> 5);
    const uint32_t t = unit / chunks, ch = unit - t * chunks;
    if (t >= tokens) return;
    const int64_t v = (int64_t)ch * 32 + (threadIdx.x & 31);
    if (v >= per_row) return;
    const int64_t s0 = (int64_t)t * k;
    float acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.f;
    for (int j0 = 0; j0 < k; j0 += kCombineSlots) {
        V r[kCombineSlots];
        float w[kCombineSlots];
        bool on[kCombineSlots];
#pragma unroll
        for (int j = 0; j < kCombineSlots; ++j) {
            const int32_t p = j0 + j < k ? pos[s0 + j0 + j] : -1;
            on[j] = p >= 0 && p < R;
            w[j] = on[j] && weights ? weights[s0 + j0 + j] : 1.f;
            if (on[j]) r[j] = ys[(int64_t)p * per_row + v];
        }
#pragma unroll
        for (int j = 0; j < kCombineSlots; ++j) {
            if (!on[j]) continue;
            float f[N];
            unpack<T, VEC>(r[j], f);
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] = fmaf(w[j], f[i], acc[i]);
        }
    }
    out[(int64_t)t * per_row + v] = pack<T, VEC>(acc);
}

constexpr int kBwdThreads = 128;
constexpr int kBwdSlots = 8;  // slots a pass over dout[t]

template <typename T, bool VEC>
__global__ void __launch_bounds__(kBwdThreads) moe_combine_bwd(const typename Row<T, VEC>::V *__restrict__ dout,
                                                               const typename Row<T, VEC>::V *__restrict__ ys,
                                                               int64_t R, const int32_t *__restrict__ pos,
                                                               const float *__restrict__ weights, int k,
                                                               int64_t per_row, typename Row<T, VEC>::V *__restrict__ dys,
                                                               float *__restrict__ dweights) {
    using V = typename Row<T, VEC>::V;
    constexpr int N = Row<T, VEC>::N;
    __shared__ float part[kBwdThreads / 32][kBwdSlots];
    const int64_t t = blockIdx.x, s0 = t * k;
    for (int j0 = 0; j0 < k; j0 += kBwdSlots) {
        int32_t p[kBwdSlots];
        float w[kBwdSlots], dot[kBwdSlots];
#pragma unroll
        for (int j = 0; j < kBwdSlots; ++j) {
            p[j] = j0 + j < k ? pos[s0 + j0 + j] : -1;
            if (p[j] >= R) p[j] = -1;
            w[j] = p[j] >= 0 ? weights[s0 + j0 + j] : 0.f;
            dot[j] = 0.f;
        }
        for (int64_t v = threadIdx.x; v < per_row; v += kBwdThreads) {
            V r[kBwdSlots];
#pragma unroll
            for (int j = 0; j < kBwdSlots; ++j)
                if (p[j] >= 0) r[j] = ys[(int64_t)p[j] * per_row + v];
            float g[N];
            unpack<T, VEC>(dout[t * per_row + v], g);
#pragma unroll
            for (int j = 0; j < kBwdSlots; ++j) {
                if (p[j] < 0) continue;
                float f[N], d[N];
                unpack<T, VEC>(r[j], f);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    dot[j] = fmaf(g[i], f[i], dot[j]);
                    d[i] = w[j] * g[i];
                }
                dys[(int64_t)p[j] * per_row + v] = pack<T, VEC>(d);
            }
        }
#pragma unroll
        for (int j = 0; j < kBwdSlots; ++j) {
#pragma unroll
            for (int o = 16; o; o >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
            if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5][j] = dot[j];
        }
        __syncthreads();
        if (threadIdx.x < kBwdSlots && j0 + (int)threadIdx.x < k) {
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < kBwdThreads / 32; ++i) sum += part[i][threadIdx.x];
            dweights[s0 + j0 + threadIdx.x] = sum;
        }
        __syncthreads();
    }
}

inline int elem_size(q4_dtype t) { return t == Q4_F32 ? 4 : 2; }
inline bool dtype_ok(q4_dtype t) { return t == Q4_F32 || t == Q4_BF16 || t == Q4_F16; }
inline bool aligned16(const void *p) { return (uintptr_t)p % 16 == 0; }

// Warps of a launch over rows x chunks, eight a CTA; 0 where the grid cannot hold them.
inline unsigned row_grid(int64_t rows, int64_t chunks) {
    if (chunks > INT32_MAX / (rows > 0 ? rows : 1)) return 0;
    return (unsigned)((rows * chunks + 7) / 8);
}

template <typename T>
cudaError_t sort_launch(const void *ids, int64_t R, int k, int E, int32_t *tokens, int32_t *pos, int32_t *offsets,
                        cudaStream_t st) {
    const size_t smem = ((size_t)kSortWarps * E + E + E + 1) * 4;
    cudaError_t e = cudaFuncSetAttribute(moe_sort_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    // up to two chunks a warp one CTA is done sooner than eight can meet
    const unsigned ctas = R <= 2 * 32 * kSortWarps ? 1 : kSortCtas;
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = ctas;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, moe_sort_kernel<T>, static_cast<const T *>(ids), R, k, E, tokens, pos, offsets);
}

template <typename T>
cudaError_t combine_launch(const void *ys, int64_t R, const int32_t *pos, const float *weights, int64_t tokens, int k,
                           int64_t D, void *out, cudaStream_t st, bool *fits) {
    const bool vec = (D * (int64_t)sizeof(T)) % 16 == 0 && aligned16(ys) && aligned16(out);
    const int64_t per_row = vec ? D * (int64_t)sizeof(T) / 16 : D, chunks = (per_row + 31) / 32;
    const unsigned grid = row_grid(tokens, chunks);
    *fits = grid != 0;
    if (!grid) return cudaSuccess;
    if (vec)
        moe_combine_kernel<T, true><<<grid, 256, 0, st>>>(static_cast<const uint4 *>(ys), R, pos, weights, tokens, k,
                                                          per_row, (uint32_t)chunks, static_cast<uint4 *>(out));
    else
        moe_combine_kernel<T, false><<<grid, 256, 0, st>>>(static_cast<const T *>(ys), R, pos, weights, tokens, k,
                                                           per_row, (uint32_t)chunks, static_cast<T *>(out));
    return cudaGetLastError();
}

template <typename T>
cudaError_t bwd_launch(const void *dout, const void *ys, int64_t R, const int32_t *pos, const float *weights,
                       int64_t tokens, int k, int64_t D, void *dys, float *dweights, cudaStream_t st) {
    const bool vec = (D * (int64_t)sizeof(T)) % 16 == 0 && aligned16(ys) && aligned16(dout) && aligned16(dys);
    if (vec)
        moe_combine_bwd<T, true><<<(unsigned)tokens, kBwdThreads, 0, st>>>(
            static_cast<const uint4 *>(dout), static_cast<const uint4 *>(ys), R, pos, weights, k,
            D * (int64_t)sizeof(T) / 16, static_cast<uint4 *>(dys), dweights);
    else
        moe_combine_bwd<T, false><<<(unsigned)tokens, kBwdThreads, 0, st>>>(
            static_cast<const T *>(dout), static_cast<const T *>(ys), R, pos, weights, k, D, static_cast<T *>(dys),
            dweights);
    return cudaGetLastError();
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
    const int64_t bytes = D * q4::elem_size(xt);
    const bool vec = bytes % 16 == 0 && q4::aligned16(x) && q4::aligned16(xs);
    const int64_t per_row = vec ? bytes / 16 : D, chunks = (per_row + 32 * q4::kGatherVecs - 1) / (32 * q4::kGatherVecs);
    const unsigned grid = q4::row_grid(R, chunks);
    if (!grid) return Q4_ERR_UNSUPPORTED;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (vec)
        q4::moe_gather_kernel<uint4><<<grid, 256, 0, st>>>(static_cast<const uint4 *>(x), T, tokens, R, per_row,
                                                           (uint32_t)chunks, static_cast<uint4 *>(xs));
    else if (xt == Q4_F32)
        q4::moe_gather_kernel<uint32_t><<<grid, 256, 0, st>>>(static_cast<const uint32_t *>(x), T, tokens, R, per_row,
                                                              (uint32_t)chunks, static_cast<uint32_t *>(xs));
    else
        q4::moe_gather_kernel<uint16_t><<<grid, 256, 0, st>>>(static_cast<const uint16_t *>(x), T, tokens, R, per_row,
                                                              (uint32_t)chunks, static_cast<uint16_t *>(xs));
    return q4::cuda_error(cudaGetLastError(), "moe_gather launch");
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
