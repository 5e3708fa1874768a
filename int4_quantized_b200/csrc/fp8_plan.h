// fp8_plan.h -- how a launch of fp8_stream (fp8_gemm.cu) is laid out: host arithmetic alone, so that it
// can be checked without a GPU.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

namespace q4 {

constexpr size_t kSmemMax = 227 * 1024;  // of a block; an SM has 1 KB more, and keeps 1 KB a block
constexpr int kStreamBufs = 8;           // tensor-memory buffers of NT columns: 128, 256 or 512 in all

// Shared memory of a block: the ring (128 weight rows and nt rows of x, 128 k each), the exchange
// buffer of the split sums, scales, barriers, the experts' tiles.
inline size_t stream_smem(int nt, int stages, int split, int64_t E) {
    return 1024 + (size_t)stages * (128 + nt) * 128 + (split > 1 ? (size_t)128 * nt * 4 : 0) +
           (size_t)kStreamBufs * nt * 4 + (2 * (size_t)stages + 3 * kStreamBufs + 2) * 8 + 16 + (size_t)(2 * E + 2) * 4;
}

struct StreamPlan {
    int split;   // CTAs of a cluster that share one tile's K
    int stages;  // ring depth
    size_t smem;
};

// For `tiles` tiles of kb blocks of k on `sms` SMs.
inline StreamPlan stream_plan(int nt, int64_t tiles, int kb, int64_t E, int sms) {
    StreamPlan p;
    // K is split over a cluster while the CTAs still fit on the machine at once, every CTA
    // keeps two blocks of k or more, and each takes whole columns of the joined sums
    p.split = 1;
    while (p.split < 8 && tiles * p.split * 2 <= sms && kb >= p.split * 4) p.split *= 2;
    const int most = (int)((kSmemMax - stream_smem(nt, 0, p.split, E)) / ((size_t)(128 + nt) * 128 + 16));
    const int64_t blocks = (int64_t)((kb + p.split - 1) / p.split) * ((tiles + sms - 1) / sms);
    p.stages = (int)std::max<int64_t>(2, std::min<int64_t>(std::min(most, 16), blocks));
    p.smem = stream_smem(nt, p.stages, p.split, E);
    // CTAs of a cluster wait for one another with their tensor memory (512 columns an SM) held: two
    // kernels that could not both have theirs must not meet on an SM, or each could hold what the
    // other's cluster waits for. Shared memory keeps them apart: blocks of 256 and 512 columns have
    // over half, so that beside one of 256 only two of 128 fit; a cluster's block of 512 leaves no
    // room for the smallest of 128; and of 128 no more than four fit at all.
    if (nt > 16) p.smem = std::max(p.smem, kSmemMax / 2 + 1024);
    if (nt == 64 && p.split > 1) p.smem = std::max(p.smem, kSmemMax - stream_smem(16, 2, 2, 1));
    return p;
}

}  // namespace q4
