// fp8_plan.h -- how the launches of fp8_gemm.cu are laid out: host arithmetic alone, so that it can be
// checked without a GPU.
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

// The tiles of fp8_wide: rows of x by weight rows, and the CTAs that make one.
enum WideShape {
    kWideSingle,  // 128 x 256, one
    kWidePair,    // 256 x 256, two
    kWideNarrow   // 128 x 128, one
};

// The shape by the rounds that its tiles take, all SMs busy: a round of 128 x 256 by single CTAs, of
// 256 x 256 by pairs and of 128 x 128 takes times as 20 : 18 : 15, and pairs 4 more in all, which
// their clusters take to start and to meet. How the rows are spread over the experts is known on the
// device only: an expert has one tile where they fill less than half of one on average, else half a
// tile more than its rows fill.
// Measured, all three on each of 1341 products (bf16 y, weights beyond L2): 94 dense ones of 8 shapes
// (N 768 to 14336, K 2048 to 11008, 65 to 4096 rows), where the chosen one took 0.4 % more than the
// fastest on average and 6 % at most; 662 by 1 to 256 experts (7 shapes, 8 to 4096 rows an expert)
// that a router with preferences fills, 0.6 % on average, over 10 % in 11 of them; and 585 with rows
// spread evenly, 1.6 %, over 10 % in 36, where nearly all experts need the same number of tiles and
// half a tile more is too much or too little. (512 x 4096 x 4096: 19.3 us single, 19.6 pairs, 15.4
// narrow; 4096 x 14336 x 4096: 249, 243, 338; 8 experts of 14336 x 4096 with 512 rows each: 300, 334,
// 385, and with 4096: 2137, 1918, 2733.)
inline WideShape wide_shape(bool grouped, int64_t E, int64_t N, int64_t R, int sms) {
    auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    auto rounds = [&](int64_t rows, int64_t width, int64_t at_once) {
        const int64_t cols = up(N, width);
        if (!grouped || E == 1) return up(up(R, rows) * cols, at_once);
        if (2 * R < E * rows) return up(std::min(R, E) * cols, at_once);
        return up((2 * R + E * rows) * cols, 2 * rows * at_once);
    };
    const int64_t single = 20 * rounds(128, 256, sms), pair = 18 * rounds(256, 256, sms / 2) + 4,
                  narrow = 15 * rounds(128, 128, sms);
    return single <= pair && single <= narrow ? kWideSingle : pair <= narrow ? kWidePair : kWideNarrow;
}

}  // namespace q4
