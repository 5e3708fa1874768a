// fp8_pack.cu -- e4m3 codes with one fp32 scale per block of 128, the format that the
// block-scaled product of fp8_gemm.cu reads.
//
// The rule is qpack's with another code: per block, scale = fl32(max|v| / 448), 0 -> 1;
// code = e4m3(fl32(v / scale)), to nearest, ties to even, at most 448 in magnitude. A block
// is 128 consecutive values of a row (activations), or 128 rows x 128 columns (weights);
// blocks at the right and lower edges hold what is left.
//
//   fp8_pack_rows   8 lanes take one block, 16 values each: one pass over x, the block's
//                   maximum by three shuffles, one 16-byte store of codes a lane. Source rows
//                   may be given by index (tokens sorted by expert on the way), and the
//                   values may be silu(gate) * up of rows that hold gate and up side by side.
//   fp8_pack_tiles  one CTA takes one 128 x 128 block, which stays in registers between the
//                   maximum and the codes.
// Both are bound by HBM: every value is read once and every code written once.
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "overlap.cuh"
#include "unaligned.cuh"

namespace q4 {

namespace {

constexpr float kE4m3Max = 448.f;
constexpr uint32_t kInf = 0x7f800000u;


// 16 bytes of T as fp32 values (NEG: negated).
template <typename T, bool NEG>
Q4_DEVINL void unpack16(const uint4 &r, float *v) {
    constexpr uint32_t sign = !NEG ? 0u : sizeof(T) == 4 ? 0x80000000u : 0x80008000u;
    const uint32_t w[4] = {r.x ^ sign, r.y ^ sign, r.z ^ sign, r.w ^ sign};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
            v[i] = __uint_as_float(w[i]);
        } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
}

// 32 bytes (a whole sector) in one load. Volatile and not .nc: it stays behind the wait for the
// kernel before (launch_overlapped), and so do the plain loads, whose pointers are not
// __restrict__.
Q4_DEVINL void ld_v8(const void *p, uint4 &a, uint4 &b) {
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
        : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
        : "l"(p));
}

// N consecutive values of a row, of which `left` (which may be negative) are inside it; zeros
// behind. The loads and their conversion are apart, so that a thread has all of its loads on
// their way before it waits for the first. NEG gives the values negated.
// VEC: a row's values are whole chunks of N at 32-byte addresses (16-byte ones for a chunk of
// 16 bytes); else rows begin anywhere and end anywhere.
template <typename T, int N, bool VEC>
struct Chunk {
    static constexpr int PER = 16 / (int)sizeof(T), WORDS = N / PER;
    uint4 raw[WORDS];
    Q4_DEVINL void load(const T *p, int left) {
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < WORDS; ++i) raw[i] = make_uint4(0, 0, 0, 0);
            if (left > 0) {
#pragma unroll
                for (int i = 0; i < WORDS; i += 2) ld_v8(p + i * PER, raw[i], raw[i + 1]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < WORDS; ++i)
                raw[i] = load_any16(p + i * PER, max(0, min(left - i * PER, PER)) * (int)sizeof(T));
        }
    }
    template <bool NEG>
    Q4_DEVINL void values(float (&v)[N]) const {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) unpack16<T, NEG>(raw[i], v + i * PER);
    }
};

// max(m, |a|, |b|) for m >= 0, NaN if any is: a block's NaN or Inf stays visible in its maximum.
Q4_DEVINL float abs_max(float m, float a, float b) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(a), "f"(b));
    return r;
}
Q4_DEVINL uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Two fp32 values in one 64-bit register, and arithmetic on both in one instruction.
Q4_DEVINL uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
Q4_DEVINL float2 halves(uint64_t p) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
    return r;
}
Q4_DEVINL uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
Q4_DEVINL uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// fl32(v / s) by the reciprocal and two residual corrections (P. Markstein, "IA-64 and
// Elementary Functions", 2000: with y = RN(1/s) and a quotient within one ulp, one more
// correction by the exact residual gives the correctly rounded quotient; the first
// correction brings RN(v y), up to two ulps off, within one). The residuals are exact while
// they stay above the subnormal range: s >= 2^-90, and quotients below 2^-11, where they
// might not, give the code 0 in any case. Other scales take the division itself.
// The values come negated (nv = -v, nr = -1/s): q = nv nr, and the residual q s - v is then
// one fma, and v = -0 keeps its sign.
Q4_DEVINL uint64_t quotients(uint64_t nv, uint64_t s, uint64_t nr) {
    const uint64_t q0 = mul2(nv, nr);
    const uint64_t q1 = fma2(fma2(q0, s, nv), nr, q0);
    return fma2(fma2(q1, s, nv), nr, q1);
}

struct BlockDiv {
    float s, nr;  // the scale; -1/s, or 0 where the division itself is taken
};
// The scale of a block whose largest magnitude is a: fl32(a / 448), by the same corrections
// with 1/448 where they are exact; 0 becomes 1.
Q4_DEVINL BlockDiv block_div(float a) {
    BlockDiv d;
    if (a >= 0x1p-80f && a < 0x1p127f) {
        constexpr float y = 1.f / kE4m3Max;  // rounded to nearest by the compiler
        const float q0 = a * y;
        const float q1 = __fmaf_rn(-__fmaf_rn(q0, kE4m3Max, -a), y, q0);
        d.s = __fmaf_rn(-__fmaf_rn(q1, kE4m3Max, -a), y, q1);
    } else {
        d.s = __fdiv_rn(a, kE4m3Max);
        if (d.s == 0.f) d.s = 1.f;
    }
    d.nr = d.s >= 0x1p-90f && d.s <= 0x1p120f ? -__frcp_rn(d.s) : 0.f;
    return d;
}
Q4_DEVINL uint32_t e4m3x4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}

// The codes of N values given negated. EXACT: of the correctly rounded quotients; else of the
// products with the reciprocal, within two units of them, for values that are no more exact
// themselves (silu, 8192 x 14336: 100 us with the corrections, 96 without).
template <int N, bool EXACT>
Q4_DEVINL void codes_of(const float (&nv)[N], const BlockDiv &d, uint32_t (&c)[N / 4]) {
    float q[N];
    if (d.nr != 0.f) {
        const uint64_t s = pair(d.s, d.s), nr = pair(d.nr, d.nr);
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const uint64_t v = pair(nv[i], nv[i + 1]);
            const float2 f = halves(EXACT ? quotients(v, s, nr) : mul2(v, nr));
            q[i] = f.x, q[i + 1] = f.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) q[i] = __fdiv_rn(-nv[i], d.s);
    }
#pragma unroll
    for (int i = 0; i < N / 4; ++i) c[i] = e4m3x4(q[4 * i], q[4 * i + 1], q[4 * i + 2], q[4 * i + 3]);
}

// silu(g) u = g u / (1 + 2^(-g log2 e)) for two values of which neither gate is below kFarGate, in
// fp32 with the hardware's exponential and reciprocal, negated where u is given negated.
// Error: t = g log2 e is off by at most |t| 2^-23 in all (its rounding and the constant's), so
// 2^-t by |g| 2^-23 relative, to which the exponential, the sum, the reciprocal and the two
// products add at most 8 x 2^-23. Of 12 million fp32 values 12 and 11 codes (two seeds) differ from
// those of 64 bits, as with fp32 exp and division (12 and 10); of fp16 values 9 and 9 (8 and 14).
// Correcting t and the reciprocal changed that by nothing and cost 17 us of 118 at 8192 x 14336.
Q4_DEVINL uint64_t silu_mul2(uint64_t g, uint64_t u) {
    constexpr float L = 1.4426950408889634f;
    const float2 t = halves(mul2(g, pair(-L, -L)));
    float2 e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(1.f + e.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(1.f + e.y));
    return mul2(mul2(g, pair(r.x, r.y)), u);
}

// Below this gate the sum above nears 2^126, from where on its reciprocal is flushed to 0 (and from
// 2^128 on the sum is infinite), however large u makes the value.
constexpr float kFarGate = -87.f;
// silu(g) u for g < kFarGate. There 1 / (1 + e^-g) is e^g to 2^-125: two factors of e^(g/2), on
// either side of u, stay inside fp32's range wherever the value does: for gates down to -182 (then
// even the largest u gives less than 2^-126) e^(g/2) is at least 2^-132, a subnormal number of 18
// bits, which the two factors' 2^-18 each leave within the bound at such gates, (10 + 1.2 |g|) 2^-23.
Q4_DEVINL float silu_mul_far(float g, float u) {
    constexpr float L = 1.4426950408889634f;
    float h;
    asm("ex2.approx.f32 %0, %1;" : "=f"(h) : "f"(0.5f * (g * L)));
    return g * h * u * h;
}
// the least of three, NaN aside
Q4_DEVINL float min3(float a, float b, float c) {
    float r;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// One value, of rows of any alignment byte by byte.
template <typename T, bool VEC>
Q4_DEVINL float load_one(const T *p) {
    if constexpr (VEC) {
        return (float)*p;
    } else {
        uint32_t v = 0;
#pragma unroll
        for (int i = 0; i < (int)sizeof(T); ++i) v |= (uint32_t)reinterpret_cast<const uint8_t *>(p)[i] << (8 * i);
        float f[16 / sizeof(T)];
        unpack16<T, false>(make_uint4(v, 0, 0, 0), f);
        return f[0];
    }
}

struct RowsArgs {
    const void *x;
    const int32_t *rows;   // source row of each output row, or null
    const int32_t *count;  // device count of output rows, or null
    uint8_t *codes;
    float *scales;
    uint32_t *status;
    int64_t x_rows, K, ldx;
    uint32_t units, kb;  // blocks in all, blocks a row
};

// CTAs an SM. Left to itself the compiler takes the registers of three, and bf16 at 8192 x 14336 with
// silu takes 102 us where five (48 registers, two-block groups spill 30 to 70 bytes) take 94, rows 76
// and 67; fp32 rows 103 and 96. fp32 with silu, whose loads alone are 64 registers in two blocks,
// spills 260 to 580 bytes at five: 282 us, with three (80 registers, 28 bytes at the most) 152.
template <typename T, bool SILU, int U>
constexpr int kRowsCtas = SILU && sizeof(T) == 4 && U == 2 ? 3 : 5;
template <typename T, bool SILU, bool VEC, int U>
__global__ void __launch_bounds__(256, (kRowsCtas<T, SILU, U>)) fp8_pack_rows(const RowsArgs a) {
    begin_overlapped();
    const int sub = threadIdx.x & 7;
    const uint32_t first = blockIdx.x * (32 * U) + (threadIdx.x >> 3);
    const uint32_t live = a.count ? (uint32_t)max(*a.count, 0) : UINT32_MAX;
    Chunk<T, 16, VEC> x[U], up[SILU ? U : 1];
    int left[U];
    uint32_t row[U], blk[U];
    bool on[U];
    row[0] = first / a.kb;
    blk[0] = first - row[0] * a.kb;
#pragma unroll
    for (int j = 0; j < U; ++j) {
        if (j > 0) {  // 32 blocks on, over as many rows as that is
            row[j] = row[j - 1];
            blk[j] = blk[j - 1] + 32;
            if (blk[j] >= a.kb) {
                row[j] += blk[j] / a.kb;
                blk[j] %= a.kb;
            }
        }
        on[j] = first + 32 * j < a.units && row[j] < live;
        left[j] = on[j] ? (int)a.K - (int)blk[j] * 128 - 16 * sub : 0;
    }
    int64_t src[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
        src[j] = row[j];
        if (a.rows && on[j]) {
            src[j] = a.rows[row[j]];
            if (src[j] < 0 || src[j] >= a.x_rows) on[j] = false, left[j] = 0, src[j] = 0;
        }
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
        const T *p = static_cast<const T *>(a.x) + src[j] * a.ldx + (blk[j] * 128 + 16 * sub);
        x[j].load(p, left[j]);
        if constexpr (SILU) up[j].load(p + a.K, left[j]);
    }
    float nv[U][16];
    uint32_t m[U];
    bool far[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
        if constexpr (SILU) {
            float g[16], u[16];
            x[j].template values<false>(g);
            up[j].template values<true>(u);
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                const float2 f = halves(silu_mul2(pair(g[i], g[i + 1]), pair(u[i], u[i + 1])));
                nv[j][i] = f.x, nv[j][i + 1] = f.y;
            }
            float least = 0.f;
#pragma unroll
            for (int i = 0; i < 16; i += 2) least = min3(least, g[i], g[i + 1]);
            far[j] = least < kFarGate;
        } else {
            x[j].template values<true>(nv[j]);
        }
    }
    if constexpr (SILU) {  // rare: those values again, read again (kept, they would cost the registers)
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if (!far[j]) continue;
            const int64_t s = a.rows ? a.rows[row[j]] : row[j];
            const T *p = static_cast<const T *>(a.x) + s * a.ldx + (blk[j] * 128 + 16 * sub);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float g = i < left[j] ? load_one<T, VEC>(p + i) : 0.f;
                if (g < kFarGate) nv[j][i] = silu_mul_far(g, -load_one<T, VEC>(p + i + a.K));
            }
        }
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
        float big = 0.f;
#pragma unroll
        for (int i = 0; i < 16; i += 2) big = abs_max(big, nv[j][i], nv[j][i + 1]);
        m[j] = abs_bits(big);
    }
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
        for (int o = 4; o; o >>= 1) m[j] = max(m[j], __shfl_xor_sync(0xffffffffu, m[j], o));
    // the scale and its reciprocal cost about as much as a lane's sixteen quotients: lane j of
    // the eight works them out for block j
    uint32_t mine = m[0];
#pragma unroll
    for (int j = 1; j < U; ++j)
        if (sub == j) mine = m[j];
    const BlockDiv own = block_div(__uint_as_float(mine));
#pragma unroll
    for (int j = 0; j < U; ++j) {
        BlockDiv d;
        d.s = __shfl_sync(0xffffffffu, own.s, j, 8);
        d.nr = __shfl_sync(0xffffffffu, own.nr, j, 8);
        if (!on[j]) continue;
        uint32_t c[4];
        codes_of<16, !SILU>(nv[j], d, c);
        uint8_t *p = a.codes + (int64_t)row[j] * a.K + (blk[j] * 128 + 16 * sub);
        if constexpr (VEC) {
            if (left[j] > 0) *reinterpret_cast<uint4 *>(p) = make_uint4(c[0], c[1], c[2], c[3]);
        } else {
            store_any16(p, make_uint4(c[0], c[1], c[2], c[3]), left[j]);
        }
        if (sub == j) {
            a.scales[(int64_t)row[j] * a.kb + blk[j]] = d.s;
            if (m[j] >= kInf && a.status) atomicOr(a.status, Q4_STATUS_NONFINITE);
        }
    }
}

// One 128 x 128 block of [.., N, K] weights a CTA. PER values (32 bytes) a lane and load; a
// row's 128 columns are 128 / PER lanes wide, so 512 threads pass over the block in 32 / PER
// steps and keep 32 values each: two CTAs an SM then have 128 KB of fp32 on their way (with 256 threads
// of 64 values one CTA filled the registers and nothing covered its loads).
constexpr int kTileThreads = 512;
template <typename T, bool VEC>
__global__ void __launch_bounds__(kTileThreads, 2) fp8_pack_tiles(const T *w, int64_t N, int64_t K, uint32_t nb,
                                                      uint32_t kb, uint8_t *codes,
                                                      float *scales, uint32_t *status) {
    constexpr int PER = 32 / sizeof(T), LANES = 128 / PER, ROWS = kTileThreads / LANES, STEPS = 128 / ROWS;
    begin_overlapped();
    const uint32_t t = blockIdx.x / kb, kblk = blockIdx.x - t * kb;  // t: (matrix, row block)
    const uint32_t e = t / nb, nblk = t - e * nb;
    const int64_t k0 = (int64_t)kblk * 128 + (threadIdx.x % LANES) * PER;
    const int64_t n0 = (int64_t)nblk * 128 + threadIdx.x / LANES;
    const T *src = w + (int64_t)e * N * K;
    Chunk<T, PER, VEC> raw[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const int64_t n = n0 + i * ROWS;
        raw[i].load(src + (n < N ? n * K + k0 : 0), n < N ? (int)(K - k0) : 0);
    }
    float big = 0.f;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        float v[PER];
        raw[i].template values<false>(v);
#pragma unroll
        for (int j = 0; j < PER; j += 2) big = abs_max(big, v[j], v[j + 1]);
    }
    uint32_t m = __reduce_max_sync(0xffffffffu, abs_bits(big));
    __shared__ uint32_t part[kTileThreads / 32];
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kTileThreads / 32; ++i) m = max(m, part[i]);
    const BlockDiv d = block_div(__uint_as_float(m));
    uint8_t *dst = codes + (int64_t)e * N * K;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const int64_t n = n0 + i * ROWS;
        if (n >= N) continue;
        float nv[PER];
        raw[i].template values<true>(nv);
        uint32_t c[PER / 4];
        codes_of<PER, true>(nv, d, c);
        uint8_t *p = dst + n * K + k0;
        uint4 out = make_uint4(c[0], c[1], 0, 0);
        if constexpr (PER == 16) out.z = c[2], out.w = c[3];
        if constexpr (VEC) {
            if (k0 < K) {
                if constexpr (PER == 16) *reinterpret_cast<uint4 *>(p) = out;
                else *reinterpret_cast<uint2 *>(p) = make_uint2(out.x, out.y);
            }
        } else {
            const int left = (int)min(K - k0, (int64_t)PER);
            if constexpr (PER == 16) {
                store_any16(p, out, left);
            } else {
#pragma unroll
                for (int j = 0; j < PER; ++j)
                    if (j < left) p[j] = (uint8_t)(c[j / 4] >> (8 * (j & 3)));
            }
        }
    }
    if (threadIdx.x == 0) {
        scales[blockIdx.x] = d.s;
        if (m >= kInf && status) atomicOr(status, Q4_STATUS_NONFINITE);
    }
}

template <typename T>
cudaError_t pack_rows(const RowsArgs &a, bool silu, cudaStream_t st) {
    // whole chunks of 16 values a row: 32-byte loads of x and 16-byte stores of codes
    const bool vec = a.K % 16 == 0 && (uintptr_t)a.x % 32 == 0 && (uintptr_t)a.codes % 16 == 0;
    // two blocks a group of lanes keep the loads in flight that HBM needs; with fewer blocks
    // than fill the machine so, one each (16 x 4096: 16 CTAs instead of 8)
    const bool two = a.units >= 148 * 32 * 2 * 2;
    const unsigned grid = (a.units + (two ? 63 : 31)) / (two ? 64 : 32);
#define Q4_ROWS(S, V, U) return launch_overlapped(fp8_pack_rows<T, S, V, U>, grid, 256, 0, st, 1, a)
    if (two) {
        if (silu) {
            if (vec) Q4_ROWS(true, true, 2);
            Q4_ROWS(true, false, 2);
        }
        if (vec) Q4_ROWS(false, true, 2);
        Q4_ROWS(false, false, 2);
    }
    if (silu) {
        if (vec) Q4_ROWS(true, true, 1);
        Q4_ROWS(true, false, 1);
    }
    if (vec) Q4_ROWS(false, true, 1);
    Q4_ROWS(false, false, 1);
#undef Q4_ROWS
}

template <typename T>
cudaError_t pack_tiles(const void *w, int64_t E, int64_t N, int64_t K, uint8_t *codes, float *scales, uint32_t *status,
                       cudaStream_t st) {
    const bool vec = (K * (int64_t)sizeof(T)) % 32 == 0 && (uintptr_t)w % 32 == 0 && (uintptr_t)codes % 16 == 0;
    const uint32_t nb = (uint32_t)((N + 127) / 128), kb = (uint32_t)((K + 127) / 128);
    const unsigned grid = (unsigned)(E * nb * kb);
    auto kern = vec ? fp8_pack_tiles<T, true> : fp8_pack_tiles<T, false>;
    return launch_overlapped(kern, grid, kTileThreads, 0, st, 1, static_cast<const T *>(w), N, K, nb, kb, codes, scales,
                             status);
}

// Blocks of a call, at most 2^31 - 1 (such codes alone would be 275 GB).
bool blocks_ok(int64_t rows, int64_t cols_blocks, int64_t *units) {
    if (rows > 0 && cols_blocks > INT32_MAX / rows) return false;
    *units = rows * cols_blocks;
    return true;
}

}  // namespace
}  // namespace q4

extern "C" {

q4_status q4_fp8_pack(const void *x, q4_dtype xt, int64_t x_rows, int64_t K, const int32_t *rows, int64_t R,
                      const int32_t *count, uint32_t flags, uint8_t *codes, float *scales, uint32_t *status_word,
                      void *stream) {
    if (xt != Q4_F32 && xt != Q4_BF16 && xt != Q4_F16) return Q4_ERR_ARG;
    if (flags & ~(uint32_t)Q4_FP8_PACK_SILU_MUL) return Q4_ERR_ARG;
    if (x_rows < 0 || R < 0 || K < 1) return Q4_ERR_ARG;
    if (!rows && R != x_rows) return Q4_ERR_ARG;
    if (K > ((int64_t)1 << 30)) return Q4_ERR_UNSUPPORTED;
    int64_t units;
    if (!q4::blocks_ok(R, (K + 127) / 128, &units)) return Q4_ERR_UNSUPPORTED;
    if (units == 0 || x_rows == 0) return Q4_OK;
    if (!x || !codes || !scales) return Q4_ERR_ARG;
    const bool silu = (flags & Q4_FP8_PACK_SILU_MUL) != 0;
    q4::RowsArgs a{x, rows, count, codes, scales, status_word, x_rows, K, silu ? 2 * K : K, (uint32_t)units,
                   (uint32_t)((K + 127) / 128)};
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = xt == Q4_F32    ? q4::pack_rows<float>(a, silu, st)
                          : xt == Q4_BF16 ? q4::pack_rows<__nv_bfloat16>(a, silu, st)
                                          : q4::pack_rows<__half>(a, silu, st);
    return q4::cuda_error(e, "fp8_pack launch");
}

q4_status q4_fp8_pack_weights(const void *w, q4_dtype wt, int64_t E, int64_t N, int64_t K, uint8_t *codes,
                              float *scales, uint32_t *status_word, void *stream) {
    if (wt != Q4_F32 && wt != Q4_BF16 && wt != Q4_F16) return Q4_ERR_ARG;
    if (E < 0 || N < 0 || K < 1) return Q4_ERR_ARG;
    if (N > ((int64_t)1 << 30) || K > ((int64_t)1 << 30)) return Q4_ERR_UNSUPPORTED;
    int64_t tiles, all;
    if (!q4::blocks_ok((N + 127) / 128, (K + 127) / 128, &tiles) || !q4::blocks_ok(E, tiles, &all))
        return Q4_ERR_UNSUPPORTED;
    if (all == 0) return Q4_OK;
    if (!w || !codes || !scales) return Q4_ERR_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = wt == Q4_F32    ? q4::pack_tiles<float>(w, E, N, K, codes, scales, status_word, st)
                          : wt == Q4_BF16 ? q4::pack_tiles<__nv_bfloat16>(w, E, N, K, codes, scales, status_word, st)
                                          : q4::pack_tiles<__half>(w, E, N, K, codes, scales, status_word, st);
    return q4::cuda_error(e, "fp8_pack_weights launch");
}

}  // extern "C"
