// unaligned.cuh -- 16 bytes at a time at addresses of any alignment, for rows whose length is
// not a multiple of 16 bytes: two aligned loads and a shift instead of one access an element.
#pragma once

#include "common.cuh"

namespace q4 {

// Bytes sh .. sh + 15 of lo and hi side by side (0 <= sh <= 15).
Q4_DEVINL uint4 shift_bytes(const uint4 &lo, const uint4 &hi, uint32_t sh) {
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    uint32_t t[7], u[5];
#pragma unroll
    for (int i = 0; i < 7; ++i) t[i] = sh & 4 ? w[i + 1] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) u[i] = sh & 8 ? t[i + 2] : t[i];
    const uint32_t b = 8 * (sh & 3);
    return make_uint4(__funnelshift_r(u[0], u[1], b), __funnelshift_r(u[1], u[2], b), __funnelshift_r(u[2], u[3], b),
                      __funnelshift_r(u[3], u[4], b));
}

// The first n of 16 bytes, zeros behind.
Q4_DEVINL uint4 first_bytes(uint4 v, int n) {
    auto mask = [n](int at) { return n >= at + 4 ? 0xffffffffu : n <= at ? 0u : (1u << (8 * (n - at))) - 1u; };
    return make_uint4(v.x & mask(0), v.y & mask(4), v.z & mask(8), v.w & mask(12));
}

// n bytes from p (0 for none, 16 or more for 16), zeros behind. Reads the aligned 16-byte
// words that hold one of these bytes and no others, so it never leaves the memory's pages.
Q4_DEVINL uint4 load_any16(const void *p, int n) {
    uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
    const uint32_t sh = (uint32_t)(uintptr_t)p & 15;
    const uint4 *a = reinterpret_cast<const uint4 *>((uintptr_t)p - sh);
    if (n > 0) lo = *a;
    if ((int)sh + min(n, 16) > 16) hi = a[1];
    const uint4 v = shift_bytes(lo, hi, sh);
    return n < 16 ? first_bytes(v, n) : v;
}

// The first n bytes of v (16 or more: all) to p, which may be any address: aligned 4-byte words
// where there are 16, and bytes at their ends.
Q4_DEVINL void store_any16(void *p, const uint4 &v, int n) {
    char *c = static_cast<char *>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    const int head = (int)(-(uintptr_t)p & 3);  // bytes before the first aligned word
    if (n < 16) {
#pragma unroll
        for (int at = 0; at < 15; ++at)
            if (at < n) c[at] = (char)(w[at / 4] >> (8 * (at & 3)));
    } else if (((uintptr_t)p & 15) == 0) {
        *reinterpret_cast<uint4 *>(p) = v;
    } else if (head == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<uint32_t *>(c + 4 * i) = w[i];
    } else {
#pragma unroll
        for (int at = 0; at < 3; ++at)
            if (at < head) c[at] = (char)(w[0] >> (8 * at));
#pragma unroll
        for (int i = 0; i < 3; ++i)
            *reinterpret_cast<uint32_t *>(c + head + 4 * i) = __funnelshift_r(w[i], w[i + 1], 8 * head);
#pragma unroll
        for (int at = 13; at < 16; ++at)
            if (at >= head + 12) c[at] = (char)(w[3] >> (8 * (at & 3)));
    }
}

}  // namespace q4
