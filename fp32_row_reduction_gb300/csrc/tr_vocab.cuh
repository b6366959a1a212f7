// Device pieces that the embedding and the linear cross entropy share.
#pragma once

#include "tr_block.cuh"

namespace tr {

// [from, to) set to zero by a warp: 16-byte stores between the ragged ends, which are whole elements of two bytes.
__device__ __forceinline__ void zero_bytes(char* from, char* to) {
    const int lane = threadIdx.x & 31;
    char* body = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(from) + 15) & ~static_cast<uintptr_t>(15));
    if (body > to) body = to;
    char* end = body + (to - body) / 16 * 16;
    for (char* p = from + 2 * lane; p < body; p += 64) *reinterpret_cast<uint16_t*>(p) = 0;
    for (char* p = body + 16 * lane; p < end; p += 512) *reinterpret_cast<uint4*>(p) = make_uint4(0, 0, 0, 0);
    for (char* p = end + 2 * lane; p < to; p += 64) *reinterpret_cast<uint16_t*>(p) = 0;
}

// The 16 bytes that begin `shift` bytes (even) into two neighbouring 16-byte words.
__device__ __forceinline__ uint4 shifted(const uint4& lo, const uint4& hi, int shift) {
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    const int bits = (shift & 2) * 8, words = shift >> 2;
    uint32_t s[8];
    // words moved by two, then by one, then the half word
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = words & 2 ? (i < 6 ? w[i + 2] : 0) : w[i];
#pragma unroll
    for (int i = 0; i < 7; ++i) s[i] = words & 1 ? s[i + 1] : s[i];
    return make_uint4(__funnelshift_r(s[0], s[1], bits), __funnelshift_r(s[1], s[2], bits), __funnelshift_r(s[2], s[3], bits),
                      __funnelshift_r(s[3], s[4], bits));
}

}  // namespace tr
