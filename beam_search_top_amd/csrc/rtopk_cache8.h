// Internal interface between the host side (rtopk_layer.cpp) of the rotation
// and of the 8-bit cache's entry points and their kernels, and the arithmetic
// of the 8-bit format. The host and a plain C++ compiler read it too, so that
// tests run the arithmetic on the CPU. Not part of the ABI.
#pragma once

#include "rtopk_pages.h"

#include <string.h>

#if !defined(RTOPK_ARITHMETIC_ONLY)
#include <hip/hip_runtime_api.h>
#endif

namespace rtopk {

constexpr int kMaxRowDim = 256; // elements of a head in these kernels

// ---- the format: a row of D elements (one token, one head) is D e4m3 codes
// and one byte s; element d is code[d] * 2^(s - 127), with s held to [1, 254].
constexpr uint32_t kMinScale = 1, kMaxScale = 254;

// The byte of a row whose largest finite |x| has these float32 bits: the smallest
// power of two, at least 2^-126, under which no element exceeds 448, the
// largest code. (A power of two costs the codes nothing: they are floating point
// themselves, and elements keep their leading bits exactly. With it a code times its
// scale is a number of float16 or bfloat16 again, so that readers round nothing.)
RTOPK_HD uint32_t scale_of(uint32_t amax_bits)
{
    const int e = (int)(amax_bits >> 23) - 8 + ((amax_bits & 0x7fffffu) > 0x600000u); // of |x| = 1.m 2^(e - 127 + 8)
    return (uint32_t)(e < (int)kMinScale ? (int)kMinScale : e);                       // at most 247
}
RTOPK_HD uint32_t held_scale(uint32_t s) { return s < kMinScale ? kMinScale : s > kMaxScale ? kMaxScale : s; }
// float32 bits of 2^(s - 127) and of its reciprocal, s held
RTOPK_HD uint32_t scale_bits(uint32_t s) { return s << 23; }
RTOPK_HD uint32_t inverse_bits(uint32_t s) { return (254u - s) << 23; } // written scales are at most 247

// Elements beyond this are held to it: the largest code times scale below the type's
// largest number. The next one, 256 times the scale, would read as infinity.
RTOPK_HD float stored_limit(int dtype) { return dtype == 1 ? 61440.f : 0x1.ep127f; }

// Tokens per workgroup of the rotation, of `row` elements each: enough to fill its lanes
// a few times, and more where T tokens would take 2^24 workgroups of 256 threads. Their
// sines and cosines fit in LDS: at most 17 tokens (kMaxRopeTokens over 2^24 - 1, rounded up) of 128.
constexpr int64_t kMaxRopeTokens = (int64_t)1 << 28;
inline int rope_tokens(int64_t T, int64_t row)
{
    const int64_t most = (1 << 24) - 1, least = (T + most - 1) / most, per = row >= 4096 ? 1 : 4096 / row > 16 ? 16 : 4096 / row;
    return (int)(per > least ? per : least);
}

#if !defined(RTOPK_ARITHMETIC_ONLY)
// Norms and rotation of queries and keys (rtopk_rope.hip); strides (token, head) in elements.
struct RopeArgs {
    const void *q, *k;
    void *q_out, *k_out;
    int64_t qs[2], ks[2], qos[2], kos[2];
    const int32_t *positions; // [T], negative: the token is skipped
    const float *freqs;       // [rot / 2] radians per position
    const void *qw, *kw;      // [D] norm weights, or null: no norm
    float eps;
    int64_t T;
    int Hq, Hkv, D, rot, interleaved;
    PageDiv heads; // Hq + Hkv
    int tpw;       // tokens per workgroup
};
hipError_t launch_rope(RopeArgs a, int dtype, bool wide, hipStream_t s);

// Store to and load from the 8-bit cache (rtopk_cache8.hip).
struct Cache8Args {
    const void *k, *v;      // store: the tokens
    void *k_out, *v_out;    // load: where they go, [T][Hkv][D]
    uint8_t *kc, *vc;       // codes
    uint8_t *ksc, *vsc;     // [num_pages][page][Hkv] scales
    const int32_t *slots;   // [T]
    int64_t T, ks[2], vs[2]; // token, head
    int64_t cs[3];          // page, token, head
    int Hkv, D, nslots, tpw;
    PageDiv heads, page;
};
hipError_t launch_cache8_store(Cache8Args a, int dtype, bool wide, hipStream_t s);
hipError_t launch_cache8_load(Cache8Args a, int dtype, bool wide, hipStream_t s);
#endif

} // namespace rtopk
