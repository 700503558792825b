// What the kernels of the 8-bit key/value cache share: the cache's layout on the
// device, its codes and the fp16 matrix instruction.
#pragma once

#include <cuda_fp16.h>

#include "zb_common.cuh"
#include "zb_host.h"

namespace zb {
namespace kv8 {

constexpr int HD = 64;
constexpr int CHUNK = 64;            // keys a warp (or a CTA's step) works on at a time
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;
// Probabilities are 2^(x - max + P_SHIFT): fp16 then holds them to 2^-11 of their
// value down to 2^-28 of the largest and to 2^-39 of it below, so that even 2^20
// keys of negligible weight each add up to what they should.
constexpr float P_SHIFT = 14.f;

// What the attention kernels (kv8_attn.cu for few query rows a head, kv8_tile.cu for
// many) and those that join their partial results are given.
struct AttnArgs {
    zb_kv8 c;
    const uint16_t* Q;
    uint16_t* O;
    float* lse;
    const int32_t* lens;
    int rows, n_q, tiles;        // query rows a head (its group's heads x n_q), items a head
    int causal;
    float scale_log2;
    long long runs;              // partial results of CTAs; those of single warps follow
    int groups;                  // weight sums a head: runs of min(block, 64) keys, or 0
    // workspace
    float* part_o;               // [runs, then one a warp][tile][64]
    float2* part_ml;             // [...][tile]: running maximum (log2 units) and sum
    int2* item;                  // [heads * tiles]: first partial run, number of runs
    float* gsum;                 // [heads][groups][rows]: log2 of a row's sum over a group
    float* lse2;                 // [heads][rows]: log2 of a row's whole sum (many rows)
    int* status;
    unsigned long long timeout_ns;
};

// Tokens of head h, cut to what the cache can hold.
ZB_DEVINL long long head_len(const int32_t* lens, int h, long long cap) {
    const long long n = __ldg(lens + h);
    return n < 0 ? 0 : n > cap ? cap : n;
}

// Slot of logical block b of head h; an entry outside the cache reads slot 0 and
// is reported.
ZB_DEVINL int slot_of(const zb_kv8& c, int h, long long b, int* status) {
    int s = c.table[static_cast<long long>(h) * c.slots + b];
    if (s < 0 || s >= c.slots) {
        flag_status(status, ZB_ERR_INDEX);
        s = 0;
    }
    return s;
}

// --------------------------------------------------------------- codes ----
// A word of four codes as two fp16 pairs, exactly.  int8: the biased byte under
// the exponent of 1024 is 1024 + code + 128.
template <int FMT>
ZB_DEVINL void unpack4(uint32_t w, uint32_t& lo, uint32_t& hi);

ZB_DEVINL uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
    return r;
}
ZB_DEVINL uint32_t fma_f16x2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
ZB_DEVINL uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// 1 x - 1152: exact, and half the latency of a subtraction here.
ZB_DEVINL uint32_t sub_1152(uint32_t h2) { return fma_f16x2(h2, 0x3C003C00u, 0xE480E480u); }
template <>
ZB_DEVINL void unpack4<ZB_KV8_INT8>(uint32_t w, uint32_t& lo, uint32_t& hi) {
    w ^= 0x80808080u;
    lo = sub_1152(prmt(w, 0x64646464u, 0x4140u));
    hi = sub_1152(prmt(w, 0x64646464u, 0x4342u));
}
template <>
ZB_DEVINL void unpack4<ZB_KV8_E4M3>(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

// Int8 codes times a power of two (a pair of fp16) that leaves them, and 1152, exact.
ZB_DEVINL void unpack4_int8(uint32_t w, uint32_t mul, uint32_t& lo, uint32_t& hi) {
    w ^= 0x80808080u;
    const uint32_t off = mul_f16x2(mul, 0xE480E480u);        // -1152
    lo = fma_f16x2(prmt(w, 0x64646464u, 0x4140u), mul, off);
    hi = fma_f16x2(prmt(w, 0x64646464u, 0x4342u), mul, off);
}

ZB_DEVINL float2 half2_floats(uint32_t h2) { return __half22float2(*reinterpret_cast<const __half2*>(&h2)); }

// Two fp32 -> fp16 pair (round to nearest even), `lo` in bits 0..15.
ZB_DEVINL uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// p = 2^(x f + add) of N fp32 values (f, add in both halves), as fp16 pairs, and their
// sum in fp32.  The steps of four pairs at a time are written one stage apart and
// kept in that order (volatile): a warp then has eight exponentials under way.  Left
// to the compiler, which runs each pair's chain to its end, 64 of them take a warp
// alone 997 to 1,109 cycles; so, 637 (the MUFU's own rate: 512).
template <int N>
ZB_DEVINL float exp_pairs(const float* x, uint64_t f, uint64_t add, uint32_t* pk) {
    constexpr int P = N / 2, B = 4;
    uint64_t y[P], acc[B];
    float u[P], v[P];
#pragma unroll
    for (int i = 0; i < B; ++i) acc[i] = 0ull;
#pragma unroll
    for (int b = 0; b < P + 2 * B; b += B) {
#pragma unroll
        for (int i = 0; i < B; ++i) {
            const int e = b + i, g = e - B, h = g - B;
            if (e < P)
                asm volatile("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(y[e]) : "l"(f2_pack(x[2 * e], x[2 * e + 1])), "l"(f), "l"(add));
            if (g >= 0 && g < P) {
                float p0, p1;
                f2_unpack(y[g], p0, p1);
                asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(u[g]) : "f"(p0));
                asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(v[g]) : "f"(p1));
            }
            if (h >= 0 && h < P) {
                asm volatile("add.rn.f32x2 %0, %0, %1;" : "+l"(acc[i]) : "l"(f2_pack(u[h], v[h])));
                asm volatile("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(pk[h]) : "f"(v[h]), "f"(u[h]));
            }
        }
    }
    float s0, s1;
    f2_unpack(f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3])), s0, s1);
    return s0 + s1;
}

// D += A B on one warp: 16 x 8 x 16, fp16 in, fp32 sums.
ZB_DEVINL void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// D = A B.
ZB_DEVINL void mma_f16_new(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// Transpose of an 8 x 8 matrix of 16-bit values, a pair of a row in each lane.
ZB_DEVINL uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// ------------------------------------------------------------ host side ----
// kv8_tile.cu: attention of many rows and the join of its parts (pair: items of 256 rows, else 128).
zb_status launch_tiles(const AttnArgs& a, bool pair, int ctas, cudaStream_t st);

inline zb_status check_cache(const zb_kv8& c, bool codes) {
    if (c.heads < 1 || c.slots < 1) return ZB_ERR_SHAPE;
    if (c.head_dim != HD) return ZB_ERR_UNSUPPORTED;
    if (c.block != 16 && c.block != 32 && c.block != 64 && c.block != 128) return ZB_ERR_UNSUPPORTED;
    if (c.format != ZB_KV8_INT8 && c.format != ZB_KV8_E4M3) return ZB_ERR_UNSUPPORTED;
    if (c.heads > 65535) return ZB_ERR_UNSUPPORTED;
    if (static_cast<long long>(c.slots) * c.block > 0x7FFFFF00ll) return ZB_ERR_UNSUPPORTED;
    if (!codes) return ZB_OK;
    if (!c.k || !c.v || !c.k_scale || !c.v_scale || !c.table) return ZB_ERR_NULL;
    if (!aligned16(c.k) || !aligned16(c.v) || !aligned16(c.k_scale) || !aligned16(c.v_scale) || !aligned16(c.table) ||
        !aligned16(c.mass))
        return ZB_ERR_ALIGN;
    return ZB_OK;
}

}  // namespace kv8
}  // namespace zb
