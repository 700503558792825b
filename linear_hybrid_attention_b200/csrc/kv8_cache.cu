// The 8-bit key/value cache: append, read back, evict.
//
// A head's cache is a list of blocks of B tokens (16 to 128).  Codes of a block
// share one scale for its keys and one for its values,
//   s = max|x| / M  (M = 127 for int8, 448 for e4m3; fp32, rounded to nearest),
//   code = the nearest to x / s (of two as near, the even one),
// and a block holding a value that is not finite gets s = NaN and reads as NaN.
// The block in progress keeps its original bf16 rows beside the codes (`tail`)
// and is quantised again whenever rows join it, so what the cache holds does not
// depend on how tokens were split over calls.  A table maps logical blocks to
// slots; eviction only reorders it: kept blocks move up, freed slots go behind
// them for later appends, and no code is touched.
//
// Rounding is decided exactly.  x / s in fp32 may land on a tie that the exact
// quotient misses by less than its rounding; where the quotient is that near a
// tie (one value in some thousands), the sign of the fused x - (k + 1/2) s,
// which no rounding can change, decides.
#include <cuda_runtime.h>

#include "kv8.cuh"

namespace zb {
namespace kv8 {

constexpr int UNIT = 128;      // rows an append CTA takes: a multiple of every block size
constexpr int A_THREADS = 256;

// ---------------------------------------------------------- quantisation ----
// Whole number nearest to x / s, ties to even; inv ~ 1 / s.
ZB_DEVINL float exact_round(float x, float s, float t) {
    const float k = floorf(t);
    const float r = fmaf(-(k + 0.5f), s, x);
    const bool odd = (static_cast<int>(k) & 1) != 0;
    return k + ((r > 0.f || (r == 0.f && odd)) ? 1.f : 0.f);
}

// From here on 1 / s is a number, half a step of any code (2^-10 s at least) is a normal one,
// and so the sign that exact_round looks at is right.
constexpr float TINY_SCALE = 0x1p-110f;

// Eight codes of x for a scale of at least TINY_SCALE.  Adding 1.5 * 2^23 rounds a
// quotient to a whole number (ties to even) whose low byte is the code: half the
// price of a conversion.  A value within 2^-13 of a tie sends the eight through
// exact_round.
ZB_DEVINL uint2 codes_int8(const float* x, float s, float inv) {
    uint32_t u[8];
    float far = 0.f;
    const uint64_t inv2 = f2_pack(inv, inv), big2 = f2_pack(12582912.f, 12582912.f);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const uint64_t t = f2_mul(f2_pack(x[i], x[i + 1]), inv2), m = f2_add(t, big2);
        float a, b, ma, mb;
        f2_unpack(f2_sub(t, f2_sub(m, big2)), a, b);
        f2_unpack(m, ma, mb);
        far = fmax3(far, fabsf(a), fabsf(b));
        u[i] = __float_as_uint(ma);
        u[i + 1] = __float_as_uint(mb);
    }
    if (far > 0.5f - 0x1p-13f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = __float_as_uint(exact_round(x[i], s, x[i] * inv) + 12582912.f);
    }
    return make_uint2(prmt(prmt(u[0], u[1], 0x0040u), prmt(u[2], u[3], 0x0040u), 0x5410u),
                      prmt(prmt(u[4], u[5], 0x0040u), prmt(u[6], u[7], 0x0040u), 0x5410u));
}

ZB_DEVINL uint32_t pack_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// The value of the e4m3 code nearest to x / s, t its quotient in fp32.
ZB_DEVINL float value_e4m3(float x, float s, float t) {
    int e = static_cast<int>((__float_as_uint(t) >> 23) & 255u) - 127;
    if (e < -6) e = -6;
    const float step = __uint_as_float(static_cast<uint32_t>(e - 3 + 127) << 23);
    const float q = exact_round(fabsf(x), s * step, fabsf(t) / step);
    return copysignf(fminf(q * step, 448.f), t);
}

// The conversion instruction rounds t correctly, and t is the quotient to some
// steps of fp32: only a value that near a tie between two codes (the 20 bits below
// the code's mantissa), or below the normal codes, needs the exact form.
ZB_DEVINL uint2 codes_e4m3(const float* x, float s, float inv) {
    float t[8];
    bool hard = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        t[i] = x[i] * inv;
        const uint32_t b = __float_as_uint(t[i]) & 0x7FFFFFFFu;
        hard |= ((b + 0x100u) & 0xFFFFFu) - 0x80000u <= 0x200u;
        hard |= b - 1u < 0x3C800000u - 1u;
    }
    if (hard) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (t[i] != 0.f) t[i] = value_e4m3(x[i], s, t[i]);
    }
    return make_uint2(pack_e4m3x2(t[0], t[1]) | pack_e4m3x2(t[2], t[3]) << 16,
                      pack_e4m3x2(t[4], t[5]) | pack_e4m3x2(t[6], t[7]) << 16);
}

template <int FMT>
ZB_DEVINL uint2 codes8(const float* x, float s, float inv) {
    if (s >= TINY_SCALE) return FMT == ZB_KV8_INT8 ? codes_int8(x, s, inv) : codes_e4m3(x, s, inv);
    // A tiny scale: both numbers times 2^64, which is exact.  A subnormal one may be rounded so far
    // that quotients pass the format's largest value: held to it.
    const float big = s * 0x1p64f;
    uint32_t w[2] = {0u, 0u};
    for (int i = 0; i < 8; ++i) {
        const float y = x[i] * 0x1p64f, t = y / big;
        uint32_t c;
        if (FMT == ZB_KV8_INT8)
            c = static_cast<uint32_t>(static_cast<int>(fminf(fmaxf(exact_round(y, big, t), -127.f), 127.f))) & 0xFFu;
        else
            c = pack_e4m3x2(t != 0.f ? value_e4m3(y, big, t) : t, 0.f) & 0xFFu;
        w[i >> 2] |= c << (8 * (i & 3));
    }
    return make_uint2(w[0], w[1]);
}

struct AppendArgs {
    zb_kv8 c;
    const uint4 *K, *V;
    int n;
    const int32_t* lens;
    int32_t* lens_out;   // NULL: written by a launch of its own
    int* status;
};

// One CTA: 128 rows from a block boundary on, of one head, keys and values.  An
// HBM stream (256 B a token in, 128 B out): each thread has its eight 16-byte
// loads in flight, a warp takes 16 rows, so a block is a whole number of warps.
template <int FMT>
__global__ void __launch_bounds__(A_THREADS, 4) append_kernel(const AppendArgs a) {
    const int h = blockIdx.y, unit = blockIdx.x;
    const zb_kv8& c = a.c;
    const int B = c.block, shift = 31 - __clz(B);   // B is a power of two
    const long long cap = static_cast<long long>(c.slots) * B;
    const long long len = __ldca(a.lens + h);       // (lens_out may be lens)
    if (len < 0 || len + a.n > cap) {          // does not fit: the head stays as it is
        if (unit == 0 && threadIdx.x == 0) {
            flag_status(a.status, ZB_ERR_INDEX);
            if (a.lens_out) a.lens_out[h] = static_cast<int32_t>(len);
        }
        return;
    }
    const int held = static_cast<int>(len) & (B - 1);
    const long long first = len >> shift;           // logical block that row 0 belongs to
    const long long rows = held + static_cast<long long>(a.n);
    const int warp = warp_id(), lane = lane_id();
    const long long blocks = (rows + B - 1) >> shift;
    const long long row0 = static_cast<long long>(unit) * UNIT + warp * 16;
    const long long blk = row0 >> shift;            // of this warp
    const bool live = blk < blocks;
    uint4* tail[2] = {reinterpret_cast<uint4*>(c.k_tail) + static_cast<long long>(h) * B * 8,
                      reinterpret_cast<uint4*>(c.v_tail) + static_cast<long long>(h) * B * 8};
    const uint4* src[2] = {a.K + static_cast<long long>(h) * a.n * 8, a.V + static_cast<long long>(h) * a.n * 8};
    // the warp's 16 rows: those before `old` come from the tail, those before `all` exist
    const int old = static_cast<int>(min(max(held - row0, 0ll), 16ll));
    const int all = static_cast<int>(min(max(rows - row0, 0ll), 16ll));
    uint4 x[2][4];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const uint4* in = src[t] + (row0 - held) * 8 + lane;   // row lane / 8, piece lane % 8
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = i * 4 + (lane >> 3);
            x[t][i] = make_uint4(0, 0, 0, 0);
            if (r >= old && r < all) x[t][i] = __ldg(in + i * 32);
        }
        if (old > 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i * 4 + (lane >> 3) < old) x[t][i] = tail[t][row0 * 8 + i * 32 + lane];
        }
    }
    // the block's largest magnitude: as integers, so that NaN is above infinity
    const int slot = live ? slot_of(c, h, first + blk, a.status) : 0;
    __shared__ uint32_t top[2][A_THREADS / 32];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m = __vmaxu2(m, __vmaxu2(__vmaxu2(x[t][i].x & 0x7FFF7FFFu, x[t][i].y & 0x7FFF7FFFu),
                                     __vmaxu2(x[t][i].z & 0x7FFF7FFFu, x[t][i].w & 0x7FFF7FFFu)));
        }
        m = __reduce_max_sync(0xffffffffu, max(m << 16, m & 0x7FFF0000u));
        if (lane == 0) top[t][warp] = m;
    }
    __syncthreads();
    if (live) {
        const long long at = static_cast<long long>(h) * c.slots + slot;
        const int w0 = warp & ~(B / 16 - 1);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            uint32_t m = 0;
            for (int w = w0; w < w0 + B / 16; ++w) m = max(m, top[t][w]);
            const bool finite = m < 0x7F800000u;
            const float s = finite ? __fdiv_rn(__uint_as_float(m), FMT == ZB_KV8_INT8 ? 127.f : 448.f)
                                   : __uint_as_float(0x7FC00000u);
            const bool codes = finite && s > 0.f;
            const float inv = codes ? 1.f / s : 0.f;
            uint2* out = reinterpret_cast<uint2*>(t ? c.v : c.k) + (at * B + row0 - blk * B) * 8 + lane;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float f[8];
                const uint32_t w[4] = {x[t][i].x, x[t][i].y, x[t][i].z, x[t][i].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    f[2 * j] = bf16_lo(w[j]);
                    f[2 * j + 1] = bf16_hi(w[j]);
                }
                out[i * 32] = codes ? codes8<FMT>(f, s, inv) : make_uint2(0, 0);
            }
            if (warp == w0 && lane == 0) (t ? c.v_scale : c.k_scale)[at] = s;
        }
        // a block that this call opens starts without weight
        if (c.mass && warp == w0 && lane == 0 && (blk > 0 || held == 0)) c.mass[at] = 0.f;
    }
    if (unit == 0) {
        // The rows of the block left in progress, once this CTA has read the old
        // ones (no other CTA reads them: they are all in the first unit).
        __syncthreads();
        const int left = static_cast<int>(rows) & (B - 1);
        const long long last = rows - left;
        for (int i = threadIdx.x; i < left * 8; i += A_THREADS) {
            const long long r = last + (i >> 3);
            if (r < held) continue;
#pragma unroll
            for (int t = 0; t < 2; ++t) tail[t][i] = __ldg(src[t] + (r - held) * 8 + (i & 7));
        }
        if (threadIdx.x == 0 && a.lens_out) a.lens_out[h] = static_cast<int32_t>(len + a.n);
    }
}

// lens + n for the heads whose append fitted (an append over several CTAs a head
// cannot advance the lengths that its CTAs are reading).
__global__ void advance_kernel(const int32_t* lens, int32_t* out, int heads, int n, long long cap) {
    const int h = blockIdx.x * blockDim.x + threadIdx.x;
    if (h >= heads) return;
    const long long len = lens[h];
    out[h] = static_cast<int32_t>(len < 0 || len + n > cap ? len : len + n);
}

// ------------------------------------------------------------------ read ----
// The newest n tokens of every head as bf16 (code * scale in fp32, rounded once);
// rows before a head's first token are zeros.  An HBM stream: 64 B of codes in,
// 128 B out a row.  A thread moves 8 values of one tensor in each of R_ROWS rows
// that lie R_STEP apart, the table's entries of all of them read before any code; a
// warp's stores are whole rows.
constexpr int R_ROWS = 4, R_STEP = 32;
template <int FMT>
__global__ void __launch_bounds__(256) read_kernel(const zb_kv8 c, const int32_t* lens, int n, uint4* Ko, uint4* Vo,
                                                   int* status) {
    const int h = blockIdx.y;
    const long long cap = static_cast<long long>(c.slots) * c.block;
    const long long len = head_len(lens, h, cap);
    const uint2* codes = reinterpret_cast<const uint2*>(blockIdx.z ? c.v : c.k);
    const float* scale = blockIdx.z ? c.v_scale : c.k_scale;
    uint4* out = (blockIdx.z ? Vo : Ko) + static_cast<long long>(h) * n * 8;
    const int shift = 31 - __clz(c.block), q = threadIdx.x & 7;
    for (long long base = static_cast<long long>(blockIdx.x) * R_STEP * R_ROWS; base < n;
         base += static_cast<long long>(gridDim.x) * R_STEP * R_ROWS) {
        long long at[R_ROWS], row[R_ROWS];
        bool on[R_ROWS];
#pragma unroll
        for (int i = 0; i < R_ROWS; ++i) {
            row[i] = base + i * R_STEP + (threadIdx.x >> 3);
            const long long tok = len - n + row[i];
            on[i] = row[i] < n && tok >= 0;
            at[i] = on[i] ? static_cast<long long>(h) * c.slots + slot_of(c, h, tok >> shift, status) : 0;
        }
        uint2 w[R_ROWS];
        float s[R_ROWS];
#pragma unroll
        for (int i = 0; i < R_ROWS; ++i) {
            w[i] = make_uint2(0, 0);
            s[i] = 0.f;
            if (on[i]) {
                const long long tok = len - n + row[i];
                w[i] = __ldcs(codes + (at[i] * c.block + (tok & (c.block - 1))) * 8 + q);
                s[i] = __ldg(scale + at[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < R_ROWS; ++i) {
            if (row[i] >= n) continue;
            const uint32_t ww[2] = {w[i].x, w[i].y};
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                uint32_t p0, p1;
                unpack4<FMT>(ww[j], p0, p1);
                const float2 f0 = half2_floats(p0), f1 = half2_floats(p1);
                o[2 * j] = pack_bf16x2(f0.x * s[i], f0.y * s[i]);
                o[2 * j + 1] = pack_bf16x2(f1.x * s[i], f1.y * s[i]);
            }
            out[row[i] * 8 + q] = on[i] ? make_uint4(o[0], o[1], o[2], o[3]) : make_uint4(0, 0, 0, 0);
        }
    }
}

// ----------------------------------------------------------------- evict ----
constexpr int E_BINS = 2048;
constexpr int E_ITEMS = 24576;   // blocks whose keys and slots fit shared memory; longer lists gather them again
constexpr int E_AHEAD = 12;      // gathers a thread has in flight

// Order-preserving key of a weight (NaN with a clear sign above +inf; -0 as +0).
ZB_DEVINL uint32_t mass_key(float m) {
    const uint32_t b = m == 0.f ? 0u : __float_as_uint(m);
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

struct EvictArgs {
    const int32_t* table;
    const float* mass;
    const int32_t* lens;
    int slots, block, budget, sinks, recent;
    int32_t *table_out, *lens_out, *kept;
    int in_smem;
    int* status;
};

// One CTA a head.  The blocks between the first `sinks` and the last `recent`
// are ranked by weight: a histogram over the range the weights span, narrowed
// to the bin that holds the last kept one until it is a single value (at most
// three rounds), then one pass that keeps everything above it and the lowest
// indices among equals, each warp writing its own contiguous part in order.
// Bound by latency: two dependent gathers (slot, weight), then rounds over a list
// of some thousand words in shared memory.  256 threads serve lists of up to 2,048
// blocks, so that several heads share an SM (384 heads of 344 blocks: 13 -> 10.6 us);
// 1,024 the longer ones (16 heads of 10,992: 15 us).
template <int THREADS>
__global__ void __launch_bounds__(THREADS) evict_kernel(const EvictArgs a) {
    extern __shared__ uint32_t items[];              // keys, then slots
    constexpr int W = THREADS / 32, PER = E_BINS / THREADS;
    __shared__ uint32_t hist[E_BINS];
    __shared__ uint32_t red[32], red2[32];
    __shared__ uint32_t s_bin, s_above;
    const int h = blockIdx.x, tid = threadIdx.x, lane = lane_id(), warp = warp_id();
    const long long row = static_cast<long long>(h) * a.slots;
    const int32_t* table = a.table + row;
    int32_t* out = a.table_out + row;
    int32_t* kept = a.kept ? a.kept + static_cast<long long>(h) * a.budget : nullptr;
    const long long had = __ldca(a.lens + h);       // (lens_out may be lens)
    const long long len = min(max(had, 0ll), static_cast<long long>(a.slots) * a.block);
    const int nb = static_cast<int>((len + a.block - 1) / a.block);
    if (nb <= a.budget) {
        for (int b = tid; b < a.slots; b += THREADS) out[b] = table[b];
        if (kept)
            for (int b = tid; b < a.budget; b += THREADS) kept[b] = b < nb ? b : -1;
        if (tid == 0) a.lens_out[h] = static_cast<int32_t>(len);
        return;
    }
    const int b0 = a.sinks, b1 = nb - a.recent;
    const int need = a.budget - a.sinks - a.recent;   // < b1 - b0
    uint32_t* keys = items;
    uint32_t* slots = items + a.slots;
    auto key_of = [&](int s) -> uint32_t {
        if (s < 0 || s >= a.slots) {
            flag_status(a.status, ZB_ERR_INDEX);
            return 0u;
        }
        return mass_key(__ldg(a.mass + row + s));
    };
    uint32_t lo = 0xFFFFFFFFu, hi = 0;
    for (int base = tid; base < a.slots; base += THREADS * E_AHEAD) {
        int s[E_AHEAD];
        uint32_t k[E_AHEAD];
#pragma unroll
        for (int i = 0; i < E_AHEAD; ++i) s[i] = base + i * THREADS < a.slots ? __ldg(table + base + i * THREADS) : 0;
#pragma unroll
        for (int i = 0; i < E_AHEAD; ++i) {
            const int b = base + i * THREADS;
            k[i] = b >= b0 && b < b1 ? key_of(s[i]) : 0u;
        }
#pragma unroll
        for (int i = 0; i < E_AHEAD; ++i) {
            const int b = base + i * THREADS;
            if (b >= a.slots) continue;
            if (b >= b0 && b < b1) {
                lo = min(lo, k[i]);
                hi = max(hi, k[i]);
            }
            if (a.in_smem) {
                keys[b] = k[i];
                slots[b] = s[i];
            }
            if (b >= nb) out[b] = s[i];              // unused slots stay
        }
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) {
        red[warp] = lo;
        red2[warp] = hi;
    }
    for (int i = tid; i < E_BINS; i += THREADS) hist[i] = 0;
    __syncthreads();
    lo = __reduce_min_sync(0xffffffffu, lane < W ? red[lane] : 0xFFFFFFFFu);
    hi = __reduce_max_sync(0xffffffffu, lane < W ? red2[lane] : 0u);
    __syncthreads();
    auto slot = [&](int b) -> int { return a.in_smem ? static_cast<int>(slots[b]) : table[b]; };
    auto key = [&](int b) -> uint32_t { return a.in_smem ? keys[b] : key_of(table[b]); };

    // invariant: `want` keys are to be kept of those in [lo, hi] (the larger ones,
    // above hi, are all kept already), 0 <= want <= their number; hist is zero
    uint32_t want = need;
    while (need > 0 && lo < hi) {
        const uint32_t span = hi - lo;
        const int bits = 32 - __clz(span);
        const int sh = bits > 11 ? bits - 11 : 0;
        for (int b = b0 + tid; b < b1; b += THREADS) {
            const uint32_t k = key(b);
            if (k >= lo && k <= hi) atomicAdd(&hist[(k - lo) >> sh], 1u);
        }
        __syncthreads();
        // PER bins a thread, from the top: the bin where the count reaches `want`
        const int top = E_BINS - 1 - PER * tid;
        uint32_t c[PER], own = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            c[i] = hist[top - i];
            own += c[i];
        }
        uint32_t incl = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) red[warp] = incl;
        __syncthreads();
        uint32_t before = __reduce_add_sync(0xffffffffu, lane < warp ? red[lane] : 0) + incl - own;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (before < want && want <= before + c[i]) {
                s_bin = top - i;
                s_above = before;
            }
            before += c[i];
            hist[top - i] = 0;
        }
        __syncthreads();
        want -= s_above;
        lo += s_bin << sh;
        const uint32_t width = (1u << sh) - 1u;
        if (hi - lo > width) hi = lo + width;
    }
    __syncthreads();
    // keep: keys above `hi` (== lo) and the first `want` equal to it
    const uint32_t edge = need > 0 ? lo : 0xFFFFFFFFu;
    if (need == 0) want = 0;
    const int per = ((nb + THREADS - 1) / THREADS) * 32;  // blocks a warp takes
    const int w0 = min(warp * per, nb), w1 = min(w0 + per, nb);
    const int w2 = w0 + (w1 - w0 + 31) / 32 * 32;         // all lanes run the same rounds
    uint32_t over = 0, ties = 0;
    for (int b = w0 + lane; b < w2; b += 32) {
        const bool in = b < w1, mid = in && b >= b0 && b < b1;
        const uint32_t k = mid ? key(b) : 0u;
        over += __popc(__ballot_sync(0xffffffffu, in && (!mid || k > edge)));
        ties += __popc(__ballot_sync(0xffffffffu, mid && k == edge));
    }
    if (lane == 0) {
        red[warp] = over;
        red2[warp] = ties;
    }
    __syncthreads();
    const uint32_t over0 = __reduce_add_sync(0xffffffffu, lane < warp ? red[lane] : 0);
    uint32_t ties0 = __reduce_add_sync(0xffffffffu, lane < warp ? red2[lane] : 0);
    uint32_t pos = over0 + min(ties0, want);              // kept before this warp's part
    for (int b = w0 + lane; b < w2; b += 32) {
        const bool in = b < w1, mid = in && b >= b0 && b < b1;
        const uint32_t k = mid ? key(b) : 0u;
        const uint32_t below = (1u << lane) - 1u;
        const uint32_t tie = __ballot_sync(0xffffffffu, mid && k == edge);
        const bool keep = in && (!mid || k > edge || (k == edge && ties0 + __popc(tie & below) < want));
        const uint32_t mask = __ballot_sync(0xffffffffu, keep);
        if (in) {
            const uint32_t r = pos + __popc(mask & below);   // kept blocks before b
            if (keep) {
                out[r] = slot(b);
                if (kept) kept[r] = b;
            } else {
                out[a.budget + (b - r)] = slot(b);
            }
        }
        pos += __popc(mask);
        ties0 += __popc(tie);
    }
    if (tid == 0) a.lens_out[h] = static_cast<int32_t>(len - static_cast<long long>(nb - a.budget) * a.block);
}

}  // namespace kv8
}  // namespace zb

using namespace zb;

extern "C" zb_status zb_kv8_append(zb_kv8 cache, const uint16_t* K, const uint16_t* V, int64_t n_new,
                                   const int32_t* lens, int32_t* lens_out, void* stream) {
    zb_status e = kv8::check_cache(cache, true);
    if (e != ZB_OK) return e;
    if (n_new < 1) return ZB_ERR_SHAPE;
    if (n_new > static_cast<long long>(cache.slots) * cache.block) return ZB_ERR_SHAPE;
    if (!K || !V || !lens || !lens_out || !cache.k_tail || !cache.v_tail) return ZB_ERR_NULL;
    if (!aligned16(K) || !aligned16(V) || !aligned16(cache.k_tail) || !aligned16(cache.v_tail) ||
        (reinterpret_cast<uintptr_t>(lens) & 3u) || (reinterpret_cast<uintptr_t>(lens_out) & 3u))
        return ZB_ERR_ALIGN;
    DeviceInfo dev;
    if ((e = current_device(&dev)) != ZB_OK) return e;
    const long long units = (cache.block - 1 + n_new + kv8::UNIT - 1) / kv8::UNIT;
    const bool apart = lens == lens_out && units > 1;
    kv8::AppendArgs a{cache, reinterpret_cast<const uint4*>(K), reinterpret_cast<const uint4*>(V),
                      static_cast<int>(n_new), lens, apart ? nullptr : lens_out, dev.status};
    const dim3 grid(static_cast<unsigned>(units), static_cast<unsigned>(cache.heads));
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (cache.format == ZB_KV8_INT8) kv8::append_kernel<ZB_KV8_INT8><<<grid, kv8::A_THREADS, 0, st>>>(a);
    else kv8::append_kernel<ZB_KV8_E4M3><<<grid, kv8::A_THREADS, 0, st>>>(a);
    if (cudaGetLastError() != cudaSuccess) return ZB_ERR_CUDA;
    if (apart) {
        kv8::advance_kernel<<<(cache.heads + 255) / 256, 256, 0, st>>>(lens, lens_out, cache.heads,
                                                                       static_cast<int>(n_new),
                                                                       static_cast<long long>(cache.slots) * cache.block);
        if (cudaGetLastError() != cudaSuccess) return ZB_ERR_CUDA;
    }
    return ZB_OK;
}

extern "C" zb_status zb_kv8_read(zb_kv8 cache, const int32_t* lens, int64_t n, uint16_t* K, uint16_t* V, void* stream) {
    zb_status e = kv8::check_cache(cache, true);
    if (e != ZB_OK) return e;
    if (n < 1 || n > 0x7FFFFFFFll) return ZB_ERR_SHAPE;
    if (!lens || !K || !V) return ZB_ERR_NULL;
    if (!aligned16(K) || !aligned16(V) || (reinterpret_cast<uintptr_t>(lens) & 3u)) return ZB_ERR_ALIGN;
    DeviceInfo dev;
    if ((e = current_device(&dev)) != ZB_OK) return e;
    long long gx = (n + kv8::R_STEP * kv8::R_ROWS - 1) / (kv8::R_STEP * kv8::R_ROWS);
    if (gx > 65536) gx = 65536;
    const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(cache.heads), 2);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    uint4 *ko = reinterpret_cast<uint4*>(K), *vo = reinterpret_cast<uint4*>(V);
    if (cache.format == ZB_KV8_INT8)
        kv8::read_kernel<ZB_KV8_INT8><<<grid, 256, 0, st>>>(cache, lens, static_cast<int>(n), ko, vo, dev.status);
    else
        kv8::read_kernel<ZB_KV8_E4M3><<<grid, 256, 0, st>>>(cache, lens, static_cast<int>(n), ko, vo, dev.status);
    return cudaGetLastError() == cudaSuccess ? ZB_OK : ZB_ERR_CUDA;
}

extern "C" zb_status zb_kv8_evict(const int32_t* table, const float* mass, const int32_t* lens, int32_t heads,
                                  int32_t slots, int32_t block, int32_t budget, int32_t sinks, int32_t recent,
                                  int32_t* table_out, int32_t* lens_out, int32_t* kept, void* stream) {
    if (heads < 1 || slots < 1 || sinks < 0 || recent < 1) return ZB_ERR_SHAPE;
    if (block != 16 && block != 32 && block != 64 && block != 128) return ZB_ERR_UNSUPPORTED;
    if (heads > 65535 || static_cast<long long>(slots) * block > 0x7FFFFF00ll) return ZB_ERR_UNSUPPORTED;
    if (budget < 1 || budget > slots || static_cast<long long>(sinks) + recent > budget) return ZB_ERR_SHAPE;
    if (!table || !mass || !lens || !table_out || !lens_out) return ZB_ERR_NULL;
    if (table == table_out) return ZB_ERR_SHAPE;
    for (const void* p : {static_cast<const void*>(table), static_cast<const void*>(mass),
                          static_cast<const void*>(lens), static_cast<const void*>(table_out),
                          static_cast<const void*>(lens_out), static_cast<const void*>(kept)})
        if (reinterpret_cast<uintptr_t>(p) & 3u) return ZB_ERR_ALIGN;
    DeviceInfo dev;
    zb_status e = current_device(&dev);
    if (e != ZB_OK) return e;
    kv8::EvictArgs a{table, mass, lens, slots, block, budget, sinks, recent, table_out, lens_out, kept,
                     slots <= kv8::E_ITEMS, dev.status};
    const int smem = a.in_smem ? slots * 8 : 0;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (slots <= 2048) {
        kv8::evict_kernel<256><<<heads, 256, smem, st>>>(a);
    } else {
        if (smem > 32 * 1024 && cudaFuncSetAttribute(kv8::evict_kernel<1024>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                     kv8::E_ITEMS * 8) != cudaSuccess)
            return ZB_ERR_CUDA;
        kv8::evict_kernel<1024><<<heads, 1024, smem, st>>>(a);
    }
    return cudaGetLastError() == cudaSuccess ? ZB_OK : ZB_ERR_CUDA;
}
