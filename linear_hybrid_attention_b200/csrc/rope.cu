// Rotary positions, and the per-head norm of queries and keys with the rotation
// in the same pass: the step between a layer's projection and its attention.
// It takes rows of 64 from wherever the projection left them (any head and
// token strides) into the layout the attention calls read.
//
//   forward   y = norm(x) * w + b            (rms: x r, layer: (x - mean) r,
//             o = rotate(y, +theta)           r = (mean of squares + eps)^-1/2)
//   backward  dy = rotate(do, -theta), g = dy * w, xh = normalised x,
//             dx = r (g - [layer: mean(g)] - xh mean(g xh)),
//             dw = sum over rows of dy xh,  db = sum over rows of dy
//
// Angles.  The frequency of pair i is held as turns a position in 64-bit fixed
// point, T_i = f_i / 2 pi * 2^64; the low 64 bits of pos * T_i are then the
// fraction of a turn, exact for any 32-bit position up to what T_i is off by: T_i comes
// from fp64 (53 bits), some 2^-56 turns a position.  Its top 32 bits go to sin and cos, so a far position
// costs no more and loses nothing against a near one.
//
// Both directions are HBM streams (a row in, a row out; backward two in, one
// out) that only reach the memory's rate if their arithmetic stays small: a row
// has 64 features and some 95 instructions a thread here.  Four lanes hold a
// row, 16 features each, chosen so that both halves of every rotated pair lie in
// one thread: no exchange but two shuffles for each of the row's sums, and one
// kernel for both pair layouts.  Features are worked on as packed pairs, and
// forward the weights and biases are turned once a token together with the sines,
// so that a row costs one rotation whatever its norm.  A thread runs over the
// heads of its token with the next rows' loads under way; the items are shared
// out evenly over the CTAs that fit at once.
//
// Measured (B200): rotation alone, 16 heads of 43,968 tokens, 32 us (27 at the
// copy rate); layer norm and rotation of 16 + 16 heads of 43,968 tokens 67 us
// (54); rms norm of 16 + 4 heads of 2 x 10,992 tokens 21 us forward, 39 + 3
// backward (17 and 25).  Before: scalar arithmetic, weights in registers and
// sincospi 37, 83, 32 and 48 + 6 us; rows copied ahead through shared memory
// instead of registers 38, 98, 35 and 57 (the shared memory's own bandwidth);
// three CTAs an SM instead of two 38 (spills); groups of tokens of four heads
// side by side 38.
#include <cuda_runtime.h>
#include <math.h>

#include "zb_common.cuh"
#include "zb_host.h"

namespace zb {
namespace rope {

constexpr int HD = 64;
constexpr int THREADS = 256;
constexpr int TOK = THREADS / 4;   // tokens a CTA works on at a time
constexpr int MAX_CTAS = 4096;     // of a backward launch (its partial sums)

struct View {
    long long b, h, t;             // strides in elements
};

// One of the two tensors of a launch (queries, keys).
struct Side {
    const uint16_t *x, *g;         // input rows; gradient of the output rows
    uint16_t* out;                 // output rows; backward: gradient of the input rows
    View xs, gs, os;
    const float *w, *bias;         // [64] or NULL
    float *dw, *db;                // [64] or NULL (backward)
    int heads, ctas;               // heads, and the CTAs that share the tensor's items
};

struct Args {
    Side side[2];
    long long tokens, n;           // batch * n, tokens of a sequence
    const int32_t* pos;
    long long pos_b;               // batch stride of pos (0: shared)
    const int64_t* turns;
    int rot, axes, half;
    float mag, eps;
    int inverse;
    float* partial;                // backward: [CTA][2][64]
};

typedef uint64_t f2;               // two fp32 in a register pair
ZB_DEVINL float total(f2 v) {
    float x, y;
    f2_unpack(v, x, y);
    return x + y;
}

// A thread's 16 features of a row, two by two: v[0..3] the first members of its
// eight rotated pairs, v[4..7] the second ones.  In the half layout those are its
// two chunks of 8, interleaved the even and the odd features of both.
template <bool HALF>
ZB_DEVINL void unpack(const uint4& x, const uint4& y, f2* v) {
    const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (HALF) {
            v[i] = f2_pack(bf16_lo(w[i]), bf16_hi(w[i]));
            v[4 + i] = f2_pack(bf16_lo(w[4 + i]), bf16_hi(w[4 + i]));
        } else {
            v[i] = f2_pack(bf16_lo(w[2 * i]), bf16_lo(w[2 * i + 1]));
            v[4 + i] = f2_pack(bf16_hi(w[2 * i]), bf16_hi(w[2 * i + 1]));
        }
    }
}
template <bool HALF>
ZB_DEVINL void pack(const f2* v, uint4& x, uint4& y) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float p0, p1, q0, q1;
        f2_unpack(v[i], p0, p1);
        f2_unpack(v[4 + i], q0, q1);
        if (HALF) {
            w[i] = pack_bf16x2(p0, p1);
            w[4 + i] = pack_bf16x2(q0, q1);
        } else {
            w[2 * i] = pack_bf16x2(p0, q0);
            w[2 * i + 1] = pack_bf16x2(p1, q1);
        }
    }
    x = make_uint4(w[0], w[1], w[2], w[3]);
    y = make_uint4(w[4], w[5], w[6], w[7]);
}
// The feature that element i of those 16 is.
template <bool HALF>
ZB_DEVINL int feature(int i, int c0, int c1) {
    if (HALF) return i < 8 ? c0 * 8 + i : c1 * 8 + i - 8;
    const int j = i & 7;
    return (j < 4 ? c0 * 8 + 2 * j : c1 * 8 + 2 * (j - 4)) + (i >> 3);
}

ZB_DEVINL float row_sum(float v) {   // over the row's four lanes
    v += __shfl_xor_sync(0xffffffffu, v, 1);
    return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

// (x, y) by the angle of (c, s): x c - y s, y c + x s.
ZB_DEVINL void rotate(f2* v, const f2* c, const f2* s) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const f2 x = v[i], y = v[4 + i];
        v[i] = f2_sub(f2_mul(x, c[i]), f2_mul(y, s[i]));
        v[4 + i] = f2_fma(y, c[i], f2_mul(x, s[i]));
    }
}

// v <- the row, centred where the norm is a layer norm; returns 1 / its deviation.  The
// variance is taken of the centred row: a second pass over registers, no cancellation.
template <int KIND>
ZB_DEVINL float centre(f2* v, float eps) {
    if (KIND == ZB_NORM_NONE) return 1.f;
    if (KIND == ZB_NORM_LAYER) {
        const float m = row_sum(total(f2_add(f2_add(f2_add(v[0], v[1]), f2_add(v[2], v[3])),
                                             f2_add(f2_add(v[4], v[5]), f2_add(v[6], v[7]))))) * (-1.f / HD);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = f2_add(v[i], f2_pack(m, m));
    }
    f2 q0 = f2_mul(v[0], v[0]), q1 = f2_mul(v[1], v[1]);
#pragma unroll
    for (int i = 2; i < 8; i += 2) {
        q0 = f2_fma(v[i], v[i], q0);
        q1 = f2_fma(v[i + 1], v[i + 1], q1);
    }
    const float ms = row_sum(total(f2_add(q0, q1))) * (1.f / HD) + eps;
    float inv = rsqrtf(ms);
    // squares that pass fp32, or are lost below it: of the row times a power of two
    if (__any_sync(0xffffffffu, !(ms >= 0x1p-90f && ms <= 0x1p100f))) {
        const float s = ms > 1.f ? 0x1p-72f : 0x1p64f;
        f2 q = 0ull;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const f2 x = f2_mul(v[i], f2_pack(s, s));
            q = f2_fma(x, x, q);
        }
        const float far = rsqrtf(fmaf(row_sum(total(q)), 1.f / HD, eps * s * s)) * s;
        if (!(ms >= 0x1p-90f && ms <= 0x1p100f)) inv = far;
    }
    return inv;
}

// sin and cos of a fraction of a turn (turns * 2^32).  After the exact reduction
// the hardware's approximation is within 2^-20 of either, eleven bits below the
// bf16 result; sincospi costs 8 pairs some 400 instructions against 100.
ZB_DEVINL void sincos_turns(int frac, float& sn, float& cs) {
    const float x = static_cast<float>(frac) * (3.14159265358979f * 0x1p-31f);
    asm("sin.approx.ftz.f32 %0, %1;" : "=f"(sn) : "f"(x));
    asm("cos.approx.ftz.f32 %0, %1;" : "=f"(cs) : "f"(x));
}

constexpr int CTAS = 2;                // an SM: 128 registers a thread; with 80 (three) most kernels spill

ZB_DEVINL void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

template <int KIND, bool BACK, bool HALF>
__global__ void __launch_bounds__(THREADS, CTAS) row_kernel(const Args a) {
    constexpr int ROWS = BACK ? 1 : 2;               // under way; forward they are worked on together
    constexpr bool NORM = KIND != ZB_NORM_NONE;
    // the next group's first rows go to L2 and its position to a register while a group is worked on
    // (rms norm of 16 + 4 heads 24 -> 21 us); the layer norm has no register left for it (67 -> 69)
    constexpr bool AHEAD = KIND != ZB_NORM_LAYER;
    if (BACK) let_next_start();                      // the sums' kernel, which waits

    // the CTA's tensor and its part of that tensor's (group of TOK tokens, head) items
    const bool second = static_cast<int>(blockIdx.x) >= a.side[0].ctas;
    const Side& sd = second ? a.side[1] : a.side[0];
    const int cta = second ? blockIdx.x - a.side[0].ctas : blockIdx.x;
    const int heads = sd.heads;
    const long long items = (a.tokens + TOK - 1) / TOK * heads;
    const long long each = items / sd.ctas, more = items - each * sd.ctas;   // the first `more` take one more
    const long long i0 = each * cta + (cta < more ? cta : more);
    long long left = each + (cta < more), group = i0 / heads;
    int h0 = static_cast<int>(i0 - group * heads);

    const int p = threadIdx.x & 3;
    const bool turned = p < a.rot / 16;
    const int pairs = a.rot / (2 * a.axes);          // of an axis
    int c0 = 2 * p, c1 = 2 * p + 1, axis = 0, pair0 = 0;
    if (turned) {
        if (HALF) {                                  // chunk c0 of an axis' part and its partner
            const int hc = pairs / 8;
            axis = p / hc;
            const int i = p - axis * hc;
            c0 = axis * 2 * hc + i;
            c1 = c0 + hc;
            pair0 = i * 8;
        } else {
            axis = p * 8 / pairs;
            pair0 = p * 8 - axis * pairs;
        }
    }
    // weights and biases in the order of the threads' elements
    __shared__ ulonglong2 weights[4][4], biases[4][4];
    if (NORM) {
        if (threadIdx.x < 4 * 16) {
            const int l = threadIdx.x & 3, i = threadIdx.x >> 2;
            const int e = feature<HALF>(i, c0, c1);  // l == p
            reinterpret_cast<float*>(weights[l])[i] = sd.w ? __ldg(sd.w + e) : 1.f;
            if (KIND == ZB_NORM_LAYER && !BACK) reinterpret_cast<float*>(biases[l])[i] = sd.bias ? __ldg(sd.bias + e) : 0.f;
        }
        __syncthreads();
    }
    auto weight = [&](int i) { return i & 1 ? weights[p][i >> 1].y : weights[p][i >> 1].x; };
    auto bias = [&](int i) { return i & 1 ? biases[p][i >> 1].y : biases[p][i >> 1].x; };
    f2 dw[8], db[8];
    if (BACK) {
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[i] = db[i] = 0ull;
    }

    const long long xh = sd.xs.h / 8, gh = sd.gs.h / 8, oh = sd.os.h / 8;
    int pos_ahead = 0;
    bool ahead = false;
#pragma unroll 1
    while (left > 0) {
        const int n = heads - h0 < left ? heads - h0 : static_cast<int>(left);   // rows of this group
        const long long u = group * TOK + (threadIdx.x >> 2);
        const bool live = u < a.tokens;              // dead lanes still join the shuffles
        long long b = 0, t = live ? u : 0;
        if (a.tokens != a.n) {
            b = (a.tokens >> 32) ? t / a.n : static_cast<uint32_t>(t) / static_cast<uint32_t>(a.n);
            t -= b * a.n;
        }
        const uint4* x = reinterpret_cast<const uint4*>(sd.x + b * sd.xs.b + t * sd.xs.t + h0 * sd.xs.h);
        const uint4* g = BACK ? reinterpret_cast<const uint4*>(sd.g + b * sd.gs.b + t * sd.gs.t + h0 * sd.gs.h) : nullptr;
        uint4* o = reinterpret_cast<uint4*>(sd.out + b * sd.os.b + t * sd.os.t + h0 * sd.os.h);
        // the next ROWS rows are on their way while these are worked on
        uint4 xv[ROWS][2], gv[BACK ? ROWS : 1][2];
        auto load = [&](int k) {
            // forward the output may be the input: not the path for memory that no one writes
            xv[k][0] = BACK ? __ldg(x + c0) : __ldca(x + c0);
            xv[k][1] = BACK ? __ldg(x + c1) : __ldca(x + c1);
            x += xh;
            if (BACK) {
                gv[k][0] = live ? __ldg(g + c0) : make_uint4(0, 0, 0, 0);
                gv[k][1] = live ? __ldg(g + c1) : make_uint4(0, 0, 0, 0);
                g += gh;
            }
        };
#pragma unroll
        for (int k = 0; k < ROWS; ++k) {
            xv[k][0] = xv[k][1] = make_uint4(0, 0, 0, 0);
            if (k == 0 || k < n) load(k);            // a row that is not there: zeros, then an old row again, not stored
        }
        if (AHEAD && left > n && live && t + TOK < a.n) {
            const uint4* xn = reinterpret_cast<const uint4*>(sd.x + b * sd.xs.b + (t + TOK) * sd.xs.t);
#pragma unroll
            for (int k = 0; k < ROWS; ++k) {
                if (k >= heads) break;
                prefetch_l2(xn + k * xh + c0);
                prefetch_l2(xn + k * xh + c1);
            }
            if (BACK) {
                const uint4* gn = reinterpret_cast<const uint4*>(sd.g + b * sd.gs.b + (t + TOK) * sd.gs.t);
                prefetch_l2(gn + c0);
                prefetch_l2(gn + c1);
            }
        }
        // forward, a row is r (x w c - y w' s) + b: weights and biases turned once a token
        f2 ca[4], cb[4], sa[4], sb[4], z[8];
        {
            float c[8], s[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                c[j] = 1.f;
                s[j] = 0.f;
            }
            if (turned) {
                const int32_t* at = a.pos + b * a.pos_b + axis * a.n + t;
                const unsigned long long pos = static_cast<long long>(ahead ? pos_ahead : __ldg(at));
                ahead = AHEAD && t + TOK < a.n;
                if (ahead) pos_ahead = __ldg(at + TOK);
                const float way = BACK || a.inverse ? -a.mag : a.mag;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const unsigned long long ph = pos * static_cast<unsigned long long>(__ldg(a.turns + pair0 + j));
                    sincos_turns(static_cast<int>(ph >> 32), s[j], c[j]);
                    c[j] *= a.mag;
                    s[j] *= way;
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                ca[i] = cb[i] = f2_pack(c[2 * i], c[2 * i + 1]);
                sa[i] = f2_pack(s[2 * i], s[2 * i + 1]);
                sb[i] = f2_pack(-s[2 * i], -s[2 * i + 1]);
                if (!BACK && KIND == ZB_NORM_LAYER) {
                    z[i] = bias(i);
                    z[4 + i] = bias(4 + i);
                }
            }
            if (!BACK && KIND == ZB_NORM_LAYER && turned) rotate(z, ca, sa);
            if (!BACK && NORM) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f2 wa = weight(i), wb = weight(4 + i);
                    ca[i] = f2_mul(ca[i], wa);
                    sa[i] = f2_mul(sa[i], wa);
                    cb[i] = f2_mul(cb[i], wb);
                    sb[i] = f2_mul(sb[i], wb);
                }
            }
        }
#pragma unroll 1
        for (int r = 0; r < n; r += ROWS) {
            f2 f[ROWS][8], e[8];
            if (!BACK) {
#pragma unroll
                for (int k = 0; k < ROWS; ++k) unpack<HALF>(xv[k][0], xv[k][1], f[k]);
#pragma unroll
                for (int k = 0; k < ROWS; ++k)
                    if (r + ROWS + k < n) load(k);
            }
#pragma unroll
            for (int k = 0; k < ROWS; ++k) {
                if (BACK) {
                    if (k && r + k >= n) break;
                    unpack<HALF>(xv[k][0], xv[k][1], f[k]);
                    unpack<HALF>(gv[BACK ? k : 0][0], gv[BACK ? k : 0][1], e);
                    if (r + ROWS + k < n) load(k);
                }
                const float inv = centre<KIND>(f[k], a.eps);
                const f2 inv2 = f2_pack(inv, inv);
                if (BACK) {
                    if (turned) rotate(e, ca, sa);
                    f2 t1 = 0ull, t0 = 0ull;
                    if (NORM) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            f[k][i] = f2_mul(f[k][i], inv2);
                            dw[i] = f2_fma(e[i], f[k][i], dw[i]);
                            if (KIND == ZB_NORM_LAYER) db[i] = f2_add(db[i], e[i]);
                            e[i] = f2_mul(e[i], weight(i));
                            t1 = f2_fma(e[i], f[k][i], t1);
                            if (KIND == ZB_NORM_LAYER) t0 = f2_add(t0, e[i]);
                        }
                        const float m1 = row_sum(total(t1)) * (-1.f / HD);
                        const float m0 = KIND == ZB_NORM_LAYER ? row_sum(total(t0)) * (-1.f / HD) : 0.f;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            if (KIND == ZB_NORM_LAYER) e[i] = f2_add(e[i], f2_pack(m0, m0));
                            e[i] = f2_mul(inv2, f2_fma(f[k][i], f2_pack(m1, m1), e[i]));
                        }
                    }
                    if (live) pack<HALF>(e, o[c0], o[c1]);
                } else {
                    f2* v = f[k];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const f2 xa = v[i], xb = v[4 + i];
                        if (turned) {
                            v[i] = f2_fma(xa, ca[i], f2_mul(xb, sb[i]));
                            v[4 + i] = f2_fma(xb, cb[i], f2_mul(xa, sa[i]));
                        } else if (NORM) {
                            v[i] = f2_mul(xa, ca[i]);
                            v[4 + i] = f2_mul(xb, cb[i]);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (KIND == ZB_NORM_LAYER) v[i] = f2_fma(v[i], inv2, z[i]);
                        if (KIND == ZB_NORM_RMS) v[i] = f2_mul(v[i], inv2);
                    }
                    if (live && (k == 0 || r + k < n)) pack<HALF>(v, o[c0], o[c1]);
                }
                o += oh;
            }
        }
        left -= n;
        h0 = 0;
        ++group;
    }
    if (BACK && KIND != ZB_NORM_NONE) {
        // the CTA's sums: rows of a warp by shuffles, warps through shared memory in order
        __shared__ float red[THREADS / 32][2][HD];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float v[4];
            f2_unpack(dw[i], v[0], v[1]);
            f2_unpack(db[i], v[2], v[3]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
#pragma unroll
                for (int l = 4; l < 32; l <<= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], l);
            }
            if (lane_id() < 4) {
#pragma unroll
                for (int k = 0; k < 4; ++k) red[warp_id()][k >> 1][feature<HALF>(2 * i + (k & 1), c0, c1)] = v[k];
            }
        }
        __syncthreads();
        if (threadIdx.x < 2 * HD) {
            float v = 0.f;
            for (int k = 0; k < THREADS / 32; ++k) v += (&red[k][0][0])[threadIdx.x];
            a.partial[static_cast<long long>(blockIdx.x) * 2 * HD + threadIdx.x] = v;
        }
    }
}

// dw and db of one tensor from the CTAs' partial sums, in a fixed order, fp64.
// Grid: 8 blocks of 8 features x 2 (dw, db) x 2 (queries, keys).
__global__ void __launch_bounds__(256) reduce_kernel(const float* partial, Args a) {
    wait_for_previous();
    const int which = blockIdx.y & 1, tensor = blockIdx.y >> 1;
    float* out = which ? a.side[tensor].db : a.side[tensor].dw;
    if (!out) return;
    const int first = tensor ? a.side[0].ctas : 0;
    const int count = a.side[tensor].ctas;
    const int f = threadIdx.x & 7, part = threadIdx.x >> 3;   // 32 parts
    double s = 0.0;
    for (int c = part; c < count; c += 32)
        s += partial[static_cast<long long>(first + c) * 2 * HD + which * HD + blockIdx.x * 8 + f];
    __shared__ double red[32][8];
    red[part][f] = s;
    __syncthreads();
    if (threadIdx.x < 8) {
        double v = 0.0;
        for (int k = 0; k < 32; ++k) v += red[k][f];
        out[blockIdx.x * 8 + f] = static_cast<float>(v);
    }
}

// ------------------------------------------------------------------ host ----
bool strides_ok(const zb_rows& r) {
    return r.batch_stride >= 0 && r.head_stride >= 0 && r.token_stride >= 0 && r.batch_stride % 8 == 0 &&
           r.head_stride % 8 == 0 && r.token_stride % 8 == 0;
}

// Rows of an output view do not overlap: with the extents in order of their
// strides, each stride spans everything below it.
bool disjoint(const zb_rows& r, long long b, long long h, long long n) {
    long long st[3] = {r.batch_stride, r.head_stride, r.token_stride}, ex[3] = {b, h, n};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (st[j] < st[i]) {
                long long x = st[i]; st[i] = st[j]; st[j] = x;
                x = ex[i]; ex[i] = ex[j]; ex[j] = x;
            }
    long long span = HD;
    for (int i = 0; i < 3; ++i) {
        if (ex[i] == 1) continue;
        if (st[i] < span) return false;
        span = st[i] * (ex[i] - 1) + span;
    }
    return true;
}

View view(const zb_rows& r) { return {r.batch_stride, r.head_stride, r.token_stride}; }
View packed(long long heads, long long n) { return {heads * n * HD, n * HD, HD}; }

zb_status check_rotation(const zb_rotation& r) {
    if (r.rotary_dim < 0 || r.rotary_dim > HD) return ZB_ERR_SHAPE;
    if (r.rotary_dim == 0) return ZB_OK;
    if (r.axes != 1 && r.axes != 2) return ZB_ERR_UNSUPPORTED;
    if (r.rotary_dim % (16 * r.axes)) return ZB_ERR_UNSUPPORTED;
    if (r.layout != ZB_ROPE_HALF && r.layout != ZB_ROPE_INTERLEAVED) return ZB_ERR_UNSUPPORTED;
    if (!(r.magnitude > 0.f) || !(r.magnitude <= 3.4e38f)) return ZB_ERR_SHAPE;
    if (r.pos_batch_stride < 0) return ZB_ERR_SHAPE;
    if (!r.pos || !r.turns) return ZB_ERR_NULL;
    if ((reinterpret_cast<uintptr_t>(r.pos) & 3u) || (reinterpret_cast<uintptr_t>(r.turns) & 7u)) return ZB_ERR_ALIGN;
    return ZB_OK;
}

zb_status check_sizes(int batch, int heads_q, int heads_k, long long n, int d) {
    if (batch < 1 || heads_q < 1 || heads_k < 0 || n < 1) return ZB_ERR_SHAPE;
    if (d != HD) return ZB_ERR_UNSUPPORTED;
    if (n > 0x7FFFFFFFll || static_cast<long long>(batch) * n > (1ll << 37)) return ZB_ERR_UNSUPPORTED;
    return ZB_OK;
}

void put_rotation(Args& a, const zb_rotation& r) {
    a.pos = r.pos;
    a.pos_b = r.pos_batch_stride;
    a.turns = r.turns;
    a.rot = r.rotary_dim;
    a.axes = r.rotary_dim ? r.axes : 1;
    a.half = r.layout == ZB_ROPE_HALF;
    a.mag = r.magnitude;
    a.inverse = r.inverse;
}

// The CTAs that fit on the device at once, shared out between the tensors by
// their items (a group of TOK tokens of one head) and within a tensor evenly:
// no last wave that leaves SMs idle.
void share_ctas(Args& a, int resident) {
    const long long groups = (a.tokens + TOK - 1) / TOK;
    const long long total = groups * (static_cast<long long>(a.side[0].heads) + a.side[1].heads);
    for (int s = 0; s < 2; ++s) {
        const long long items = groups * a.side[s].heads;
        long long k = total <= resident ? items : static_cast<long long>(static_cast<double>(items) / total * resident + 0.5);
        if (k > items) k = items;
        a.side[s].ctas = items ? static_cast<int>(k < 1 ? 1 : k) : 0;
    }
}

template <int KIND, bool BACK, bool HALF>
zb_status launch_layout(Args& a, const DeviceInfo& dev, cudaStream_t st) {
    share_ctas(a, CTAS * dev.sm_count);
    row_kernel<KIND, BACK, HALF><<<a.side[0].ctas + a.side[1].ctas, THREADS, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? ZB_OK : ZB_ERR_CUDA;
}

template <int KIND, bool BACK>
zb_status launch_kind(Args& a, const DeviceInfo& dev, cudaStream_t st) {
    return a.half ? launch_layout<KIND, BACK, true>(a, dev, st) : launch_layout<KIND, BACK, false>(a, dev, st);
}

template <bool BACK>
zb_status launch(Args& a, int kind, const DeviceInfo& dev, cudaStream_t st) {
    switch (kind) {
        case ZB_NORM_RMS: return launch_kind<ZB_NORM_RMS, BACK>(a, dev, st);
        case ZB_NORM_LAYER: return launch_kind<ZB_NORM_LAYER, BACK>(a, dev, st);
        default: return launch_kind<ZB_NORM_NONE, BACK>(a, dev, st);
    }
}

}  // namespace rope
}  // namespace zb

using namespace zb;

extern "C" zb_status zb_rope_frequencies(int32_t pairs, double base, int32_t scaling, double factor,
                                         double original_len, double low, double high, int64_t* turns,
                                         double* radians, float* magnitude) {
    if (pairs < 1 || pairs > rope::HD / 2) return ZB_ERR_SHAPE;
    if (!(base > 1.0) || !(base < 1e30)) return ZB_ERR_SHAPE;
    if (!turns) return ZB_ERR_NULL;
    if (scaling < ZB_ROPE_PLAIN || scaling > ZB_ROPE_PARTS) return ZB_ERR_UNSUPPORTED;
    if (scaling != ZB_ROPE_PLAIN && (!(factor >= 1.0) || !(factor < 1e9))) return ZB_ERR_SHAPE;
    if (scaling == ZB_ROPE_PARTS && (!(original_len > 0.0) || !(low < high))) return ZB_ERR_SHAPE;
    if (scaling == ZB_ROPE_NTK && pairs < 2) return ZB_ERR_SHAPE;
    const double two_pi = 6.283185307179586476925286766559;
    if (scaling == ZB_ROPE_NTK) base *= pow(factor, static_cast<double>(pairs) / (pairs - 1));
    for (int i = 0; i < pairs; ++i) {
        double f = pow(base, -static_cast<double>(i) / pairs);
        if (scaling == ZB_ROPE_LINEAR) f /= factor;
        if (scaling == ZB_ROPE_PARTS) {
            const double rotations = original_len * f / two_pi;
            double keep = (rotations - low) / (high - low);
            keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
            f = (1.0 - keep) * f / factor + keep * f;
        }
        // f <= 1 radian: less than a sixth of a turn, far from the sign bit
        turns[i] = static_cast<int64_t>(llrint(f / two_pi * 0x1p64));
        if (radians) radians[i] = f;
    }
    if (magnitude) *magnitude = scaling == ZB_ROPE_PARTS ? static_cast<float>(0.1 * log(factor) + 1.0) : 1.f;
    return ZB_OK;
}

extern "C" zb_status zb_rope(const uint16_t* X, zb_rows x_rows, int32_t batch, int32_t heads, int64_t n_tokens,
                             int32_t head_dim, zb_rotation rot, uint16_t* Y, zb_rows y_rows, void* stream) {
    zb_status e = rope::check_sizes(batch, heads, 0, n_tokens, head_dim);
    if (e != ZB_OK) return e;
    if ((e = rope::check_rotation(rot)) != ZB_OK) return e;
    if (!rope::strides_ok(x_rows) || !rope::strides_ok(y_rows)) return ZB_ERR_ALIGN;
    if (!rope::disjoint(y_rows, batch, heads, n_tokens)) return ZB_ERR_SHAPE;
    if (!X || !Y) return ZB_ERR_NULL;
    if (!aligned16(X) || !aligned16(Y)) return ZB_ERR_ALIGN;
    DeviceInfo dev;
    if ((e = current_device(&dev)) != ZB_OK) return e;
    rope::Args a{};
    a.side[0] = {X, nullptr, Y, rope::view(x_rows), {}, rope::view(y_rows), nullptr, nullptr, nullptr, nullptr, heads, 0};
    a.tokens = static_cast<long long>(batch) * n_tokens;
    a.n = n_tokens;
    rope::put_rotation(a, rot);
    return rope::launch<false>(a, ZB_NORM_NONE, dev, static_cast<cudaStream_t>(stream));
}

namespace {
zb_status check_norm(const zb_qk_norm& norm, const zb_rotation& rot) {
    if (rot.inverse) return ZB_ERR_UNSUPPORTED;
    if (norm.kind < ZB_NORM_NONE || norm.kind > ZB_NORM_LAYER) return ZB_ERR_UNSUPPORTED;
    if (norm.kind != ZB_NORM_NONE && (!(norm.eps >= 0.f) || !(norm.eps < 1e30f))) return ZB_ERR_SHAPE;
    if (norm.kind != ZB_NORM_LAYER && (norm.bq || norm.bk)) return ZB_ERR_UNSUPPORTED;
    for (const float* p : {norm.wq, norm.wk, norm.bq, norm.bk})
        if (reinterpret_cast<uintptr_t>(p) & 3u) return ZB_ERR_ALIGN;
    return ZB_OK;
}
}  // namespace

extern "C" zb_status zb_qk_norm_rope(const uint16_t* Q, zb_rows q_rows, int32_t heads_q, const uint16_t* K,
                                     zb_rows k_rows, int32_t heads_k, int32_t batch, int64_t n_tokens,
                                     int32_t head_dim, zb_qk_norm norm, zb_rotation rot, uint16_t* Qo, uint16_t* Ko,
                                     void* stream) {
    zb_status e = rope::check_sizes(batch, heads_q, heads_k, n_tokens, head_dim);
    if (e != ZB_OK) return e;
    if ((e = rope::check_rotation(rot)) != ZB_OK) return e;
    if ((e = check_norm(norm, rot)) != ZB_OK) return e;
    if (!rope::strides_ok(q_rows) || (heads_k && !rope::strides_ok(k_rows))) return ZB_ERR_ALIGN;
    if (!Q || !Qo || (heads_k && (!K || !Ko))) return ZB_ERR_NULL;
    if (!aligned16(Q) || !aligned16(Qo) || (heads_k && (!aligned16(K) || !aligned16(Ko)))) return ZB_ERR_ALIGN;
    DeviceInfo dev;
    if ((e = current_device(&dev)) != ZB_OK) return e;
    rope::Args a{};
    a.side[0] = {Q, nullptr, Qo, rope::view(q_rows), {}, rope::packed(heads_q, n_tokens),
                 norm.wq, norm.bq, nullptr, nullptr, heads_q, 0};
    a.side[1] = {K, nullptr, Ko, rope::view(k_rows), {}, rope::packed(heads_k, n_tokens),
                 norm.wk, norm.bk, nullptr, nullptr, heads_k, 0};
    a.tokens = static_cast<long long>(batch) * n_tokens;
    a.n = n_tokens;
    a.eps = norm.eps;
    rope::put_rotation(a, rot);
    return rope::launch<false>(a, norm.kind, dev, static_cast<cudaStream_t>(stream));
}

extern "C" size_t zb_qk_norm_rope_backward_workspace_bytes(void) {
    return static_cast<size_t>(rope::MAX_CTAS) * 2 * rope::HD * sizeof(float);
}

extern "C" zb_status zb_qk_norm_rope_backward(const uint16_t* dQo, const uint16_t* dKo, const uint16_t* Q,
                                              zb_rows q_rows, int32_t heads_q, const uint16_t* K, zb_rows k_rows,
                                              int32_t heads_k, int32_t batch, int64_t n_tokens, int32_t head_dim,
                                              zb_qk_norm norm, zb_rotation rot, uint16_t* dQ, zb_rows dq_rows,
                                              uint16_t* dK, zb_rows dk_rows, float* dwq, float* dwk, float* dbq,
                                              float* dbk, void* ws, size_t ws_bytes, void* stream) {
    zb_status e = rope::check_sizes(batch, heads_q, heads_k, n_tokens, head_dim);
    if (e != ZB_OK) return e;
    if ((e = rope::check_rotation(rot)) != ZB_OK) return e;
    if ((e = check_norm(norm, rot)) != ZB_OK) return e;
    if (!rope::strides_ok(q_rows) || !rope::strides_ok(dq_rows) ||
        (heads_k && (!rope::strides_ok(k_rows) || !rope::strides_ok(dk_rows))))
        return ZB_ERR_ALIGN;
    if (!rope::disjoint(dq_rows, batch, heads_q, n_tokens) ||
        (heads_k && !rope::disjoint(dk_rows, batch, heads_k, n_tokens)))
        return ZB_ERR_SHAPE;
    if (!dQo || !Q || !dQ || (heads_k && (!dKo || !K || !dK))) return ZB_ERR_NULL;
    if (!aligned16(dQo) || !aligned16(Q) || !aligned16(dQ) ||
        (heads_k && (!aligned16(dKo) || !aligned16(K) || !aligned16(dK))))
        return ZB_ERR_ALIGN;
    if ((norm.kind == ZB_NORM_NONE && (dwq || dwk)) || (norm.kind != ZB_NORM_LAYER && (dbq || dbk)))
        return ZB_ERR_UNSUPPORTED;
    for (const float* p : {dwq, dwk, dbq, dbk})
        if (reinterpret_cast<uintptr_t>(p) & 3u) return ZB_ERR_ALIGN;
    if (!ws || ws_bytes < zb_qk_norm_rope_backward_workspace_bytes()) return ZB_ERR_WORKSPACE;
    if (!aligned16(ws)) return ZB_ERR_ALIGN;
    DeviceInfo dev;
    if ((e = current_device(&dev)) != ZB_OK) return e;
    rope::Args a{};
    a.side[0] = {Q, dQo, dQ, rope::view(q_rows), rope::packed(heads_q, n_tokens), rope::view(dq_rows),
                 norm.wq, nullptr, dwq, dbq, heads_q, 0};
    a.side[1] = {K, dKo, dK, rope::view(k_rows), rope::packed(heads_k, n_tokens), rope::view(dk_rows),
                 norm.wk, nullptr, heads_k ? dwk : nullptr, heads_k ? dbk : nullptr, heads_k, 0};
    a.tokens = static_cast<long long>(batch) * n_tokens;
    a.n = n_tokens;
    a.eps = norm.eps;
    rope::put_rotation(a, rot);
    a.partial = static_cast<float*>(ws);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    e = rope::launch<true>(a, norm.kind, dev, st);
    if (e != ZB_OK) return e;
    if (a.side[0].dw || a.side[0].db || a.side[1].dw || a.side[1].db) {
        return launch_behind(rope::reduce_kernel, dim3(8, 4), 256, st, static_cast<const float*>(a.partial), a);
    }
    return ZB_OK;
}
