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
// fraction of a turn, exact for any 32-bit position up to the rounding of T_i
// (2^-65 turns a position).  Its top 32 bits go to sincospi, so a far position
// costs no more and loses nothing against a near one.
//
// Both directions are HBM streams (a row in, a row out; backward two in, one
// out).  Four lanes hold a row, 16 features each, chosen so that both halves of
// every rotated pair lie in one thread: no exchange but two shuffles for the
// row's sums, and one kernel for both pair layouts.  A thread keeps the sines
// of its 8 pairs and runs over HEADS heads of its token with the loads of
// UNROLL rows in flight.
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
constexpr long long MAX_GX = 1 << 24;  // of a forward launch (a CTA then takes several groups of tokens)

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
    int heads, slices;             // heads, and CTAs along y that share them
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

ZB_DEVINL void unpack8(const uint4& v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
    }
}
ZB_DEVINL uint4 pack8(const float* f) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}
ZB_DEVINL float row_sum(float v) {   // over the row's four lanes
    v += __shfl_xor_sync(0xffffffffu, v, 1);
    return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

// Rotate the thread's 16 features by its 8 angles: pairs (f[j], f[8 + j]) in the
// half layout, (f[2j], f[2j + 1]) interleaved.
ZB_DEVINL void rotate(float* f, const float* c, const float* s, bool half, bool back) {
    if (half) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float sj = back ? -s[j] : s[j];
            const float a = f[j], b = f[8 + j];
            f[j] = a * c[j] - b * sj;
            f[8 + j] = b * c[j] + a * sj;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float sj = back ? -s[j] : s[j];
            const float a = f[2 * j], b = f[2 * j + 1];
            f[2 * j] = a * c[j] - b * sj;
            f[2 * j + 1] = b * c[j] + a * sj;
        }
    }
}

// Normalise in place; returns r.
template <int KIND>
ZB_DEVINL float normalise(float* f, float eps) {
    if (KIND == ZB_NORM_NONE) return 1.f;
    if (KIND == ZB_NORM_LAYER) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) m += f[i];
        m = row_sum(m) * (1.f / HD);
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] -= m;
    }
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) q += f[i] * f[i];
    const float r = rsqrtf(row_sum(q) * (1.f / HD) + eps);
#pragma unroll
    for (int i = 0; i < 16; ++i) f[i] *= r;
    return r;
}

template <int KIND, bool BACK, int UNROLL>
__global__ void __launch_bounds__(THREADS, 2) row_kernel(const Args a) {
    // y index -> tensor and its slice of heads
    const bool second = static_cast<int>(blockIdx.y) >= a.side[0].slices;
    const Side& sd = second ? a.side[1] : a.side[0];
    const int slice = second ? blockIdx.y - a.side[0].slices : blockIdx.y;
    const int h0 = static_cast<int>(static_cast<long long>(sd.heads) * slice / sd.slices);
    const int h1 = static_cast<int>(static_cast<long long>(sd.heads) * (slice + 1) / sd.slices);

    const int p = threadIdx.x & 3;
    const bool half = a.half != 0;
    const bool turned = p < a.rot / 16;
    const int pairs = a.rot / (2 * a.axes);          // of an axis
    int c0 = 2 * p, c1 = 2 * p + 1, axis = 0, pair0 = 0;
    if (turned) {
        if (half) {                                  // chunk c0 of an axis' part and its partner
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
    float w[16], bias[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int e = (i < 8 ? c0 * 8 : c1 * 8 - 8) + i;
        w[i] = (KIND != ZB_NORM_NONE && sd.w) ? __ldg(sd.w + e) : 1.f;
        if (!BACK) bias[i] = (KIND == ZB_NORM_LAYER && sd.bias) ? __ldg(sd.bias + e) : 0.f;
    }
    float dw[16], db[16];
    if (BACK) {
#pragma unroll
        for (int i = 0; i < 16; ++i) dw[i] = db[i] = 0.f;
    }

    const long long step = static_cast<long long>(gridDim.x) * TOK;
    for (long long base = static_cast<long long>(blockIdx.x) * TOK; base < a.tokens; base += step) {
        const long long u = base + (threadIdx.x >> 2);
        const bool live = u < a.tokens;              // dead lanes still join the shuffles
        const long long b = live ? u / a.n : 0, t = live ? u - b * a.n : 0;
        float cs[8], sn[8];
        if (turned && live) {
            const int pos = __ldg(a.pos + b * a.pos_b + axis * a.n + t);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const unsigned long long ph = static_cast<unsigned long long>(static_cast<long long>(pos)) *
                                              static_cast<unsigned long long>(__ldg(a.turns + pair0 + j));
                sincospif(static_cast<float>(static_cast<int>(ph >> 32)) * 0x1p-31f, &sn[j], &cs[j]);
                sn[j] *= a.mag;
                cs[j] *= a.mag;
            }
        }
        const uint16_t* x = sd.x + b * sd.xs.b + t * sd.xs.t;
        const uint16_t* g = BACK ? sd.g + b * sd.gs.b + t * sd.gs.t : nullptr;
        uint16_t* o = sd.out + b * sd.os.b + t * sd.os.t;
        for (int h = h0; h < h1; h += UNROLL) {
            uint4 xv[UNROLL][2], gv[UNROLL][2];
#pragma unroll
            for (int k = 0; k < UNROLL; ++k) {
                const bool on = live && h + k < h1;
                const uint4* r = reinterpret_cast<const uint4*>(x + (h + k) * sd.xs.h);
                xv[k][0] = on ? __ldg(r + c0) : make_uint4(0, 0, 0, 0);
                xv[k][1] = on ? __ldg(r + c1) : make_uint4(0, 0, 0, 0);
                if (BACK) {
                    const uint4* q = reinterpret_cast<const uint4*>(g + (h + k) * sd.gs.h);
                    gv[k][0] = on ? __ldg(q + c0) : make_uint4(0, 0, 0, 0);
                    gv[k][1] = on ? __ldg(q + c1) : make_uint4(0, 0, 0, 0);
                }
            }
#pragma unroll
            for (int k = 0; k < UNROLL; ++k) {
                float f[16], e[16];
                unpack8(xv[k][0], f);
                unpack8(xv[k][1], f + 8);
                const bool on = live && h + k < h1;
                // a row that is not there is zeros: with 1 for eps it stays zeros and adds
                // nothing to the sums
                const float r = normalise<KIND>(f, on ? a.eps : 1.f);
                if (BACK) {
                    unpack8(gv[k][0], e);
                    unpack8(gv[k][1], e + 8);
                    if (turned) rotate(e, cs, sn, half, true);
                    float m1 = 0.f, m0 = 0.f;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        if (KIND != ZB_NORM_NONE) dw[i] += e[i] * f[i];
                        if (KIND == ZB_NORM_LAYER) db[i] += e[i];
                        e[i] *= w[i];
                        m1 += e[i] * f[i];
                        m0 += e[i];
                    }
                    m1 = KIND != ZB_NORM_NONE ? row_sum(m1) * (1.f / HD) : 0.f;
                    m0 = KIND == ZB_NORM_LAYER ? row_sum(m0) * (1.f / HD) : 0.f;
#pragma unroll
                    for (int i = 0; i < 16; ++i) f[i] = r * (e[i] - m0 - f[i] * m1);
                } else {
                    if (KIND != ZB_NORM_NONE) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) f[i] = KIND == ZB_NORM_LAYER ? f[i] * w[i] + bias[i] : f[i] * w[i];
                    }
                    if (turned) rotate(f, cs, sn, half, a.inverse != 0);
                }
                if (on) {
                    uint4* q = reinterpret_cast<uint4*>(o + (h + k) * sd.os.h);
                    q[c0] = pack8(f);
                    q[c1] = pack8(f + 8);
                }
            }
        }
    }
    if (BACK && KIND != ZB_NORM_NONE) {
        // the CTA's sums: rows of a warp by shuffles, warps through shared memory in order
        __shared__ float red[THREADS / 32][2][HD];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                dw[i] += __shfl_xor_sync(0xffffffffu, dw[i], o);
                db[i] += __shfl_xor_sync(0xffffffffu, db[i], o);
            }
        }
        if (lane_id() < 4) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int e = (i < 8 ? c0 * 8 : c1 * 8 - 8) + i;
                red[warp_id()][0][e] = dw[i];
                red[warp_id()][1][e] = db[i];
            }
        }
        __syncthreads();
        if (threadIdx.x < 2 * HD) {
            float s = 0.f;
            for (int k = 0; k < THREADS / 32; ++k) s += (&red[k][0][0])[threadIdx.x];
            a.partial[(static_cast<long long>(blockIdx.y) * gridDim.x + blockIdx.x) * 2 * HD + threadIdx.x] = s;
        }
    }
}

// dw and db of one tensor from the CTAs' partial sums, in a fixed order, fp64.
// Grid: 8 blocks of 8 features x 2 (dw, db) x 2 (queries, keys).
__global__ void __launch_bounds__(256) reduce_kernel(const float* partial, int gx, Args a) {
    const int which = blockIdx.y & 1, tensor = blockIdx.y >> 1;
    float* out = which ? a.side[tensor].db : a.side[tensor].dw;
    if (!out) return;
    const int first = tensor ? a.side[0].slices * gx : 0;
    const int count = a.side[tensor].slices * gx;
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

// Heads are shared out over y so that the launch has about eight CTAs an SM
// where the tokens alone do not give them; every slice pays for the sines of
// its tokens again.
void slice_heads(Args& a, long long gx, int sms) {
    const int total = a.side[0].heads + a.side[1].heads;
    long long want = (8ll * sms + gx - 1) / gx;
    if (want > total) want = total;
    for (int s = 0; s < 2; ++s) {
        const int h = a.side[s].heads;
        long long k = (want * h + total - 1) / total;
        if (k > h) k = h;
        if (k > 16000) k = 16000;
        a.side[s].slices = h ? static_cast<int>(k < 1 ? 1 : k) : 0;
    }
}

template <bool BACK, int UNROLL>
zb_status launch(const Args& a, int kind, dim3 grid, cudaStream_t st) {
    switch (kind) {
        case ZB_NORM_RMS: row_kernel<ZB_NORM_RMS, BACK, UNROLL><<<grid, THREADS, 0, st>>>(a); break;
        case ZB_NORM_LAYER: row_kernel<ZB_NORM_LAYER, BACK, UNROLL><<<grid, THREADS, 0, st>>>(a); break;
        default: row_kernel<ZB_NORM_NONE, BACK, UNROLL><<<grid, THREADS, 0, st>>>(a); break;
    }
    return cudaGetLastError() == cudaSuccess ? ZB_OK : ZB_ERR_CUDA;
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
    long long gx = (a.tokens + rope::TOK - 1) / rope::TOK;
    if (gx > rope::MAX_GX) gx = rope::MAX_GX;
    rope::slice_heads(a, gx, dev.sm_count);
    return rope::launch<false, 4>(a, ZB_NORM_NONE, dim3(static_cast<unsigned>(gx), a.side[0].slices),
                                  static_cast<cudaStream_t>(stream));
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
    long long gx = (a.tokens + rope::TOK - 1) / rope::TOK;
    if (gx > rope::MAX_GX) gx = rope::MAX_GX;
    rope::slice_heads(a, gx, dev.sm_count);
    return rope::launch<false, 4>(a, norm.kind,
                                  dim3(static_cast<unsigned>(gx), a.side[0].slices + a.side[1].slices),
                                  static_cast<cudaStream_t>(stream));
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
    long long gx = (a.tokens + rope::TOK - 1) / rope::TOK;
    if (gx > 2ll * dev.sm_count) gx = 2ll * dev.sm_count;   // the CTAs that fit at once: few partial sums
    rope::slice_heads(a, gx, dev.sm_count);
    while (gx * (a.side[0].slices + a.side[1].slices) > rope::MAX_CTAS) {
        if (a.side[0].slices > 1 || a.side[1].slices > 1) {
            a.side[0].slices = (a.side[0].slices + 1) / 2;
            a.side[1].slices = (a.side[1].slices + 1) / 2;
        } else {
            gx = rope::MAX_CTAS / 2;
        }
    }
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    e = rope::launch<true, 2>(a, norm.kind, dim3(static_cast<unsigned>(gx), a.side[0].slices + a.side[1].slices), st);
    if (e != ZB_OK) return e;
    if (a.side[0].dw || a.side[0].db || a.side[1].dw || a.side[1].db) {
        rope::reduce_kernel<<<dim3(8, 4), 256, 0, st>>>(a.partial, static_cast<int>(gx), a);
        if (cudaGetLastError() != cudaSuccess) return ZB_ERR_CUDA;
    }
    return ZB_OK;
}
