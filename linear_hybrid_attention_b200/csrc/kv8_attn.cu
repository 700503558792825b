// Softmax attention over the 8-bit key/value cache for few query rows a head
// (decoding), and the join of partial results.
//
//   x_rj = scale q_r . code_j s_k[block of j],   p = softmax over the row's keys,
//   O_r = sum_j p_rj s_v[block of j] code_j,     weight of block b = sum of p over
//   its keys and the head's rows.
//
// Bound by the cache's bytes (128 a token): every byte is read once, with 17 to 32 rows a
// head twice (an item has at most 16).  Work is cut
// into chunks of 64 keys, laid end to end over all heads (and 16-row tiles of
// their queries); each warp takes an equal run of chunks, whatever the heads'
// lengths, the 12 warps of a CTA neighbouring ones.  Lengths are read on the
// device, so a captured graph serves all of them.  A warp streams its chunks
// through a ring of its own of STAGES bulk copies (4 KB of keys, 4 KB of values
// each) across the heads it meets, and writes what lies wholly in its run at once:
// the warps meet only at the end, where the CTA joins the parts of heads that
// several of them hold.  (Joining at every head's end instead cost a batch with
// some one-token sequences 3 us for each of them.)  Starting on a head costs a warp
// about as much as a chunk, so runs are equal in chunks and heads begun together.
// What several CTAs hold goes to the workspace, and the join kernel adds it up.
//
// The codes go to the matrix instruction as fp16, which holds both formats
// exactly; the scales stay in fp32 (s_k multiplies the logits, s_v the chunk's
// product).  Queries are scaled by a power of two per row to fp16's range.  Keys and
// features are the instruction's 16 rows and queries its 8 columns (S^T = K Q^T,
// O^T = V^T P^T, P^T by an 8 x 8 transpose between the two): 8 query rows then cost
// half of what they do as half-empty rows, and a code is unpacked once for 16.  The
// features and keys a lane holds are chosen so that it reads its 16 bytes of a key
// and its 8 bytes of four values in one piece each.
#include <cuda_runtime.h>

#include <atomic>

#include "kv8.cuh"

namespace zb {
namespace kv8 {

// Twelve warps of two stages, not eight of three: the ring holds as much (192 KB),
// and three warps a scheduler hide what two leave open (256 views, one token:
// 145 -> 130 us then; 117 with what came after).
constexpr int WARPS = 12;
constexpr int STAGES = 2;
constexpr int TILE = 16;                         // most query rows of an item (8 if there are no more)
constexpr uint32_t HALF_STAGE = CHUNK * HD;      // 4 KB of codes
// Sums of weights (up to 2^P_SHIFT a key) times values pass fp32 where values near the end
// of bf16's range meet many keys.  From the first value scale above VAST on, a part's sums
// are held times VAST_MUL (what that takes off values below 2^-62 is nothing beside those),
// and all parts leave theirs times O_UNIT: room for 2^18 keys of the largest weight and value.
constexpr float VAST = 0x1p64f, VAST_MUL = 0x1p-64f, O_UNIT = 0x1p-32f;

// A warp's part of an item that others hold parts of too (item -1: none).  Entry 2 w
// is the part that warp w's run starts with, in its row of part_o; entry 2 w + 1 the
// part it ends with, in its ring.
struct Piece {
    long long item;
    int from_start, to_end;      // it begins / ends the item
};

struct __align__(128) AttnSmem {
    uint8_t ring[WARPS][STAGES][2][HALF_STAGE];
    float m[2 * WARPS][TILE], l[2 * WARPS][TILE];
    Piece piece[2 * WARPS];
    uint64_t full[WARPS][STAGES];
    unsigned long long wsum[WARPS];
    long long start_before;
    int start_head;
    int abort_flag;
};

// Where a warp stands in its run: the current item and the chunks of it that fall
// into the run.  Runs are measured in units: an item has one for its start and one
// a chunk.
struct Cursor {
    int h, tile;
    int c, c1;            // next chunk, end of the item's part
    int c0;               // first chunk of the item's part
    int nc;               // chunks of the item
    long long len;        // tokens of the head
    long long left;       // units of the run after this part
};

ZB_DEVINL int chunks_of(long long len) { return static_cast<int>((len + CHUNK - 1) / CHUNK); }
// Units of a head.
ZB_DEVINL long long units_of(long long len, int tiles) {
    return len > 0 ? static_cast<long long>(chunks_of(len) + 1) * tiles : 0;
}

// NT: groups of 8 query rows an item has.  GK: 16-key steps that share a value
// scale (block / 16, at most 4).
template <int FMT, int NT, int GK>
__global__ void __launch_bounds__(WARPS * 32, 1) attn_kernel(const AttnArgs a) {
    constexpr int TR = 8 * NT;
    let_next_start();
    extern __shared__ uint8_t smem_raw[];
    AttnSmem& sm = *reinterpret_cast<AttnSmem*>(smem_raw);
    const int warp = warp_id(), lane = lane_id(), g = lane >> 2, c4 = lane & 3;
    const zb_kv8& c = a.c;
    const int B = c.block, shift = 31 - __clz(B);
    const long long cap = static_cast<long long>(c.slots) * B;
    constexpr int PIECES = 4 / GK;                  // blocks a chunk spans
    constexpr int PIECE_ROWS = CHUNK / PIECES;
    constexpr uint32_t PIECE_BYTES = PIECE_ROWS * HD;

    // ---- this CTA's run: the units of all heads, end to end -----------------
    const int per = (c.heads + WARPS * 32 - 1) / (WARPS * 32);
    const int ha = min(static_cast<int>(threadIdx.x) * per, c.heads), hb = min(ha + per, c.heads);
    long long mine = 0;
    for (int h = ha; h < hb; ++h) mine += units_of(head_len(a.lens, h, cap), a.tiles);
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) sm.wsum[warp] = incl;
    if (threadIdx.x == 0) sm.abort_flag = 0;
    if (lane == 0)
        for (int s = 0; s < STAGES; ++s) mbar_init(smem_addr(&sm.full[warp][s]), 1);
    fence_mbar_init();
    __syncthreads();
    long long total = 0, before = incl - mine;
    for (int w = 0; w < WARPS; ++w) {
        if (w < warp) before += sm.wsum[w];
        total += sm.wsum[w];
    }
    const long long ctas = min(static_cast<long long>(gridDim.x), total);
    if (blockIdx.x >= ctas) return;
    // (a 64-bit division is some hundred instructions, and the first copy waits for these)
    auto share = [&](unsigned i) -> long long {
        if (total < (1 << 24)) return static_cast<uint32_t>(total) * i / static_cast<uint32_t>(ctas);
        return total * i / ctas;
    };
    const long long at = share(blockIdx.x), end = share(blockIdx.x + 1);
    if (before <= at && at < before + mine) {
        long long b = before;
        for (int h = ha; h < hb; ++h) {
            const long long n = units_of(head_len(a.lens, h, cap), a.tiles);
            if (at < b + n) {
                sm.start_head = h;
                sm.start_before = b;
                break;
            }
            b += n;
        }
    }
    __syncthreads();

    auto open = [&](Cursor& k, int h, long long into, long long left) {
        // unit `into` of head h, `left` units to go in the run
        k.h = h;
        k.len = head_len(a.lens, h, cap);
        k.nc = chunks_of(k.len);
        k.tile = a.tiles == 1 ? 0 : static_cast<int>(into / (k.nc + 1));
        const int u = static_cast<int>(into - static_cast<long long>(k.tile) * (k.nc + 1));
        const int here = static_cast<int>(min(left, static_cast<long long>(k.nc + 1 - u)));
        k.c0 = max(u - 1, 0);
        k.c1 = u + here - 1;
        k.c = k.c0;
        k.left = left - here;
    };
    auto next_part = [&](Cursor& k) -> bool {       // the run's next item (a start without a chunk is none)
        do {
            if (k.left == 0) return false;
            int h = k.h, t = k.tile + 1;
            if (t == a.tiles) {
                t = 0;
                do ++h; while (head_len(a.lens, h, cap) == 0);
            }
            open(k, h, static_cast<long long>(t) * (chunks_of(head_len(a.lens, h, cap)) + 1), k.left);
        } while (k.c0 >= k.c1);
        return true;
    };
    // this warp's run within the CTA's, and the head it starts in
    auto part = [&](int w) -> long long {
        if (end - at < (1 << 24)) return at + static_cast<uint32_t>(end - at) * w / WARPS;
        return at + (end - at) * w / WARPS;
    };
    const long long wa = part(warp), wb = part(warp + 1);
    if (lane < 2) sm.piece[2 * warp + lane].item = -1;
    Cursor cur, iss;
    bool running = wa < wb;
    if (running) {
        int h = sm.start_head;
        long long b = sm.start_before;
        for (;; ++h) {
            const long long n = units_of(head_len(a.lens, h, cap), a.tiles);
            if (wa < b + n) break;
            b += n;
        }
        open(cur, h, wa - b, wb - wa);
        if (cur.c0 >= cur.c1) running = next_part(cur);
        iss = cur;
    }
    bool more = running;                             // the issue cursor stands on a chunk
    auto settle = [&]() {
        if (iss.c < iss.c1) return;
        more = next_part(iss);
        // the next item's queries, ahead of their use
        const int r = iss.tile * TR + lane;
        if (more && lane < TR && r < a.rows)
            asm volatile("prefetch.global.L1 [%0];" ::"l"(a.Q + (static_cast<long long>(iss.h) * a.rows + r) * HD));
    };

    const WaitCtx wc{a.status, &sm.abort_flag, a.timeout_ns};
    uint8_t(*ring)[2][HALF_STAGE] = sm.ring[warp];
    uint32_t issued = 0, used = 0;
    float ks_q[STAGES], vs_q[STAGES];                // scales of the chunks in the ring (lane: piece)
    for (int s = 0; s < STAGES; ++s) ks_q[s] = vs_q[s] = 0.f;
    float ks_new = 0.f, vs_new = 0.f;
    int entry = 0;                                   // table entry of the lane's piece of the next chunk to issue
    bool dead = false;
    auto fetch = [&]() {
        if (!more) return;
        const long long key = static_cast<long long>(iss.c) * CHUNK + lane * PIECE_ROWS;
        if (lane < PIECES && key < iss.len)
            entry = __ldg(c.table + static_cast<long long>(iss.h) * c.slots + (key >> shift));
    };
    fetch();

    // Start the copies of the issue cursor's chunk; its scales land in ks_new, vs_new.
    auto issue = [&]() {
        const long long key0 = static_cast<long long>(iss.c) * CHUNK;
        const int have = static_cast<int>((min(iss.len - key0, static_cast<long long>(CHUNK)) + PIECE_ROWS - 1) / PIECE_ROWS);
        const int s = issued % STAGES;
        const uint32_t bar = smem_addr(&sm.full[warp][s]);
        ks_new = vs_new = 0.f;
        if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(have) * 2 * PIECE_BYTES);
        __syncwarp();
        if (lane < have) {
            const long long key = key0 + lane * PIECE_ROWS;
            int slot = entry;
            if (slot < 0 || slot >= c.slots) {       // as slot_of
                flag_status(a.status, ZB_ERR_INDEX);
                slot = 0;
            }
            const long long blk = static_cast<long long>(iss.h) * c.slots + slot;
            const long long byte = (blk * B + (key & (B - 1))) * HD;
            bulk_load(smem_addr(&ring[s][0][lane * PIECE_BYTES]), c.k + byte, PIECE_BYTES, bar);
            bulk_load(smem_addr(&ring[s][1][lane * PIECE_BYTES]), c.v + byte, PIECE_BYTES, bar);
            ks_new = __ldg(c.k_scale + blk);
            vs_new = __ldg(c.v_scale + blk);
        }
        ++issued;
        ++iss.c;
        settle();
        fetch();
    };
#pragma unroll
    for (int s = 0; s < STAGES; ++s) {
        if (more) {
            issue();
            ks_q[s] = ks_new;
            vs_q[s] = vs_new;
        }
    }

    while (running) {
        // ---- one item's part of the run ------------------------------------
        const long long len = cur.len;
        const int row0 = cur.tile * TR, live_rows = min(TR, a.rows - row0);
        const uint16_t* Q = a.Q + (static_cast<long long>(cur.h) * a.rows + row0) * HD;
        uint32_t qb[NT][4][2];                       // row 8 n + g, features 16 c4 ..
        float qf[NT][2];                             // of the lane's columns: rows 8 n + 2 c4 + e
        long long lim[NT][2];                        // keys they see
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = 8 * n + g;
            uint4 w[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
            if (r < live_rows) {
                w[0] = __ldg(reinterpret_cast<const uint4*>(Q + r * HD) + c4 * 2);
                w[1] = __ldg(reinterpret_cast<const uint4*>(Q + r * HD) + c4 * 2 + 1);
            }
            const uint32_t ww[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) top = max(top, max((ww[i] & 0x7FFFu) << 16, ww[i] & 0x7FFF0000u));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // row largest to [2^14, 2^15): exact in fp16 down to 2^-28 of it, and to 2^-39 of it below
            const bool finite = top < 0x7F800000u;
            const int e = max(static_cast<int>(top >> 23) - 127, -100);
            const float up = finite ? __uint_as_float(static_cast<uint32_t>(14 - e + 127) << 23) : 0.f;
            // a row that is not finite has NaN logits throughout
            const float down = finite ? __uint_as_float(static_cast<uint32_t>(e - 14 + 127) << 23) * a.scale_log2
                                      : __uint_as_float(0x7FC00000u);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t v = ww[2 * s + i];
                    qb[n][s][i] = finite ? pack_f16x2(bf16_lo(v) * up, bf16_hi(v) * up) : 0u;
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                qf[n][i] = __shfl_sync(0xffffffffu, down, (2 * c4 + i) * 4);
                lim[n][i] = a.causal ? len - a.n_q + 1 + (row0 + 8 * n + 2 * c4 + i) % a.n_q : len;
            }
        }
        float o[NT][4][4];                           // features 8 g + 2 j + (0, 0, 1, 1), rows 8 n + 2 c4 + (0, 1, 0, 1)
        float m[NT][2], l[NT][2];
        float v_mul = 1.f;                           // of the sums: VAST_MUL once a value is vast
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int j = 0; j < 4; ++j) o[n][j][0] = o[n][j][1] = o[n][j][2] = o[n][j][3] = 0.f;
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.f;
        }

        for (; cur.c < cur.c1; ++cur.c) {
            const int st = used % STAGES;
            if (!dead && !mbar_wait_warp(smem_addr(&sm.full[warp][st]), (used / STAGES) & 1, wc)) dead = true;
            if (dead) break;                         // nothing more is issued; drained below
            ++used;
            const float ksl = ks_q[0], vsl = vs_q[0];
            const long long key0 = static_cast<long long>(cur.c) * CHUNK;
            const uint8_t* kc = ring[st][0];
            uint8_t* vc = ring[st][1];
            // keys of the chunk that each row sees: all of them but at a head's end
            int end[NT][2];
            bool edge = false;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    end[n][i] = static_cast<int>(max(min(lim[n][i] - key0, 64ll), 0ll));
                    edge |= end[n][i] < CHUNK;
                }
            }
            edge = __any_sync(0xffffffffu, edge);
            const int valid = static_cast<int>(min(len - key0, 64ll));
            if (valid < CHUNK) {
                // rows behind the last token: what the ring held before could be any code
                for (int i = valid * (HD / 8) + lane; i < CHUNK * HD / 8; i += 32)
                    reinterpret_cast<uint2*>(vc)[i] = make_uint2(0, 0);
                fence_proxy_async_smem();            // before a later copy into this stage
                __syncwarp();
            }
            // ---- logits: the instruction's row i of step t is key 16 t + 8 (i / 8) + 4 (i & 1) + i % 8 / 2
            const int mine = 4 * (g & 1) + (g >> 1);
            float x[NT][4][4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const uint4 w0 = *reinterpret_cast<const uint4*>(kc + (16 * t + mine) * HD + c4 * 16);
                const uint4 w1 = *reinterpret_cast<const uint4*>(kc + (16 * t + 8 + mine) * HD + c4 * 16);
                const uint32_t lo[4] = {w0.x, w0.y, w0.z, w0.w}, hi[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    uint32_t ka[4];
                    unpack4<FMT>(lo[s], ka[0], ka[2]);
                    unpack4<FMT>(hi[s], ka[1], ka[3]);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        if (s == 0) mma_f16_new(x[n][t], ka, qb[n][s][0], qb[n][s][1]);
                        else mma_f16(x[n][t], ka, qb[n][s][0], qb[n][s][1]);
                    }
                }
            }
            // ---- softmax over the chunk: x[n][t][2 b + i] is key 16 t + 8 b + mine, row 8 n + 2 c4 + i
            float ks[PIECES];
#pragma unroll
            for (int p = 0; p < PIECES; ++p) ks[p] = __shfl_sync(0xffffffffu, ksl, p);
            uint32_t pb[NT][4][2];
            float corr[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float mx = m[n][i];
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        const float f = ks[t / GK] * qf[n][i];
                        x[n][t][i] *= f;
                        x[n][t][2 + i] *= f;
                    }
                    if (edge) {
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            x[n][t][i] = 16 * t + mine < end[n][i] ? x[n][t][i] : -INFINITY;
                            x[n][t][2 + i] = 16 * t + 8 + mine < end[n][i] ? x[n][t][2 + i] : -INFINITY;
                        }
                    }
#pragma unroll
                    for (int t = 0; t < 4; ++t) mx = fmax3(mx, x[n][t][i], x[n][t][2 + i]);
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                    const float ref = mx == -INFINITY ? 0.f : mx - P_SHIFT;
                    corr[n][i] = m[n][i] == -INFINITY ? 0.f : ex2(m[n][i] - mx);
                    m[n][i] = mx;
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        x[n][t][i] = ex2(x[n][t][i] - ref);
                        x[n][t][2 + i] = ex2(x[n][t][2 + i] - ref);
                    }
                    float part[PIECES];              // the pieces' sums of this lane's keys
#pragma unroll
                    for (int p = 0; p < PIECES; ++p) {
                        part[p] = 0.f;
#pragma unroll
                        for (int t = p * GK; t < (p + 1) * GK; ++t) part[p] += x[n][t][i] + x[n][t][2 + i];
                    }
                    float sum = 0.f;
#pragma unroll
                    for (int p = 0; p < PIECES; ++p) sum += part[p];
                    l[n][i] = fmaf(l[n][i], corr[n][i], sum);
                    if (a.groups) {
                        const int r = 8 * n + 2 * c4 + i;
                        const long long grp0 = static_cast<long long>(cur.c) * PIECES;
#pragma unroll
                        for (int p = 0; p < PIECES; ++p) {
                            float s = part[p];
                            s += __shfl_xor_sync(0xffffffffu, s, 4);
                            s += __shfl_xor_sync(0xffffffffu, s, 8);
                            s += __shfl_xor_sync(0xffffffffu, s, 16);
                            if (g == 0 && r < live_rows && grp0 + p < a.groups)
                                a.gsum[(static_cast<long long>(cur.h) * a.groups + grp0 + p) * a.rows + row0 + r] =
                                    __log2f(s) + ref;
                        }
                    }
                }
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    pb[n][t][0] = transpose8(pack_f16x2(x[n][t][0], x[n][t][1]));
                    pb[n][t][1] = transpose8(pack_f16x2(x[n][t][2], x[n][t][3]));
                }
            }
            bool moved = vsl * v_mul > VAST;
#pragma unroll
            for (int n = 0; n < NT; ++n) moved |= corr[n][0] != 1.f || corr[n][1] != 1.f;
            if (__any_sync(0xffffffffu, moved)) {    // rare once the maxima settle
                float down = 1.f;
                if (__any_sync(0xffffffffu, vsl * v_mul > VAST)) v_mul = down = VAST_MUL;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[n][j][e] *= corr[n][e & 1] * down;
                    }
                }
            }
            // ---- values: row i of the instruction's tile j is feature 8 (i % 8) + 2 j + i / 8 ----
#pragma unroll
            for (int p = 0; p < PIECES; ++p) {
                float acc[NT][4][4];
#pragma unroll
                for (int t = p * GK; t < (p + 1) * GK; ++t) {
                    uint2 w[4];                      // keys 2 c4, 2 c4 + 1, 2 c4 + 8, 2 c4 + 9 of the step
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        w[i] = *reinterpret_cast<const uint2*>(vc + (16 * t + 4 * i + c4) * HD + g * 8);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t sel = j & 1 ? 0x7362u : 0x5140u;
                        uint32_t va[4];
                        unpack4<FMT>(j < 2 ? prmt(w[0].x, w[1].x, sel) : prmt(w[0].y, w[1].y, sel), va[0], va[1]);
                        unpack4<FMT>(j < 2 ? prmt(w[2].x, w[3].x, sel) : prmt(w[2].y, w[3].y, sel), va[2], va[3]);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            if (t == p * GK) mma_f16_new(acc[n][j], va, pb[n][t][0], pb[n][t][1]);
                            else mma_f16(acc[n][j], va, pb[n][t][0], pb[n][t][1]);
                        }
                    }
                }
                const float vs = __shfl_sync(0xffffffffu, vsl, p) * v_mul;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    // a row that sees nothing of the piece takes nothing of it, whatever its scale is
                    const float v[2] = {end[n][0] > p * PIECE_ROWS ? vs : 0.f, end[n][1] > p * PIECE_ROWS ? vs : 0.f};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[n][j][e] = fmaf(acc[n][j][e], v[e & 1], o[n][j][e]);
                    }
                }
            }
            __syncwarp();                            // the stage has been read
            // ---- next copy into the stage, and the scales move up ----------
#pragma unroll
            for (int s = 0; s + 1 < STAGES; ++s) {
                ks_q[s] = ks_q[s + 1];
                vs_q[s] = vs_q[s + 1];
            }
            ks_new = vs_new = 0.f;
            if (more) issue();
            ks_q[STAGES - 1] = ks_new;
            vs_q[STAGES - 1] = vs_new;
        }

        // ---- the part's result ---------------------------------------------
        const long long it = static_cast<long long>(cur.h) * a.tiles + cur.tile;
        const bool starts = cur.c0 == 0, ends = cur.c1 == cur.nc, last = cur.left == 0;
        const bool whole = starts && ends;           // nobody else's: the outputs themselves
        const long long run = it + blockIdx.x;
        // else the run goes on: to the warp's row of the workspace; or its ring, now idle, has room
        // (after a wait that gave up this may hold anything, and the status says so)
        const int e2 = 2 * warp + (last ? 1 : 0);
        float* dst = last ? reinterpret_cast<float*>(&ring[0][0][0])
                          : a.part_o + (a.runs + static_cast<long long>(blockIdx.x) * WARPS + warp) * TR * HD;
        const float unit = v_mul == 1.f ? O_UNIT : O_UNIT / VAST_MUL;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][j][e] *= unit;
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float L = l[n][i];
                L += __shfl_xor_sync(0xffffffffu, L, 4);
                L += __shfl_xor_sync(0xffffffffu, L, 8);
                L += __shfl_xor_sync(0xffffffffu, L, 16);
                const float M = m[n][i];
                const int r = 8 * n + 2 * c4 + i;
                if (whole) {
                    if (r < live_rows) {
                        const long long row = static_cast<long long>(cur.h) * a.rows + row0 + r;
                        const float inv = L == 0.f ? 0.f : 1.f / O_UNIT / L;   // no key: zeros; NaN stays
                        uint32_t w[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) w[j] = pack_bf16x2(o[n][j][i] * inv, o[n][j][2 + i] * inv);
                        reinterpret_cast<uint4*>(a.O + row * HD)[g] = make_uint4(w[0], w[1], w[2], w[3]);
                        if (g == 0) {
                            if (a.lse) a.lse[row] = L == 0.f ? -INFINITY : (M - P_SHIFT + log2f(L)) * LN2;
                            a.part_ml[run * TR + r] = make_float2(M, L);
                        }
                    }
                } else {
                    if (g == 0) {
                        sm.m[e2][r] = M;
                        sm.l[e2][r] = L;
                    }
                    float4* d = reinterpret_cast<float4*>(dst + r * HD + 8 * g);
                    d[0] = make_float4(o[n][0][i], o[n][0][2 + i], o[n][1][i], o[n][1][2 + i]);
                    d[1] = make_float4(o[n][2][i], o[n][2][2 + i], o[n][3][i], o[n][3][2 + i]);
                }
            }
        }
        if (lane == 0) {
            if (whole) a.item[it] = make_int2(static_cast<int>(run), 1);
            else sm.piece[e2] = Piece{it, starts, ends};
        }
        running = next_part(cur);
    }
    // copies of a warp that gave up are still writing its ring
    for (; used < issued; ++used) {
        const uint64_t t0 = globaltimer_ns(), limit = drain_timeout_ns(a.timeout_ns);
        while (!mbar_try_wait(smem_addr(&sm.full[warp][used % STAGES]), (used / STAGES) & 1))
            if (globaltimer_ns() - t0 > limit) break;
    }
    __threadfence_block();
    __syncthreads();
    // ---- parts of one item that neighbouring warps hold ---------------------
    for (int e0 = 0; e0 < 2 * WARPS;) {
        const long long it = sm.piece[e0].item;
        int e1 = e0 + 1, tail = e0;                  // entries of the item: [e0, e1), unused ones among them
        if (it >= 0)
            for (; e1 < 2 * WARPS && (sm.piece[e1].item == it || sm.piece[e1].item < 0); ++e1)
                if (sm.piece[e1].item == it) tail = e1;
        if (it >= 0) {
            const int h = a.tiles == 1 ? static_cast<int>(it) : static_cast<int>(it / a.tiles);
            const int row0 = static_cast<int>(it - static_cast<long long>(h) * a.tiles) * TR;
            const int live_rows = min(TR, a.rows - row0);
            const long long run = it + blockIdx.x;
            const bool whole = sm.piece[e0].from_start && sm.piece[tail].to_end;
            for (int i = threadIdx.x; i < live_rows * (HD / 4); i += WARPS * 32) {
                const int r = i / (HD / 4), q = i % (HD / 4);
                float M = -INFINITY, L = 0.f;
                for (int e = e0; e <= tail; ++e)
                    if (sm.piece[e].item == it) M = fmaxf(M, sm.m[e][r]);
                float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                for (int e = e0; e <= tail; ++e) {
                    const bool on = sm.piece[e].item == it;
                    const float f = !on || sm.m[e][r] == -INFINITY ? 0.f : ex2(sm.m[e][r] - M);
                    const float* src = (e & 1) ? reinterpret_cast<const float*>(&sm.ring[e >> 1][0][0][0])
                                               : a.part_o + (a.runs + static_cast<long long>(blockIdx.x) * WARPS + (e >> 1)) * TR * HD;
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (on) v = *reinterpret_cast<const float4*>(src + r * HD + 4 * q);
                    L = fmaf(on ? sm.l[e][r] : 0.f, f, L);
                    s.x = fmaf(v.x, f, s.x);
                    s.y = fmaf(v.y, f, s.y);
                    s.z = fmaf(v.z, f, s.z);
                    s.w = fmaf(v.w, f, s.w);
                }
                if (q == 0) a.part_ml[run * TR + r] = make_float2(M, L);
                if (whole) {
                    const float inv = L == 0.f ? 0.f : 1.f / O_UNIT / L;
                    const long long row = static_cast<long long>(h) * a.rows + row0 + r;
                    reinterpret_cast<uint2*>(a.O + row * HD)[q] =
                        make_uint2(pack_bf16x2(s.x * inv, s.y * inv), pack_bf16x2(s.z * inv, s.w * inv));
                    if (q == 0 && a.lse) a.lse[row] = L == 0.f ? -INFINITY : (M - P_SHIFT + log2f(L)) * LN2;
                } else {
                    reinterpret_cast<float4*>(a.part_o + (run * TR + r) * HD)[q] = s;
                }
            }
        }
        e0 = e1;
    }
    // the runs of the items that begin in this one: from this CTA to the one with the last chunk
    if (lane < 2 && sm.piece[2 * warp + lane].item >= 0 && sm.piece[2 * warp + lane].from_start) {
        const Piece p = sm.piece[2 * warp + lane];
        // a part that begins an item is the warp's last, and ends where its run ends
        const long long len = head_len(a.lens, static_cast<int>(p.item / a.tiles), cap);
        const long long final = wb - (cur.c1 - cur.c0) + chunks_of(len) - 1;   // the last chunk's unit
        const long long to = ((final + 1) * ctas - 1) / total;
        a.item[p.item] = make_int2(static_cast<int>(p.item + blockIdx.x), static_cast<int>(to - blockIdx.x + 1));
    }
}

// ------------------------------------------------------------------ join ----
// Adds up the partial runs of each item (rows without a token: zeros, -inf) and,
// with a.groups, turns the rows' group sums into the blocks' weight.  Grid: (heads,
// parts): every part works out the rows' log-sum-exp again, part 0 writes the
// outputs, and the blocks are shared out over the parts.
// Most rows a head that this kernel takes; kv8_tile.cu takes more.  This kernel / that one
// (us a call, int8 in blocks of 64): 16 heads of 43,968 tokens 74 / 67 at 33 to 48 rows
// and 96 / 67 at 64; 16 of 1,024 20 / 17 and 22 / 17; 64 of 1,024 23 / 24 and 28 / 25; but
// 256 of 300 26 / 40 and 33 / 41, 1,024 of 300 59 / 114 and 71 / 115: with many heads of a
// few hundred tokens each 128-row tile costs more than the second reading of the cache.  The
// lengths are on the device, so the rule does not follow them.
constexpr int FEW_ROWS = 32;
constexpr int JOIN_ROWS = FEW_ROWS;

// One row's runs added up, by the 16 threads (one half warp) that hold 4 of its
// features each: each thread reads the maximum and sum of one run in sixteen, so a
// row's runs cost two dependent reads, not two a run.
template <int TR>
ZB_DEVINL void add_runs(const AttnArgs& a, int2 it, int r, int q, bool outputs, float& M, float& L, float4& s) {
    const uint32_t half = 0xFFFFu << (lane_id() & 16);
    M = -INFINITY;
    for (int i = q; i < it.y; i += 16) M = fmaxf(M, a.part_ml[static_cast<long long>(it.x + i) * TR + r].x);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(half, M, o));
    L = 0.f;
    s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < it.y; i0 += 16) {
        float f = 0.f, l = 0.f;
        if (i0 + q < it.y) {
            const float2 ml = a.part_ml[static_cast<long long>(it.x + i0 + q) * TR + r];
            if (ml.y != 0.f) {
                f = ex2(ml.x - M);
                l = ml.y * f;
            }
        }
        const int n = min(16, it.y - i0);
        const float4* v = reinterpret_cast<const float4*>(a.part_o + (static_cast<long long>(it.x + i0) * TR + r) * HD) + q;
        const bool read = outputs && it.y > 1;
#pragma unroll 4
        for (int i = 0; i < n; ++i) {
            L += __shfl_sync(half, l, i, 16);
            const float fi = __shfl_sync(half, f, i, 16);
            if (read) {                              // (a part without weight too: its values may be NaN)
                const float4 w = v[static_cast<long long>(i) * TR * (HD / 4)];
                s.x = fmaf(w.x, fi, s.x);
                s.y = fmaf(w.y, fi, s.y);
                s.z = fmaf(w.z, fi, s.z);
                s.w = fmaf(w.w, fi, s.w);
            }
        }
    }
}

template <int TR>
__global__ void __launch_bounds__(256) join_kernel(const AttnArgs a) {
    __shared__ float lse2[JOIN_ROWS];
    const zb_kv8& c = a.c;
    const int h = blockIdx.x, part = blockIdx.y;
    const long long cap = static_cast<long long>(c.slots) * c.block;
    const long long len = head_len(a.lens, h, cap);
    const int blocks = static_cast<int>((len + c.block - 1) >> (31 - __clz(c.block)));
    const int per_block = c.block > CHUNK ? c.block / CHUNK : 1;
    const int live = static_cast<int>((len + min(c.block, CHUNK) - 1) / min(c.block, CHUNK));
    const int first = part * 256 + threadIdx.x;      // this thread's first block
    // what the attention kernel does not write is read while it still runs
    float* mass = nullptr;
    float old = 0.f;
    if (a.groups && first < blocks) {
        mass = c.mass + static_cast<long long>(h) * c.slots + slot_of(c, h, first, a.status);
        old = *mass;
    }
    wait_for_previous();
    // and the block's group sums while the rows' sums are added up
    constexpr int AHEAD = 16;
    const bool few = per_block * a.rows <= AHEAD;
    float gs[AHEAD];
    const int sums = a.groups && first < blocks ? (min((first + 1) * per_block, live) - first * per_block) * a.rows : 0;
    const float* gsum = a.gsum + (static_cast<long long>(h) * a.groups + static_cast<long long>(first) * per_block) * a.rows;
    if (few) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) gs[i] = i < sums ? gsum[i] : -INFINITY;
    }
    if (len == 0) {
        if (part) return;
        for (int i = threadIdx.x; i < a.rows * (HD / 8); i += 256) {
            const long long row = static_cast<long long>(h) * a.rows + i / (HD / 8);
            reinterpret_cast<uint4*>(a.O + row * HD)[i % (HD / 8)] = make_uint4(0, 0, 0, 0);
            if (i % (HD / 8) == 0 && a.lse) a.lse[row] = -INFINITY;
        }
        return;
    }
    // 16 threads a row, 4 features each
    const int r = threadIdx.x >> 4, q = threadIdx.x & 15;
    for (int r0 = 0; r0 < a.rows; r0 += 16) {
        const int row = r0 + r;
        if (row < a.rows) {
            const int2 it = a.item[static_cast<long long>(h) * a.tiles + row / TR];
            float M, L;
            float4 s;
            add_runs<TR>(a, it, row % TR, q, part == 0, M, L, s);
            const float t = L == 0.f ? -INFINITY : M - P_SHIFT + log2f(L);
            if (q == 0) lse2[row] = t;
            if (part == 0 && it.y > 1) {
                const float inv = L == 0.f ? 0.f : 1.f / O_UNIT / L;
                const long long out = static_cast<long long>(h) * a.rows + row;
                reinterpret_cast<uint2*>(a.O + out * HD)[q] =
                    make_uint2(pack_bf16x2(s.x * inv, s.y * inv), pack_bf16x2(s.z * inv, s.w * inv));
                if (q == 0 && a.lse) a.lse[out] = t * LN2;
            }
        }
    }
    if (!a.groups) return;
    __syncthreads();
    for (int b = first; b < blocks; b += gridDim.y * 256) {
        float s = 0.f;
        if (few && b == first) {
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                if (i >= sums) break;
                const float t = lse2[i % a.rows];
                if (t != -INFINITY) s += ex2(gs[i] - t);
            }
        } else {
            for (int k = b * per_block; k < min((b + 1) * per_block, live); ++k) {
                const float* gk = a.gsum + (static_cast<long long>(h) * a.groups + k) * a.rows;
                for (int i = 0; i < a.rows; ++i)
                    if (lse2[i] != -INFINITY) s += ex2(gk[i] - lse2[i]);
            }
        }
        if (b != first) {
            mass = c.mass + static_cast<long long>(h) * c.slots + slot_of(c, h, b, a.status);
            old = *mass;
        }
        *mass = old + s;
    }
}

// The weights for more rows (kv8_tile.cu): a warp a block, whose rows' sums are
// contiguous and read in eights.  A causal row's sums end where its keys do; only
// the last groups have rows that do not see them.
__global__ void __launch_bounds__(256) mass_kernel(const AttnArgs a) {
    wait_for_previous();
    const zb_kv8& c = a.c;
    const int h = blockIdx.x;
    const long long len = head_len(a.lens, h, static_cast<long long>(c.slots) * c.block);
    const int blocks = static_cast<int>((len + c.block - 1) >> (31 - __clz(c.block)));
    const int per_block = c.block > CHUNK ? c.block / CHUNK : 1;
    const int live = static_cast<int>((len + min(c.block, CHUNK) - 1) / min(c.block, CHUNK));
    const int size = min(c.block, CHUNK);
    const float* lse2 = a.lse2 + static_cast<long long>(h) * a.rows;
    for (int b = blockIdx.y * 8 + warp_id(); b < blocks; b += gridDim.y * 8) {
        float s = 0.f;
        for (int k = b * per_block; k < min((b + 1) * per_block, live); ++k) {
            const float* gs = a.gsum + (static_cast<long long>(h) * a.groups + k) * a.rows;
            const long long beyond = static_cast<long long>(k) * size - (len - a.n_q);   // of the first query's last key
            if (!a.causal || beyond <= 0) {
#pragma unroll 8
                for (int i = lane_id(); i < a.rows; i += 32) {
                    const float t = lse2[i], x = ex2(gs[i] - t);
                    if (t != -INFINITY) s += x;
                }
            } else {
                for (int i = lane_id(); i < a.rows; i += 32) {
                    const float t = lse2[i];
                    if (i % a.n_q >= beyond && t != -INFINITY) s += ex2(gs[i] - t);
                }
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane_id() == 0) {
            const int slot = slot_of(c, h, b, a.status);
            c.mass[static_cast<long long>(h) * c.slots + slot] += s;
        }
    }
}

// ------------------------------------------------------------------ host ----
struct Plan {
    bool few, pair;       // the streaming kernel; else 256 rows an item, or 128
    long long rows, tile, tiles, runs, groups;
    size_t o, ml, item, gsum, lse2, total;
};

size_t up256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

constexpr int MAX_SMS = 160;

Plan plan(const zb_kv8& c, int heads_q, long long n_q, int add_mass) {
    Plan p{};
    p.rows = static_cast<long long>(heads_q / c.heads) * n_q;
    p.few = p.rows <= FEW_ROWS;
    p.pair = p.rows > 128;
    p.tile = p.few ? (p.rows <= 8 ? 8 : TILE) : p.pair ? 256 : 128;
    p.tiles = (p.rows + p.tile - 1) / p.tile;
    // few rows: an item and a CTA, their sum is its run, and a row a warp; many: two places a CTA
    p.runs = p.few ? p.tiles * c.heads + MAX_SMS : 2 * MAX_SMS;
    p.groups = add_mass ? static_cast<long long>(c.slots) * (c.block > CHUNK ? c.block / CHUNK : 1) : 0;
    p.o = up256(static_cast<size_t>(p.runs + (p.few ? MAX_SMS * WARPS : 0)) * p.tile * HD * sizeof(float));
    p.ml = up256(static_cast<size_t>(p.runs) * p.tile * sizeof(float2));
    p.item = up256(static_cast<size_t>(p.tiles) * c.heads * sizeof(int2));
    p.gsum = up256(static_cast<size_t>(p.groups) * c.heads * p.rows * sizeof(float));
    p.lse2 = !p.few && add_mass ? up256(static_cast<size_t>(c.heads) * p.rows * sizeof(float)) : 0;
    p.total = p.o + p.ml + p.item + p.gsum + p.lse2;
    return p;
}

template <int FMT, int NT, int GK>
zb_status launch_attn(const AttnArgs& a, int ctas, cudaStream_t st) {
    auto* fn = attn_kernel<FMT, NT, GK>;
    static std::atomic<unsigned long long> done{0};  // devices that have the attribute set
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return ZB_ERR_CUDA;
    if (!(done.load(std::memory_order_relaxed) >> dev & 1)) {
        if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(AttnSmem)) != cudaSuccess)
            return ZB_ERR_CUDA;
        done.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    fn<<<ctas, WARPS * 32, sizeof(AttnSmem), st>>>(a);
    return cudaGetLastError() == cudaSuccess ? ZB_OK : ZB_ERR_CUDA;
}
template <int FMT, int NT>
zb_status launch_block(const AttnArgs& a, int ctas, cudaStream_t st) {
    switch (a.c.block) {
        case 16: return launch_attn<FMT, NT, 1>(a, ctas, st);
        case 32: return launch_attn<FMT, NT, 2>(a, ctas, st);
        default: return launch_attn<FMT, NT, 4>(a, ctas, st);
    }
}
template <int FMT>
zb_status launch_rows(const AttnArgs& a, int ctas, cudaStream_t st) {
    return a.rows <= 8 ? launch_block<FMT, 1>(a, ctas, st) : launch_block<FMT, 2>(a, ctas, st);
}

}  // namespace kv8
}  // namespace zb

using namespace zb;

extern "C" size_t zb_kv8_attn_workspace_bytes(zb_kv8 cache, int32_t heads_q, int64_t n_q, int32_t add_mass) {
    if (kv8::check_cache(cache, false) != ZB_OK || heads_q < 1 || heads_q % cache.heads || n_q < 1) return 0;
    return kv8::plan(cache, heads_q, n_q, add_mass).total;
}

extern "C" zb_status zb_kv8_attn(const uint16_t* Q, int32_t heads_q, int64_t n_q, zb_kv8 cache, const int32_t* lens,
                                 int32_t causal, float scale, uint16_t* O, float* lse, int32_t add_mass, void* ws,
                                 size_t ws_bytes, void* stream) {
    zb_status e = kv8::check_cache(cache, true);
    if (e != ZB_OK) return e;
    if (heads_q < 1 || heads_q % cache.heads || n_q < 1) return ZB_ERR_SHAPE;
    if (!(scale > 0.f) || !(scale <= 3.4e38f)) return ZB_ERR_SHAPE;
    if (n_q > 0x7FFFFFFFll || static_cast<long long>(heads_q / cache.heads) * n_q > 0x7FFFFFFFll) return ZB_ERR_UNSUPPORTED;
    if (!Q || !lens || !O || (add_mass && !cache.mass)) return ZB_ERR_NULL;
    if (!aligned16(Q) || !aligned16(O) || (reinterpret_cast<uintptr_t>(lens) & 3u) ||
        (reinterpret_cast<uintptr_t>(lse) & 3u))
        return ZB_ERR_ALIGN;
    const kv8::Plan p = kv8::plan(cache, heads_q, n_q, add_mass);
    // items, and a CTA's share of all items' tiles, in 32 bits
    const long long tiles = static_cast<long long>(cache.slots) * cache.block / 64 + 3;
    if (p.tiles * cache.heads > (1ll << 30) || p.tiles * cache.heads > (1ll << 37) / tiles) return ZB_ERR_UNSUPPORTED;
    if (!ws || ws_bytes < p.total) return ZB_ERR_WORKSPACE;
    if (!aligned16(ws)) return ZB_ERR_ALIGN;
    if (O == Q) return ZB_ERR_SHAPE;                 // a row's output is written while others' parts read its queries
    DeviceInfo dev;
    if ((e = current_device(&dev)) != ZB_OK) return e;
    if (dev.sm_count > kv8::MAX_SMS) return ZB_ERR_DEVICE;
    uint8_t* w = static_cast<uint8_t*>(ws);
    kv8::AttnArgs a{};
    a.c = cache;
    a.Q = Q;
    a.O = O;
    a.lse = lse;
    a.lens = lens;
    a.rows = static_cast<int>(p.rows);
    a.n_q = static_cast<int>(n_q);
    a.tiles = static_cast<int>(p.tiles);
    a.causal = causal != 0;
    a.scale_log2 = scale * kv8::LOG2E;
    a.runs = p.runs;
    a.groups = static_cast<int>(p.groups);
    a.part_o = reinterpret_cast<float*>(w);
    a.part_ml = reinterpret_cast<float2*>(w + p.o);
    a.item = reinterpret_cast<int2*>(w + p.o + p.ml);
    a.gsum = reinterpret_cast<float*>(w + p.o + p.ml + p.item);
    a.status = dev.status;
    a.timeout_ns = wait_timeout_ns();
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (!p.few) {
        if (add_mass) a.lse2 = reinterpret_cast<float*>(w + p.o + p.ml + p.item + p.gsum);
        e = kv8::launch_tiles(a, p.pair, dev.sm_count, st);
        if (e != ZB_OK || !add_mass) return e;
        const int parts = cache.slots / 8 + 1 < 512 ? cache.slots / 8 + 1 : 512;
        return launch_behind(kv8::mass_kernel, dim3(static_cast<unsigned>(cache.heads), static_cast<unsigned>(parts)),
                                  256, st, a);
    }
    e = cache.format == ZB_KV8_INT8 ? kv8::launch_rows<ZB_KV8_INT8>(a, dev.sm_count, st)
                                    : kv8::launch_rows<ZB_KV8_E4M3>(a, dev.sm_count, st);
    if (e != ZB_OK) return e;
    int parts = 1;
    if (a.groups) {
        parts = (cache.slots + 255) / 256;
        if (parts > 64) parts = 64;
    }
    const dim3 grid(static_cast<unsigned>(cache.heads), static_cast<unsigned>(parts));
    return launch_behind(p.tile == 8 ? kv8::join_kernel<8> : kv8::join_kernel<kv8::TILE>, grid, 256, st, a);
}
