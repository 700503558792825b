// Softmax attention over the 8-bit key/value cache for many query rows a head (a
// view's or a prompt's tokens at once), on the tcgen05 tensor cores.
//
// The same mathematics as kv8_attn.cu, bound by the exponentials and the
// instructions around them rather than by the cache's bytes.  One persistent CTA
// per SM, 512 threads:
//   warp 0        loader: bulk copies of a 128-key tile's codes into a ring
//   warp 3        the tiles' scales, up to eight tiles ahead
//   warps 1, 2    MMA issuers of row tiles ("slots") 0 and 1: S = Q K^T, O += P V
//   warps 4..7    converters (two for K, two for V): codes to fp16, exactly, in the
//                 128-byte-swizzle layout the MMAs read
//   warps 8..11, 12..15  softmax of slots 0 and 1, one thread a row
// Work items are 256 query rows of a head, 128 in each slot, both slots reading
// every converted tile (half the conversions a row); or 128 rows, where a head has
// no more, with the tiles dealt to the slots in turn.  Items are laid end to end in
// tiles, and each CTA takes an equal run, as in kv8_attn.cu; a causal item ends
// with its last row's last key.  Only the first and the last part of a run can be
// less than an item: those go to the workspace, to the CTA's two places there, and a
// second kernel adds them up.
//
// Scales.  s_k multiplies the logits, 64 or 16 columns at a time.  s_v = f 2^e, 1/2 <= f < 1:
// 2^(e - r) goes into the converted values, which it leaves exact, and f into the
// exponent, P = 2^(x + log2 f - m), so that O += P V needs no further product, and the
// softmax sum takes those columns' sum of P times 1 / f.  r is the part's reference for its
// values, the e of its first block that is not all zeros, raised where a block is 2^K_MAX
// larger; O is multiplied by 2^-(what it grew by) then.  So fp16 holds a weight relative to
// its row's largest weight, whatever the values' sizes.  (With all of s_v in the exponent it
// held weight times scale relative to the largest such product: a block of large values
// that had most of a row's weight took the bits of all others.)  m is the running maximum
// of x, raised only when it grows by more than RAISE.
//
// Measured at 16 heads x 1,374 rows (12 row tiles with the last) against 43,968 int8
// tokens: 465 us without weights, 532 TFLOP/s (510 us causal with weights and both
// joins); 1,280 rows 391 us, 589 TFLOP/s; 64 rows 70 us.  e4m3 in blocks of 16: 528 us,
// 756, 445 and 78.  Keeping the values' powers of two apart from the weights costs 2% of that
// without weights (e4m3 in blocks of 16: 12%), nothing with them.  A pair of 128 x 128 tiles takes about
// 3,500 cycles, 2,048 of them the MUFU's 256 exponentials a scheduler, the tensor
// pipe's some 1,050; what is left is a warp's own chain (read S, maximum, write P, and
// waits of some 150 cycles each even where the phase is there: answering them by one
// vote took 507 us to 462), which the other slot's warp covers only in part.  Also
// built, and slower by 2 to 20%: three slots of 64 keys; four slots of 64 keys with P
// in S's columns; the two slots' exponentials taking turns (a hand-over costs what it
// saves); P V in halves under the other half's exponentials.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <type_traits>

#include "kv8.cuh"

namespace zb {
namespace kv8 {
namespace {

constexpr int BM = 128, BN = 128;
constexpr int THREADS = 512;
constexpr int RAW = 3, K16 = 3, V16 = 3, SC = 8;   // ring stages
constexpr uint32_t RAW_BYTES = BN * HD;            // 8 KB of codes
constexpr uint32_t TILE_BYTES = BN * HD * 2;       // 16 KB of fp16
constexpr uint32_t TMEM_COLS = 512, SLOT_COLS = 256, TM_S = 0, TM_P = 128, TM_O = 192;
constexpr uint32_t SLEEP_NS = 20000;
// 128 threads each of roles and converters, 256 of softmax; adds up to the launch's 512 x 128
constexpr int LAUNCH_REGS = 128, ROLE_REGS = 64, CONVERT_REGS = 96, SOFTMAX_REGS = 176;
static_assert(128 * (ROLE_REGS + CONVERT_REGS) + 256 * SOFTMAX_REGS == THREADS * LAUNCH_REGS, "register split");
// P is at most 2^(SHIFT + RAISE) in fp16, and a row's largest weight at least 2^(SHIFT - 1):
// weights are rounded to 2^-11 of themselves down to 2^-(SHIFT + 13) of the largest, to
// 2^-(SHIFT + 24) of it below.
constexpr float SHIFT = 7.f, RAISE = 8.f;
// Powers of two that a format's codes can be multiplied by in fp16: up to the largest value,
// and down to where the smallest step of a code is fp16's smallest number.  (1152 as well,
// which the conversion of int8 multiplies.)  Scales below K_MIN take up to K_REST of what is
// missing off the weights, where fp16 then loses bits; a block below that counts as zeros.
template <int FMT>
constexpr int K_MAX = FMT == ZB_KV8_INT8 ? 5 : 7;
template <int FMT>
constexpr int K_MIN = FMT == ZB_KV8_INT8 ? -24 : -15;
constexpr int K_REST = 16;
constexpr int NO_REF = -96;       // the smallest reference, and that of a part without values yet
ZB_DEVINL uint32_t ref_word(int ref) { return static_cast<uint32_t>(ref + 256) << 8; }
ZB_DEVINL int word_ref(uint32_t word) { return static_cast<int>(word >> 8) - 256; }

struct __align__(1024) TileSmem {
    uint8_t q[2][TILE_BYTES];
    uint8_t k16[K16][TILE_BYTES];
    uint8_t v16[V16][TILE_BYTES];
    uint8_t raw[RAW][2][RAW_BYTES];
    float4 other[HD / 4][BM];         // slot 1's sums where it shares slot 0's rows
    float4 other_ml[BM];              // maximum, sum, what the sums are to be multiplied by
    float4 sc[SC][8];                 // s_k, log2 f, 1 / f of 64 or 16 keys
    uint32_t v_mul[SC][8];            // the power of two of their values, a pair of fp16
    uint32_t sc_word[SC];             // bit g: s_v of group g is not finite; above: the reference of the values
    uint64_t raw_full[RAW], raw_empty[RAW];
    uint64_t k_full[K16], k_empty[K16], v_full[V16], v_empty[V16];
    uint64_t sc_full[SC], sc_empty[SC];
    uint64_t other_full, other_empty;
    uint64_t q_full[2], s_full[2], s_free[2], p_full[2], p_free[2], o_free[2], drain[2];
    unsigned long long wsum[THREADS / 32];
    long long start_before;
    int start_item;
    uint32_t tmem_base;
    int abort_flag;
};

template <int N>
ZB_DEVINL void reg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
ZB_DEVINL void reg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// 32 lanes x consecutive 32-bit columns, moved and waited for in one piece: with the wait
// apart, tying the registers to it costs a move each.
ZB_DEVINL void tmem_load(uint32_t taddr, uint32_t (&r)[64]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%64];\n\t"
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%65];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(taddr), "r"(taddr + 32)
        : "memory");
}
ZB_DEVINL void tmem_store(uint32_t taddr, const uint32_t (&r)[64]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33};\n\t"
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%1], {%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63,%64,%65};\n\t"
        "tcgen05.wait::st.sync.aligned;" ::"r"(taddr), "r"(taddr + 32), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(r[32]), "r"(r[33]), "r"(r[34]), "r"(r[35]), "r"(r[36]), "r"(r[37]), "r"(r[38]), "r"(r[39]), "r"(r[40]), "r"(r[41]), "r"(r[42]), "r"(r[43]), "r"(r[44]), "r"(r[45]), "r"(r[46]), "r"(r[47]), "r"(r[48]), "r"(r[49]), "r"(r[50]), "r"(r[51]), "r"(r[52]), "r"(r[53]), "r"(r[54]), "r"(r[55]), "r"(r[56]), "r"(r[57]), "r"(r[58]), "r"(r[59]), "r"(r[60]), "r"(r[61]), "r"(r[62]), "r"(r[63])
        : "memory");
}
ZB_DEVINL void tmem_store(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n\t"
        "tcgen05.wait::st.sync.aligned;" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

// 2^n of n <= 127 (0 below -126).
ZB_DEVINL float pow2(int n) { return n < -126 ? 0.f : __uint_as_float(static_cast<uint32_t>(n + 127) << 23); }

// mbar_wait_warp for phases that cannot come round again before this warp arrives: most are
// there already, and then one vote answers, without a branch that lanes could part at.
ZB_DEVINL bool wait_warp(uint32_t bar, uint32_t parity, const WaitCtx& w) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return mbar_wait_warp(bar, parity, w);
}
ZB_DEVINL bool wait_warp(uint32_t bar0, uint32_t parity0, uint32_t bar1, uint32_t parity1, const WaitCtx& w) {
    const bool first = mbar_try_wait(bar0, parity0), second = mbar_try_wait(bar1, parity1);
    if (__all_sync(0xffffffffu, first && second)) return true;
    return mbar_wait_warp(bar0, parity0, w) && mbar_wait_warp(bar1, parity1, w);
}

// Instruction descriptor: fp16 A and B, fp32 accumulator (b_mn: B stored along N).
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int b_mn) {
    return (1u << 4) | (static_cast<uint32_t>(b_mn) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
           (static_cast<uint32_t>(M >> 4) << 24);
}

// Tiles of an item: those its last-reaching row sees.
ZB_DEVINL int item_tiles(const AttnArgs& a, int len, int tile, int item_rows) {
    if (a.causal) {
        const int r0 = tile * item_rows, r1 = min(r0 + item_rows, a.rows) - 1;
        const int reach = r0 / a.n_q == r1 / a.n_q ? r1 % a.n_q : a.n_q - 1;
        len = min(len, max(len - a.n_q + 1 + reach, 0));
    }
    return static_cast<int>((static_cast<unsigned>(len) + BN - 1) / BN);
}

// Units of an item in the runs: two for its start (Q, and a pipeline that runs
// empty) and one a tile.
constexpr int START = 2;
ZB_DEVINL int item_units(int tiles) { return tiles ? tiles + START : 0; }

// The parts of items that make up a CTA's run, in order; every role walks them.
// The host refuses calls whose runs could pass 32 bits.
struct Walk {
    int h, tile, len;
    int c0, c1, nc;           // the part's tiles, the item's
    int left;                 // units of the run after this part
};

template <bool PAIR>
struct Items {
    static constexpr int ROWS = PAIR ? 256 : 128;
    const AttnArgs& a;
    int cap;
    ZB_DEVINL int len(int h) const { return static_cast<int>(head_len(a.lens, h, cap)); }
    ZB_DEVINL void load(Walk& w, int into, int left) const {
        w.len = len(w.h);
        w.nc = item_tiles(a, w.len, w.tile, ROWS);
        const int here = min(left, item_units(w.nc) - into);
        w.c0 = max(into - START, 0);
        w.c1 = max(into + here - START, 0);
        w.left = left - here;
    }
    // To the next part with a tile in it; false at the run's end.
    ZB_DEVINL bool next(Walk& w) const {
        do {
            if (w.left <= 0) return false;
            do {
                if (++w.tile == a.tiles) {
                    w.tile = 0;
                    ++w.h;
                }
            } while (item_tiles(a, len(w.h), w.tile, ROWS) == 0);
            load(w, 0, w.left);
        } while (w.c0 >= w.c1);
        return true;
    }
    ZB_DEVINL long long index(const Walk& w) const { return static_cast<long long>(w.h) * a.tiles + w.tile; }
};

// A place in a ring of N stages.
template <int N>
struct Ring {
    int st = 0;
    uint32_t ph = 0;
    ZB_DEVINL void step() {
        if (++st == N) {
            st = 0;
            ph ^= 1u;
        }
    }
    ZB_DEVINL void back() {
        if (--st < 0) {
            st = N - 1;
            ph ^= 1u;
        }
    }
};

// G: scales a tile has (2 for blocks of 64 and 128, 8 for smaller ones).
template <int FMT, bool PAIR, bool MASS, int G>
__global__ void __launch_bounds__(THREADS, 1) tile_kernel(const AttnArgs a) {
    let_next_start();
    extern __shared__ uint8_t smem_raw[];
    TileSmem& sm = *reinterpret_cast<TileSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = warp_id(), lane = lane_id();
    const zb_kv8& c = a.c;
    const int B = c.block, shift = 31 - __clz(B);
    const Items<PAIR> items{a, c.slots * B};
    const WaitCtx wc{a.status, &sm.abort_flag, a.timeout_ns};

    // ---- this CTA's run ------------------------------------------------------
    const int n_items = c.heads * a.tiles;
    const int per = (n_items + THREADS - 1) / THREADS;
    const int ia = static_cast<int>(min(static_cast<long long>(threadIdx.x) * per, static_cast<long long>(n_items)));
    const int ib = min(ia + per, n_items);
    auto units = [&](int i) { return item_units(item_tiles(a, items.len(i / a.tiles), i % a.tiles, Items<PAIR>::ROWS)); };
    long long mine = 0;
    for (int i = ia; i < ib; ++i) mine += units(i);
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) sm.wsum[warp] = incl;
    if (threadIdx.x == 0) {
        sm.abort_flag = 0;
        for (int i = 0; i < RAW; ++i) {
            mbar_init(smem_addr(&sm.raw_full[i]), 1);
            mbar_init(smem_addr(&sm.raw_empty[i]), 4);
        }
        for (int i = 0; i < K16; ++i) {
            mbar_init(smem_addr(&sm.k_full[i]), 2);
            mbar_init(smem_addr(&sm.k_empty[i]), PAIR ? 2 : 1);
        }
        for (int i = 0; i < V16; ++i) {
            mbar_init(smem_addr(&sm.v_full[i]), 2);
            mbar_init(smem_addr(&sm.v_empty[i]), PAIR ? 2 : 1);
        }
        for (int i = 0; i < SC; ++i) {
            mbar_init(smem_addr(&sm.sc_full[i]), 1);
            mbar_init(smem_addr(&sm.sc_empty[i]), (PAIR ? 8 : 4) + 2);   // softmax warps, and those that convert V
        }
        mbar_init(smem_addr(&sm.other_full), 128);
        mbar_init(smem_addr(&sm.other_empty), 128);
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_addr(&sm.q_full[s]), 128);
            mbar_init(smem_addr(&sm.s_full[s]), 1);
            mbar_init(smem_addr(&sm.s_free[s]), 128);
            mbar_init(smem_addr(&sm.p_full[s]), 128);
            mbar_init(smem_addr(&sm.p_free[s]), 1);
            mbar_init(smem_addr(&sm.o_free[s]), 128);
            mbar_init(smem_addr(&sm.drain[s]), 1);
        }
        fence_mbar_init();
    }
    __syncthreads();
    long long total = 0, before = incl - mine;
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += sm.wsum[w];
        total += sm.wsum[w];
    }
    const long long ctas = min(static_cast<long long>(gridDim.x), total);
    if (blockIdx.x >= ctas) return;
    const long long at = total * blockIdx.x / ctas, end = total * (blockIdx.x + 1) / ctas;
    if (before <= at && at < before + mine) {
        long long b = before;
        for (int i = ia; i < ib; ++i) {
            const int n = units(i);
            if (at < b + n) {
                sm.start_item = i;
                sm.start_before = b;
                break;
            }
            b += n;
        }
    }
    if (warp == 1) tmem_alloc(smem_addr(&sm.tmem_base), TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    Walk walk;
    walk.h = sm.start_item / a.tiles;
    walk.tile = sm.start_item % a.tiles;
    items.load(walk, static_cast<int>(at - sm.start_before), static_cast<int>(end - at));
    bool running = walk.c0 < walk.c1 || items.next(walk);

    if (warp < 4) {
        reg_dec<ROLE_REGS>();
        if (warp == 0) {
            // ==================================================== loader ====
            const int piece_rows = min(B, BN);
            const uint32_t piece_bytes = static_cast<uint32_t>(piece_rows) * HD;
            Ring<RAW> raw;
            int issued = 0;
            bool ok = true;
            for (; running && ok; running = items.next(walk)) {
                for (int t = walk.c0; t < walk.c1; ++t) {
                    const int key0 = t * BN;
                    const int have = (min(walk.len - key0, BN) + piece_rows - 1) / piece_rows;
                    int slot = 0;
                    if (lane < have) slot = slot_of(c, walk.h, (key0 + lane * piece_rows) >> shift, a.status);
                    if (!(ok = wait_warp(smem_addr(&sm.raw_empty[raw.st]), raw.ph ^ 1u, wc))) break;
                    const uint32_t bar = smem_addr(&sm.raw_full[raw.st]);
                    if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(have) * 2 * piece_bytes);
                    __syncwarp();
                    if (lane < have) {
                        const long long byte = ((static_cast<long long>(walk.h) * c.slots + slot) * B +
                                                ((key0 + lane * piece_rows) & (B - 1))) * HD;
                        bulk_load(smem_addr(&sm.raw[raw.st][0][lane * piece_bytes]), c.k + byte, piece_bytes, bar);
                        bulk_load(smem_addr(&sm.raw[raw.st][1][lane * piece_bytes]), c.v + byte, piece_bytes, bar);
                    }
                    raw.step();
                    ++issued;
                }
            }
            // copies in flight still write the ring
            volatile int no_abort = 0;
            const WaitCtx w2{a.status, &no_abort, drain_timeout_ns(a.timeout_ns)};
            for (int i = 0; i < min(issued, RAW); ++i) {       // back from the newest
                raw.back();
                mbar_wait(smem_addr(&sm.raw_full[raw.st]), raw.ph, w2);
            }
        } else if (warp < 3) {
            // ================================================ MMA issuer ====
            const int s = warp - 1;
            if (lane == 0) {
                constexpr uint32_t IDESC_QK = idesc_f16(BM, BN, 0), IDESC_PV = idesc_f16(BM, HD, 1);
                const uint32_t s_tmem = tmem + s * SLOT_COLS + TM_S, p_tmem = tmem + s * SLOT_COLS + TM_P;
                const uint32_t o_tmem = tmem + s * SLOT_COLS + TM_O;
                Ring<K16> kr;              // this slot's next tile (a slot of its own rows skips the other's)
                Ring<V16> vr;
                uint32_t g = 0, part = 0;  // this slot's steps and parts so far
                bool ok = true;
                constexpr int STEP = PAIR ? 1 : 2;
                const uint64_t qd = sdesc_sw128(smem_addr(sm.q[s]), 16, 1024);
                for (; running && ok; running = items.next(walk)) {
                    const int n = walk.c1 - walk.c0;
                    const int j0 = PAIR ? 0 : s;
                    if (!PAIR && s) {
                        kr.step();
                        vr.step();
                    }
                    if (j0 < n) {
                        if (!(ok = mbar_wait_sleep(smem_addr(&sm.q_full[s]), part & 1, wc, SLEEP_NS))) break;
                        auto issue_qk = [&](uint32_t step) -> bool {
                            if (!mbar_wait_sleep(smem_addr(&sm.k_full[kr.st]), kr.ph, wc, SLEEP_NS)) return false;
                            if (!mbar_wait_sleep(smem_addr(&sm.s_free[s]), (step & 1) ^ 1, wc, SLEEP_NS)) return false;
                            tc_fence_after();
                            const uint64_t kd = sdesc_sw128(smem_addr(sm.k16[kr.st]), 16, 1024);
#pragma unroll
                            for (int kk = 0; kk < HD / 16; ++kk) umma_ss(s_tmem, qd + kk * 2, kd + kk * 2, IDESC_QK, kk > 0 ? 1u : 0u);
                            umma_commit(smem_addr(&sm.s_full[s]));
                            umma_commit(smem_addr(&sm.k_empty[kr.st]));
                            kr.step();
                            if (!PAIR) kr.step();
                            return true;
                        };
                        if (!(ok = issue_qk(g))) break;
                        for (int j = j0; j < n; j += STEP, ++g) {
                            if (j + STEP < n && !(ok = issue_qk(g + 1))) break;
                            if (!(ok = mbar_wait_sleep(smem_addr(&sm.v_full[vr.st]), vr.ph, wc, SLEEP_NS))) break;
                            if (j == j0 && !(ok = mbar_wait_sleep(smem_addr(&sm.o_free[s]), (part & 1) ^ 1, wc, SLEEP_NS))) break;
                            if (!(ok = mbar_wait_sleep(smem_addr(&sm.p_full[s]), g & 1, wc, SLEEP_NS))) break;
                            tc_fence_after();
                            const uint64_t vd = sdesc_sw128(smem_addr(sm.v16[vr.st]), 0, 1024);
#pragma unroll
                            for (int kk = 0; kk < BN / 16; ++kk)
                                umma_ts(o_tmem, p_tmem + kk * 8, vd + kk * 128, IDESC_PV, (j > j0 || kk > 0) ? 1u : 0u);
                            umma_commit(smem_addr(&sm.v_empty[vr.st]));
                            umma_commit(smem_addr(&sm.p_free[s]));
                            vr.step();
                            if (!PAIR) vr.step();
                        }
                        if (!ok) break;
                        ++part;
                    }
                    if (!PAIR) {           // to the next part's first tile (each slot has gone past its last by two)
                        const int over = j0 < n ? ((n - j0 + 1) / 2) * 2 + j0 - n : j0 - n;
                        for (int i = 0; i < over; ++i) {
                            kr.back();
                            vr.back();
                        }
                    }
                }
                // no MMA of this thread may still run when TMEM is released
                umma_commit(smem_addr(&sm.drain[s]));
                volatile int no_abort = 0;
                const WaitCtx w2{a.status, &no_abort, drain_timeout_ns(a.timeout_ns)};
                mbar_wait(smem_addr(&sm.drain[s]), 0, w2);
            }
        } else {
            // ==================================================== scales ====
            constexpr int AHEAD = 32 / G;                      // tiles whose scales the lanes read at once
            constexpr int KEYS = BN / G;
            Ring<SC> sc;
            bool ok = true;
            for (int part = 0; running; running = items.next(walk), ++part) {
                int ref = NO_REF;
                auto fetch = [&](int t, float& ks, float& vs) {
                    const long long key = static_cast<long long>(t) * BN + lane * KEYS;   // (t + lane / G, group lane % G)
                    ks = vs = 0.f;
                    if (t + lane / G < walk.c1 && key < walk.len) {
                        const long long blk = static_cast<long long>(walk.h) * c.slots + slot_of(c, walk.h, key >> shift, a.status);
                        ks = __ldg(c.k_scale + blk);
                        vs = __ldg(c.v_scale + blk);
                    }
                };
                float ks = 0.f, vs = 0.f, ks_next = 0.f, vs_next = 0.f;
                if (ok) fetch(walk.c0, ks, vs);
                for (int t0 = walk.c0; t0 < walk.c1 && ok; t0 += AHEAD) {
                    if (t0 + AHEAD < walk.c1) fetch(t0 + AHEAD, ks_next, vs_next);
                    const bool bad = !(fabsf(vs) <= 3.4e38f), some = !bad && vs > 0.f;
                    const uint32_t nan = __ballot_sync(0xffffffffu, bad);
                    const int e = static_cast<int>(__float_as_uint(vs) >> 23) - 126;   // subnormal: -126
                    const float frac = e > 2 ? vs * 0.25f * pow2(2 - e) : vs * pow2(-e);
                    int top = some ? min(max(e, NO_REF), 127) : NO_REF;   // of the lane's tile; 2^top is a number
#pragma unroll
                    for (int o = 1; o < G; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                    const int n = min(AHEAD, walk.c1 - t0);
                    for (int i = 0; i < n; ++i) {
                        const int now = __shfl_sync(0xffffffffu, top, i * G);
                        if (t0 + i == walk.c0 || now > ref + K_MAX<FMT>) ref = now;
                        if (!(ok = wait_warp(smem_addr(&sm.sc_empty[sc.st]), sc.ph ^ 1u, wc))) break;
                        if (lane / G == i) {
                            const int k = max(e - ref, K_MIN<FMT>), rest = e - ref - k;
                            // Zeros, and values that 2^-40 of the largest (e4m3: 2^-31) is more than: no values.  A
                            // scale that is not finite has a path of its own (nan_value).
                            const bool on = some && rest >= -K_REST;
                            const float lv = on ? log2f(frac) + static_cast<float>(rest) : 0.f;
                            // 1 in the place of a key scale of 0 keeps -inf * s_k what it is
                            sm.sc[sc.st][lane % G] = make_float4(ks == 0.f ? 1.f : ks, lv, ex2(-lv), 0.f);
                            const uint32_t mul = !on ? 0u : k >= -14 ? static_cast<uint32_t>(k + 15) << 10 : 1u << (k + 24);
                            sm.v_mul[sc.st][lane % G] = mul << 16 | mul;
                        }
                        if (lane == 0) sm.sc_word[sc.st] = ref_word(ref) | (nan >> (i * G) & ((1u << G) - 1u));
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_addr(&sm.sc_full[sc.st]));
                        sc.step();
                    }
                    ks = ks_next;
                    vs = vs_next;
                }
                // (behind the scales, which others wait for; and after a wait that gave up too: the join reads it)
                if (walk.c0 == 0 && lane == 0) {
                    // where the join finds the partial results of an item that begins in this run: this CTA's
                    // place and how many CTAs hold parts, 0 for an item held whole.  The part's first tile and
                    // the item's last one, in units of all items:
                    const long long first = end - walk.left - (walk.c1 - walk.c0);
                    const long long to = ((first + walk.nc) * ctas - 1) / total;
                    a.item[items.index(walk)] = make_int2(blockIdx.x * 2 + (part > 0 ? 1 : 0),
                                                          walk.c1 == walk.nc ? 0 : static_cast<int>(to - blockIdx.x + 1));
                }
            }
        }
        __syncwarp();
    } else if (warp < 8) {
        reg_dec<CONVERT_REGS>();
        // ================================================== converters ====
        const int half = warp & 1, which = (warp >> 1) & 1;   // rows 64 half .., 0: K, 1: V
        const int rot = lane >> 2, piece = lane & 3;          // row within 8, 16-byte piece of it
        constexpr int HG = G / 2;                             // scales of these rows
        static_assert(K16 == V16, "one ring walk for both");
        Ring<RAW> raw;
        Ring<K16> to;
        Ring<SC> sc;
        uint64_t* const full = which ? sm.v_full : sm.k_full;
        uint64_t* const empty = which ? sm.v_empty : sm.k_empty;
        uint8_t* const tiles = which ? sm.v16[0] : sm.k16[0];
        bool ok = true;
        for (; running && ok; running = items.next(walk)) {
            for (int t = walk.c0; t < walk.c1; ++t) {
                if (!(ok = wait_warp(smem_addr(&sm.raw_full[raw.st]), raw.ph, wc))) break;
                const uint8_t* src = sm.raw[raw.st][which];
                uint4 w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    w[i] = *reinterpret_cast<const uint4*>(src + (half * 64 + i * 8 + rot) * HD + piece * 16);
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&sm.raw_empty[raw.st]));
                raw.step();
                if (!(ok = wait_warp(smem_addr(empty + to.st), to.ph ^ 1u, wc))) break;
                uint32_t mul[HG];
                if (which) {
                    if (!(ok = wait_warp(smem_addr(&sm.sc_full[sc.st]), sc.ph, wc))) break;
#pragma unroll
                    for (int i = 0; i < HG; ++i) mul[i] = sm.v_mul[sc.st][half * HG + i];
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&sm.sc_empty[sc.st]));
                    sc.step();
                } else {
#pragma unroll
                    for (int i = 0; i < HG; ++i) mul[i] = 0x3C003C00u;
                }
                uint8_t* dst = tiles + to.st * TILE_BYTES;
                // values behind the last token must be finite: what the ring holds there is anything
                const int valid = which ? min(walk.len - t * BN, BN) : BN;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int row = half * 64 + i * 8 + rot;
                    const uint32_t by = mul[i / (8 / HG)];
                    uint32_t o[8];
                    if (FMT == ZB_KV8_INT8) {                  // the factor costs nothing here
                        unpack4_int8(w[i].x, by, o[0], o[1]);
                        unpack4_int8(w[i].y, by, o[2], o[3]);
                        unpack4_int8(w[i].z, by, o[4], o[5]);
                        unpack4_int8(w[i].w, by, o[6], o[7]);
                    } else {
                        unpack4<FMT>(w[i].x, o[0], o[1]);
                        unpack4<FMT>(w[i].y, o[2], o[3]);
                        unpack4<FMT>(w[i].z, o[4], o[5]);
                        unpack4<FMT>(w[i].w, o[6], o[7]);
#pragma unroll
                        for (int k = 0; k < 8; ++k) o[k] = mul_f16x2(o[k], by);
                    }
                    if (row >= valid) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) o[k] = 0u;
                    }
                    *reinterpret_cast<uint4*>(dst + row * 128 + ((2 * piece) ^ rot) * 16) = make_uint4(o[0], o[1], o[2], o[3]);
                    *reinterpret_cast<uint4*>(dst + row * 128 + ((2 * piece + 1) ^ rot) * 16) = make_uint4(o[4], o[5], o[6], o[7]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(full + to.st));
                to.step();
            }
        }
    } else {
        reg_inc<SOFTMAX_REGS>();
        // ========================================= softmax of a slot ====
        const int s = (warp >> 2) - 2;
        const int row = (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t tm_s = tmem + lanes + s * SLOT_COLS + TM_S;
        const uint32_t tm_p = tmem + lanes + s * SLOT_COLS + TM_P;
        const uint32_t tm_o = tmem + lanes + s * SLOT_COLS + TM_O;
        const int per_sum = G == 2 ? 1 : B / 16;               // scales to a weight sum
        uint32_t base = 0, g = 0, part = 0;   // tiles of earlier parts; this slot's steps; parts
        bool ok = true;
        constexpr int STEP = PAIR ? 1 : 2;
        for (; running && ok; running = items.next(walk), ++part) {
            const int n = walk.c1 - walk.c0;
            const int j0 = PAIR ? 0 : s;
            const int r_head = walk.tile * Items<PAIR>::ROWS + (PAIR ? s * BM : 0) + row;
            const bool live = r_head < a.rows;
            const long long out_row = static_cast<long long>(walk.h) * a.rows + r_head;
            float m = -INFINITY, l = 0.f;
            uint32_t last = ref_word(NO_REF);                  // the reference of the values so far
            bool nan_value = false;
            if (j0 < n) {
                // Q: the row's largest to [2^14, 2^15), as in kv8_attn.cu.  All of the slot's earlier
                // Q K^T are done (their S has been read), so its tile is free.
                float qf;
                {
                    uint32_t top = 0;
                    const uint4* src = reinterpret_cast<const uint4*>(a.Q + out_row * HD);
                    uint4 w[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        w[i] = live ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
                        top = __vmaxu2(top, __vmaxu2(__vmaxu2(w[i].x & 0x7FFF7FFFu, w[i].y & 0x7FFF7FFFu),
                                                     __vmaxu2(w[i].z & 0x7FFF7FFFu, w[i].w & 0x7FFF7FFFu)));
                    }
                    top = max(top << 16, top & 0x7FFF0000u);
                    const bool finite = top < 0x7F800000u;
                    const int e = max(static_cast<int>(top >> 23) - 127, -100);
                    const float up = finite ? __uint_as_float(static_cast<uint32_t>(14 - e + 127) << 23) : 0.f;
                    qf = finite ? __uint_as_float(static_cast<uint32_t>(e - 14 + 127) << 23) * a.scale_log2
                                : __uint_as_float(0x7FC00000u);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t ww[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
                        uint32_t o[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) o[k] = finite ? pack_f16x2(bf16_lo(ww[k]) * up, bf16_hi(ww[k]) * up) : 0u;
                        *reinterpret_cast<uint4*>(sm.q[s] + row * 128 + (i ^ (row & 7)) * 16) = make_uint4(o[0], o[1], o[2], o[3]);
                    }
                    fence_proxy_async_smem();
                    mbar_arrive(smem_addr(&sm.q_full[s]));
                }
                const int lim = a.causal ? walk.len - a.n_q + 1 + r_head % a.n_q : walk.len;
                // weight sums of this part's tiles, in order (where slots share rows: every second tile)
                const int per_tile = G / per_sum;
                int gsum_left = a.groups - (walk.c0 + j0) * per_tile;
                float* gsum = a.gsum + (static_cast<long long>(walk.h) * a.groups + static_cast<long long>(walk.c0 + j0) * per_tile) * a.rows + r_head;
                for (int j = j0; j < n; j += STEP, ++g) {
                    const uint32_t t = base + j;
                    const int sc = t % SC;
                    if (!(ok = wait_warp(smem_addr(&sm.s_full[s]), g & 1, smem_addr(&sm.sc_full[sc]), (t / SC) & 1, wc))) break;
                    tc_fence_after();
                    const int seen = max(min(lim - (walk.c0 + j) * BN, BN), 0);
                    float alpha = 1.f, nm = 0.f, weight = 0.f;
                    bool raise = false;
                    int grown = 0;                             // less what the values' reference grew by
                    // A tile is read in halves, the first half twice: for the maximum, and again for its
                    // exponentials after the second half's.  Held whole, its 128 values left the compiler so
                    // few registers that it moved each about once more than needed.  Tiles that every row
                    // sees to their end (all but the last few of an item) get code without a mask.
                    constexpr int HALF = BN / 2, HG = G / 2, COLS = BN / G;
                    auto step = [&](auto edge_tag) -> bool {
                        constexpr bool EDGE = decltype(edge_tag)::value;
                        auto load = [&](int h, float (&x)[HALF]) {
                            uint32_t raw[HALF];
                            tmem_load(tm_s + h * HALF, raw);
#pragma unroll
                            for (int e = 0; e < HALF; ++e) {
                                x[e] = __uint_as_float(raw[e]);
                                if (EDGE) x[e] = h * HALF + e < seen ? x[e] : -INFINITY;
                            }
                        };
                        // logits are x f, COLS columns to a scale.  At an edge -inf must stay -inf: f is
                        // kept off zero, and is 1 where nothing is seen, whatever the scale there is.
                        auto factor = [&](float ks, int q) {
                            float f = ks * qf;
                            if (EDGE) {
                                f = f < 1e-37f ? 1e-37f : f;
                                f = q * COLS >= seen ? 1.f : f;
                            }
                            return f;
                        };
                        auto maximum = [&](int h, const float (&x)[HALF]) {
                            float mx = -INFINITY;
#pragma unroll
                            for (int q = 0; q < HG; ++q) {
                                const float ks = sm.sc[sc][h * HG + q].x;
                                float v = -INFINITY;
#pragma unroll
                                for (int k = 0; k < COLS; k += 16) { // a tree of 3-input maxima
                                    float u = fmax3(x[COLS * q + k], x[COLS * q + k + 1], x[COLS * q + k + 2]);
#pragma unroll
                                    for (int e = 3; e < 15; e += 2) u = fmax3(u, x[COLS * q + k + e], x[COLS * q + k + e + 1]);
                                    v = fmax3(v, u, x[COLS * q + k + 15]);
                                }
                                mx = fmaxf(mx, v * factor(ks, h * HG + q));
                            }
                            return mx;
                        };
                        // P of a half to TMEM, its sums to l and the weights (their order: see the caller)
                        auto exponentials = [&](int h, const float (&x)[HALF]) {
                            uint32_t pk[HALF / 2];
                            float add_l = 0.f;
                            float* dst = gsum + static_cast<long long>(h) * (per_tile / 2) * a.rows;
#pragma unroll
                            for (int q = 0; q < HG; ++q) {
                                const float4 w = sm.sc[sc][h * HG + q];
                                const float f = factor(w.x, h * HG + q), add = nm + w.y;
                                const float sum = exp_pairs<COLS>(x + COLS * q, f2_pack(f, f), f2_pack(add, add), pk + COLS / 2 * q) * w.z;
                                add_l += sum;
                                if (MASS) {
                                    // log2 of the sums of each 64 keys, or of a smaller block
                                    weight += sum;
                                    if (G == 2 || ((q + 1) & (per_sum - 1)) == 0) {
                                        const int k = h * (per_tile / 2) + q / per_sum;
                                        if (live && k < gsum_left) *dst = __log2f(weight) - nm;
                                        dst += a.rows;
                                        weight = 0.f;
                                    }
                                }
                            }
                            l += add_l;
                            tmem_store(tm_p + h * (HALF / 2), pk);
                        };
                        float x[HALF];
                        load(0, x);
                        float mx = maximum(0, x);
                        load(1, x);
                        mx = fmaxf(mx, maximum(1, x));
                        if (const uint32_t word = sm.sc_word[sc]; word != last) {
                            nan_value |= (word & 0xFFu & ((1u << ((seen + COLS - 1) / COLS)) - 1u)) != 0;
                            if (j > j0) grown = word_ref(last) - word_ref(word);
                            last = word & ~0xFFu;
                        }
                        raise = mx > m + RAISE || (m == -INFINITY && mx > m);
                        if (raise) {
                            alpha = m == -INFINITY ? 0.f : ex2(m - mx);
                            m = mx;
                            l *= alpha;
                        }
                        nm = (m == -INFINITY ? 0.f : -m) + SHIFT;
                        // P is free once P V of the step before is done; O then holds every earlier step
                        if (!wait_warp(smem_addr(&sm.p_free[s]), (g & 1) ^ 1, wc)) return false;
                        tc_fence_after();
                        exponentials(1, x);
                        load(0, x);
                        tc_fence_before();
                        mbar_arrive(smem_addr(&sm.s_free[s]));
                        exponentials(0, x);
                        return true;
                    };
                    if (!(ok = __any_sync(0xffffffffu, seen < BN) ? step(std::true_type{}) : step(std::false_type{}))) break;
                    if (__any_sync(0xffffffffu, (raise && j > j0) || grown != 0)) {
                        const float al = (raise && j > j0 ? alpha : 1.f) * pow2(grown);
                        uint32_t ro[HD];
                        tmem_load(tm_o, ro);
#pragma unroll
                        for (int e = 0; e < HD; ++e) ro[e] = __float_as_uint(__uint_as_float(ro[e]) * al);
                        tmem_store(tm_o, ro);
                    }
                    tc_fence_before();
                    mbar_arrive(smem_addr(&sm.p_full[s]));
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_addr(&sm.sc_empty[sc]));
                    if (MASS) {                                      // past this tile, and the other slot's
                        gsum += static_cast<long long>(per_tile) * STEP * a.rows;
                        gsum_left -= per_tile * STEP;
                    }
                }
                if (!ok) break;
                // the last P V
                if (!(ok = wait_warp(smem_addr(&sm.p_free[s]), (g & 1) ^ 1, wc))) break;
                tc_fence_after();
            }
            base += n;
            // ---- the part's result ------------------------------------------
            float o[HD];
            if (j0 < n) {
                uint32_t ro[HD];
                tmem_load(tm_o, ro);
#pragma unroll
                for (int e = 0; e < HD; ++e) o[e] = __uint_as_float(ro[e]);
                tc_fence_before();
                mbar_arrive(smem_addr(&sm.o_free[s]));
            } else {
#pragma unroll
                for (int e = 0; e < HD; ++e) o[e] = 0.f;
            }
            // o times this and the share of the softmax sum: the outputs
            const float size = nan_value ? __uint_as_float(0x7FC00000u) : pow2(word_ref(last));
            if (PAIR) {
                const float f = l == 0.f ? 0.f * size : size / l;  // no key: zeros; NaN stays
#pragma unroll
                for (int e = 0; e < HD; ++e) o[e] *= f;
            } else {
                // the slots hold the same rows: slot 1 hands its sums to slot 0
                if (s == 1) {
                    if (!(ok = wait_warp(smem_addr(&sm.other_empty), (part & 1) ^ 1, wc))) break;
#pragma unroll
                    for (int i = 0; i < HD / 4; ++i)
                        sm.other[i][row] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                    sm.other_ml[row] = make_float4(m, l, size, 0.f);
                    mbar_arrive(smem_addr(&sm.other_full));
                    continue;
                }
                if (!(ok = wait_warp(smem_addr(&sm.other_full), part & 1, wc))) break;
                const float4 ml = sm.other_ml[row];
                const float M = fmaxf(m, ml.x);
                const float w0 = m == -INFINITY ? 1.f : ex2(m - M), w1 = ml.x == -INFINITY ? 1.f : ex2(ml.x - M);
                m = M;
                l = l * w0 + ml.y * w1;
                const float inv = l == 0.f ? 0.f : 1.f / l, f0 = w0 * inv * size, f1 = w1 * inv * ml.z;
#pragma unroll
                for (int i = 0; i < HD / 4; ++i) {
                    const float4 w = sm.other[i][row];
                    o[4 * i] = o[4 * i] * f0 + w.x * f1;
                    o[4 * i + 1] = o[4 * i + 1] * f0 + w.y * f1;
                    o[4 * i + 2] = o[4 * i + 2] * f0 + w.z * f1;
                    o[4 * i + 3] = o[4 * i + 3] * f0 + w.w * f1;
                }
                mbar_arrive(smem_addr(&sm.other_empty));
            }
            if (!live) continue;
            if (walk.c0 == 0 && walk.c1 == walk.nc) {          // the whole item: the outputs themselves
                uint4* out = reinterpret_cast<uint4*>(a.O + out_row * HD);
#pragma unroll
                for (int i = 0; i < HD / 8; ++i)
                    out[i] = make_uint4(pack_bf16x2(o[8 * i], o[8 * i + 1]), pack_bf16x2(o[8 * i + 2], o[8 * i + 3]),
                                        pack_bf16x2(o[8 * i + 4], o[8 * i + 5]), pack_bf16x2(o[8 * i + 6], o[8 * i + 7]));
                const float total2 = l == 0.f ? -INFINITY : m - SHIFT + log2f(l);
                if (a.lse) a.lse[out_row] = total2 * LN2;
                if (a.lse2) a.lse2[out_row] = total2;
            } else {
                const long long place = (static_cast<long long>(blockIdx.x) * 2 + (part > 0 ? 1 : 0)) * (PAIR ? 2 : 1) + (PAIR ? s : 0);
                float4* dst = reinterpret_cast<float4*>(a.part_o + (place * BM + row) * HD);
#pragma unroll
                for (int i = 0; i < HD / 4; ++i) dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                a.part_ml[place * BM + row] = make_float2(m, l);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

// The parts of items that several CTAs hold, each the outputs over its own keys, added
// up by their shares of the softmax sum; rows of items without a tile become zeros and
// -inf.  Grid: (row tiles, 8): 16 rows a CTA, 16 threads a row.  A row's thread reads
// one part's maximum and sum in sixteen and 4 features of all.
template <bool PAIR>
__global__ void __launch_bounds__(256) join_tiles_kernel(const AttnArgs a) {
    const int per_item = PAIR ? 2 : 1, row_tiles = a.tiles * per_item;
    const int h = blockIdx.x / row_tiles, rt = blockIdx.x % row_tiles, s = PAIR ? rt & 1 : 0;
    const int len = static_cast<int>(head_len(a.lens, h, static_cast<long long>(a.c.slots) * a.c.block));
    const bool none = item_tiles(a, len, rt / per_item, BM * per_item) == 0;
    wait_for_previous();
    let_next_start();
    const int2 it = none ? make_int2(0, 0) : a.item[static_cast<long long>(h) * a.tiles + rt / per_item];
    if (!none && it.y == 0) return;                  // written whole
    const int q = threadIdx.x & 15, r = blockIdx.y * 16 + (threadIdx.x >> 4);
    const int r_head = rt * BM + r;
    if (r_head >= a.rows) return;                    // (half warps are rows: the shuffles below stay whole)
    const uint32_t half = 0xFFFFu << (lane_id() & 16);
    auto at = [&](int i) {                           // the i-th CTA's place: its first part, but for the item's own start
        const long long place = i == 0 ? it.x : (it.x / 2 + i) * 2;
        return (place * per_item + s) * BM + r;
    };
    auto part = [&](int i, int k) {
        return i + k < it.y ? reinterpret_cast<const float4*>(a.part_o + at(i + k) * HD)[q] : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    // most rows have few parts: all loads of the first ones are under way before any is needed
    const float2 ml = q < it.y ? a.part_ml[at(q)] : make_float2(-INFINITY, 0.f);
    float4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = part(0, k);
    float M = ml.x;
    for (int i = q + 16; i < it.y; i += 16) M = fmaxf(M, a.part_ml[at(i)].x);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(half, M, o));
    // a part's share of the softmax sum, over 2^M
    auto share = [&](float2 p) { return p.y == 0.f ? 0.f : p.y * ex2(p.x - M); };
    const float first = share(ml);
    float L = first;
    for (int i = q + 16; i < it.y; i += 16) L += share(a.part_ml[at(i)]);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) L += __shfl_xor_sync(half, L, o);
    const float inv = L == 0.f ? 0.f : 1.f / L;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < it.y; i0 += 16) {
        const float f = (i0 == 0 ? first : i0 + q < it.y ? share(a.part_ml[at(i0 + q)]) : 0.f) * inv;
        const int n = min(16, it.y - i0);
        for (int i1 = 0; i1 < n; i1 += 4) {
            if (i0 + i1 > 0) {
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] = part(i0 + i1, k);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {            // lanes past the last part hold zeros
                const float fk = __shfl_sync(half, f, (i1 + k) & 15, 16);
                sum.x = fmaf(v[k].x, fk, sum.x);
                sum.y = fmaf(v[k].y, fk, sum.y);
                sum.z = fmaf(v[k].z, fk, sum.z);
                sum.w = fmaf(v[k].w, fk, sum.w);
            }
        }
    }
    const float total2 = L == 0.f ? -INFINITY : M - SHIFT + log2f(L);
    const long long row = static_cast<long long>(h) * a.rows + r_head;
    reinterpret_cast<uint2*>(a.O + row * HD)[q] =
        make_uint2(pack_bf16x2(sum.x, sum.y), pack_bf16x2(sum.z, sum.w));
    if (q == 0) {
        if (a.lse) a.lse[row] = total2 * LN2;
        if (a.lse2) a.lse2[row] = total2;
    }
}

template <int FMT, bool PAIR, bool MASS, int G>
zb_status launch_one(const AttnArgs& a, int ctas, cudaStream_t st) {
    auto* fn = tile_kernel<FMT, PAIR, MASS, G>;
    constexpr int bytes = sizeof(TileSmem) + 1024;
    static std::atomic<unsigned long long> done{0};  // devices that have the attribute set
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return ZB_ERR_CUDA;
    if (!(done.load(std::memory_order_relaxed) >> dev & 1)) {
        if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return ZB_ERR_CUDA;
        done.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    fn<<<ctas, THREADS, bytes, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? ZB_OK : ZB_ERR_CUDA;
}

template <int FMT, bool PAIR>
zb_status launch(const AttnArgs& a, int ctas, cudaStream_t st) {
    const bool wide = a.c.block >= CHUNK;
    const zb_status e = a.groups ? wide ? launch_one<FMT, PAIR, true, 2>(a, ctas, st) : launch_one<FMT, PAIR, true, 8>(a, ctas, st)
                        : wide   ? launch_one<FMT, PAIR, false, 2>(a, ctas, st)
                                 : launch_one<FMT, PAIR, false, 8>(a, ctas, st);
    if (e != ZB_OK) return e;
    return launch_behind(join_tiles_kernel<PAIR>, dim3(static_cast<unsigned>(a.c.heads * a.tiles * (PAIR ? 2 : 1)), 8), 256,
                         st, a);
}

}  // namespace

zb_status launch_tiles(const AttnArgs& a, bool pair, int ctas, cudaStream_t st) {
    if (a.c.format == ZB_KV8_INT8)
        return pair ? launch<ZB_KV8_INT8, true>(a, ctas, st) : launch<ZB_KV8_INT8, false>(a, ctas, st);
    return pair ? launch<ZB_KV8_E4M3, true>(a, ctas, st) : launch<ZB_KV8_E4M3, false>(a, ctas, st);
}

}  // namespace kv8
}  // namespace zb
