// k_prefix_tc.cu -- attention over shared prefixes on the tensor cores (tcgen05, TMEM,
// TMA): bf16 pools in blocks of 8 rows or more.  See k_prefix.cu for what is computed and
// rkv_prefix.cuh for the line of work.
//
// The queries of all sequences of a prefix that use a KV head are the rows of two products
// with the prefix's keys and values: S = Q K^T, O += P V, each 128 queries x 64 rows a
// step, accumulated in TMEM.  One block an SM, eleven warps:
//   * warp 10: TMA producer, a ring of tiles of 64 rows (K and V in the order in which
//     they are used) through the prefix's block table, one copy per block (of up to 64
//     rows) and 64 columns, 128-byte swizzle.  Rows past the prefix in its last block are
//     cleared in V, where they would meet a probability of 0.
//   * warps 8 and 9: issue the MMAs, one warp for each group of 128 queries.  S from shared
//     memory; O += P V with P as the operand in TMEM and V as it lies, its rows being the
//     contracted index (an MN-major operand).
//   * warps 0-3 and 4-7: softmax of a group, one query a thread, which is a row of TMEM:
//     maxima, sums and scales take no exchange between threads.  P is written over S as
//     bf16 (one part, 2^-8 of it: a second would take the tensor cores half as long
//     again).  O is brought to a new maximum only where a logit passes the old one by more
//     than 8 (log2), so that hardly ever anybody waits for it.
// With more than 128 queries a prefix the groups take 128 each, all rows; with fewer
// (SPLIT) the same queries, every other unit of rows each, and join at a piece's end
// through shared memory.
//
// Why units of 64 rows: at head_dim 128 O takes half of TMEM, and the other half holds two
// buffers of S for each group only if they are 64 columns wide.  With one buffer of 128 the
// next S waits until P V is done with it, 340 cycles behind the pipe's own time, and the
// softmax waits for that S: 241 us for the case below where two buffers took 212 when the
// step was measured by itself, although S in steps of 64 costs the pipe half as much again
// (48 cycles an MMA, the operands' shared memory, where 128 columns take 64).
//
// Measured (one GB300, head_dim 128, 8 KV heads): 128 samples of 131071 rows, G = 4, 275
// GFLOP: 173 us from the first piece to the last, 1.6 PFLOP/s; about 1600 cycles a step of
// 2 x 128 queries, of which the products take 1280.  The whole call takes 220 us over many
// calls on the same inputs, 227 with inputs that change from call to call.  A piece's beginning
// (its place on the line, queries, first tiles) and end take about 4 us each, which bounds short
// prefixes.
// Every wait is bounded; one that runs out records a device error, and all roles end.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "rkv_prefix.cuh"
#include "tcgen05.cuh"

namespace rkv {
namespace prefix {
namespace {

using namespace tc;

constexpr int kUnit = 64;             // rows of a step
constexpr int kChunk = kUnit * 128;   // 64 rows of 64 bf16
constexpr int kQChunk = 128 * 128;    // 128 queries of 64 bf16
constexpr float kFar = 0x1p20f;       // (see the softmax)
constexpr int kThreads = 352;

template <int D>
struct Cfg {
    static constexpr int KC = D / 64;
    static constexpr int TILE = KC * kChunk;    // 64 rows of K or V
    static constexpr int QTILE = KC * kQChunk;  // the queries of a group
    static constexpr int STAGES = D == 128 ? 10 : 12;
    static constexpr int RING = 2 * QTILE;      // behind the queries of both groups
    static constexpr int BARS = RING + STAGES * TILE;
    static constexpr int NUM_BARS = 2 * STAGES + 2 + 4 + 4 + 4 + 5;
    static constexpr int ML = BARS + NUM_BARS * 8 + 16;
    static constexpr int BYTES = 1024 + ML + 128 * 8;
};

// Shared-memory matrix descriptor of a tile whose rows are the contracted index: 64
// columns (128 bytes, swizzled) of 8 rows are 1024 bytes, the next 8 rows behind them
// (stride byte offset), the next 64 columns `chunk` bytes on (leading byte offset).
RKV_DEV uint64_t sdesc_rows(const void* p, uint32_t chunk) {
    const uint64_t a = smem_u32(p);
    uint64_t d = (a >> 4) & 0x3FFFull;
    d |= (uint64_t)(chunk >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= 1ull << 46;
    d |= 2ull << 61;
    return d;
}
// D = A B (+ D) with A in TMEM.
RKV_DEV void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                         uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
RKV_DEV void tmem_st_32cols(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
        "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
        "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
RKV_DEV void tmem_st_16cols(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
RKV_DEV void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
RKV_DEV void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
RKV_DEV uint64_t pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
RKV_DEV uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
RKV_DEV uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
RKV_DEV void unpair(uint64_t v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
RKV_DEV uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}
// One lane of a converged warp.  (The issuing warp stays together around its MMAs, so
// that what they are given is uniform: issued by a lane of its own they took 100 cycles
// each where the product takes 64.)
RKV_DEV bool elect_one() {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok != 0;
}
RKV_DEV void commit_to(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// A bounded wait of a whole warp.  Without a suspend hint: with one a wait costs 200
// cycles even where the phase is over (17 without), and a step has eight in a row.
RKV_DEV bool wait_at(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
    long long since = 0;
    for (;;) {
        uint32_t over;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(over)
            : "r"(bar), "r"(parity)
            : "memory");
        if (__all_sync(0xffffffffu, over != 0)) return true;
        const long long now = clock64();
        if (since == 0) since = now;
        if (__any_sync(0xffffffffu, *abort_flag != 0 || now - since > kWaitCycles)) return false;
    }
}
RKV_DEV bool wait_all(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    return wait_at(smem_u32(bar), parity, abort_flag);
}

// Whoever waits for a tile has waited for the one that was in its place before: a
// parity tells a phase that is over from the one before it, not from the one behind it.
// So with SPLIT each group has a ring of its own (its share of the stages), and without
// it both issuing warps go through all tiles, those of a piece without queries for the
// second group as well.
template <int D, bool SPLIT> constexpr int kRing = Cfg<D>::STAGES / (SPLIT ? 2 : 1);
// Two units' K go into a ring before V of the first (S has two buffers a group).  The
// places of K and V of the ring's unit q among its 2 n tiles of a piece.
RKV_DEV uint32_t place_k(int q) { return q + max(0, q - 1); }
RKV_DEV uint32_t place_v(int q, int n) { return q + min(q + 2, n); }

// The products of a group's n units of a piece, by its issuing warp.  (One for each
// group: what a warp does between two MMAs, waits that are over take 100 cycles, is time
// in which the other's fill the tensor cores; one warp for both: 2090 cycles for 64 rows
// of 2 x 128 queries.)
struct Issue {
    uint32_t bars;  // full, empty, .. as in the kernel
    uint32_t s, o;  // TMEM of the group's S and O
    uint32_t tile;  // tiles of earlier pieces in the group's ring
    uint32_t ph;    // phases of p_full and o_done, a bit a buffer
};
template <int D, bool SPLIT>
RKV_DEV bool issue_piece(Issue& w, int x, int n, uint64_t q0, uint64_t k0, uint64_t v0,
                         volatile int* abort_flag) {
    using C = Cfg<D>;
    constexpr int RING = kRing<D, SPLIT>;
    constexpr uint32_t kIdescS = idesc_bf16(128, kUnit);
    constexpr uint32_t kIdescO = idesc_bf16(128, D) | (1u << 16);  // B by rows
    constexpr uint32_t kEmpty = 8 * C::STAGES, kS = 2 * kEmpty + 16, kP = kS + 32, kO = kP + 32;
    uint32_t st;
    const auto find = [&](uint32_t t) {
        t += w.tile;
        st = (SPLIT ? x * RING : 0) + t % RING;
        return wait_at(w.bars + 8 * st, (t / RING) & 1u, abort_flag);
    };
    const auto logits = [&](uint32_t b) {  // S into buffer b
        if (elect_one()) {
            const uint64_t k = k0 + st * (C::TILE >> 4);
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
                mma_bf16(w.s + b * 64, q0 + (i >> 2) * (kQChunk >> 4) + 2 * (i & 3),
                         k + (i >> 2) * (kChunk >> 4) + 2 * (i & 3), kIdescS, i != 0);
            commit_to(w.bars + kS + 16 * x + 8 * b);
            commit_to(w.bars + kEmpty + 8 * st);
        }
        __syncwarp();
    };
    for (int q = 0; q < 2 && q < n; ++q) {
        if (!find(place_k(q))) return false;
        logits(q);
    }
    for (int q = 0; q < n; ++q) {
        const uint32_t b = q & 1;
        if (!find(place_v(q, n))) return false;
        if (!wait_at(w.bars + kP + 16 * x + 8 * b, (w.ph >> b) & 1u, abort_flag)) return false;
        tc_fence_after();
        if (elect_one()) {  // O += P V, P from buffer b
            const uint64_t v = v0 + st * (C::TILE >> 4);
#pragma unroll
            for (int k = 0; k < kUnit / 16; ++k)
                mma_bf16_ts(w.o, w.s + b * 64 + 8 * k, v + (2048 >> 4) * k, kIdescO, q != 0 || k != 0);
            commit_to(w.bars + kO + 16 * x + 8 * b);
            commit_to(w.bars + kEmpty + 8 * st);
        }
        __syncwarp();
        if (q + 2 < n) {
            // the S of two units on takes the place of this P, which the product has to be done with
            if (!find(place_k(q + 2))) return false;
            if (!wait_at(w.bars + kO + 16 * x + 8 * b, (w.ph >> b) & 1u, abort_flag)) return false;
            logits(b);
        }
        w.ph ^= 1u << b;
    }
    return true;
}

// Logits of columns from `col` on that no row stands behind become -inf: those past
// the piece, and those of blocks (of 1 << log2box columns) that are not there.  Their
// maximum.
RKV_DEV float hide(uint32_t (&z)[32], int col, int left, uint32_t have, int log2box) {
    const int n = left - col;
    uint32_t keep = n >= 32 ? 0xffffffffu : (n <= 0 ? 0u : (1u << n) - 1u);
    have >>= col >> log2box;
    if (log2box >= 5) {
        if (!(have & 1u)) keep = 0u;
    } else {
        for (int b = 0; b < 32 >> log2box; ++b)
            if (!((have >> b) & 1u)) keep &= ~(((1u << (1 << log2box)) - 1u) << (b << log2box));
    }
    float top = -INFINITY;
#pragma unroll
    for (int k = 0; k < 32; ++k) {
        if (!((keep >> k) & 1u)) z[k] = 0xff800000u;
        top = fmaxf(top, __uint_as_float(z[k]));
    }
    return top;
}
RKV_DEV int units_in(const Piece& c) { return (c.c1 - c.c0 + kUnit - 1) / kUnit; }

template <int D, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
prefix_tc_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                 const __grid_constant__ Params p) {
    using C = Cfg<D>;
    constexpr int STEP = SPLIT ? 2 : 1;  // units between two of a group
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint8_t* ring = smem + C::RING;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BARS);
    uint64_t* empty = full + C::STAGES;
    uint64_t* q_full = empty + C::STAGES;  // [group]
    uint64_t* s_full = q_full + 2;         // [group][buffer]
    uint64_t* p_full = s_full + 4;         // [group][buffer]
    // O += P V done, by the buffer of P: a phase is then never more than one ahead of who
    // waits for it (the next product from a buffer waits for the group's next P in it)
    uint64_t* o_done = p_full + 4;         // [group][buffer]
    uint64_t* tail_bar = o_done + 4;       // a tile that has rows to clear
    uint64_t* drain_bar = tail_bar + 1;    // [group]
    uint64_t* x_full = drain_bar + 2;      // SPLIT: half of the second group's output is there
    uint64_t* x_empty = x_full + 1;
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(x_empty + 1);
    volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
    float2* sh_ml = reinterpret_cast<float2*>(smem + C::ML);
    // [D / 2][128], in the place of the second group's queries, which are the first's then
    float* sh_x = reinterpret_cast<float*>(smem + C::QTILE);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t run = blockIdx.x / p.team;
    const int member = blockIdx.x - run * p.team;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], SPLIT ? 1 : 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], 4);
            mbar_init(&drain_bar[i], 1);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
            mbar_init(&o_done[i], 1);
        }
        mbar_init(tail_bar, 1);
        mbar_init(x_full, 4);
        mbar_init(x_empty, 4);
        *s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&kmap)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&vmap)) : "memory");
    }
    if (warp == 8) {
        tmem_alloc(s_tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    // (Begins while the own rows' pass ends, every block of which has waited for everything before
    // it, so queries, pools and tables are there; its sums are waited for where they are read.
    // See launch_early.)
    Place place = find_place<kUnit>(p, run);
    Piece c{};
    bool ok = true;

    if (warp == 10) {
        // ------------------------------------------------------- producer --
        // lane i copies 64 columns of a block (of up to 64 rows)
        const int log2box = p.log2bs < 6 ? p.log2bs : 6, box = 1 << log2box;
        const int b = lane / C::KC, ch = lane - b * C::KC, own = b << log2box;
        const bool copies = lane < (kUnit >> log2box) * C::KC;  // 16 at most
        const uint32_t to = ch * kChunk + own * 128;
        constexpr int RING = kRing<D, SPLIT>;
        uint32_t tiles = 0, tiles1 = 0, tails = 0;  // tiles in the (first) ring, SPLIT: in the second
        // the block of the lane's rows of unit u, asked for one tile ahead (-1: rows past the piece)
        auto look_up = [&](int u) {
            const int r = c.c0 + u * kUnit + own;
            return copies && r < c.c1 ? p.table[(int64_t)c.i * p.max_blocks + (r >> p.log2bs)] : -1;
        };
        auto load = [&](const CUtensorMap* map, int u, int block, bool is_v) {
            const int r0 = c.c0 + u * kUnit;
            const bool there = (unsigned)block < (unsigned)p.num_blocks, second = SPLIT && (u & 1);
            const uint32_t t = second ? tiles1 : tiles, st = (second ? RING : 0) + t % RING;
            if (copies && !there && !is_v && ch == 0 && r0 + own < c.c1)
                set_error(p.status, kDevErrIndex, (unsigned)(r0 + own));
            if (!wait_all(&empty[st], ((t / RING) & 1u) ^ 1u, s_abort)) return false;
            uint8_t* dst = ring + st * C::TILE;
            const bool clear = is_v && r0 + kUnit > c.c1 && (c.c1 & (box - 1)) != 0;
            uint64_t* bar = clear ? tail_bar : &full[st];
            // (bytes that land before they are expected leave the count below zero for a while)
            if (lane == 0) mbar_arrive_expect_tx(bar, C::TILE);
            // an outer coordinate past the pool reads as zeros
            if (copies)
                tma_load_3d(dst + to, map, bar, ch * 64, (r0 + own) & ((1 << p.log2bs) - 1),
                            there ? block * p.H + c.h : p.num_blocks * p.H);
            if (clear) {
                if (!wait_all(tail_bar, tails++ & 1, s_abort)) return false;
                const int from = c.c1 - r0, end = (from + box) & ~(box - 1);
                for (int e = lane; e < (end - from) * 8 * C::KC; e += 32) {
                    const int row = from + e / (8 * C::KC), x = e % (8 * C::KC);
                    *reinterpret_cast<uint4*>(dst + (x >> 3) * kChunk + row * 128 + (x & 7) * 16) =
                        make_uint4(0u, 0u, 0u, 0u);
                }
                fence_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[st]);
            }
            tiles += !second;
            tiles1 += second;
            return true;
        };
        while (ok && next_piece<kUnit>(p, run, member, place, c)) {
            const int n = c.rows > 0 ? units_in(c) : 0;
            int k = 0, next_k = look_up(0), next_v = next_k;
            for (; ok && k < (SPLIT ? 4 : 2) && k < n; ++k) {
                const int block = next_k;
                next_k = look_up(k + 1);
                ok = load(&kmap, k, block, false);
            }
            for (int u = 0; ok && u < n; ++u) {
                int block = next_v;
                next_v = look_up(u + 1);
                ok = load(&vmap, u, block, true);
                if (ok && k < n) {
                    block = next_k;
                    next_k = look_up(k + 1);
                    ok = load(&kmap, k++, block, false);
                }
            }
        }
        if (!ok) {
            *s_abort = 1;
            if (lane == 0) set_error(p.status, kDevErrTimeout, 1u);
        }
        // every copy issued has landed before the block may end
        volatile int never = 0;
        for (uint32_t t = tiles > RING ? tiles - RING : 0; t < tiles; ++t)
            mbar_wait(&full[t % RING], (t / RING) & 1, &never);
        for (uint32_t t = tiles1 > RING ? tiles1 - RING : 0; t < tiles1; ++t)
            mbar_wait(&full[RING + t % RING], (t / RING) & 1, &never);
    } else if (warp >= 8) {
        // ---------------------------------------------------- MMA issuers --
        const int x = warp - 8;
        uint32_t asked = 0;
        Issue w{smem_u32(full), tmem + x * 128, tmem + 256 + x * D, 0u, 0u};
        const uint64_t q0 = sdesc_sw128(smem + (SPLIT ? 0 : x * C::QTILE)), k0 = sdesc_sw128(ring),
                       v0 = sdesc_rows(ring, kChunk);
        while (ok && next_piece<kUnit>(p, run, member, place, c)) {
            const int n = c.rows > 0 ? units_in(c) : 0;
            const int mine = SPLIT ? (n + 1 - x) >> 1 : n;
            if (SPLIT || c.rows > 128 * x) {
                if (mine == 0) continue;
                if (!(ok = wait_all(&q_full[x], asked++ & 1, s_abort))) break;
                tc_fence_after();
                ok = issue_piece<D, SPLIT>(w, x, mine, q0, k0, v0, s_abort);
            } else {
                for (int t = 0; ok && t < 2 * mine; ++t) {
                    const uint32_t st = (w.tile + t) % C::STAGES;
                    ok = wait_all(&full[st], ((w.tile + t) / C::STAGES) & 1, s_abort);
                    if (ok && lane == 0) mbar_arrive(&empty[st]);
                }
            }
            w.tile += 2 * mine;
        }
        if (!ok) {
            *s_abort = 1;
            if (lane == 0) set_error(p.status, kDevErrTimeout, 2u);
        }
        // every MMA issued so far is done before TMEM is released
        if (elect_one()) mma_commit(&drain_bar[x]);
        __syncwarp();
        volatile int never = 0;
        mbar_wait(&drain_bar[x], 0, &never);
    } else {
        // -------------------------------------------------------- softmax --
        const int x = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t t_x = tmem + ((uint32_t)(warp & 3) << 21) + x * 128;
        const uint32_t t_o = tmem + ((uint32_t)(warp & 3) << 21) + 256 + x * D;
        const int log2box = p.log2bs < 6 ? p.log2bs : 6, boxes = kUnit >> log2box;
        bool waited = false;
        uint32_t seen = 0, halves = 0;  // phases of s_full and o_done (a bit a buffer), x_full
        while (ok && next_piece<kUnit>(p, run, member, place, c)) {
            if (!SPLIT && c.rows <= 128 * x) continue;
            const int n = units_in(c);
            const int r = (SPLIT ? 0 : x * 128) + row;
            const bool valid = r < c.rows;
            int s = 0, tk = 0, hd = 0;
            if (valid) place_of_row(p, c.seq0, c.h, c.row0 + r, s, tk, hd);
            if (n > 0 && (!SPLIT || x == 0)) {
                // a row of queries by D / 8 neighbouring lanes, all rows of the warp on their way
                // before the first is stored
                constexpr int LANES = D / 8;
                const int u = lane % LANES;
                const int64_t mine = valid ? s * p.q_seq + tk * p.q_tok + hd * p.q_head : -1;
                uint4 y[LANES];
#pragma unroll
                for (int i = 0; i < LANES; ++i) {
                    const int64_t at = __shfl_sync(0xffffffffu, mine, i * (32 / LANES) + lane / LANES);
                    y[i] = make_uint4(0u, 0u, 0u, 0u);
                    if (at >= 0)
                        y[i] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + at + 8 * u);
                }
#pragma unroll
                for (int i = 0; i < LANES; ++i) {
                    const int to = (warp & 3) * 32 + i * (32 / LANES) + lane / LANES;
                    y[i].x ^= p.flip; y[i].y ^= p.flip; y[i].z ^= p.flip; y[i].w ^= p.flip;
                    *reinterpret_cast<uint4*>(smem + x * C::QTILE + (u >> 3) * kQChunk + to * 128 +
                                              (((u & 7) ^ (to & 7)) << 4)) = y[i];
                }
                fence_async();
                mbar_arrive_warp(&q_full[x]);
                if (SPLIT && n > 1) mbar_arrive_warp(&q_full[1]);
            }
            if (threadIdx.x == 0 && bad_length(p, c)) set_error(p.status, kDevErrIndex, (unsigned)c.i);
            // m: running maximum of q . k; sums are relative to 2^base, base the fp32 nearest
            // to m * scale and rest what that leaves, so that z * scale - base is one FMA and
            // exact up to its rounding.  Past kFar, where base is coarse, they are relative to
            // 2^(m * scale) (rest 0), and differences of q . k are taken; far: some query of
            // the warp is there.
            float m = kNone, l = 0.f, base = -INFINITY, rest = 0.f;
            bool far = true;
            bool begin = true;
            int buf = 1;
            // the block of this lane's rows of a unit, looked at one unit later, when the load has
            // come back (0, which there is, for lanes without rows)
            const auto look_up = [&](int u) {
                const int rb = c.c0 + u * kUnit + (lane << log2box);
                return lane < boxes && rb < c.c1 ? p.table[(int64_t)c.i * p.max_blocks + (rb >> p.log2bs)] : 0;
            };
            int block = look_up(SPLIT ? x : 0);
            for (int u = SPLIT ? x : 0; u < n; u += STEP) {
                buf ^= 1;
                const uint32_t t_s = t_x + buf * 64;
                const int r0 = c.c0 + u * kUnit, left = c.c1 - r0;
                const uint32_t have = __ballot_sync(0xffffffffu, (unsigned)block < (unsigned)p.num_blocks);
                block = look_up(u + STEP);
                if (!(ok = wait_all(&s_full[2 * x + buf], (seen >> buf) & 1, s_abort))) break;
                seen ^= 1u << buf;
                tc_fence_after();
                uint32_t z[2][32];
                float top[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) tmem_ld_32cols_max(t_s + 32 * i, z[i], top[i]);
                tmem_ld_wait();
                if (left < kUnit || have != 0xffffffffu) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) top[i] = hide(z[i], 32 * i, left, have, log2box);
                }
                const float mx = fmaxf(top[0], top[1]);
                const bool grow = mx > m + p.slack;
                if (__any_sync(0xffffffffu, grow)) {
                    float f = 1.f;
                    if (grow) {
                        // from the old reference to the new one
                        const float z = __fmul_rn(mx, p.scale);
                        const float r = fabsf(z) < kFar ? fmaf(mx, p.scale, -z) : 0.f;
                        f = m == kNone ? 0.f : ex2(fmaf(m - mx, p.scale, r - rest));
                        m = mx;
                        base = z;
                        rest = r;
                    }
                    far = __any_sync(0xffffffffu, !(fabsf(base) < kFar));
                    l *= f;
                    if (!begin) {
                        if (!(ok = wait_all(&o_done[2 * x + (buf ^ 1)], ((seen >> (buf ^ 1)) & 1) ^ 1, s_abort))) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int i = 0; i < D / 32; ++i) {
                            uint32_t o[32];
                            tmem_ld_32cols(t_o + 32 * i, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                            tmem_st_32cols(t_o + 32 * i, o);
                        }
                    }
                }
                begin = false;
                uint64_t sum[2] = {0ull, 0ull};
                const uint64_t by = pair(p.scale, p.scale);
                if (far) {
                    // (logits past kFar: differences of q . k)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            z[i][k] = __float_as_uint(fmaf(__uint_as_float(z[i][k]) - m, p.scale, rest));
                } else {
                    const uint64_t less = pair(-base, -base);
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int k = 0; k < 32; k += 2) {
                            float a, b;
                            unpair(fma2(pair(__uint_as_float(z[i][k]), __uint_as_float(z[i][k + 1])), by, less), a, b);
                            z[i][k] = __float_as_uint(a);
                            z[i][k + 1] = __float_as_uint(b);
                        }
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t y[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const float a = ex2(__uint_as_float(z[i][2 * k])), b = ex2(__uint_as_float(z[i][2 * k + 1]));
                        sum[k & 1] = add2(sum[k & 1], pair(a, b));
                        y[k] = pack_bf16(a, b);
                    }
                    tmem_st_16cols(t_s + 16 * i, y);
                }
                float a, b;
                unpair(add2(sum[0], sum[1]), a, b);
                l += a + b;
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive_warp(&p_full[2 * x + buf]);
            }
            if (!ok) break;
            float fix = 1.f;
            if (!(fabsf(base) < kFar)) base = base_of(m, p.scale, fix);
            l *= fix;
            if (!begin) {
                if (!(ok = wait_all(&o_done[2 * x], (seen & 1) ^ 1, s_abort))) break;
                if (!(ok = wait_all(&o_done[2 * x + 1], ((seen >> 1) & 1) ^ 1, s_abort))) break;
                tc_fence_after();
            }
            // SPLIT: the second group's sums join the first's, half of the dimensions at a time
            float other = 0.f;  // what they count
            if (SPLIT && n > 1) {
                if (x == 1) {
                    for (int h = 0; ok && h < 2; ++h) {
                        if (!(ok = wait_all(x_empty, (halves++ & 1) ^ 1, s_abort))) break;
                        if (h == 0) sh_ml[row] = make_float2(base, l);
#pragma unroll 1
                        for (int i = 0; i < D / 64; ++i) {
                            uint32_t o[32];
                            tmem_ld_32cols(t_o + h * (D / 2) + 32 * i, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                sh_x[(32 * i + k) * 128 + row] = __uint_as_float(o[k]) * fix;
                        }
                        mbar_arrive_warp(x_full);
                    }
                    if (!ok) break;
                    tc_fence_before();
                    continue;
                }
                if (!(ok = wait_all(x_full, halves & 1, s_abort))) break;
                const float2 ml = sh_ml[row];
                const float mx = fmaxf(base, ml.x);
                const float f = weight(base, l, mx);
                other = weight(ml.x, ml.y, mx);
                l = l * f + ml.y * other;
                fix *= f;
                base = mx;
            } else if (SPLIT && x == 1) {
                continue;
            }
            if (!waited) {
                wait_for_last();
                waited = true;
            }
            Joined j{};
            const int64_t at = ((int64_t)s * p.T + tk) * p.H * p.G + hd;
            if (c.whole && valid) {
                j = join_own(base, l, p.own_ml[at]);
                if (p.lse) p.lse[at] = j.lse;
            }
            __syncwarp();
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + s * p.o_seq + tk * p.o_tok + hd * p.o_head;
#pragma unroll 1
            for (int i = 0; i < D / 32; ++i) {
                uint32_t o[32];
                if (!begin) {
                    tmem_ld_32cols(t_o + 32 * i, o);
                    tmem_ld_wait();
                }
                float v[32];
#pragma unroll
                for (int k = 0; k < 32; ++k) v[k] = begin ? 0.f : __uint_as_float(o[k]) * fix;
                if (SPLIT && n > 1) {
                    if (i > 0 && i * 32 % (D / 2) == 0) {
                        mbar_arrive_warp(x_empty);
                        if (!(ok = wait_all(x_full, ++halves & 1, s_abort))) break;
                    }
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        v[k] += sh_x[((32 * i) % (D / 2) + k) * 128 + row] * other;
                }
                if (c.whole && valid) {
                    const float4* own = reinterpret_cast<const float4*>(p.own + at * D + 32 * i);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float4 a = join4(j, make_float4(v[8 * k], v[8 * k + 1], v[8 * k + 2], v[8 * k + 3]), own[2 * k]);
                        const float4 b = join4(j, make_float4(v[8 * k + 4], v[8 * k + 5], v[8 * k + 6], v[8 * k + 7]), own[2 * k + 1]);
                        *reinterpret_cast<uint4*>(out + 32 * i + 8 * k) =
                            make_uint4(pack_bf16(a.x, a.y), pack_bf16(a.z, a.w), pack_bf16(b.x, b.y), pack_bf16(b.z, b.w));
                    }
                } else if (valid) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        p.partial[((int64_t)c.slot * (D / 4) + 8 * i + k) * p.tile + r] =
                            make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                }
                __syncwarp();
            }
            if (!ok) break;
            if (SPLIT && n > 1) {
                mbar_arrive_warp(x_empty);
                ++halves;
            }
            if (!c.whole && valid) p.partial_ml[(int64_t)c.slot * p.tile + r] = make_float2(base, l);
            tc_fence_before();  // the next piece's products overwrite O
        }
        if (!ok) {
            *s_abort = 1;
            if (lane == 0) set_error(p.status, kDevErrTimeout, 3u);
        }
        if (!waited) wait_for_last();
        if (threadIdx.x == 0) {
            p.joins[blockIdx.x] = make_int4(c.seq0, c.h, c.row0, ok && c.rows > 0 ? join_of(c.rows, c.parts) : 0);
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 8) tmem_dealloc(tmem, 512);
}

template <int D, bool SPLIT>
cudaError_t go(const Params& p, cudaStream_t s) {
    const int bs = 1 << p.log2bs, box = bs < kUnit ? bs : kUnit;
    const int64_t outer = (int64_t)p.num_blocks * p.H;
    CUtensorMap k, v;
    if (!make_map_3d_bf16(&k, p.k, D, bs, outer, D, (int64_t)bs * D, box) ||
        !make_map_3d_bf16(&v, p.v, D, bs, outer, D, (int64_t)bs * D, box))
        return cudaErrorInvalidValue;
    auto kern = prefix_tc_kernel<D, SPLIT>;
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(kern, Cfg<D>::BYTES, done);
    if (e != cudaSuccess) return e;
    return launch_early(kern, (unsigned)(p.runs * p.team), kThreads, Cfg<D>::BYTES, s, k, v, p);
}

}  // namespace

bool tc_takes(const PrefixArgs& a) {
    return a.own.dtype == RKV_DTYPE_BF16 && a.own.pg.log2bs >= 3 && encode_fn() != nullptr;
}

cudaError_t launch_tc(const Params& p, int d, cudaStream_t s) {
    if (p.tile == 128) return d == 128 ? go<128, true>(p, s) : go<64, true>(p, s);
    return d == 128 ? go<128, false>(p, s) : go<64, false>(p, s);
}

}  // namespace prefix
}  // namespace rkv
