// k_prefix_tc.cu -- attention over shared prefixes on the tensor cores (tcgen05, TMEM,
// TMA): bf16 pools in blocks of 8 rows or more.  See k_prefix.cu for what is computed and
// rkv_prefix.cuh for the line of work.
//
// The queries of all sequences of a prefix that use a KV head are the rows of two products
// with the prefix's keys and values: S = Q K^T, O += P V, each 128 queries x 128 rows a
// step, accumulated in TMEM.  One block an SM, ten warps:
//   * warp 9: TMA producer, a ring of tiles of 128 rows (K and V in the order in which
//     they are used) through the prefix's block table, one copy per block (of up to 128
//     rows) and 64 columns, 128-byte swizzle.  Rows past the prefix in its last block are
//     cleared in V, where they would meet a probability of 0.
//   * warp 8: issues the MMAs.  S from shared memory; O += P V with P as the operand in
//     TMEM and V as it lies, its rows being the contracted index (an MN-major operand).
//   * warps 0-3 and 4-7: softmax, one query a thread, which is a row of TMEM: maxima, sums
//     and scales take no exchange between threads.  P is
//     written over S as bf16 (one part, 2^-8 of it: a second would take the tensor cores
//     half as long again).  O is brought to a new maximum only where a logit passes the old
//     one by more than 8 (log2), so that hardly ever anybody waits for it.
// The two softmax groups keep each other's products off the critical path.  With more
// than 128 queries a prefix they take 128 each, all rows; with fewer (SPLIT) the same
// queries, every other unit of rows each, and join at a piece's end through shared memory.
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

constexpr int kUnit = 128;
constexpr int kChunk = kUnit * 128;  // 128 rows of 64 bf16
constexpr int kThreads = 320;

template <int D>
struct Cfg {
    static constexpr int KC = D / 64;
    static constexpr int TILE = KC * kChunk;  // 128 rows
    static constexpr int STAGES = D == 128 ? 5 : 8;
    static constexpr int RING = 2 * TILE;     // behind the queries of both groups
    static constexpr int BARS = RING + STAGES * TILE;
    static constexpr int NUM_BARS = 2 * STAGES + 8 + 4;
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
RKV_DEV uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
RKV_DEV void unpair(uint64_t v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
RKV_DEV uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}
RKV_DEV bool wait_all(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag));
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
    constexpr int LOOK = SPLIT ? 2 : 1;  // units of S ahead of P V
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint8_t* ring = smem + C::RING;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BARS);
    uint64_t* empty = full + C::STAGES;
    uint64_t* q_full = empty + C::STAGES;  // [2]
    uint64_t* s_full = q_full + 2;         // [2]
    uint64_t* p_full = s_full + 2;         // [2]
    uint64_t* o_done = p_full + 2;         // [2]
    uint64_t* tail_bar = o_done + 2;
    uint64_t* drain_bar = tail_bar + 1;
    uint64_t* x_full = drain_bar + 1;  // SPLIT: half of the second group's output is there
    uint64_t* x_empty = x_full + 1;
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(x_empty + 1);
    volatile int* s_abort = reinterpret_cast<volatile int*>(s_tmem + 1);
    float2* sh_ml = reinterpret_cast<float2*>(smem + C::ML);
    float* sh_x = reinterpret_cast<float*>(smem + C::TILE);  // [D / 2][128] (the second group's queries are the first's)

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t run = blockIdx.x;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], 4);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
            mbar_init(&o_done[i], 1);
        }
        mbar_init(tail_bar, 1);
        mbar_init(drain_bar, 1);
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
    wait_for_last();
    Place place = find_place<kUnit>(p, run);
    Piece c{};
    bool ok = true;

    if (warp == 9) {
        // ------------------------------------------------------- producer --
        const int log2box = p.log2bs < 7 ? p.log2bs : 7, box = 1 << log2box;
        const int copies = (kUnit >> log2box) * C::KC;  // of a tile, at most 32
        uint32_t kt = 0, tails = 0;
        auto load = [&](const CUtensorMap* map, int u, bool is_v) {
            const int st = kt % C::STAGES, r0 = c.c0 + u * kUnit;
            const int b = lane / C::KC, ch = lane - b * C::KC, r = r0 + (b << log2box);
            // an outer coordinate past the pool reads as zeros
            int z = p.num_blocks * p.H;
            if (lane < copies && r < c.c1) {
                const int blk = p.table[(int64_t)c.i * p.max_blocks + (r >> p.log2bs)];
                if ((unsigned)blk < (unsigned)p.num_blocks)
                    z = blk * p.H + c.h;
                else if (!is_v && ch == 0)
                    set_error(p.status, kDevErrIndex, (unsigned)r);
            }
            if (!wait_all(&empty[st], ((kt / C::STAGES) & 1) ^ 1, s_abort)) return false;
            uint8_t* dst = ring + st * C::TILE;
            const bool clear = is_v && r0 + kUnit > c.c1 && (c.c1 & (box - 1)) != 0;
            uint64_t* bar = clear ? tail_bar : &full[st];
            if (lane == 0) mbar_arrive_expect_tx(bar, C::TILE);
            __syncwarp();
            if (lane < copies)
                tma_load_3d(dst + ch * kChunk + (b << log2box) * 128, map, bar, ch * 64,
                            r & ((1 << p.log2bs) - 1), z);
            ++kt;
            if (clear) {
                if (!wait_all(tail_bar, tails++ & 1, s_abort)) return false;
                const int from = c.c1 - r0, to = (from + box) & ~(box - 1);
                for (int e = lane; e < (to - from) * 8 * C::KC; e += 32) {
                    const int row = from + e / (8 * C::KC), x = e % (8 * C::KC);
                    *reinterpret_cast<uint4*>(dst + (x >> 3) * kChunk + row * 128 + (x & 7) * 16) =
                        make_uint4(0u, 0u, 0u, 0u);
                }
                fence_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[st]);
            }
            return true;
        };
        while (ok && next_piece<kUnit>(p, run, place, c)) {
            const int n = units_in(c);
            for (int u = 0; ok && u < LOOK && u < n; ++u) ok = load(&kmap, u, false);
            for (int u = 0; ok && u < n; ++u) {
                ok = load(&vmap, u, true);
                if (ok && u + LOOK < n) ok = load(&kmap, u + LOOK, false);
            }
        }
        if (!ok) {
            *s_abort = 1;
            if (lane == 0) set_error(p.status, kDevErrTimeout, 1u);
        }
        // every copy issued has landed before the block may end
        volatile int never = 0;
        for (uint32_t u = kt > (uint32_t)C::STAGES ? kt - C::STAGES : 0; u < kt; ++u)
            mbar_wait(&full[u % C::STAGES], (u / C::STAGES) & 1, &never);
    } else if (warp == 8) {
        // ----------------------------------------------------- MMA issuer --
        constexpr uint32_t kIdescS = idesc_bf16(128, kUnit);
        constexpr uint32_t kIdescO = idesc_bf16(128, D) | (1u << 16);  // B by rows
        if (lane == 0) {
            uint32_t kt = 0, pieces = 0, done[2] = {0, 0}, filled[2] = {0, 0}, second = 0;
            auto logits = [&](int x, const uint8_t* tile) {
                const uint8_t* q = smem + (SPLIT ? 0 : x * C::TILE);
#pragma unroll
                for (int ch = 0; ch < C::KC; ++ch) {
                    const uint64_t a = sdesc_sw128(q + ch * kChunk), b = sdesc_sw128(tile + ch * kChunk);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_bf16(tmem + x * 128, a + 2 * k, b + 2 * k, kIdescS, (ch | k) != 0);
                }
                mma_commit(&s_full[x]);
            };
            auto values = [&](int x, const uint8_t* tile, bool begin) {
                const uint64_t b = sdesc_rows(tile, kChunk);
#pragma unroll
                for (int k = 0; k < kUnit / 16; ++k)
                    mma_bf16_ts(tmem + 256 + x * D, tmem + x * 128 + 8 * k, b + (2048 >> 4) * k, kIdescO,
                                !begin || k != 0);
                mma_commit(&o_done[x]);
                ++done[x];
            };
            while (ok && next_piece<kUnit>(p, run, place, c)) {
                const int n = units_in(c);
                if (n == 0) continue;
                const bool two = !SPLIT && c.rows > 128;
                if (!(ok = mbar_wait(&q_full[0], pieces++ & 1, s_abort))) break;
                if (two && !(ok = mbar_wait(&q_full[1], second++ & 1, s_abort))) break;
                tc_fence_after();
                for (int u = 0; ok && u < LOOK && u < n; ++u, ++kt) {
                    const int st = kt % C::STAGES;
                    if (!(ok = mbar_wait(&full[st], (kt / C::STAGES) & 1, s_abort))) break;
                    logits(SPLIT ? u : 0, ring + st * C::TILE);
                    if (two) logits(1, ring + st * C::TILE);
                    mma_commit(&empty[st]);
                }
                for (int u = 0; ok && u < n; ++u) {
                    const int sv = kt % C::STAGES, sk = (kt + 1) % C::STAGES;
                    const bool more = u + LOOK < n;
                    if (!(ok = mbar_wait(&full[sv], (kt / C::STAGES) & 1, s_abort))) break;
                    for (int i = 0; i < (two ? 2 : 1); ++i) {
                        const int x = SPLIT ? u & 1 : i;
                        if (!(ok = mbar_wait(&p_full[x], filled[x]++ & 1, s_abort))) break;
                        tc_fence_after();
                        values(x, ring + sv * C::TILE, SPLIT ? u < 2 : u == 0);
                        if (i == (two ? 1 : 0)) mma_commit(&empty[sv]);
                        if (!more) continue;
                        if (i == 0 &&
                            !(ok = mbar_wait(&full[sk], ((kt + 1) / C::STAGES) & 1, s_abort)))
                            break;
                        // S takes the place of P, which the product has to be done with
                        if (!(ok = mbar_wait(&o_done[x], (done[x] - 1) & 1, s_abort))) break;
                        logits(x, ring + sk * C::TILE);
                        if (i == (two ? 1 : 0)) mma_commit(&empty[sk]);
                    }
                    kt += more ? 2 : 1;
                }
            }
            if (!ok) {
                *s_abort = 1;
                set_error(p.status, kDevErrTimeout, 2u);
            }
            // every MMA issued so far is done before TMEM is released
            mma_commit(drain_bar);
            volatile int never = 0;
            mbar_wait(drain_bar, 0, &never);
        }
    } else {
        // -------------------------------------------------------- softmax --
        const int x = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t t_s = tmem + ((uint32_t)(warp & 3) << 21) + x * 128;
        const uint32_t t_o = tmem + ((uint32_t)(warp & 3) << 21) + 256 + x * D;
        const int log2box = p.log2bs < 7 ? p.log2bs : 7, boxes = kUnit >> log2box;
        uint32_t seen = 0, done = 0, halves = 0;  // phases of s_full, o_done, x_full
        while (ok && next_piece<kUnit>(p, run, place, c)) {
            if (!SPLIT && x == 1 && c.rows <= 128) continue;
            if (threadIdx.x == 0 && bad_length(p, c)) set_error(p.status, kDevErrIndex, (unsigned)c.i);
            const int n = units_in(c);
            const int r = (SPLIT ? 0 : x * 128) + row;
            const bool valid = r < c.rows;
            int s = 0, tk = 0, hd = 0;
            if (valid) place_of_row(p, c.seq0, c.h, c.row0 + r, s, tk, hd);
            if (n > 0 && (!SPLIT || x == 0)) {
                const uint4* q = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) +
                                                                s * p.q_seq + tk * p.q_tok + hd * p.q_head);
                uint8_t* dst = smem + x * C::TILE + row * 128;
#pragma unroll
                for (int u = 0; u < D / 8; ++u) {
                    uint4 y = make_uint4(0u, 0u, 0u, 0u);
                    if (valid) y = q[u];
                    y.x ^= p.flip; y.y ^= p.flip; y.z ^= p.flip; y.w ^= p.flip;
                    *reinterpret_cast<uint4*>(dst + (u >> 3) * kChunk + (((u & 7) ^ (row & 7)) << 4)) = y;
                }
                fence_async();
                mbar_arrive_warp(&q_full[x]);
            }
            // m: running maximum of q . k; sums are relative to 2^(m * scale)
            float m = kNone, l = 0.f;
            bool begin = true;
            for (int u = SPLIT ? x : 0; u < n; u += LOOK) {
                const int r0 = c.c0 + u * kUnit, left = c.c1 - r0;
                bool there = true;
                if (lane < boxes && (lane << log2box) < left) {
                    const int rb = r0 + (lane << log2box);
                    const int blk = p.table[(int64_t)c.i * p.max_blocks + (rb >> p.log2bs)];
                    there = (unsigned)blk < (unsigned)p.num_blocks;
                }
                const uint32_t have = __ballot_sync(0xffffffffu, there);
                if (!(ok = wait_all(&s_full[x], seen++ & 1, s_abort))) break;
                tc_fence_after();
                // the row's maximum; the values come again below, 32 at a time (all at once
                // they would take more registers than there are)
                const bool masked = left < kUnit || have != 0xffffffffu;
                float mx = -INFINITY;
#pragma unroll
                for (int i = 0; i < 4; i += 2) {
                    uint32_t z0[32], z1[32];
                    float t0, t1;
                    tmem_ld_32cols_max(t_s + 32 * i, z0, t0);
                    tmem_ld_32cols_max(t_s + 32 * i + 32, z1, t1);
                    tmem_ld_wait();
                    if (masked) {
                        t0 = hide(z0, 32 * i, left, have, log2box);
                        t1 = hide(z1, 32 * i + 32, left, have, log2box);
                    }
                    mx = fmaxf(mx, fmaxf(t0, t1));
                }
                const bool grow = mx > m + p.slack;
                if (__any_sync(0xffffffffu, grow)) {
                    const float f = grow ? (m == kNone ? 0.f : ex2((m - mx) * p.scale)) : 1.f;
                    if (grow) m = mx;
                    l *= f;
                    if (!begin) {
                        if (!(ok = wait_all(&o_done[x], (done - 1) & 1, s_abort))) break;
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
                const uint64_t less = pair(-m, -m), by = pair(p.scale, p.scale);
                uint64_t sum[2] = {0ull, 0ull};
                uint32_t z[2][32];
                tmem_ld_32cols(t_s, z[0]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    tmem_ld_wait();
                    if (i < 3) tmem_ld_32cols(t_s + 32 * i + 32, z[(i + 1) & 1]);
                    uint32_t (&at)[32] = z[i & 1];
                    if (masked) hide(at, 32 * i, left, have, log2box);
                    uint32_t y[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        float a, b;
                        unpair(mul2(add2(pair(__uint_as_float(at[2 * k]), __uint_as_float(at[2 * k + 1])), less), by), a, b);
                        a = ex2(a);
                        b = ex2(b);
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
                mbar_arrive_warp(&p_full[x]);
                ++done;
            }
            if (!ok) break;
            float fix;
            float base = base_of(m, p.scale, fix);
            l *= fix;
            if (!begin) {
                if (!(ok = wait_all(&o_done[x], (done - 1) & 1, s_abort))) break;
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
        if (threadIdx.x == 0) {
            p.joins[2 * run] = make_int4(c.seq0, c.rows, c.h, c.row0);
            p.joins[2 * run + 1] = make_int4(ok ? (int)c.parts : 0, 0, 0, 0);
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
    return launch_early(kern, (unsigned)p.runs, kThreads, Cfg<D>::BYTES, s, k, v, p);
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
