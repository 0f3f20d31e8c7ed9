// k_tokens.cu -- new tokens on their way to the cache: rotary positions, the
// append to a paged pool, and the append to a 4-bit pool, in one kernel; and
// reading 4-bit rows back.
//
// Rotation: pair i of a head is turned by pos * f_i.  The plan holds f_i /
// (2 pi) as a 64-bit fixed-point part of a turn, so the low 64 bits of
// pos * turns[i] are the angle modulo one turn, exactly; the upper 32 of them go to
// the nearest quarter turn in whole numbers and from there, at most pi / 4, through
// the Taylor series of sine and cosine (sine_of: within 2 ulp).
//
// Every value is read and written once, 16 bytes (eight bf16) a step, so many
// tokens are bound by HBM and a decode step by launch and load latency.  A
// thread takes the same pairs of several heads of one token: it issues all of
// its loads first, then finds the position (and, with an append, the row: a
// warp searches the ragged sequences 32 ways) and computes eight sines once for
// its heads; nothing waits on a table of sines.  Measured (one GB300): 16384
// tokens of 48 heads, 403 MB: 61 us, 6.6 TB/s; 28.9 thousand ragged tokens
// appended with their queries, 730 MB: 107 us, 6.8 TB/s; 64 tokens of 40 heads
// 3.1 us, appended 3.7 us (one after the other in a captured graph).
//
// 4 bits: four neighbouring lanes own one row; lane t holds values 32 w + 8 t
// .. + 7 of every group w, so a group's minimum and maximum take two shuffles
// and the lane's codes of all groups are one store of 16 bytes (8 at head_dim
// 64).  With t = x - low rounded to fp32, t * r + 1.5 * 2^23 in one FMA rounds the
// exact product to a whole number (halves to even) and leaves it in the low
// mantissa bits.  16.8
// thousand tokens with their queries, written and read back, 473 MB: 80 us,
// 5.9 TB/s (the blocks wait for their rows' places).
#include <float.h>

#include "rkv_common.cuh"
#include "rkv_internal.h"

namespace rkv {
namespace {

// Threads of a block: few enough that its tokens' places and sines hold up few
// others (16384 tokens appended: 61.6 us, at 4 bits 62.1; 256 threads: 62.6 and
// 64.5; 64: 61.9 and 64.5), and as many as a plan has pairs.
constexpr int kThreads = 128;
static_assert(kThreads >= RKV_MAX_ROT_DIM / 2, "a thread per pair of the plan");

struct Div {  // n / d for 0 <= n < 2^31
    uint32_t d, mul, shift;
};
Div make_div(uint32_t d) {
    uint32_t l = 0;
    while ((1ull << l) < d) ++l;
    const uint64_t m = ((1ull << (31 + l)) + d - 1) / d;
    return Div{d, (uint32_t)m, 31 + l};
}
RKV_DEV uint32_t div_by(uint32_t n, const Div& v) {
    return (uint32_t)(((uint64_t)n * v.mul) >> v.shift);
}

struct Params {
    TokenArgs a;
    int half;          // rot / 2
    int iph, ipv;      // items of a rotated head, of a copied head
    int uq, uk, ukv;   // a token's units: those of q, of k, of k and v
    int tokens;        // tokens a block may meet
    // Blocks take the q of some tokens, or k and v.  In an append, of `period`
    // blocks in a row the last is one of the `minor` rarer kind (q where minor_q),
    // while there are any, so that both kinds are on an SM at a time: q streams
    // while the blocks of k and v wait for their rows' places (28.9 thousand
    // tokens 118 -> 110 us, 16.8 thousand at 4 bits 95 -> 86 us).  Where nothing
    // waits, q_blocks of q come first (rotation alone: 64.4 us against 65.5).
    uint32_t minor, q_blocks;
    int minor_q;
    int64_t total_q, total_kv;
    Div div_q, div_kv, div_iph, div_ipv, div_seq, div_half, period;
};

// What a block knows of each of its tokens.
struct Token {
    int64_t row;  // pool row of head 0 (heads are 1 << log2bs rows apart), or -1
    int pos;
    int live;     // 0: padding behind the last sequence
};

// Eight elements as loaded.
template <typename T> struct Eight;
template <> struct Eight<__nv_bfloat16> {
    uint4 u;
    RKV_DEV void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
    RKV_DEV void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = u; }
    RKV_DEV void get(float* o) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            o[2 * t] = __uint_as_float(w[t] << 16);
            o[2 * t + 1] = __uint_as_float(w[t] & 0xffff0000u);
        }
    }
    static RKV_DEV uint32_t pack(float lo, float hi) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&b);
    }
    RKV_DEV void set(const float* v) {
        u = make_uint4(pack(v[0], v[1]), pack(v[2], v[3]), pack(v[4], v[5]), pack(v[6], v[7]));
    }
};
template <> struct Eight<float> {
    float4 a, b;
    RKV_DEV void load(const float* p) {
        a = reinterpret_cast<const float4*>(p)[0];
        b = reinterpret_cast<const float4*>(p)[1];
    }
    RKV_DEV void store(float* p) const {
        reinterpret_cast<float4*>(p)[0] = a;
        reinterpret_cast<float4*>(p)[1] = b;
    }
    RKV_DEV void get(float* o) const {
        o[0] = a.x; o[1] = a.y; o[2] = a.z; o[3] = a.w;
        o[4] = b.x; o[5] = b.y; o[6] = b.z; o[7] = b.w;
    }
    RKV_DEV void set(const float* v) {
        a = make_float4(v[0], v[1], v[2], v[3]);
        b = make_float4(v[4], v[5], v[6], v[7]);
    }
};
// One element (the rotated part does not split into steps of eight).
template <typename T> RKV_DEV T one_of(float v);
template <> RKV_DEV float one_of<float>(float v) { return v; }
template <> RKV_DEV __nv_bfloat16 one_of<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// (cos, sin) of an angle in units of 2^-32 turn.  The angle is taken to the
// nearest quarter turn in whole numbers, and what is left, at most pi / 4, goes
// through the Taylor series of both functions (to x^9 and x^10: the next terms
// are below 2^-28 of the result); the quarter turns swap and change signs.
RKV_DEV void sine_of(uint32_t turn, float& c, float& s) {
    const uint32_t near = turn + 0x20000000u;
    const float x = (float)(int32_t)(turn - (near & 0xc0000000u)) * 1.4629180792671596e-9f;  // 2 pi 2^-32
    const float t = x * x;
    float u = fmaf(t, 2.7557319e-6f, -1.9841270e-4f);  // 1 / 9!, -1 / 7!
    u = fmaf(t, u, 8.3333333e-3f);
    u = fmaf(t, u, -1.6666667e-1f);
    u = fmaf(x * t, u, x);
    float v = fmaf(t, -2.7557319e-7f, 2.4801587e-5f);  // -1 / 10!, 1 / 8!
    v = fmaf(t, v, -1.3888889e-3f);
    v = fmaf(t, v, 4.1666667e-2f);
    v = fmaf(t, v, -0.5f);
    v = fmaf(t, v, 1.f);
    const bool swap = (near & 0x40000000u) != 0;
    const uint32_t cs = (near + 0x40000000u) & 0x80000000u, sn = near & 0x80000000u;
    c = __uint_as_float(__float_as_uint(swap ? u : v) ^ cs);
    s = __uint_as_float(__float_as_uint(swap ? v : u) ^ sn);
}
// The plan's turns in shared memory (lanes ask for different pairs, which
// constant memory would serve one after another), so that neighbouring lanes'
// first, second, .. pairs lie side by side: PAIRS pairs a lane.
constexpr int kTurns = RKV_MAX_ROT_DIM / 2;
template <int PAIRS>
RKV_DEV int turn_slot(int i) {
    return (i % PAIRS) * (kTurns / PAIRS) + i / PAIRS;
}
// (cos, sin) times the factor of pair i at a position.
template <int PAIRS>
RKV_DEV void turn_of(const TokenArgs& a, const uint64_t* turns, int pos, int i, float& c, float& s) {
    const uint64_t turn = (uint64_t)(int64_t)pos * turns[turn_slot<PAIRS>(i)];
    sine_of((uint32_t)(turn >> 32), c, s);
    c *= a.factor;
    s *= a.inverse ? -a.factor : a.factor;
}

// The last s with cu[s] <= j, searched 32 ways by a warp (cu[0] <= j).
RKV_DEV int64_t find_seq(const int32_t* cu, int64_t n, int64_t j) {
    int64_t lo = 0, hi = n;
    const int lane = threadIdx.x & 31;
    while (hi - lo > 1) {
        const int64_t step = (hi - lo + 31) / 32, at = lo + step * (lane + 1);
        const bool below = at < hi && cu[at] <= j;
        const int c = __popc(__ballot_sync(0xffffffffu, below));
        lo += step * c;
        if (lo + step < hi) hi = lo + step;
    }
    return lo;
}

// The place of token j in an append (by a whole warp).
RKV_DEV Token place_token(const TokenArgs& a, int64_t j) {
    const int lane = threadIdx.x & 31;
    Token t;
    t.live = 1;
    t.row = -1;
    t.pos = a.positions ? a.positions[j] : 0;
    int64_t s, first, count, len;
    if (a.cu == nullptr) {
        s = (uint32_t)j / (uint32_t)a.per_seq;
        first = s * a.per_seq;
        count = a.per_seq;
        len = a.lens[s];
    } else if (a.num_seqs <= 32) {
        // one look at all sequences: those that end at or before j come before its own
        const bool in = lane < a.num_seqs;
        const int c0 = in ? a.cu[lane] : 0, c1 = in ? a.cu[lane + 1] : 0, n = in ? a.lens[lane] : 0;
        const int before = __popc(__ballot_sync(0xffffffffu, in && c1 <= j));
        t.live = before < a.num_seqs && j >= __shfl_sync(0xffffffffu, c0, 0);
        s = before < a.num_seqs ? before : 0;
        first = __shfl_sync(0xffffffffu, c0, (int)s);
        count = __shfl_sync(0xffffffffu, c1, (int)s) - first;
        len = __shfl_sync(0xffffffffu, n, (int)s);
    } else {
        t.live = j < a.cu[a.num_seqs] && j >= a.cu[0];
        s = t.live ? find_seq(a.cu, a.num_seqs, j) : 0;
        first = a.cu[s];
        count = a.cu[s + 1] - first;
        len = a.lens[s];
    }
    if (!t.live) return t;
    const int64_t r = len - count + (j - first);
    if (!a.positions) t.pos = (int)r;
    bool ok = r >= 0 && r < ((int64_t)a.pg.max_blocks << a.pg.log2bs);
    if (ok) {
        const int blk = a.pg.table[s * a.pg.max_blocks + (r >> a.pg.log2bs)];
        ok = (unsigned)blk < (unsigned)a.pg.num_blocks;
        t.row = (((int64_t)blk * a.pg.H) << a.pg.log2bs) + (r & ((1 << a.pg.log2bs) - 1));
    }
    if (!ok) {
        t.row = -1;
        if (lane == 0) set_error(a.status, kDevErrIndex, (unsigned)s);
    }
    return t;
}

// Smallest and largest; NaN where any is NaN.
RKV_DEV float min_of(float a, float b, float c) {
    float y;
    asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}
RKV_DEV float max_of(float a, float b, float c) {
    float y;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}
// x / 15 rounded to nearest for 0 <= x < infinity (NaN for infinity): a quotient
// by the divisor's reciprocal and one correction by its remainder (division by a
// divisor known in advance, Brisebarre, Muller and Raina, 2004; compared with the
// division for every such x).
RKV_DEV float fifteenth(float x) {
    constexpr float c = 1.f / 15.f;
    const float q = x * c;
    return fmaf(fmaf(-15.f, q, x), c, q);
}

// One 4-bit row's share of a lane: values of W groups.  The four lanes of the
// row take part.
template <int W>
RKV_DEV void quantise_store(const float (&v)[W][8], int t, bool write, uint8_t* codes,
                            uint32_t* scales) {
    const uint32_t quad = 0xfu << (threadIdx.x & 28);
    uint32_t h[W][2], pair = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        float mn = min_of(v[w][0], v[w][1], v[w][2]), mx = max_of(v[w][0], v[w][1], v[w][2]);
        mn = min_of(min_of(mn, v[w][3], v[w][4]), v[w][5], v[w][6]);
        mx = max_of(max_of(mx, v[w][3], v[w][4]), v[w][5], v[w][6]);
        mn = min_of(mn, mn, v[w][7]);
        mx = max_of(mx, mx, v[w][7]);
#pragma unroll
        for (int o = 1; o <= 2; o <<= 1) {
            mn = min_of(mn, mn, __shfl_xor_sync(quad, mn, o));
            mx = max_of(mx, mx, __shfl_xor_sync(quad, mx, o));
        }
        __nv_bfloat16 lo = __float2bfloat16_rd(mn);
        float lof = __bfloat162float(lo);
        __nv_bfloat16 sc = __float2bfloat16_ru(fifteenth(mx - lof));
        float sf = __bfloat162float(sc);
        // (an infinity is the smallest or the largest and makes the difference one, or NaN)
        if (!(sf <= FLT_MAX)) {
            sc = lo = __ushort_as_bfloat16(0x7fff);
            sf = 0.f;
        }
        const float r = sf >= FLT_MIN ? __frcp_rn(sf) : 0.f;
        if (sf < FLT_MIN) lof = 0.f;
        uint32_t c[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            c[i] = __float_as_uint(fmaf(v[w][i] - lof, r, 12582912.f));
#pragma unroll
        for (int k = 0; k < 2; ++k)
            h[w][k] = (c[4 * k] + 16u * c[4 * k + 1] + 256u * c[4 * k + 2] + 4096u * c[4 * k + 3]) &
                      0xffffu;
        if (t == w)
            pair = (uint32_t)__bfloat16_as_ushort(sc) | ((uint32_t)__bfloat16_as_ushort(lo) << 16);
    }
    if (!write) return;
    if constexpr (W == 4) {
        reinterpret_cast<uint4*>(codes)[t] =
            make_uint4(h[0][0] | (h[1][0] << 16), h[2][0] | (h[3][0] << 16),
                       h[0][1] | (h[1][1] << 16), h[2][1] | (h[3][1] << 16));
    } else {
        reinterpret_cast<uint2*>(codes)[t] =
            make_uint2(h[0][0] | (h[1][0] << 16), h[0][1] | (h[1][1] << 16));
    }
    if (t < W) scales[t] = pair;
}

// The lane's part of a K row turned in place: values 32 w + 8 t .. of group w;
// cs, sn: the token's cosines and sines, x: the row (partners that may lie in
// another lane are read again).
template <typename T, bool VEC, bool INTER, int W>
RKV_DEV void turn_row(float (&v)[W][8], const T* x, int t, const Params& p, const float* cs,
                      const float* sn) {
    const int rot = p.a.rot, half = p.half;
    if constexpr (VEC && !INTER) {
        // halves that are whole groups: both elements of a pair are the lane's own
        const auto pairs = [&](float (&x)[8], float (&y)[8], int i0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float c = cs[i0 + i], s = sn[i0 + i], a = x[i], b = y[i];
                x[i] = a * c - b * s;
                y[i] = b * c + a * s;
            }
        };
        if (half == 16 * W) {
#pragma unroll
            for (int w = 0; w < W / 2; ++w) pairs(v[w], v[w + W / 2], 32 * w + 8 * t);
            return;
        }
        if (W == 4 && half == 32) {
            pairs(v[0], v[1], 8 * t);
            return;
        }
    }
#pragma unroll
    for (int w = 0; w < W; ++w) {
        const int e = 32 * w + 8 * t;
        if (e >= rot) continue;
        if constexpr (VEC && INTER) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float c = cs[e / 2 + i], s = sn[e / 2 + i], a = v[w][2 * i], b = v[w][2 * i + 1];
                v[w][2 * i] = a * c - b * s;
                v[w][2 * i + 1] = b * c + a * s;
            }
        } else if constexpr (VEC) {
            const bool first = e < half;
            const int i0 = first ? e : e - half;
            Eight<T> other;
            other.load(x + (first ? e + half : e - half));
            float o[8];
            other.get(o);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float c = cs[i0 + i], s = first ? -sn[i0 + i] : sn[i0 + i];
                v[w][i] = v[w][i] * c + o[i] * s;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int at = e + i;
                if (at < rot) {
                    const bool first = INTER ? (at & 1) == 0 : at < half;
                    const int k = INTER ? at >> 1 : (first ? at : at - half);
                    const int other = INTER ? at ^ 1 : (first ? at + half : at - half);
                    const float o = Elem<T>::to_f(x[other]);
                    v[w][i] = v[w][i] * cs[k] + (first ? -o : o) * sn[k];
                }
            }
        }
    }
}

// Heads that a thread takes together.
template <typename T> constexpr int kHeads = sizeof(T) == 2 ? 4 : 2;

// VEC: the rotated part splits into whole steps of eight.  A unit is one item
// (the eight pairs, or eight elements, that a thread holds; without VEC one
// pair or element) of kHeads heads, or a lane of a 4-bit row.
// 64 registers, eight blocks an SM, where the compiler would take more (28.9
// thousand tokens appended at 80: 127 us against 122; 16384 at 4 bits 72 against
// 64.5; at 56 and less these spill: 81 and 78); the others are left to it (the
// interleaved rotation of 16384 x 48 heads 67.5 us, 69.6 bounded).
template <typename T, bool INTER, bool Q4>
constexpr int kBlocks = Q4 || (sizeof(T) == 2 && !INTER) ? 8 : 0;
template <typename T, bool VEC, bool INTER, bool Q4, int W>
__global__ void __launch_bounds__(kThreads, kBlocks<T, INTER, Q4>) tokens_kernel(const __grid_constant__ Params p) {
    extern __shared__ __align__(16) uint8_t smem[];
    Token* tok = reinterpret_cast<Token*>(smem);                          // [tokens]
    float* sines = reinterpret_cast<float*>(smem + sizeof(Token) * p.tokens);  // 4 bits: [tokens][2][half]
    __shared__ uint64_t turns[kTurns];
    constexpr int HG = kHeads<T>, PAIRS = VEC ? (INTER ? 4 : 8) : 1;
    const TokenArgs& a = p.a;
    let_next_begin();
    wait_for_last();
    const int tid = threadIdx.x;
    const bool append = a.pg.table != nullptr;
    bool is_q;
    uint32_t block;  // of its kind
    if (append) {
        const uint32_t turn = div_by(blockIdx.x, p.period);
        const bool rare = turn < p.minor && blockIdx.x - turn * p.period.d == p.period.d - 1;
        is_q = rare == (p.minor_q != 0);
        block = rare ? turn : blockIdx.x - min(turn, p.minor);
    } else {
        is_q = blockIdx.x < p.q_blocks;
        block = blockIdx.x - (is_q ? 0 : p.q_blocks);
    }
    const int64_t id0 = (int64_t)block * kThreads;
    const int units = is_q ? p.uq : p.ukv;
    const int64_t total = is_q ? p.total_q : p.total_kv;
    const int64_t j0 = id0 / units;
    const uint32_t e = (uint32_t)(id0 - j0 * units) + tid;  // unit counted from token j0
    const bool on = id0 + tid < total;
    const uint32_t tl = div_by(e, is_q ? p.div_q : p.div_kv);
    const int64_t j = j0 + tl;
    const uint32_t unit = e - tl * units;

    // sources: tokens by sequence, or numbered through
    const int64_t seq = a.cu ? 0 : div_by((uint32_t)j, p.div_seq), within = j - seq * a.per_seq;
    const bool is_k = !Q4 && !is_q && unit < (uint32_t)p.uk;
    const RowsView& src = is_q ? a.q : (is_k ? a.k : a.v);
    uint32_t item = 0, head = 0;
    bool turning = false;  // the item is turned (else copied)
    int at = 0;            // its first element
    Eight<T> x[HG], y[HG];
    [[maybe_unused]] Eight<T> row4[W];
    T one_x[HG], one_y[HG];
    [[maybe_unused]] bool is_v4 = false;
    const T* from = nullptr;
    if (!Q4 || is_q) {
        const uint32_t u = is_q || is_k ? unit : unit - p.uk;
        const bool rotated = is_q || is_k;
        const uint32_t g = div_by(u, rotated ? p.div_iph : p.div_ipv);
        item = u - g * (rotated ? p.iph : p.ipv);
        head = g * HG;
        if (!rotated) {
            at = item * 8;
        } else if constexpr (VEC) {
            const uint32_t n = INTER ? a.rot / 8 : p.half / 8;
            turning = item < n;
            at = turning ? item * 8 : a.rot + (item - n) * 8;
        } else {
            turning = item < (uint32_t)p.half;
            at = turning ? (INTER ? 2 * item : item) : a.rot + (item - p.half);
        }
        from = static_cast<const T*>(src.data) + seq * src.seq + within * src.tok + head * src.head + at;
#pragma unroll
        for (int k = 0; k < HG; ++k) {
            if (!on || head + k >= (uint32_t)src.heads) continue;
            const T* f = from + k * src.head;
            if (VEC || !rotated) {
                x[k].load(f);
                if (!INTER && turning) y[k].load(f + p.half);
            } else {
                one_x[k] = *f;
                if (turning) one_y[k] = f[INTER ? 1 : p.half];
            }
        }
    } else if constexpr (Q4) {
        // K of all heads, then V: a warp rarely holds both
        const uint32_t r = unit >> 2;
        is_v4 = r >= (uint32_t)a.k.heads;
        head = r - (is_v4 ? a.k.heads : 0);
        const RowsView& v = is_v4 ? a.v : a.k;
        from = static_cast<const T*>(v.data) + seq * v.seq + within * v.tok + head * v.head;
        if (on)
#pragma unroll
            for (int w = 0; w < W; ++w) row4[w].load(from + 32 * w + 8 * (unit & 3));
    }

    if (tid < p.half) turns[turn_slot<PAIRS>(tid)] = a.turns[tid];
    // positions and rows (q wants the rows only where they are its positions)
    Token t;
    t.live = 1;
    t.row = -1;
    t.pos = 0;
    if (append && (!is_q || (a.rot > 0 && !a.positions))) {
        const int warp = tid >> 5;
        const int64_t last = min(id0 + kThreads, total) - 1;
        const int n = (int)(last / units - j0) + 1;
        for (int i = warp; i < n; i += kThreads / 32) {
            const Token x = place_token(a, j0 + i);
            if ((tid & 31) == 0) tok[i] = x;
        }
        __syncthreads();
        if constexpr (Q4) {
            if (!is_q) {
#pragma unroll 1  // (unrolled, the append takes 78 us instead of 64.5)
                for (int q = tid; q < n * p.half; q += kThreads) {
                    const int i = div_by(q, p.div_half), k = q - i * p.half;
                    float c, s;
                    turn_of<PAIRS>(a, turns, tok[i].pos, k, c, s);
                    sines[i * 2 * p.half + k] = c;
                    sines[i * 2 * p.half + p.half + k] = s;
                }
                __syncthreads();
            }
        }
        if (on) t = tok[tl];
    } else {
        if (on && a.positions) t.pos = a.positions[j];
        if (on && a.cu) t.live = j < a.cu[a.num_seqs] && j >= a.cu[0];
        if (p.half > 0) __syncthreads();  // the turns
    }
    if (!on || !t.live) return;  // (a 4-bit row's four lanes leave together)

    const int64_t hs = (int64_t)1 << a.pg.log2bs;  // rows between heads of a block
    if (!Q4 || is_q) {
        if (!is_q && append && t.row < 0) return;
        T* to;
        int64_t step;
        if (is_q || !append) {
            const RowsView& dst = is_q ? a.out_q : a.out_k;
            to = static_cast<T*>(dst.data) + seq * dst.seq + within * dst.tok + head * dst.head + at;
            step = dst.head;
        } else {
            to = static_cast<T*>(is_k ? a.k_pool : a.v_pool) + (t.row + head * hs) * a.d + at;
            step = hs * a.d;
        }
        const bool rotated = is_q || is_k;
        if (VEC || !rotated) {
            constexpr int N = INTER ? 4 : 8;
            float cs[N], sn[N];
            if (VEC && turning) {
#pragma unroll
                for (int i = 0; i < N; ++i)
                    turn_of<PAIRS>(a, turns, t.pos, item * N + i, cs[i], sn[i]);
            }
#pragma unroll
            for (int k = 0; k < HG; ++k) {
                if (head + k >= (uint32_t)src.heads) break;
                T* q = to + k * step;
                if (turning) {
                    float u[8], v[8], o[8];
                    x[k].get(u);
                    if constexpr (INTER) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            o[2 * i] = u[2 * i] * cs[i] - u[2 * i + 1] * sn[i];
                            o[2 * i + 1] = u[2 * i + 1] * cs[i] + u[2 * i] * sn[i];
                        }
                        x[k].set(o);
                    } else {
                        y[k].get(v);
#pragma unroll
                        for (int i = 0; i < 8; ++i) o[i] = u[i] * cs[i] - v[i] * sn[i];
                        x[k].set(o);
#pragma unroll
                        for (int i = 0; i < 8; ++i) o[i] = v[i] * cs[i] + u[i] * sn[i];
                        y[k].set(o);
                        y[k].store(q + p.half);
                    }
                }
                x[k].store(q);
            }
        } else {
            float c = 1.f, s = 0.f;
            if (turning) turn_of<PAIRS>(a, turns, t.pos, item, c, s);
#pragma unroll
            for (int k = 0; k < HG; ++k) {
                if (head + k >= (uint32_t)src.heads) break;
                T* q = to + k * step;
                if (!turning) {
                    *q = one_x[k];
                    continue;
                }
                const float u = Elem<T>::to_f(one_x[k]), v = Elem<T>::to_f(one_y[k]);
                *q = one_of<T>(u * c - v * s);
                q[INTER ? 1 : p.half] = one_of<T>(v * c + u * s);
            }
        }
    } else if constexpr (Q4) {
        const int l = unit & 3;
        float v[W][8];
#pragma unroll
        for (int w = 0; w < W; ++w) row4[w].get(v[w]);
        if (!is_v4 && p.half > 0) {
            const float* cs = sines + tl * 2 * p.half;
            turn_row<T, VEC, INTER, W>(v, from, l, p, cs, cs + p.half);
        }
        const int64_t row = t.row + head * hs;
        quantise_store<W>(v, l, t.row >= 0, (is_v4 ? a.q4p.v_codes : a.q4p.k_codes) + row * (a.d / 2),
                          (is_v4 ? a.q4p.v_scales : a.q4p.k_scales) + row * W);
    }
}

template <typename T, bool VEC, bool INTER>
cudaError_t go(const Params& p, unsigned grid, size_t smem, cudaStream_t s) {
    if (!p.a.q4)
        return launch_early(tokens_kernel<T, VEC, INTER, false, 2>, grid, kThreads, smem, s, p);
    return p.a.d == 128 ? launch_early(tokens_kernel<T, VEC, INTER, true, 4>, grid, kThreads, smem, s, p)
                        : launch_early(tokens_kernel<T, VEC, INTER, true, 2>, grid, kThreads, smem, s, p);
}
template <typename T>
cudaError_t go(Params& p, cudaStream_t s) {
    const TokenArgs& a = p.a;
    const bool vec = a.rot == 0 || (a.interleaved ? a.rot % 8 == 0 : a.rot % 16 == 0);
    // without a rotation every item is a copy of eight
    p.iph = !vec ? p.half + (a.d - a.rot)
                 : (a.interleaved ? a.rot / 8 : p.half / 8) + (a.d - a.rot) / 8;
    p.ipv = a.d / 8;
    constexpr int HG = kHeads<T>;
    const auto groups = [&](int heads) { return (heads + HG - 1) / HG; };
    p.uq = a.q.data ? groups(a.q.heads) * p.iph : 0;
    p.uk = a.k.data && !a.q4 ? groups(a.k.heads) * p.iph : 0;
    p.ukv = a.q4 ? a.k.heads * 2 * 4 : p.uk + (a.v.data ? groups(a.v.heads) * p.ipv : 0);
    p.total_q = a.num_tokens * p.uq;
    p.total_kv = a.num_tokens * p.ukv;
    const int least = p.uq > 0 && (p.ukv == 0 || p.uq < p.ukv) ? p.uq : p.ukv;
    p.tokens = (kThreads - 1) / least + 2;
    p.div_q = make_div(p.uq > 0 ? p.uq : 1);
    p.div_kv = make_div(p.ukv > 0 ? p.ukv : 1);
    p.div_iph = make_div(p.iph);
    p.div_ipv = make_div(p.ipv);
    p.div_seq = make_div((uint32_t)a.per_seq);
    p.div_half = make_div(p.half > 0 ? p.half : 1);
    const int64_t qb = (p.total_q + kThreads - 1) / kThreads;
    const int64_t kb = (p.total_kv + kThreads - 1) / kThreads, blocks = qb + kb;
    if (blocks >= ((int64_t)1 << 31)) return cudaErrorInvalidConfiguration;
    p.q_blocks = (uint32_t)qb;
    p.minor_q = qb < kb;
    p.minor = (uint32_t)(p.minor_q ? qb : kb);
    p.period = make_div(p.minor ? (uint32_t)((p.minor_q ? kb : qb) / p.minor) + 1 : 1);
    const size_t smem = a.pg.table ? sizeof(Token) * p.tokens +
                                         (a.q4 ? sizeof(float) * 2 * p.half * p.tokens : 0)
                                   : 0;
    const unsigned g = (unsigned)blocks;
    if (a.interleaved)
        return vec ? go<T, true, true>(p, g, smem, s) : go<T, false, true>(p, g, smem, s);
    return vec ? go<T, true, false>(p, g, smem, s) : go<T, false, false>(p, g, smem, s);
}

// ------------------------------------------------------------- q4 read --

// A lane's 32 (W = 4) or 16 values of a row; four lanes a row as in the append.
template <typename T, int W>
__global__ void __launch_bounds__(kThreads) q4_read_kernel(const __grid_constant__ Q4ReadArgs a,
                                                           int64_t total, int both, Div by_rows,
                                                           Div by_heads) {
    let_next_begin();
    wait_for_last();
    const int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (e >= total) return;
    const int t = (int)(e & 3);
    uint32_t r = div_by((uint32_t)(e >> 2), by_rows);  // problem (and tensor)
    const int i = (int)((uint32_t)(e >> 2) - r * (uint32_t)a.n_rows);
    bool is_v = a.out_k == nullptr;
    if (both) {
        is_v = r & 1;
        r >>= 1;
    }
    const uint32_t s = div_by(r, by_heads), h = r - s * (uint32_t)a.pg.H;
    const int64_t row = (a.first ? a.first[s] : 0) + (int64_t)i;
    if (row >= a.lens[s]) return;
    int64_t phys = -1;
    if (row >= 0 && row < ((int64_t)a.pg.max_blocks << a.pg.log2bs)) {
        const int blk = a.pg.table[(int64_t)s * a.pg.max_blocks + (row >> a.pg.log2bs)];
        if ((unsigned)blk < (unsigned)a.pg.num_blocks)
            phys = (((int64_t)blk * a.pg.H + h) << a.pg.log2bs) | (row & ((1 << a.pg.log2bs) - 1));
    }
    if (phys < 0) {
        set_error(a.status, kDevErrIndex, (unsigned)s);
        return;
    }
    const uint8_t* codes = (is_v ? a.p.v_codes : a.p.k_codes) + phys * (W * 16);
    const uint32_t* scales = (is_v ? a.p.v_scales : a.p.k_scales) + phys * W;
    uint32_t half[2][W];
    if constexpr (W == 4) {
        const uint4 c = reinterpret_cast<const uint4*>(codes)[t];
        half[0][0] = c.x & 0xffffu; half[0][1] = c.x >> 16; half[0][2] = c.y & 0xffffu; half[0][3] = c.y >> 16;
        half[1][0] = c.z & 0xffffu; half[1][1] = c.z >> 16; half[1][2] = c.w & 0xffffu; half[1][3] = c.w >> 16;
    } else {
        const uint2 c = reinterpret_cast<const uint2*>(codes)[t];
        half[0][0] = c.x & 0xffffu; half[0][1] = c.x >> 16;
        half[1][0] = c.y & 0xffffu; half[1][1] = c.y >> 16;
    }
    T* dst = static_cast<T*>(is_v ? a.out_v : a.out_k) + ((int64_t)r * a.n_rows + i) * (W * 32);
#pragma unroll
    for (int w = 0; w < W; ++w) {
        const uint32_t pr = scales[w];
        const float sc = __uint_as_float(pr << 16), lo = __uint_as_float(pr & 0xffff0000u);
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            v[k] = fmaf(sc, (float)((half[k >> 2][w] >> (4 * (k & 3))) & 15u), lo);
        Eight<T> o;
        o.set(v);
        o.store(dst + 32 * w + 8 * t);
    }
}

}  // namespace

cudaError_t launch_tokens(const TokenArgs& a, cudaStream_t s) {
    if (a.num_tokens == 0) return cudaSuccess;
    Params p;
    p.a = a;
    p.half = a.rot / 2;
    return a.dtype == RKV_DTYPE_BF16 ? go<__nv_bfloat16>(p, s) : go<float>(p, s);
}

cudaError_t launch_q4_read(const Q4ReadArgs& a, cudaStream_t s) {
    const int both = a.out_k && a.out_v;
    const int64_t total = a.num_seqs * a.pg.H * (int64_t)a.n_rows * 4 * (both ? 2 : 1);
    if (total == 0) return cudaSuccess;
    const int64_t blocks = (total + kThreads - 1) / kThreads;
    const unsigned g = (unsigned)blocks;
    const Div rows = make_div((uint32_t)a.n_rows), heads = make_div((uint32_t)a.pg.H);
    if (a.dtype == RKV_DTYPE_BF16) {
        return launch_early(a.d == 128 ? q4_read_kernel<__nv_bfloat16, 4> : q4_read_kernel<__nv_bfloat16, 2>,
                            g, kThreads, 0, s, a, total, both, rows, heads);
    }
    return launch_early(a.d == 128 ? q4_read_kernel<float, 4> : q4_read_kernel<float, 2>, g, kThreads,
                        0, s, a, total, both, rows, heads);
}

}  // namespace rkv
