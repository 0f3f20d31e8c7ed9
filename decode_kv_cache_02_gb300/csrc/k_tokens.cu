// k_tokens.cu -- new tokens on their way to the cache: rotary positions, the
// append to a paged pool, and the append to a 4-bit pool, in one kernel.
//
// Rotation: pair i of a head is turned by pos * f_i.  The plan holds f_i /
// (2 pi) as a 64-bit fixed-point part of a turn, so the low 64 bits of
// pos * turns[i] are the angle modulo one turn, exactly; the upper 32 of them,
// read as a signed number, go through sincospif.  A block computes the sines
// of its tokens once into shared memory and all heads of the token use them.
//
// Every value is read and written once, 16 bytes (eight bf16) a step: the
// rotation and the append are bound by HBM for many tokens and by launch and
// load latency for a decode step.
//
// 4 bits: four neighbouring lanes own one row; lane t holds values 32 w + 8 t
// .. + 7 of every group w, so a group's minimum and maximum take two shuffles
// and the lane's codes of all groups are one store of 16 bytes (8 at head_dim
// 64).  (x - low) * r + 1.5 * 2^23 in one FMA rounds the exact product to a
// whole number (halves to even) and leaves it in the low mantissa bits.
#include <float.h>

#include "rkv_common.cuh"
#include "rkv_internal.h"
#include "rkv_paged.cuh"

namespace rkv {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 32;  // tokens per block

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
    int half;             // rot / 2
    int tpb;              // tokens per block
    int items_q, items_k; // items per token: the heads of q; of k (and v)
    int items;
    Div div_items, div_iph, div_ipv, div_units;
    int iph, ipv;         // items per rotated head, per copied head
    int units;            // 4-bit lanes per token
};

// What a block knows of each of its tokens.
struct Token {
    int64_t seq, within;  // sequence and place in it (0 and the token itself where numbered through)
    int64_t row;          // pool row of head 0 (head stride 1 << log2bs rows), or -1
    int pos;
    int live;
};

RKV_DEV void store8(float* p, const float* v) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
RKV_DEV uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}
RKV_DEV void store8(__nv_bfloat16* p, const float* v) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                              pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}
RKV_DEV void copy8(const float* x, float* y) {
    const float4 a = reinterpret_cast<const float4*>(x)[0], b = reinterpret_cast<const float4*>(x)[1];
    reinterpret_cast<float4*>(y)[0] = a;
    reinterpret_cast<float4*>(y)[1] = b;
}
RKV_DEV void copy8(const __nv_bfloat16* x, __nv_bfloat16* y) {
    *reinterpret_cast<uint4*>(y) = *reinterpret_cast<const uint4*>(x);
}
RKV_DEV float from_f(float, float v) { return v; }
RKV_DEV __nv_bfloat16 from_f(__nv_bfloat16, float v) { return __float2bfloat16_rn(v); }

// One item of a rotated head: eight pairs (VEC: two runs of eight elements,
// or eight elements of neighbouring pairs), or one pair, or what passes
// through.  An item owns what it writes, so x may be y.
template <typename T, bool VEC, bool INTER>
RKV_DEV void rotate_item(const T* x, T* y, int item, const Params& p, const float* cs,
                         const float* sn) {
    const int rot = p.a.rot, half = p.half;
    if constexpr (VEC) {
        const int turning = INTER ? rot / 8 : half / 8;
        if (item >= turning) {
            const int e = rot + (item - turning) * 8;
            if (x != y) copy8(x + e, y + e);
            return;
        }
        if constexpr (INTER) {
            float v[8], o[8];
            load8(x + item * 8, v);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float c = cs[item * 4 + i], s = sn[item * 4 + i];
                o[2 * i] = v[2 * i] * c - v[2 * i + 1] * s;
                o[2 * i + 1] = v[2 * i + 1] * c + v[2 * i] * s;
            }
            store8(y + item * 8, o);
        } else {
            float u[8], v[8], o[8], r[8];
            load8(x + item * 8, u);
            load8(x + half + item * 8, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float c = cs[item * 8 + i], s = sn[item * 8 + i];
                o[i] = u[i] * c - v[i] * s;
                r[i] = v[i] * c + u[i] * s;
            }
            store8(y + item * 8, o);
            store8(y + half + item * 8, r);
        }
    } else {
        if (item >= half) {
            const int e = rot + (item - half);
            if (x != y) y[e] = x[e];
            return;
        }
        const int e = INTER ? 2 * item : item, f = INTER ? e + 1 : e + half;
        const float u = Elem<T>::to_f(x[e]), v = Elem<T>::to_f(x[f]);
        const float c = cs[item], s = sn[item];
        y[e] = from_f(T(), u * c - v * s);
        y[f] = from_f(T(), v * c + u * s);
    }
}

RKV_DEV int64_t view_at(const RowsView& v, const Token& t, int head) {
    return t.seq * v.seq + t.within * v.tok + (int64_t)head * v.head;
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

// One 4-bit row's share of a lane: values of W groups.
template <int W>
RKV_DEV void quantise_store(float (&v)[W][8], int t, uint8_t* codes, uint32_t* scales) {
    uint32_t h[W][2], pair = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        float mn = v[w][0], mx = v[w][0], bad = v[w][0] * 0.f;
#pragma unroll
        for (int i = 1; i < 8; ++i) {
            mn = fminf(mn, v[w][i]);
            mx = fmaxf(mx, v[w][i]);
            bad += v[w][i] * 0.f;  // NaN once any value is NaN or infinite
        }
#pragma unroll
        for (int o = 1; o <= 2; o <<= 1) {
            mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            bad += __shfl_xor_sync(0xffffffffu, bad, o);
        }
        __nv_bfloat16 lo = __float2bfloat16_rd(mn);
        float lof = __bfloat162float(lo);
        __nv_bfloat16 sc = __float2bfloat16_ru(__fdiv_rn(mx - lof, 15.f));
        float sf = __bfloat162float(sc);
        if (bad != 0.f || !(sf <= FLT_MAX) || !(lof >= -FLT_MAX)) {
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
    if (codes == nullptr) return;
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

// Eight elements of x at e, turned where they lie below rot (out of place:
// the partners are read again, from L1).
template <typename T, bool VEC, bool INTER>
RKV_DEV void load_turned(const T* x, int e, const Params& p, const float* cs, const float* sn,
                         float* o) {
    const int rot = p.a.rot, half = p.half;
    load8(x + e, o);
    if (e >= rot) return;
    if constexpr (VEC && INTER) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float c = cs[e / 2 + i], s = sn[e / 2 + i], u = o[2 * i], v = o[2 * i + 1];
            o[2 * i] = u * c - v * s;
            o[2 * i + 1] = v * c + u * s;
        }
    } else if constexpr (VEC) {
        const bool first = e < half;
        const int i0 = first ? e : e - half;
        float v[8];
        load8(x + (first ? e + half : e - half), v);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float c = cs[i0 + i], s = first ? -sn[i0 + i] : sn[i0 + i];
            o[i] = o[i] * c + v[i] * s;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int at = e + i;
            if (at < rot) {
                const bool first = INTER ? (at & 1) == 0 : at < half;
                const int k = INTER ? at >> 1 : (first ? at : at - half);
                const int other = INTER ? at ^ 1 : (first ? at + half : at - half);
                const float v = Elem<T>::to_f(x[other]);
                o[i] = o[i] * cs[k] + (first ? -v : v) * sn[k];
            }
        }
    }
}

// VEC: the rotated part splits into whole steps of eight.
template <typename T, bool VEC, bool INTER, bool Q4, int W>
__global__ void __launch_bounds__(kThreads) tokens_kernel(const __grid_constant__ Params p) {
    extern __shared__ float sines[];  // [tpb][2][half]
    __shared__ Token tok[kMaxTokens];
    const TokenArgs& a = p.a;
    const int tid = threadIdx.x, lane = tid & 31;
    const int64_t j0 = (int64_t)blockIdx.x * p.tpb;
    const int n_tok = (int)(a.num_tokens - j0 < p.tpb ? a.num_tokens - j0 : p.tpb);
    const bool append = a.pg.table != nullptr;

    for (int i = tid >> 5; i < n_tok; i += kThreads / 32) {
        const int64_t j = j0 + i;
        Token t;
        t.live = 1;
        t.row = -1;
        t.pos = 0;
        if (!append) {
            t.seq = j / a.per_seq;
            t.within = j - t.seq * a.per_seq;
        } else {
            int64_t s, first, count;
            if (a.cu == nullptr) {
                s = j / a.per_seq;
                first = s * a.per_seq;
                count = a.per_seq;
                t.seq = s;
                t.within = j - first;
            } else {
                t.live = j < a.cu[a.num_seqs] && j >= a.cu[0];
                s = t.live ? find_seq(a.cu, a.num_seqs, j) : 0;
                first = a.cu[s];
                count = a.cu[s + 1] - first;
                t.seq = 0;
                t.within = j;
            }
            const int64_t r = (int64_t)a.lens[s] - count + (j - first);
            if (t.live) {
                t.pos = (int)r;
                bool ok = r >= 0 && r < ((int64_t)a.pg.max_blocks << a.pg.log2bs);
                if (ok) {
                    const int blk = a.pg.table[s * a.pg.max_blocks + (r >> a.pg.log2bs)];
                    ok = (unsigned)blk < (unsigned)a.pg.num_blocks;
                    t.row = (((int64_t)blk * a.pg.H) << a.pg.log2bs) +
                            (r & ((1 << a.pg.log2bs) - 1));
                }
                if (!ok) {
                    t.row = -1;
                    if (lane == 0) set_error(a.status, kDevErrIndex, (unsigned)s);
                }
            }
        }
        if (t.live && a.positions) t.pos = a.positions[j];
        if (lane == 0) tok[i] = t;
    }
    __syncthreads();
    for (int e = tid; e < n_tok * p.half; e += kThreads) {
        const int i = e / p.half, k = e - i * p.half;
        const uint64_t turn = (uint64_t)(int64_t)tok[i].pos * a.turns[k];
        float s, c;
        sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &s, &c);
        float* cs = sines + i * 2 * p.half;
        cs[k] = c * a.factor;
        cs[p.half + k] = (a.inverse ? -s : s) * a.factor;
    }
    __syncthreads();

    const T* q = static_cast<const T*>(a.q.data);
    const T* kk = static_cast<const T*>(a.k.data);
    const T* vv = static_cast<const T*>(a.v.data);
    const int64_t hs = (int64_t)1 << a.pg.log2bs;  // rows between heads of a block
    const int step = kThreads * gridDim.y;
    for (uint32_t e = blockIdx.y * kThreads + tid; e < (uint32_t)(n_tok * p.items); e += step) {
        const uint32_t i = div_by(e, p.div_items);
        uint32_t it = e - i * p.items;
        const Token& t = tok[i];
        if (!t.live) continue;
        [[maybe_unused]] const float* cs = sines + i * 2 * p.half;
        if (it < (uint32_t)p.items_q) {
            const uint32_t h = div_by(it, p.div_iph);
            rotate_item<T, VEC, INTER>(q + view_at(a.q, t, h),
                                       static_cast<T*>(a.out_q.data) + view_at(a.out_q, t, h),
                                       it - h * p.iph, p, cs, cs + p.half);
            continue;
        }
        it -= p.items_q;
        if constexpr (!Q4) {
            if (it < (uint32_t)p.items_k) {
                const uint32_t h = div_by(it, p.div_iph);
                T* dst;
                if (append) {
                    if (t.row < 0) continue;
                    dst = static_cast<T*>(a.k_pool) + (t.row + h * hs) * a.d;
                } else {
                    dst = static_cast<T*>(a.out_k.data) + view_at(a.out_k, t, h);
                }
                rotate_item<T, VEC, INTER>(kk + view_at(a.k, t, h), dst, it - h * p.iph, p, cs,
                                           cs + p.half);
            } else {
                it -= p.items_k;
                const uint32_t h = div_by(it, p.div_ipv);
                const int at = (it - h * p.ipv) * 8;
                if (t.row < 0) continue;
                copy8(vv + view_at(a.v, t, h) + at,
                      static_cast<T*>(a.v_pool) + (t.row + h * hs) * a.d + at);
            }
        }
    }
    if constexpr (Q4) {
        // whole warps take part in every step: the shuffles need all lanes
        const uint32_t total = (uint32_t)(n_tok * p.units);
        for (uint32_t e0 = blockIdx.y * kThreads + (tid & ~31); e0 < total; e0 += step) {
            const uint32_t e = e0 + lane, u = e < total ? e : total - 1;
            const uint32_t i = div_by(u, p.div_units), it = u - i * p.units;
            const Token& t = tok[i];
            const int tl = lane & 3;
            // K of all heads, then V: a warp rarely holds both
            const bool is_v = (it >> 2) >= (uint32_t)a.k.heads;
            const uint32_t h = (it >> 2) - (is_v ? a.k.heads : 0);
            const bool ok = e < total && t.live && t.row >= 0;
            float x[W][8];
            if (t.live) {
                const float* cs = sines + i * 2 * p.half;
                const T* src = is_v ? vv + view_at(a.v, t, h) : kk + view_at(a.k, t, h);
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    if (is_v)
                        load8(src + 32 * w + 8 * tl, x[w]);
                    else
                        load_turned<T, VEC, INTER>(src, 32 * w + 8 * tl, p, cs, cs + p.half, x[w]);
                }
            } else {
#pragma unroll
                for (int w = 0; w < W; ++w)
#pragma unroll
                    for (int k = 0; k < 8; ++k) x[w][k] = 0.f;
            }
            const int64_t row = ok ? t.row + h * hs : 0;
            quantise_store<W>(x, tl,
                              ok ? (is_v ? a.q4p.v_codes : a.q4p.k_codes) + row * (a.d / 2) : nullptr,
                              (is_v ? a.q4p.v_scales : a.q4p.k_scales) + row * W);
        }
    }
}

template <typename T, bool VEC, bool INTER>
cudaError_t go(const Params& p, dim3 grid, size_t smem, cudaStream_t s) {
    if (!p.a.q4)
        tokens_kernel<T, VEC, INTER, false, 4><<<grid, kThreads, smem, s>>>(p);
    else if (p.a.d == 128)
        tokens_kernel<T, VEC, INTER, true, 4><<<grid, kThreads, smem, s>>>(p);
    else
        tokens_kernel<T, VEC, INTER, true, 2><<<grid, kThreads, smem, s>>>(p);
    return cudaGetLastError();
}
template <typename T>
cudaError_t go(const Params& p, bool vec, dim3 grid, size_t smem, cudaStream_t s) {
    if (p.a.interleaved)
        return vec ? go<T, true, true>(p, grid, smem, s) : go<T, false, true>(p, grid, smem, s);
    return vec ? go<T, true, false>(p, grid, smem, s) : go<T, false, false>(p, grid, smem, s);
}

// ------------------------------------------------------------- q4 read --

// A lane's 32 (W = 4) or 16 values of a row; four lanes a row as in the append.
template <typename T, int W>
__global__ void __launch_bounds__(kThreads) q4_read_kernel(const __grid_constant__ Q4ReadArgs a,
                                                           int64_t total, int both) {
    const int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (e >= total) return;
    const int t = (int)(e & 3);
    int64_t r = e >> 2;
    const int i = (int)(r % a.n_rows);
    r /= a.n_rows;  // problem (and tensor)
    bool is_v = a.out_k == nullptr;
    if (both) {
        is_v = r & 1;
        r >>= 1;
    }
    const int64_t s = r / a.pg.H;
    const int64_t row = (a.first ? a.first[s] : 0) + (int64_t)i;
    if (row >= a.lens[s]) return;
    bool ok = row >= 0 && row < ((int64_t)a.pg.max_blocks << a.pg.log2bs);
    int64_t phys = -1;
    if (ok) phys = paged_phys_row(a.pg, r, (int)row);
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
    T* dst = static_cast<T*>(is_v ? a.out_v : a.out_k) + (r * a.n_rows + i) * (W * 32);
#pragma unroll
    for (int w = 0; w < W; ++w) {
        const uint32_t pr = scales[w];
        const float sc = __uint_as_float(pr << 16), lo = __uint_as_float(pr & 0xffff0000u);
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            v[k] = fmaf(sc, (float)((half[k >> 2][w] >> (4 * (k & 3))) & 15u), lo);
        store8(dst + 32 * w + 8 * t, v);
    }
}

}  // namespace

cudaError_t launch_tokens(const TokenArgs& a, cudaStream_t s) {
    if (a.num_tokens == 0) return cudaSuccess;
    Params p;
    p.a = a;
    p.half = a.rot / 2;
    const bool vec = a.rot == 0 || (a.interleaved ? a.rot % 8 == 0 : a.rot % 16 == 0);
    // without a rotation every item is a copy of eight
    p.iph = !vec ? p.half + (a.d - a.rot)
                 : (a.interleaved ? a.rot / 8 : p.half / 8) + (a.d - a.rot) / 8;
    p.ipv = a.d / 8;
    p.items_q = a.q.data ? a.q.heads * p.iph : 0;
    p.items_k = (a.k.data && !a.q4) ? a.k.heads * p.iph : 0;
    p.items = p.items_q + p.items_k + (a.v.data && !a.q4 ? a.v.heads * p.ipv : 0);
    p.units = a.q4 ? a.k.heads * 2 * 4 : 0;
    p.div_items = make_div(p.items ? p.items : 1);
    p.div_iph = make_div(p.iph);
    p.div_ipv = make_div(p.ipv);
    p.div_units = make_div(p.units ? p.units : 1);
    // a block takes enough tokens for about two steps of its threads, and a
    // token with many heads is shared by several blocks while tokens are few
    const int per_token = p.items + p.units;
    int tpb = 2 * kThreads / per_token;
    tpb = tpb < 1 ? 1 : (tpb > kMaxTokens ? kMaxTokens : tpb);
    while (tpb > 1 && (a.num_tokens + tpb - 1) / tpb < 304) tpb /= 2;
    p.tpb = tpb;
    const int64_t blocks = (a.num_tokens + tpb - 1) / tpb;
    int64_t split = 1;
    while (blocks * split < 152 && split * kThreads < per_token) split *= 2;
    const dim3 grid((unsigned)blocks, (unsigned)split);
    const size_t smem = sizeof(float) * (size_t)tpb * 2 * (p.half ? p.half : 1);
    return a.dtype == RKV_DTYPE_BF16 ? go<__nv_bfloat16>(p, vec, grid, smem, s)
                                     : go<float>(p, vec, grid, smem, s);
}

cudaError_t launch_q4_read(const Q4ReadArgs& a, cudaStream_t s) {
    const int both = a.out_k && a.out_v;
    const int64_t total = a.num_seqs * a.pg.H * (int64_t)a.n_rows * 4 * (both ? 2 : 1);
    if (total == 0) return cudaSuccess;
    const int64_t blocks = (total + kThreads - 1) / kThreads;
    const unsigned g = (unsigned)blocks;
    if (a.dtype == RKV_DTYPE_BF16) {
        if (a.d == 128) q4_read_kernel<__nv_bfloat16, 4><<<g, kThreads, 0, s>>>(a, total, both);
        else q4_read_kernel<__nv_bfloat16, 2><<<g, kThreads, 0, s>>>(a, total, both);
    } else {
        if (a.d == 128) q4_read_kernel<float, 4><<<g, kThreads, 0, s>>>(a, total, both);
        else q4_read_kernel<float, 2><<<g, kThreads, 0, s>>>(a, total, both);
    }
    return cudaGetLastError();
}

}  // namespace rkv
