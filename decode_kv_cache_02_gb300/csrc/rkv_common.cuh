// rkv_common.cuh -- device helpers shared by the librkv kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#define RKV_DEV __device__ __forceinline__

namespace rkv {

// Device error word, stored at the start of the caller's workspace.
struct DeviceStatus {
    unsigned int code;  // 0 = ok, else one of the kDevErr* codes
    unsigned int info;  // kernel-specific detail (which wait / which index)
};

enum : unsigned int {
    kDevErrNone = 0,
    kDevErrTimeout = 1,  // a bounded mbarrier wait gave up
    kDevErrIndex = 2,    // an index was found outside its buffer
};

// Record an error; the first one wins.
RKV_DEV void set_error(DeviceStatus* st, unsigned int code, unsigned int info) {
    if (st == nullptr) return;
    if (atomicCAS(&st->code, 0u, code) == 0u) atomicExch(&st->info, info);
}

// Element loads as fp32 (bf16 -> fp32 is exact).
template <typename T> struct Elem;
template <> struct Elem<float> {
    static RKV_DEV float to_f(float x) { return x; }
};
template <> struct Elem<__nv_bfloat16> {
    static RKV_DEV float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
};

// 8 consecutive elements as fp32 from a 16-byte (bf16) or two 16-byte (fp32)
// aligned loads.
RKV_DEV void load8(const __nv_bfloat16* p, float* o) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        o[2 * t] = __uint_as_float(w[t] << 16);
        o[2 * t + 1] = __uint_as_float(w[t] & 0xffff0000u);
    }
}
RKV_DEV void load8(const float* p, float* o) {
    const float4 a = *reinterpret_cast<const float4*>(p);
    const float4 b = *reinterpret_cast<const float4*>(p + 4);
    o[0] = a.x; o[1] = a.y; o[2] = a.z; o[3] = a.w;
    o[4] = b.x; o[5] = b.y; o[6] = b.z; o[7] = b.w;
}

// Monotone map float -> uint32: a < b  <=>  key(a) < key(b).  -0 is mapped
// to the key of +0 so that the two compare equal, as they do as floats.
RKV_DEV uint32_t orderable(float z) {
    uint32_t b = __float_as_uint(z + 0.0f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

RKV_DEV float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
RKV_DEV float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// A launch that may begin while the stream's last kernel ends (launch_early)
// waits for that kernel before its first look at memory, and may let the launch
// behind it begin, which waits in turn.  Call after call on a stream this takes
// 2 us off each (16384 tokens rotated: 53.8 -> 51.2 us, appended 64.9 -> 62.6);
// captured, an append and an attention of one sequence of 1152 take 9.4 us
// instead of 10.2.  The join of a plain attention lets nothing begin: what began there
// would hold its SMs up (16 sequences of 16384 at 4 bits 57.4 -> 58.4 us).
//
// One kernel looks before it waits: the pass over shared prefixes on the tensor cores
// reads its tables, queries and pools at once and waits where it takes the sums over the
// own rows.  What came before the call is over by then, because of what stands between:
// it begins once every block of the attention over the own rows has let it (or the join
// between, which passes that on before its own wait) or has ended, and those blocks
// have waited before either.  So in attn_kernel and attn_f32_kernel wait_for_last()
// stays first and let_next_begin() behind it, and no kernel that lets the next begin
// before its own wait (as the token kernels do) may come in place of them.
RKV_DEV void wait_for_last() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
RKV_DEV void let_next_begin() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
template <typename... P, typename... A>
cudaError_t launch_early(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s,
                         A&&... args) {
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, P(args)...);
}

// Dynamic shared memory past 48 KB has to be asked for once per kernel and
// device (half a microsecond, so not at every call).
template <typename K>
cudaError_t allow_smem(K kern, int bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (dev < 64 && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

}  // namespace rkv
