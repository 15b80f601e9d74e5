// rows.cuh -- what the operators on matrices of binary32, float16 or bfloat16 entries share:
// conversions, packed loads and stores, argument checks, and launches.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "dgc_device.cuh"

namespace dgc {

constexpr int64_t kMaxExtent = 1 << 24;  // rows or columns of a matrix

// up2, down2: two neighbours in one 32-bit register, the first in its low half. Rounded to nearest
// even. (binary32 has no such pairs.)
template <typename T>
struct Num;
template <>
struct Num<float> {
    __device__ static float up(float x) { return x; }
    __device__ static float down(float x) { return x; }
    __device__ static float2 up2(uint32_t) { return {0.0f, 0.0f}; }
    __device__ static uint32_t down2(float, float) { return 0; }
};
template <>
struct Num<__half> {
    __device__ static float up(__half x) { return __half2float(x); }
    __device__ static __half down(float x) { return __float2half_rn(x); }
    __device__ static float2 up2(uint32_t w) {
        return __half22float2(*reinterpret_cast<const __half2*>(&w));
    }
    __device__ static uint32_t down2(float a, float b) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
};
template <>
struct Num<__nv_bfloat16> {
    __device__ static float up(__nv_bfloat16 x) { return __bfloat162float(x); }
    __device__ static __nv_bfloat16 down(float x) { return __float2bfloat16_rn(x); }
    __device__ static float2 up2(uint32_t w) {
        return {__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)};
    }
    __device__ static uint32_t down2(float a, float b) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
};

// kN entries as they lie in memory, in 32-bit registers.
template <typename T, int kN>
struct Packed {
    static constexpr int kWords = (kN * (int)sizeof(T) + 3) / 4;
    uint32_t w[kWords];
};

// Coherent loads, since a result may lie where an operand does. kOnce: the entries are used once
// and need no place in the caches.
template <bool kOnce, typename W>
__device__ __forceinline__ W load_word(const W* p) {
    if constexpr (kOnce) return __ldcs(p);
    else return *p;
}
// kN entries from an address on a boundary of min(16, kN entries) bytes.
template <typename T, int kN, bool kOnce = true>
__device__ __forceinline__ Packed<T, kN> load_packed(const T* p) {
    constexpr int kBytes = kN * (int)sizeof(T);
    Packed<T, kN> r;
    if constexpr (kBytes >= 16) {
        static_assert(kBytes % 16 == 0, "whole 16-byte pieces");
#pragma unroll
        for (int i = 0; i < kBytes / 16; ++i) {
            const uint4 v = load_word<kOnce>(reinterpret_cast<const uint4*>(p) + i);
            r.w[4 * i] = v.x;
            r.w[4 * i + 1] = v.y;
            r.w[4 * i + 2] = v.z;
            r.w[4 * i + 3] = v.w;
        }
    } else if constexpr (kBytes == 8) {
        const uint2 v = load_word<kOnce>(reinterpret_cast<const uint2*>(p));
        r.w[0] = v.x;
        r.w[1] = v.y;
    } else if constexpr (kBytes == 4) {
        r.w[0] = load_word<kOnce>(reinterpret_cast<const uint32_t*>(p));
    } else {
        static_assert(kBytes == 2, "a power of two");
        r.w[0] = load_word<kOnce>(reinterpret_cast<const uint16_t*>(p));
    }
    return r;
}

// The first `n` of kN entries one by one, zeros behind them.
template <typename T, int kN, bool kOnce = true>
__device__ __forceinline__ Packed<T, kN> load_some(const T* p, uint32_t n) {
    Packed<T, kN> r;
#pragma unroll
    for (int i = 0; i < Packed<T, kN>::kWords; ++i) r.w[i] = 0;
#pragma unroll
    for (int i = 0; i < kN; ++i)
        if ((uint32_t)i < n) {
            if constexpr (sizeof(T) == 4)
                r.w[i] = load_word<kOnce>(reinterpret_cast<const uint32_t*>(p) + i);
            else
                r.w[i / 2] |= (uint32_t)load_word<kOnce>(reinterpret_cast<const uint16_t*>(p) + i)
                              << (16 * (i & 1));
        }
    return r;
}

template <typename T, int kN>
__device__ __forceinline__ void unpack(const Packed<T, kN>& p, float (&f)[kN]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < kN; ++i) f[i] = __uint_as_float(p.w[i]);
    } else if constexpr (kN == 1) {
        f[0] = Num<T>::up2(p.w[0]).x;
    } else {
#pragma unroll
        for (int i = 0; i < kN / 2; ++i) {
            const float2 v = Num<T>::up2(p.w[i]);
            f[2 * i] = v.x;
            f[2 * i + 1] = v.y;
        }
    }
}

// Entries 2 i and 2 i + 1.
template <typename T, int kN>
__device__ __forceinline__ float2 pair_of(const Packed<T, kN>& p, int i) {
    if constexpr (sizeof(T) == 4)
        return {__uint_as_float(p.w[2 * i]), __uint_as_float(p.w[2 * i + 1])};
    else
        return Num<T>::up2(p.w[i]);
}
template <typename T, int kN>
__device__ __forceinline__ void set_pair(Packed<T, kN>& p, int i, float2 v) {
    if constexpr (sizeof(T) == 4) {
        p.w[2 * i] = __float_as_uint(v.x);
        p.w[2 * i + 1] = __float_as_uint(v.y);
    } else {
        p.w[i] = Num<T>::down2(v.x, v.y);
    }
}

template <typename T, int kN>
__device__ __forceinline__ Packed<T, kN> pack(const float (&f)[kN]) {
    Packed<T, kN> r;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < kN; ++i) r.w[i] = __float_as_uint(f[i]);
    } else if constexpr (kN == 1) {
        r.w[0] = Num<T>::down2(f[0], 0.0f);
    } else {
#pragma unroll
        for (int i = 0; i < kN / 2; ++i) r.w[i] = Num<T>::down2(f[2 * i], f[2 * i + 1]);
    }
    return r;
}

template <typename T, int kN>
__device__ __forceinline__ void store_packed(T* p, const Packed<T, kN>& r) {
    constexpr int kBytes = kN * (int)sizeof(T);
    if constexpr (kBytes >= 16) {
#pragma unroll
        for (int i = 0; i < kBytes / 16; ++i)
            __stcs(reinterpret_cast<uint4*>(p) + i,
                   make_uint4(r.w[4 * i], r.w[4 * i + 1], r.w[4 * i + 2], r.w[4 * i + 3]));
    } else if constexpr (kBytes == 8) {
        __stcs(reinterpret_cast<uint2*>(p), make_uint2(r.w[0], r.w[1]));
    } else if constexpr (kBytes == 4) {
        __stcs(reinterpret_cast<uint32_t*>(p), r.w[0]);
    } else {
        __stcs(reinterpret_cast<uint16_t*>(p), (uint16_t)r.w[0]);
    }
}

template <typename T, int kN>
__device__ __forceinline__ void store_some(T* p, const Packed<T, kN>& r, uint32_t n) {
#pragma unroll
    for (int i = 0; i < kN; ++i)
        if ((uint32_t)i < n) {
            if constexpr (sizeof(T) == 4)
                __stcs(reinterpret_cast<uint32_t*>(p) + i, r.w[i]);
            else
                __stcs(reinterpret_cast<uint16_t*>(p) + i, (uint16_t)(r.w[i / 2] >> (16 * (i & 1))));
        }
}

// kN entries of a row of which `n` are left (n may pass kN): whole where kWide says that the
// address allows it.
template <bool kWide, typename T, int kN, bool kOnce = true>
__device__ __forceinline__ Packed<T, kN> load_piece(const T* p, uint32_t n) {
    if (kWide && n >= (uint32_t)kN) return load_packed<T, kN, kOnce>(p);
    return load_some<T, kN, kOnce>(p, n);
}
template <bool kWide, typename T, int kN>
__device__ __forceinline__ void store_piece(T* p, const Packed<T, kN>& r, uint32_t n) {
    if (kWide && n >= (uint32_t)kN)
        store_packed<T, kN>(p, r);
    else
        store_some<T, kN>(p, r, n);
}

// Two binary32 numbers in one instruction, each rounded as alone.
__device__ __forceinline__ uint64_t bits2(float2 a) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
    return r;
}
__device__ __forceinline__ float2 floats2(uint64_t r) {
    float2 a;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a.x), "=f"(a.y) : "l"(r));
    return a;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
    return floats2(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
    return floats2(r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
    return floats2(r);
}
__device__ __forceinline__ float2 both(float a) { return {a, a}; }

// The first index i in [lo, lo + len) with a[i] >= key, lo + len if there is none, by all lanes of a
// warp, 32 probes a step; any contents (where they do not rise, any index of the range).
template <typename T>
__device__ __forceinline__ uint32_t first_from(const T* a, uint32_t lo, uint32_t len, T key) {
    const uint32_t lane = threadIdx.x & 31;
    while (len > 0) {
        const uint32_t step = (len + 31) / 32;
        const uint32_t i = lo + min((lane + 1) * step, len) - 1;
        const uint32_t not_less = ~__ballot_sync(kFull, a[i] < key);
        if (not_less == 0) return lo + len;
        const uint32_t less = __ffs(not_less) - 1;
        lo += less * step;
        if (step == 1) return lo;
        len = min(step, len - less * step) - 1;  // its last one is known not to be less
    }
    return lo;
}

// Copies to shared memory that run behind the thread's back: kBytes (4, 8 or 16) of which the first
// `n` are read and the rest become zeros. Every thread reads what it copied itself, after
// copy_wait<k>: all but its last k groups of copies have arrived (the hardware's wait, no loop).
template <int kBytes>
__device__ __forceinline__ void copy_async(void* smem, const void* p, uint32_t n) {
    if constexpr (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(smem)), "l"(p),
                     "r"(n)
                     : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(smem_addr(smem)), "l"(p),
                     "n"(kBytes), "r"(n)
                     : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

// The pieces of a matrix, `per_row` to a row, walked by blocks of kThreads threads that take kSteps
// pieces a thread, kThreads apart: row and place in the row by one division, then by additions.
struct PieceWalk {
    uint64_t total;            // rows * per_row
    uint32_t per_row, dq, dr;  // kThreads / per_row and what is left
};
template <int kThreads, int kSteps>
struct Pieces {
    uint64_t row;
    uint32_t at;
    __device__ Pieces(const PieceWalk& w, uint64_t tile) {
        const uint64_t first = tile * (kThreads * kSteps);
        row = first / w.per_row;
        const uint32_t c = (uint32_t)(first - row * w.per_row) + threadIdx.x;
        const uint32_t q = c / w.per_row;
        row += q;
        at = c - q * w.per_row;
    }
    __device__ void next(const PieceWalk& w) {
        row += w.dq;
        at += w.dr;
        if (at >= w.per_row) {
            at -= w.per_row;
            ++row;
        }
    }
};
inline PieceWalk piece_walk(uint64_t rows, uint32_t per_row, uint32_t threads) {
    return {rows * per_row, per_row, threads / per_row, threads % per_row};
}

// ----------------------------------------------------------------------------------- host
struct Rows {  // a checked matrix
    void* p;
    uint64_t rows, cols, ld;
    int32_t dtype;
    size_t entry() const { return dtype == DGC_F32 ? 4 : 2; }
    // whether every row starts on a boundary of `bytes` (a power of two)
    bool on(size_t bytes) const {
        return rows == 0 || cols == 0 ||
               ((((uintptr_t)p | (rows > 1 ? ld * entry() : 0)) & (bytes - 1)) == 0);
    }
    bool shaped(uint64_t r, uint64_t c) const { return rows == r && cols == c; }
};

// A matrix argument; dtype -1: any of the three types.
inline int check_rows(const dgc_matrix* m, Rows* out, int32_t dtype) {
    if (!m || m->rows < 0 || m->cols < 0 || m->reserved != 0) return DGC_EINVAL;
    if (m->dtype != DGC_F32 && m->dtype != DGC_F16 && m->dtype != DGC_BF16) return DGC_EINVAL;
    if (dtype >= 0 && m->dtype != dtype) return DGC_EINVAL;
    if (m->rows > kMaxExtent || m->cols > kMaxExtent) return DGC_EUNSUPPORTED;
    *out = Rows{m->data, (uint64_t)m->rows, (uint64_t)m->cols, (uint64_t)m->ld, m->dtype};
    if (m->rows == 0 || m->cols == 0) return DGC_OK;
    if (!m->data || ((uintptr_t)m->data & (out->entry() - 1))) return DGC_EINVAL;
    if (m->rows == 1) {
        out->ld = (uint64_t)m->cols;  // not read
        return DGC_OK;
    }
    if (m->ld < m->cols) return DGC_EINVAL;
    if (m->ld > (1ll << 36)) return DGC_EUNSUPPORTED;
    return DGC_OK;
}

// A vector argument of n entries of one type.
inline int check_vector(const dgc_tensor* t, uint64_t n, int32_t dtype) {
    if (!t || t->n < 0 || t->reserved != 0 || t->dtype != dtype || (uint64_t)t->n != n)
        return DGC_EINVAL;
    const size_t size = dtype == DGC_I64 ? 8 : dtype == DGC_F32 || dtype == DGC_I32 ? 4 : 2;
    if (n && (!t->data || ((uintptr_t)t->data & (size - 1)))) return DGC_EINVAL;
    return DGC_OK;
}

// A launch that may start while the kernel ahead of it ends (every kernel waits before it reads or
// writes).
template <typename... A>
int launch_shared_kernel(void (*kernel)(A...), dim3 grid, unsigned threads, size_t smem,
                         cudaStream_t s, const std::decay_t<A>&... args) {
    void* ptrs[] = {const_cast<void*>(static_cast<const void*>(&args))...};
    if (smem > 32 * 1024 &&  // 48 KB with the static part need no leave
        cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)smem) != cudaSuccess) {
        cudaGetLastError();
        return DGC_ECUDA;
    }
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    c.attrs = at;
    c.numAttrs = 1;
    if (cudaLaunchKernelExC(&c, reinterpret_cast<const void*>(kernel), ptrs) != cudaSuccess) {
        cudaGetLastError();
        return DGC_ECUDA;
    }
    dgc_internal_count_launches(1);
    return DGC_OK;
}

template <typename... A>
int launch_rows_kernel(void (*kernel)(A...), dim3 grid, unsigned threads, cudaStream_t s,
                       const std::decay_t<A>&... args) {
    return launch_shared_kernel(kernel, grid, threads, 0, s, args...);
}

// f with the type of the entries: f(T{}).
template <typename F>
int with_type(int32_t dtype, F f) {
    if (dtype == DGC_F32) return f(float{});
    if (dtype == DGC_F16) return f(__half{});
    return f(__nv_bfloat16{});
}

}  // namespace dgc
