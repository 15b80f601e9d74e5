// grad.cu -- the global norm of a step's gradient tensors, and clipping by it (sm_103a).
//
//   k_grad_table   writes the table of tensors into the workspace when it is too long for a
//                  kernel's parameters (a launch per kTableCap tensors).
//   k_grad_norm    one pass over all tensors: partial sums of squares, one binary64 per block.
//   k_grad_finish  joins the partial sums: norm and scale.
//   k_grad_scale   dst = src * scale (dgc_grad_clip).
//
// The work unit is a warp tile of 4 KB of one tensor. In the sum, warps take every so many-th tile
// (which tiles is fixed by the list and the GPU's SM count, so the sum's order is too), looking
// their first tensor up and stepping through the table from there.
#include <cmath>
#include <cstring>
#include <type_traits>

#include "dgc_device.cuh"
#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace dgc {
namespace {

constexpr int kGradThreads = 256;
constexpr int kGradWarps = kGradThreads / 32;
// Entries of a warp tile: 4 KB of the source, 8 loads of 16 bytes a lane.
constexpr uint32_t kTileBytes = 4096;
template <typename T>
constexpr uint32_t kTile = kTileBytes / sizeof(T);
constexpr int kTableCap = 960;      // tensors in one kernel's parameters (27 KB of 32 KB)
constexpr int kMidTable = 192;      // ... of the variants for shorter lists, whose launches
constexpr int kSmallTable = 24;     // copy fewer bytes
constexpr int kBlocksPerSm = 3;      // 85 registers a thread: at 64 the norm kernel spills
constexpr int64_t kMaxTensors = 1 << 20;

// One tensor: source, destination (0 for the norm alone), entries, types, first warp tile.
struct GradEntry {
    const void* src;
    void* dst;
    uint64_t n;          // entries in bits 0..55, source type in 56..59, destination in 60..63
    __host__ __device__ uint64_t count() const { return n & ((1ull << 56) - 1); }
    __host__ __device__ int src_type() const { return (int)(n >> 56) & 15; }
    __host__ __device__ int dst_type() const { return (int)(n >> 60) & 15; }
};

template <int kCap>
struct GradTable {
    GradEntry e[kCap];
    uint32_t first[kCap + 1];  // first[count] = number of warp tiles
};

struct GradArgs {
    const GradEntry* entries;  // in the workspace; null: the table is in the parameters
    const uint32_t* first;
    int32_t count;
    uint32_t tiles;
    double* partial;           // one per block of k_grad_norm
    int32_t nparts;
    float max_norm;            // 0: no clipping
    int32_t in_place, twice;   // twice: clipping, which reads the list again
    float *norm, *scale;
};

__global__ void __launch_bounds__(256) k_grad_table(const __grid_constant__ GradTable<kTableCap> t,
                                                    int32_t n, GradEntry* entries,
                                                    uint32_t* first) {
    for (int i = threadIdx.x; i < n; i += blockDim.x) entries[i] = t.e[i];
    for (int i = threadIdx.x; i <= n; i += blockDim.x) first[i] = t.first[i];
}

template <typename T>
struct Cvt;
template <>
struct Cvt<float> {
    __device__ static float up(float x) { return x; }
    __device__ static float down(float x) { return x; }
};
template <>
struct Cvt<__half> {
    __device__ static float up(__half x) { return __half2float(x); }
    __device__ static __half down(float x) { return __float2half_rn(x); }
};
template <>
struct Cvt<__nv_bfloat16> {
    __device__ static float up(__nv_bfloat16 x) { return __bfloat162float(x); }
    __device__ static __nv_bfloat16 down(float x) { return __float2bfloat16_rn(x); }
};

template <typename T, int kN>
struct alignas(sizeof(T) * kN) Vec {
    T v[kN];
};

// Priorities in L2. When the list is read twice (clipping), the first pass reads the entries before
// the last 48 MB so that they are the first to leave, and those at the normal priority; the second
// pass starts with them, and reads everything for the last time. No line is kept above the normal
// priority (evict_last): nothing takes that back, and the work behind the call would find so much
// less of L2 (six passes over 90 MB: 145 us for 112), for 0.4 to 2.5 us of the call's own. Against one
// priority for all: 411M bf16 entries 493 -> 483 us, 25.6M binary32 entries 49.9 -> 48.0.
constexpr uint32_t kKeepTiles = (48u << 20) / kTileBytes;

__device__ __forceinline__ uint64_t l2_first() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ uint64_t l2_normal() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}
template <typename T, int kN>
__device__ __forceinline__ Vec<T, kN> load_vec(const T* p, uint64_t policy) {
    static_assert(sizeof(T) * kN == 16 || sizeof(T) * kN == 8, "8 or 16 bytes");
    Vec<T, kN> v;
    if constexpr (sizeof(T) * kN == 16) {
        uint4 w;
        asm volatile("ld.global.L2::cache_hint.v4.u32 {%0, %1, %2, %3}, [%4], %5;"
                     : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                     : "l"(p), "l"(policy));
        memcpy(&v, &w, 16);
    } else {
        uint2 w;
        asm volatile("ld.global.L2::cache_hint.v2.u32 {%0, %1}, [%2], %3;"
                     : "=r"(w.x), "=r"(w.y)
                     : "l"(p), "l"(policy));
        memcpy(&v, &w, 8);
    }
    return v;
}

template <typename T, int kN>
__device__ __forceinline__ void store_vec(T* p, const Vec<T, kN>& v) {
    static_assert(sizeof(T) * kN == 16 || sizeof(T) * kN == 8, "8 or 16 bytes");
    if constexpr (sizeof(T) * kN == 16) {
        uint4 w;
        memcpy(&w, &v, 16);
        __stcs(reinterpret_cast<uint4*>(p), w);
    } else {
        uint2 w;
        memcpy(&w, &v, 8);
        __stcs(reinterpret_cast<uint2*>(p), w);
    }
}

// ------------------------------------------------------------------------------- the sum
// A lane's squares of up to 64 entries, as one binary64 number. The squares are summed in
// binary32: four chains of at most 16 fused multiply-adds and two additions that join them, all of
// positive terms, so that at most 18 * 2^-24 of the sum is lost, and half of that, 5.4e-7, of the
// norm. From there on sums are binary64: for every entry it would be bound by its arithmetic, 1/64
// of binary32's rate. A sum outside [2^-90, 2^126]
// may have lost squares to underflow or overflow: it is taken again with the entries scaled by
// 2^90 or 2^-70, where neither can happen to any finite entry (below the first limit every entry
// is under 2^-45, and the least subnormal's square becomes 2^-118; above the second limit the
// largest square becomes 2^116). What is still not finite there holds an infinity or a NaN.
template <typename T, int kV, int kN>
__device__ __forceinline__ float chain_sum(const Vec<T, kV> (&w)[kN], float f) {
    static_assert(kV * kN <= 64, "four chains of at most 16");
    float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < kN; ++i)
#pragma unroll
        for (int j = 0; j < kV; ++j) {
            const float y = Cvt<T>::up(w[i].v[j]) * f;
            s[(i * kV + j) & 3] = fmaf(y, y, s[(i * kV + j) & 3]);
        }
    return (s[0] + s[1]) + (s[2] + s[3]);
}

template <typename T, int kV, int kN>
__device__ __forceinline__ double squares(const Vec<T, kV> (&w)[kN]) {
    const float s = chain_sum(w, 1.0f);
    if (s >= 0x1p-90f && s <= 0x1p126f) return (double)s;
    if (s < 0x1p-90f) return (double)chain_sum(w, 0x1p90f) * 0x1p-180;
    return (double)chain_sum(w, 0x1p-70f) * 0x1p140;
}

// One tile of a tensor, from entry `begin`, by one warp: 16-byte loads where the address allows (kV
// entries each), entry by entry at the ends and for unaligned tensors.
template <typename T>
__device__ __forceinline__ double tile_squares(const T* p, uint64_t n, uint64_t begin,
                                               uint64_t policy) {
    constexpr int kV = 16 / sizeof(T);
    constexpr int kLoads = kTile<T> / 32 / kV;  // 8, in flight together
    const int lane = threadIdx.x & 31;
    const uint32_t m = (uint32_t)umin64(kTile<T>, n - begin);
    const T* q = p + begin;
    double sum = 0.0;
    if (m == kTile<T> && ((uintptr_t)q & 15u) == 0) {
        Vec<T, kV> w[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            w[i] = load_vec<T, kV>(q + (i * 32 + lane) * kV, policy);
        return squares(w);
    }
    for (uint32_t h = 0; h < m; h += 32 * 8) {
        Vec<T, 1> x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t at = h + i * 32 + lane;
            x[i].v[0] = at < m ? q[at] : Cvt<T>::down(0.0f);
        }
        sum += squares(x);
    }
    return sum;
}

// The block's sum of one binary64 per thread, in a fixed order; valid in every thread.
__device__ __forceinline__ double block_sum(double x, double* sm) {
    x = warp_sum(x);
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = x;
    __syncthreads();
    double s = 0.0;
#pragma unroll
    for (int w = 0; w < kGradWarps; ++w) s += sm[w];
    __syncthreads();
    return s;
}

// Bound by HBM: one read of every entry, one multiply-add each (16-bit types: and a conversion).
// 575 us for 2^30 binary32 entries, 7.5 TB/s.
template <int kCap>
__global__ void __launch_bounds__(kGradThreads, kBlocksPerSm)
    k_grad_norm(const __grid_constant__ GradArgs a, const __grid_constant__ GradTable<kCap> tab) {
    __shared__ double sm[kGradWarps];
    grid_dep_wait();
    grid_dep_launch();
    const GradEntry* entries = a.entries ? a.entries : tab.e;
    const uint32_t* first = a.entries ? a.first : tab.first;
    const uint32_t step = gridDim.x * kGradWarps;
    const uint32_t leave = a.twice && a.tiles > kKeepTiles ? a.tiles - kKeepTiles : 0;
    const uint64_t early = l2_first(), late = l2_normal();
    double sum = 0.0;
    uint32_t t = blockIdx.x * kGradWarps + (threadIdx.x >> 5);
    if (t < a.tiles) {
        int e = upper_bound_minus1(first, a.count, t);
        for (; t < a.tiles; t += step) {
            while (t >= first[e + 1]) ++e;
            const GradEntry g = entries[e];
            const uint64_t i = t - first[e];
            const uint64_t l2 = t < leave ? early : late;
            if (g.src_type() == DGC_F32)
                sum += tile_squares((const float*)g.src, g.count(), i * kTile<float>, l2);
            else if (g.src_type() == DGC_F16)
                sum += tile_squares((const __half*)g.src, g.count(), i * kTile<__half>, l2);
            else
                sum += tile_squares((const __nv_bfloat16*)g.src, g.count(),
                                    i * kTile<__nv_bfloat16>, l2);
        }
    }
    sum = block_sum(sum, sm);
    if (threadIdx.x == 0) a.partial[blockIdx.x] = sum;
}

// norm = sqrt(sum of the partial sums), scale = max_norm / norm where norm > max_norm, else 1
// (a NaN norm compares false: scale 1; an infinite one gives 0). Binary64, rounded once.
__device__ __forceinline__ float join(const GradArgs& a, double* sm, bool write) {
    double s = 0.0;
    for (int i = threadIdx.x; i < a.nparts; i += kGradThreads) s += a.partial[i];
    const double norm = sqrt(block_sum(s, sm));
    const float scale =
        (a.max_norm > 0.0f && norm > (double)a.max_norm) ? (float)((double)a.max_norm / norm) : 1.0f;
    if (write && threadIdx.x == 0) {
        *a.norm = (float)norm;
        *a.scale = scale;
    }
    return scale;
}

__global__ void __launch_bounds__(kGradThreads) k_grad_finish(const __grid_constant__ GradArgs a) {
    __shared__ double sm[kGradWarps];
    grid_dep_wait();
    join(a, sm, true);
}

// ------------------------------------------------------------------------------- clipping
template <typename S, typename D>
__device__ __forceinline__ void tile_scale(const S* p, D* d, uint64_t n, uint64_t begin, float f) {
    constexpr int kV = (sizeof(S) == 4 || sizeof(D) == 4) ? 4 : 8;
    constexpr int kSteps = kTile<S> / 32 / kV;  // 8 or 16
    constexpr int kStep = 8;                    // loads in flight together
    const uint64_t policy = l2_first();         // their last use
    const int lane = threadIdx.x & 31;
    const uint32_t m = (uint32_t)umin64(kTile<S>, n - begin);
    const S* q = p + begin;
    D* o = d + begin;
    if (m == kTile<S> && ((uintptr_t)q & (sizeof(S) * kV - 1)) == 0 &&
        ((uintptr_t)o & (sizeof(D) * kV - 1)) == 0) {
#pragma unroll 1
        for (int h = 0; h < kSteps; h += kStep) {
            Vec<S, kV> w[kStep];
#pragma unroll
            for (int i = 0; i < kStep; ++i)
                w[i] = load_vec<S, kV>(q + ((h + i) * 32 + lane) * kV, policy);
#pragma unroll
            for (int i = 0; i < kStep; ++i) {
                Vec<D, kV> r;
#pragma unroll
                for (int j = 0; j < kV; ++j) r.v[j] = Cvt<D>::down(Cvt<S>::up(w[i].v[j]) * f);
                store_vec(o + ((h + i) * 32 + lane) * kV, r);
            }
        }
        return;
    }
    for (uint32_t h = 0; h < m; h += 32 * 8) {
        S x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t at = h + i * 32 + lane;
            x[i] = at < m ? q[at] : Cvt<S>::down(0.0f);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t at = h + i * 32 + lane;
            if (at < m) o[at] = Cvt<D>::down(Cvt<S>::up(x[i]) * f);
        }
    }
}

template <typename S>
__device__ __forceinline__ void tile_scale_to(const GradEntry& g, uint64_t tile, float f) {
    const S* p = (const S*)g.src;
    const uint64_t begin = tile * kTile<S>;
    if (g.dst_type() == DGC_F32)
        tile_scale(p, (float*)g.dst, g.count(), begin, f);
    else if (g.dst_type() == DGC_F16)
        tile_scale(p, (__half*)g.dst, g.count(), begin, f);
    else
        tile_scale(p, (__nv_bfloat16*)g.dst, g.count(), begin, f);
}

// Bound by HBM: every entry read again and written. Many small blocks, a tile a warp, which the
// hardware hands to the SMs as they come free, from the list's end back: what the norm read last is
// still in L2 (in the list's order 25.6M binary32 entries take 55.6 us, both kernels; from the end
// 50.2). Persistent blocks with even shares took 8% longer on 411M bf16 entries, with loads through
// shared memory or without: SMs do not all reach memory equally fast. kJoin: every block joins the
// partial sums itself, for lists that need few blocks; else k_grad_finish has done it.
template <int kCap, bool kJoin>
__global__ void __launch_bounds__(kGradThreads)
    k_grad_scale(const __grid_constant__ GradArgs a, const __grid_constant__ GradTable<kCap> tab) {
    __shared__ double sm[kGradWarps];
    const GradEntry* entries = a.entries ? a.entries : tab.e;
    const uint32_t* first = a.entries ? a.first : tab.first;
    const uint32_t t = (gridDim.x - 1 - blockIdx.x) * kGradWarps + (threadIdx.x >> 5);
    grid_dep_wait();
    const int e = t < a.tiles ? upper_bound_minus1(first, a.count, t) : 0;
    const float f = kJoin ? join(a, sm, blockIdx.x == 0) : *a.scale;
    if (t >= a.tiles || (a.in_place && f == 1.0f)) return;
    const GradEntry g = entries[e];
    const uint64_t i = t - first[e];
    if (g.src_type() == DGC_F32)
        tile_scale_to<float>(g, i, f);
    else if (g.src_type() == DGC_F16)
        tile_scale_to<__half>(g, i, f);
    else
        tile_scale_to<__nv_bfloat16>(g, i, f);
}

// ----------------------------------------------------------------------------------- host
size_t type_size(int32_t t) { return t == DGC_F32 ? 4 : 2; }
uint64_t tiles_of(const dgc_tensor& t) {
    const uint64_t per = kTileBytes / type_size(t.dtype);
    return ((uint64_t)t.n + per - 1) / per;
}

// Checks a list and counts its warp tiles.
int check_list(const dgc_tensor* t, int32_t count, uint64_t* tiles) {
    if (count < 0 || (count > 0 && !t)) return DGC_EINVAL;
    if (count > kMaxTensors) return DGC_EUNSUPPORTED;
    uint64_t sum = 0;
    for (int32_t i = 0; i < count; ++i) {
        if (t[i].n < 0 || t[i].reserved != 0) return DGC_EINVAL;
        if (t[i].dtype != DGC_F32 && t[i].dtype != DGC_F16 && t[i].dtype != DGC_BF16)
            return DGC_EINVAL;
        if (t[i].n > 0 && (!t[i].data || ((uintptr_t)t[i].data & (type_size(t[i].dtype) - 1))))
            return DGC_EINVAL;
        if (t[i].n > (1ll << 42)) return DGC_EUNSUPPORTED;
        sum += tiles_of(t[i]);
        if (sum > 0x7FFFFFFFull) return DGC_EUNSUPPORTED;
    }
    *tiles = sum;
    return DGC_OK;
}

struct GradLayout {
    size_t partial, entries, first, total;
};
GradLayout grad_layout(int32_t count) {
    auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
    GradLayout L{};
    L.partial = 0;
    L.entries = up(sizeof(double) * 4096);  // blocks of k_grad_norm: at most 4096
    L.first = L.entries;
    L.total = L.entries;
    if (count > kTableCap) {
        L.first = up(L.entries + sizeof(GradEntry) * (size_t)count);
        L.total = up(L.first + sizeof(uint32_t) * ((size_t)count + 1));
    }
    return L;
}

// A launch that may start while the kernel ahead of it ends (it waits before it reads).
template <typename... A>
int launch(void (*kernel)(A...), unsigned grid, cudaStream_t s, const std::decay_t<A>&... args) {
    void* ptrs[] = {const_cast<void*>(static_cast<const void*>(&args))...};
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(grid);
    c.blockDim = dim3(kGradThreads);
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

template <int kCap>
void fill(GradTable<kCap>* t, const dgc_tensor* src, const dgc_tensor* dst, int32_t count,
          uint32_t* tile) {
    for (int32_t i = 0; i < count; ++i) {
        const dgc_tensor& d = dst ? dst[i] : src[i];
        t->e[i].src = src[i].data;
        t->e[i].dst = d.data;
        t->e[i].n = (uint64_t)src[i].n | ((uint64_t)src[i].dtype << 56) | ((uint64_t)d.dtype << 60);
        t->first[i] = *tile;
        *tile += (uint32_t)tiles_of(src[i]);
    }
    t->first[count] = *tile;
}

template <int kCap>
int run(const dgc_tensor* src, const dgc_tensor* dst, int32_t count, bool clip, GradArgs a,
        unsigned grid, cudaStream_t s) {
    GradTable<kCap> tab;
    if (!a.entries) {
        uint32_t tile = 0;
        fill(&tab, src, dst, count, &tile);
    }
    int rc = launch(k_grad_norm<kCap>, grid, s, a, tab);
    if (rc) return rc;
    const unsigned blocks = (a.tiles + kGradWarps - 1) / kGradWarps;
    if (clip && blocks <= grid)
        return launch(k_grad_scale<kCap, true>, blocks ? blocks : 1, s, a, tab);
    rc = launch(k_grad_finish, 1, s, a);
    if (rc || !clip) return rc;
    return launch(k_grad_scale<kCap, false>, blocks, s, a, tab);
}

int grad_call(const dgc_tensor* src, const dgc_tensor* dst, int32_t count, float max_norm,
              bool clip, float* norm, float* scale, void* ws, size_t ws_bytes,
              dgc_stream_t stream) {
    uint64_t tiles = 0, dst_tiles = 0;
    if (std::isnan(max_norm) || !norm || !scale || !ws || ((uintptr_t)ws & 255u)) return DGC_EINVAL;
    int rc = check_list(src, count, &tiles);
    if (rc) return rc;
    bool in_place = true;
    if (clip && dst) {
        rc = check_list(dst, count, &dst_tiles);
        if (rc) return rc;
        for (int32_t i = 0; i < count; ++i) {
            if (dst[i].n != src[i].n) return DGC_EINVAL;
            if (src[i].n == 0) continue;
            if (dst[i].data != src[i].data)
                in_place = false;
            else if (dst[i].dtype != src[i].dtype)
                return DGC_EINVAL;
        }
    }
    const GradLayout L = grad_layout(count);
    if (ws_bytes < L.total) return DGC_EINVAL;
    const int sms = dgc_internal_sm_count();
    if (sms <= 0) return DGC_ECUDA;

    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    char* w = static_cast<char*>(ws);
    GradArgs a{};
    a.count = count;
    a.tiles = (uint32_t)tiles;
    a.partial = reinterpret_cast<double*>(w + L.partial);
    a.max_norm = (max_norm > 0.0f && !std::isinf(max_norm)) ? max_norm : 0.0f;
    a.in_place = in_place;
    a.twice = clip;
    a.norm = norm;
    a.scale = scale;
    const uint64_t want = (tiles + kGradWarps - 1) / kGradWarps;
    const uint64_t most = umin64(4096, (uint64_t)sms * kBlocksPerSm);
    const unsigned grid = (unsigned)umin64(want ? want : 1, most);
    a.nparts = (int32_t)grid;
    if (count <= kSmallTable) return run<kSmallTable>(src, dst, count, clip, a, grid, s);
    if (count <= kMidTable) return run<kMidTable>(src, dst, count, clip, a, grid, s);
    if (count <= kTableCap) return run<kTableCap>(src, dst, count, clip, a, grid, s);

    // a long list: its table goes to the workspace in the parameters of a launch per part
    GradEntry* entries = reinterpret_cast<GradEntry*>(w + L.entries);
    uint32_t* first = reinterpret_cast<uint32_t*>(w + L.first);
    uint32_t tile = 0;
    for (int32_t at = 0; at < count; at += kTableCap) {
        GradTable<kTableCap> tab;
        const int32_t m = count - at < kTableCap ? count - at : kTableCap;
        fill(&tab, src + at, dst ? dst + at : nullptr, m, &tile);
        k_grad_table<<<1, 256, 0, s>>>(tab, m, entries + at, first + at);
        if (cudaPeekAtLastError() != cudaSuccess) {
            cudaGetLastError();
            return DGC_ECUDA;
        }
        dgc_internal_count_launches(1);
    }
    a.entries = entries;
    a.first = first;
    return run<kSmallTable>(src, dst, count, clip, a, grid, s);
}

}  // namespace
}  // namespace dgc

using namespace dgc;

extern "C" int dgc_grad_workspace(const dgc_tensor* src, int32_t count, size_t* bytes) {
    uint64_t tiles = 0;
    if (!bytes) return DGC_EINVAL;
    const int rc = check_list(src, count, &tiles);
    if (rc) return rc;
    *bytes = grad_layout(count).total;
    return DGC_OK;
}

extern "C" int dgc_grad_norm(const dgc_tensor* src, int32_t count, float max_norm, float* norm,
                             float* scale, void* ws, size_t ws_bytes, dgc_stream_t stream) {
    return grad_call(src, nullptr, count, max_norm, false, norm, scale, ws, ws_bytes, stream);
}

extern "C" int dgc_grad_clip(const dgc_tensor* src, const dgc_tensor* dst, int32_t count,
                             float max_norm, float* norm, float* scale, void* ws, size_t ws_bytes,
                             dgc_stream_t stream) {
    return grad_call(src, dst, count, max_norm, true, norm, scale, ws, ws_bytes, stream);
}
