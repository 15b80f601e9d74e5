// recurrence.cu -- a gated linear recurrence over packed sequences and its backward pass (sm_103a).
//
//   a = 1 / (1 + e^-gate);  h_t = a_t h_{t-1} + (1 - a_t) x_t;  y_t = h_t
//   u_t = a_t G_t;  G_t = dy_t + u_{t+1};  dx_t = G_t (1 - a_t)
//   dgate_t = G_t (h_{t-1} - x_t) a_t (1 - a_t)
//
// Columns are independent; rows are a scan. A step, and any run of steps, is an affine map of the
// state, h -> A h + B, so a run's map is known before the state that enters it. A block takes 64
// columns of a chunk of rows, each of its 8 warps kS rows of it, two columns a lane, all in
// registers:
//   1. each warp composes its rows' map; the first warp composes the warps' and publishes the
//      chunk's (A, B);
//   2. 32 chunks are a group: the first warp takes the state that enters the group, which the last
//      chunk of the group ahead publishes, and applies the maps of the chunks before its own, in
//      order. (Which maps are joined is fixed, so the rounding is too: results are the same bits on
//      every run. A chain from chunk to chunk would cost its latency 32 times.)
//   3. each warp walks its rows again from the state it enters with, and writes.
// The data is read once. Blocks take their chunks by a ticket, in order, so a block only waits for
// blocks that run; waits are bounded all the same.
//
// A sequence's first row has no predecessor: its map is h -> B with B = a h0 + (1 - a) x, kept as
// A = kReset, so that nothing of what is ahead, infinities and NaNs among it, comes through.
//
// The backward pass is the same scan from the end (u_{t+1} -> u_t = a_t u_{t+1} + a_t dy_t). It needs
// h_{t-1}, which it walks again from the state ahead of each piece of 64 rows that the forward pass
// left.
#include <algorithm>

#include "rows.cuh"

namespace dgc {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCols = 64;        // of a block
constexpr uint32_t kGroup = 32;  // chunks
constexpr uint32_t kPiece = 64;  // rows between two saved states
constexpr float kReset = -1.0f;  // no run of steps has a negative A

struct ScanArgs {
    const void *x, *gate, *dy;
    void *y, *dx, *dgate;
    uint64_t ldx, ldg, lddy, ldy, lddx, lddg;
    const float *h0, *d_last;
    float *h_last, *d_h0, *saved;
    uint64_t ldh0, ldd_last, ldh_last, ldd_h0, lds;
    const int64_t* offsets;
    uint32_t nseq, rows, cols, tiles, chunks;
    // the workspace: a ticket, whether a wait gave up, a flag of every chunk and of every group of a column tile, their
    // maps {A, A, B, B} and states of a lane's two columns. ticket null: one chunk, nothing shared.
    uint32_t *ticket, *abort, *chunk_flag, *group_flag;
    float4* maps;
    float2* states;
    uint32_t spin_limit, lost;  // lost: self-test, a chunk that publishes nothing
    int32_t* status;
};

__device__ __forceinline__ uint32_t ld_acquire(const uint32_t* p) {
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void st_release(uint32_t* p, uint32_t v) {
    asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// Two columns of a row: kPair whole, where the address allows it and both are there.
template <typename T>
struct Two {
    Packed<T, 2> p;
    template <bool kPair>
    __device__ static Two load(const void* m, uint64_t ld, uint64_t row, uint32_t col, uint32_t n) {
        return {load_piece<kPair, T, 2>(static_cast<const T*>(m) + row * ld + col, n)};
    }
    __device__ float2 up() const {
        float f[2];
        unpack<T, 2>(p, f);
        return {f[0], f[1]};
    }
};
template <typename T, bool kPair>
__device__ __forceinline__ void store_two(void* m, uint64_t ld, uint64_t row, uint32_t col,
                                          uint32_t n, float2 v) {
    const float f[2] = {v.x, v.y};
    store_piece<kPair, T, 2>(static_cast<T*>(m) + row * ld + col, pack<T, 2>(f), n);
}
__device__ __forceinline__ float2 load_state(const float* m, uint64_t ld, uint64_t row,
                                             uint32_t col, uint32_t n) {
    const float* p = m + row * ld + col;
    return {n > 0 ? p[0] : 0.0f, n > 1 ? p[1] : 0.0f};
}
__device__ __forceinline__ void store_state(float* m, uint64_t ld, uint64_t row, uint32_t col,
                                            uint32_t n, float2 v) {
    float* p = m + row * ld + col;
    if (n > 0) p[0] = v.x;
    if (n > 1) p[1] = v.y;
}

// a = 1 / (1 + e^-g) and 1 - a = e^-g / (1 + e^-g), neither by a subtraction. e^-g is held below
// 2^126, where the reciprocal is still a normal number; a gate of -infinity closes the state off.
__device__ __forceinline__ void sigmoid2(float g, float& a, float& keep) {
    const float e = expf(-g);
    const float r = __fdividef(1.0f, 1.0f + fminf(e, 0x1p125f));
    a = e < INFINITY ? r : 0.0f;
    keep = e < 0x1p125f ? e * r : 1.0f;
    if (g != g) a = keep = g;
}

// h -> A h + B, two columns.
struct Map {
    float4 m;  // A, A, B, B
    __device__ float2 operator()(float2 h) const {
        return {m.x < 0.0f ? m.z : fmaf(m.x, h.x, m.z), m.y < 0.0f ? m.w : fmaf(m.y, h.y, m.w)};
    }
};

// The first index i in [0, n) with off[i] >= key, n if there is none. All lanes of a warp; any
// contents (where they do not rise, any index).
__device__ __forceinline__ uint32_t first_from(const int64_t* off, uint32_t n, int64_t key) {
    const uint32_t lane = threadIdx.x & 31;
    uint32_t lo = 0, len = n;
    while (len > 0) {
        const uint32_t step = (len + 31) / 32;
        const uint32_t i = lo + min((lane + 1) * step, len) - 1;
        const uint32_t not_less = ~__ballot_sync(kFull, off[i] < key);
        if (not_less == 0) return lo + len;
        const uint32_t less = __ffs(not_less) - 1;
        lo += less * step;
        if (step == 1) return lo;
        len = min(step, len - less * step) - 1;  // its last one is known not to be less
        if (len == 0) return lo;
    }
    return lo;
}

// Marks the rows of a chunk where a sequence starts or ends. starts, ends: the sequence, or -1.
template <int kRows>
__device__ __forceinline__ void mark_rows(const ScanArgs& a, uint32_t row0, int32_t* starts,
                                          int32_t* ends) {
    const int lane = threadIdx.x & 31;
    for (int i = lane; i < kRows; i += 32) starts[i] = ends[i] = -1;
    __syncwarp();
    const uint32_t n = a.nseq + 1;
    for (uint32_t i0 = first_from(a.offsets, n, row0);; i0 += 32) {
        const uint32_t i = i0 + lane;
        const int64_t off = i < n ? a.offsets[i] : INT64_MAX;
        if (off >= (int64_t)row0 && off <= (int64_t)row0 + kRows) {
            const int r = (int)(off - row0);
            if (r < kRows && i + 1 < n && a.offsets[i + 1] > off) starts[r] = (int32_t)i;
            if (r > 0 && i > 0 && a.offsets[i - 1] < off) ends[r - 1] = (int32_t)i - 1;
        }
        if (!__all_sync(kFull, off <= (int64_t)row0 + kRows)) break;
    }
}

// What has no row: sequences of length 0 pass their state on; and the table's check. By the first
// chunk's blocks.
__device__ __forceinline__ void empty_sequences(const ScanArgs& a, uint32_t tile, const float* from,
                                                uint64_t ld_from, float* to, uint64_t ld_to) {
    const int lane = threadIdx.x & 31;
    const uint32_t col = tile * kCols + 2 * lane, n = col < a.cols ? min(2u, a.cols - col) : 0;
    bool bad = false;
    for (uint32_t q0 = (threadIdx.x >> 5) * 32; q0 < a.nseq; q0 += kThreads) {
        const uint32_t q = q0 + lane;
        const int64_t b = q < a.nseq ? a.offsets[q] : 0, e = q < a.nseq ? a.offsets[q + 1] : 1;
        bad |= q < a.nseq && (b > e || b < 0 || e > (int64_t)a.rows);
        uint32_t todo = __ballot_sync(kFull, b == e);
        for (; to && todo; todo &= todo - 1) {
            const uint32_t s = q0 + __ffs(todo) - 1;
            store_state(to, ld_to, s, col, n,
                        from ? load_state(from, ld_from, s, col, n) : make_float2(0.0f, 0.0f));
        }
    }
    if (tile == 0 && bad) report(a.status, DGC_EINVAL);
}

// The chunk and the column tile of this block.
__device__ __forceinline__ uint32_t take_ticket(const ScanArgs& a, uint32_t* slot) {
    if (!a.ticket) return blockIdx.x;
    if (threadIdx.x == 0) *slot = atomicAdd(a.ticket, 1u);
    __syncthreads();
    return *slot;
}

// By the first warp: publishes the chunk's map, if the last of a group the state behind it too, and
// returns the state that enters the chunk. order: the chunk's place in the scan's direction.
// no_carry: nothing enters (a sequence begins with the chunk).
__device__ __forceinline__ void publish_map(const ScanArgs& a, uint32_t order, uint32_t tile,
                                            const Map& m) {
    const int lane = threadIdx.x & 31;
    if (!a.ticket || order == a.lost) return;
    a.maps[((uint64_t)order * a.tiles + tile) * 32 + lane] = m.m;
    __threadfence();
    __syncwarp();
    if (lane == 0) st_release(&a.chunk_flag[(uint64_t)tile * a.chunks + order], 1);
}
__device__ __forceinline__ float2 enter_chunk(const ScanArgs& a, uint32_t order, uint32_t tile,
                                              const Map& m, bool no_carry) {
    const uint32_t lane = threadIdx.x & 31;
    const uint32_t group = order / kGroup, k = order % kGroup;
    const uint32_t groups = (a.chunks + kGroup - 1) / kGroup;
    float2 h = {0.0f, 0.0f};
    if (!a.ticket) return h;
    if (!no_carry) {
        const uint32_t* flag = nullptr;
        if (lane < k)
            flag = &a.chunk_flag[(uint64_t)tile * a.chunks + group * kGroup + lane];
        else if (lane == 31 && group > 0)
            flag = &a.group_flag[(uint64_t)tile * groups + group];
        bool ready = flag == nullptr;
        for (uint32_t spins = 0;; ++spins) {
            if (!ready) ready = ld_acquire(flag) != 0;
            if (__all_sync(kFull, ready)) break;
            if (spins > a.spin_limit || ((spins & 63) == 63 && ld_acquire(a.abort) != 0)) {
                if (lane == 0) {
                    report(a.status, DGC_ETIMEOUT);
                    atomicExch(a.abort, 1u);
                }
                break;
            }
            __nanosleep(20);
        }
        __threadfence();
        if (group > 0) h = __ldcg(&a.states[((uint64_t)group * a.tiles + tile) * 32 + lane]);
        const float4* maps = a.maps + ((uint64_t)group * kGroup * a.tiles + tile) * 32 + lane;
        const uint64_t step = (uint64_t)a.tiles * 32;
        for (uint32_t i = 0; i < k; i += 8) {
            Map p[8];
#pragma unroll
            for (uint32_t j = 0; j < 8; ++j)
                if (i + j < k) p[j].m = __ldcg(maps + (i + j) * step);
#pragma unroll
            for (uint32_t j = 0; j < 8; ++j)
                if (i + j < k) h = p[j](h);
        }
    }
    if (k == kGroup - 1 && group + 1 < groups && order != a.lost) {
        a.states[((uint64_t)(group + 1) * a.tiles + tile) * 32 + lane] = m(h);
        __threadfence();
        __syncwarp();
        if (lane == 0) st_release(&a.group_flag[(uint64_t)tile * groups + group + 1], 1);
    }
    return h;
}

// Composes the maps of the warps before (or, from the end, behind) one.
struct WarpMaps {
    float4 m[kWarps][32];
};

__global__ void __launch_bounds__(256) k_scan_clear(uint32_t* words, uint64_t n) {
    grid_dep_wait();
    grid_dep_launch();
    for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (uint64_t)gridDim.x * 256)
        words[i] = 0;
}

// --------------------------------------------------------------------------------- forward
// Bound by HBM: x and gate read once, y written once.
template <typename T, bool kPair, int kS>
__global__ void __launch_bounds__(kThreads) k_scan(const __grid_constant__ ScanArgs a) {
    constexpr int kRows = kWarps * kS;
    __shared__ int32_t starts[kRows], ends[kRows];
    __shared__ WarpMaps maps;
    __shared__ float2 enter[32];
    __shared__ uint32_t slot;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_dep_wait();
    grid_dep_launch();
    const uint32_t ticket = take_ticket(a, &slot);
    const uint32_t chunk = ticket / a.tiles, tile = ticket % a.tiles;
    const uint32_t row0 = chunk * kRows, first = row0 + warp * kS;
    const uint32_t col = tile * kCols + 2 * lane, n = col < a.cols ? min(2u, a.cols - col) : 0;
    Two<T> px[kS], pg[kS];
#pragma unroll
    for (int s = 0; s < kS; ++s) {
        const uint32_t here = first + s < a.rows ? n : 0;
        pg[s] = Two<T>::template load<kPair>(a.gate, a.ldg, first + s, col, here);
        px[s] = Two<T>::template load<kPair>(a.x, a.ldx, first + s, col, here);
    }
    const int64_t valid0 = a.offsets[0], valid1 = a.offsets[a.nseq];
    if (warp == kWarps - 1) mark_rows<kRows>(a, row0, starts, ends);
    if (chunk == 0) empty_sequences(a, tile, a.h0, a.ldh0, a.h_last, a.ldh_last);
    __syncthreads();
    uint32_t start_bits = 0, end_bits = 0;
    {
        const int r = warp * kS + (lane < kS ? lane : 0);
        start_bits = __ballot_sync(kFull, lane < kS && starts[r] >= 0);
        end_bits = __ballot_sync(kFull, lane < kS && ends[r] >= 0);
    }
    // rows as h -> A h + B
    float2 A[kS], B[kS];
#pragma unroll
    for (int s = 0; s < kS; ++s) {
        const float2 g = pg[s].up(), x = px[s].up();
        float2 keep;
        sigmoid2(g.x, A[s].x, keep.x);
        sigmoid2(g.y, A[s].y, keep.y);
        B[s] = {keep.x * x.x, keep.y * x.y};
    }
    if (start_bits && a.h0) {
        float2 h[kS];
#pragma unroll
        for (int s = 0; s < kS; ++s)
            h[s] = load_state(a.h0, a.ldh0, start_bits >> s & 1 ? starts[warp * kS + s] : 0, col,
                              start_bits >> s & 1 ? n : 0);
#pragma unroll
        for (int s = 0; s < kS; ++s)
            if (start_bits >> s & 1) {
                B[s].x = fmaf(A[s].x, h[s].x, B[s].x);
                B[s].y = fmaf(A[s].y, h[s].y, B[s].y);
            }
    }
    Map m{{1.0f, 1.0f, 0.0f, 0.0f}};
#pragma unroll
    for (int s = 0; s < kS; ++s) {
        if (start_bits >> s & 1) {
            m.m = {kReset, kReset, B[s].x, B[s].y};
        } else {
            m.m.z = fmaf(A[s].x, m.m.z, B[s].x);
            m.m.w = fmaf(A[s].y, m.m.w, B[s].y);
            m.m.x = m.m.x < 0.0f ? kReset : m.m.x * A[s].x;
            m.m.y = m.m.y < 0.0f ? kReset : m.m.y * A[s].y;
        }
    }
    maps.m[warp][lane] = m.m;
    __syncthreads();
    if (warp == 0) {
        Map all = m;
        for (int w = 1; w < kWarps; ++w) {
            const Map q{maps.m[w][lane]};
            const float2 b = q({all.m.z, all.m.w});
            all.m = {q.m.x < 0.0f || all.m.x < 0.0f ? kReset : q.m.x * all.m.x,
                     q.m.y < 0.0f || all.m.y < 0.0f ? kReset : q.m.y * all.m.y, b.x, b.y};
        }
        publish_map(a, chunk, tile, all);
        enter[lane] = enter_chunk(a, chunk, tile, all, starts[0] >= 0);
    }
    __syncthreads();
    float2 h = enter[lane];
    for (int w = 0; w < warp; ++w) h = Map{maps.m[w][lane]}(h);
    if (a.saved && first % kPiece == 0 && first < a.rows)
        store_state(a.saved, a.lds, first / kPiece, col, n, h);
#pragma unroll
    for (int s = 0; s < kS; ++s) {
        const uint32_t row = first + s;
        if (start_bits >> s & 1) {
            h = B[s];
        } else {
            h.x = fmaf(A[s].x, h.x, B[s].x);
            h.y = fmaf(A[s].y, h.y, B[s].y);
        }
        if (row < a.rows && row >= valid0 && row < valid1)
            store_two<T, kPair>(a.y, a.ldy, row, col, n, h);
        if (a.h_last && (end_bits >> s & 1) && row < a.rows)
            store_state(a.h_last, a.ldh_last, ends[warp * kS + s], col, n, h);
    }
}

// -------------------------------------------------------------------------------- backward
// Bound by HBM: x, gate and dy read once, dx and dgate written once, the states of every 64th row.
template <typename T, bool kPair, int kS>
__global__ void __launch_bounds__(kThreads) k_scan_back(const __grid_constant__ ScanArgs a) {
    constexpr int kRows = kWarps * kS;
    static_assert(kRows % kPiece == 0 && kPiece % kS == 0, "a chunk begins at a saved state");
    __shared__ int32_t starts[kRows], ends[kRows];
    __shared__ WarpMaps maps, back;
    __shared__ float2 enter[32];
    __shared__ uint32_t slot;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_dep_wait();
    grid_dep_launch();
    const uint32_t ticket = take_ticket(a, &slot);
    const uint32_t order = ticket / a.tiles, tile = ticket % a.tiles;
    const uint32_t chunk = a.chunks - 1 - order;
    const uint32_t row0 = chunk * kRows, first = row0 + warp * kS;
    const uint32_t col = tile * kCols + 2 * lane, n = col < a.cols ? min(2u, a.cols - col) : 0;
    Two<T> px[kS], pg[kS], pd[kS];
#pragma unroll
    for (int s = 0; s < kS; ++s) {
        const uint32_t here = first + s < a.rows ? n : 0;
        pg[s] = Two<T>::template load<kPair>(a.gate, a.ldg, first + s, col, here);
        px[s] = Two<T>::template load<kPair>(a.x, a.ldx, first + s, col, here);
        pd[s] = Two<T>::template load<kPair>(a.dy, a.lddy, first + s, col, here);
    }
    float2 h = row0 < a.rows ? load_state(a.saved, a.lds, row0 / kPiece, col, n)
                             : make_float2(0.0f, 0.0f);
    const int64_t valid0 = a.offsets[0], valid1 = a.offsets[a.nseq];
    if (warp == kWarps - 1) mark_rows<kRows>(a, row0, starts, ends);
    if (chunk == 0) empty_sequences(a, tile, a.d_last, a.ldd_last, a.d_h0, a.ldd_h0);
    __syncthreads();
    uint32_t start_bits = 0, end_bits = 0;
    {
        const int r = warp * kS + (lane < kS ? lane : 0);
        start_bits = __ballot_sync(kFull, lane < kS && starts[r] >= 0);
        end_bits = __ballot_sync(kFull, lane < kS && ends[r] >= 0);
    }
    float2 A[kS], keep[kS], q[kS], G[kS];  // q: x, then (h_{t-1} - x) a (1 - a)
#pragma unroll
    for (int s = 0; s < kS; ++s) {
        const float2 g = pg[s].up();
        q[s] = px[s].up();
        G[s] = pd[s].up();
        sigmoid2(g.x, A[s].x, keep[s].x);
        sigmoid2(g.y, A[s].y, keep[s].y);
    }
    if (end_bits && a.d_last)
#pragma unroll
        for (int s = 0; s < kS; ++s)
            if (end_bits >> s & 1) {
                const float2 d = load_state(a.d_last, a.ldd_last, ends[warp * kS + s], col, n);
                G[s].x += d.x;
                G[s].y += d.y;
            }
    // the rows' map of h, and from the end that of u
    Map m{{1.0f, 1.0f, 0.0f, 0.0f}}, u{{1.0f, 1.0f, 0.0f, 0.0f}};
    float2 first_h[kS];  // a sequence's first state where one starts
#pragma unroll
    for (int s = 0; s < kS; ++s) {
        first_h[s] = {0.0f, 0.0f};
        if ((start_bits >> s & 1) && a.h0)
            first_h[s] = load_state(a.h0, a.ldh0, starts[warp * kS + s], col, n);
        const float2 b = {keep[s].x * q[s].x, keep[s].y * q[s].y};
        if (start_bits >> s & 1) {
            m.m = {kReset, kReset, fmaf(A[s].x, first_h[s].x, b.x), fmaf(A[s].y, first_h[s].y, b.y)};
        } else {
            m.m.z = fmaf(A[s].x, m.m.z, b.x);
            m.m.w = fmaf(A[s].y, m.m.w, b.y);
            m.m.x = m.m.x < 0.0f ? kReset : m.m.x * A[s].x;
            m.m.y = m.m.y < 0.0f ? kReset : m.m.y * A[s].y;
        }
    }
#pragma unroll
    for (int s = kS - 1; s >= 0; --s) {
        if (end_bits >> s & 1) {
            u.m = {kReset, kReset, A[s].x * G[s].x, A[s].y * G[s].y};
        } else {
            u.m.z = A[s].x * (G[s].x + u.m.z);
            u.m.w = A[s].y * (G[s].y + u.m.w);
            u.m.x = u.m.x < 0.0f ? kReset : u.m.x * A[s].x;
            u.m.y = u.m.y < 0.0f ? kReset : u.m.y * A[s].y;
        }
    }
    maps.m[warp][lane] = m.m;
    back.m[warp][lane] = u.m;
    __syncthreads();
    Map all = u;  // of the last warp, which is the first one from the end
    if (warp == kWarps - 1) {
        for (int w = kWarps - 2; w >= 0; --w) {
            const Map p{back.m[w][lane]};
            const float2 b = p({all.m.z, all.m.w});
            all.m = {p.m.x < 0.0f || all.m.x < 0.0f ? kReset : p.m.x * all.m.x,
                     p.m.y < 0.0f || all.m.y < 0.0f ? kReset : p.m.y * all.m.y, b.x, b.y};
        }
        publish_map(a, order, tile, all);
    }
    for (int w = 0; w < warp; ++w) h = Map{maps.m[w][lane]}(h);
#pragma unroll
    for (int s = 0; s < kS; ++s) {
        if (start_bits >> s & 1) h = first_h[s];
        const float2 x = q[s];
        q[s] = {(h.x - x.x) * A[s].x * keep[s].x, (h.y - x.y) * A[s].y * keep[s].y};
        h.x = fmaf(A[s].x, h.x, keep[s].x * x.x);
        h.y = fmaf(A[s].y, h.y, keep[s].y * x.y);
    }
    if (warp == kWarps - 1)
        enter[lane] = enter_chunk(a, order, tile, all, ends[kRows - 1] >= 0);
    __syncthreads();
    float2 v = enter[lane];  // u of the row behind
    for (int w = kWarps - 1; w > warp; --w) v = Map{back.m[w][lane]}(v);
#pragma unroll
    for (int s = kS - 1; s >= 0; --s) {
        const uint32_t row = first + s;
        if (end_bits >> s & 1) v = {0.0f, 0.0f};
        const float2 g = {G[s].x + v.x, G[s].y + v.y};
        if (row < a.rows && row >= valid0 && row < valid1) {
            store_two<T, kPair>(a.dx, a.lddx, row, col, n, {g.x * keep[s].x, g.y * keep[s].y});
            store_two<T, kPair>(a.dgate, a.lddg, row, col, n, {g.x * q[s].x, g.y * q[s].y});
        }
        v = {A[s].x * g.x, A[s].y * g.y};
        if (a.d_h0 && (start_bits >> s & 1) && row < a.rows)
            store_state(a.d_h0, a.ldd_h0, starts[warp * kS + s], col, n, v);
    }
}

// ----------------------------------------------------------------------------------- host
constexpr uint32_t kBackRows = 64;     // of a chunk of the backward pass
constexpr uint32_t kForwardRows = 128; // of the forward pass

struct ScanLayout {
    size_t flags, flag_words, maps, states, total;
    uint32_t chunks, groups, tiles;
};
ScanLayout scan_layout(uint64_t rows, uint64_t cols, uint32_t chunk_rows) {
    auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
    ScanLayout L{};
    L.chunks = (uint32_t)std::max<uint64_t>(1, (rows + chunk_rows - 1) / chunk_rows);
    L.groups = (L.chunks + kGroup - 1) / kGroup;
    L.tiles = (uint32_t)((cols + kCols - 1) / kCols);
    if (L.chunks == 1) return L;
    L.flag_words = 2 + (size_t)L.tiles * (L.chunks + L.groups);
    L.maps = up(L.flag_words * 4);
    L.states = L.maps + (size_t)L.chunks * L.tiles * 32 * sizeof(float4);
    L.total = up(L.states + (size_t)L.groups * L.tiles * 32 * sizeof(float2));
    return L;
}
size_t scan_workspace(uint64_t rows, uint64_t cols) {
    return std::max(scan_layout(rows, cols, kForwardRows).total,
                    scan_layout(rows, cols, kBackRows).total);
}

// A state of binary32, one row a sequence; may be missing.
int check_state(const dgc_matrix* m, uint64_t nseq, uint64_t cols, const float** p, uint64_t* ld) {
    if (!m) return DGC_OK;
    Rows r;
    const int rc = check_rows(m, &r, DGC_F32);
    if (rc) return rc;
    if (!r.shaped(nseq, cols)) return DGC_EINVAL;
    *p = static_cast<const float*>(r.p);
    *ld = r.ld;
    return DGC_OK;
}

int start_scan(ScanArgs& a, const ScanLayout& L, void* ws, cudaStream_t s) {
    a.tiles = L.tiles;
    a.chunks = L.chunks;
    if (!a.spin_limit) {
        a.spin_limit = kDefaultSpinLimit;
        a.lost = ~0u;
    }
    if (L.chunks == 1) return DGC_OK;
    char* w = static_cast<char*>(ws);
    a.ticket = reinterpret_cast<uint32_t*>(w);
    a.abort = a.ticket + 1;
    a.chunk_flag = a.ticket + 2;
    a.group_flag = a.chunk_flag + (size_t)L.tiles * L.chunks;
    a.maps = reinterpret_cast<float4*>(w + L.maps);
    a.states = reinterpret_cast<float2*>(w + L.states);
    const unsigned blocks = (unsigned)std::min<size_t>(1024, (L.flag_words + 1023) / 1024);
    return launch_rows_kernel(k_scan_clear, dim3(blocks), 256, s, a.ticket,
                              (uint64_t)L.flag_words);
}

int check_common(const dgc_matrix* x, const dgc_matrix* gate, const int64_t* offsets, int32_t nseq,
                 const int32_t* status, Rows* mx, Rows* mg) {
    int rc;
    if (!x || !status || nseq < 0 || !offsets || ((uintptr_t)offsets & 7u)) return DGC_EINVAL;
    if (nseq > kMaxExtent) return DGC_EUNSUPPORTED;
    if ((rc = check_rows(x, mx, -1)) || (rc = check_rows(gate, mg, mx->dtype))) return rc;
    return mg->shaped(mx->rows, mx->cols) ? DGC_OK : DGC_EINVAL;
}
bool bad_workspace(void* ws, size_t ws_bytes, size_t need) {
    return ws_bytes < need || (need && (!ws || ((uintptr_t)ws & 255u)));
}

int recurrence(const dgc_matrix* x, const dgc_matrix* gate, const int64_t* offsets, int32_t nseq,
               const dgc_matrix* h0, const dgc_matrix* y, const dgc_matrix* h_last,
               const dgc_matrix* saved, int32_t* status, void* ws, size_t ws_bytes,
               dgc_stream_t stream, uint32_t test_spins) {
    Rows mx, mg, my;
    ScanArgs a{};
    const float *last = nullptr, *states = nullptr;
    int rc;
    if ((rc = check_common(x, gate, offsets, nseq, status, &mx, &mg)) ||
        (rc = check_rows(y, &my, mx.dtype)))
        return rc;
    if (!my.shaped(mx.rows, mx.cols)) return DGC_EINVAL;
    if ((rc = check_state(h0, nseq, mx.cols, &a.h0, &a.ldh0)) ||
        (rc = check_state(h_last, nseq, mx.cols, &last, &a.ldh_last)) ||
        (rc = check_state(saved, (mx.rows + kPiece - 1) / kPiece, mx.cols, &states, &a.lds)))
        return rc;
    if (bad_workspace(ws, ws_bytes, scan_workspace(mx.rows, mx.cols))) return DGC_EINVAL;
    if (mx.cols == 0 || nseq == 0) return DGC_OK;
    a.h_last = const_cast<float*>(last);
    a.saved = const_cast<float*>(states);
    a.x = mx.p;
    a.ldx = mx.ld;
    a.gate = mg.p;
    a.ldg = mg.ld;
    a.y = my.p;
    a.ldy = my.ld;
    a.offsets = offsets;
    a.nseq = (uint32_t)nseq;
    a.rows = (uint32_t)mx.rows;
    a.cols = (uint32_t)mx.cols;
    a.status = status;
    if (test_spins) a.spin_limit = test_spins;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const ScanLayout L = scan_layout(mx.rows, mx.cols, kForwardRows);
    if ((uint64_t)L.tiles * L.chunks > 0x7FFFFFFFull) return DGC_EUNSUPPORTED;
    if ((rc = start_scan(a, L, ws, s))) return rc;
    const bool pair = mx.on(2 * mx.entry()) && mg.on(2 * mx.entry()) && my.on(2 * mx.entry());
    const dim3 grid(L.tiles * L.chunks);
    return with_type(mx.dtype, [&](auto t) {
        using T = decltype(t);
        return launch_rows_kernel(pair ? k_scan<T, true, kForwardRows / kWarps>
                                       : k_scan<T, false, kForwardRows / kWarps>,
                                  grid, kThreads, s, a);
    });
}

}  // namespace
}  // namespace dgc

using namespace dgc;

extern "C" int dgc_recurrence_workspace(int64_t rows, int64_t cols, size_t* bytes) {
    if (!bytes || rows < 0 || cols < 0) return DGC_EINVAL;
    if (rows > kMaxExtent || cols > kMaxExtent) return DGC_EUNSUPPORTED;
    *bytes = scan_workspace((uint64_t)rows, (uint64_t)cols);
    return DGC_OK;
}

extern "C" int dgc_recurrence_saved_rows(int64_t rows, int64_t* saved_rows) {
    if (!saved_rows || rows < 0) return DGC_EINVAL;
    if (rows > kMaxExtent) return DGC_EUNSUPPORTED;
    *saved_rows = (rows + kPiece - 1) / kPiece;
    return DGC_OK;
}

extern "C" int dgc_recurrence(const dgc_matrix* x, const dgc_matrix* gate, const int64_t* offsets,
                              int32_t nseq, const dgc_matrix* h0, const dgc_matrix* y,
                              const dgc_matrix* h_last, const dgc_matrix* saved, int32_t* status,
                              void* ws, size_t ws_bytes, dgc_stream_t stream) {
    return recurrence(x, gate, offsets, nseq, h0, y, h_last, saved, status, ws, ws_bytes, stream,
                      0);
}

extern "C" int dgc_selftest_recurrence_timeout(const dgc_matrix* x, const dgc_matrix* gate,
                                               const int64_t* offsets, int32_t nseq,
                                               const dgc_matrix* y, int32_t* status, void* ws,
                                               size_t ws_bytes, uint32_t spin_limit,
                                               dgc_stream_t stream) {
    if (spin_limit == 0 || spin_limit > kDefaultSpinLimit) return DGC_EINVAL;
    return recurrence(x, gate, offsets, nseq, nullptr, y, nullptr, nullptr, status, ws, ws_bytes,
                      stream, spin_limit);
}

extern "C" int dgc_recurrence_backward(const dgc_matrix* dy, const dgc_matrix* x,
                                       const dgc_matrix* gate, const int64_t* offsets, int32_t nseq,
                                       const dgc_matrix* h0, const dgc_matrix* saved,
                                       const dgc_matrix* d_last, const dgc_matrix* dx,
                                       const dgc_matrix* dgate, const dgc_matrix* d_h0,
                                       int32_t* status, void* ws, size_t ws_bytes,
                                       dgc_stream_t stream) {
    Rows mx, mg, my, md, me;
    ScanArgs a{};
    const float *first = nullptr, *states = nullptr;
    int rc;
    if ((rc = check_common(x, gate, offsets, nseq, status, &mx, &mg)) ||
        (rc = check_rows(dy, &my, mx.dtype)) || (rc = check_rows(dx, &md, mx.dtype)) ||
        (rc = check_rows(dgate, &me, mx.dtype)))
        return rc;
    if (!saved || !my.shaped(mx.rows, mx.cols) || !md.shaped(mx.rows, mx.cols) ||
        !me.shaped(mx.rows, mx.cols))
        return DGC_EINVAL;
    if ((rc = check_state(h0, nseq, mx.cols, &a.h0, &a.ldh0)) ||
        (rc = check_state(saved, (mx.rows + kPiece - 1) / kPiece, mx.cols, &states, &a.lds)) ||
        (rc = check_state(d_last, nseq, mx.cols, &a.d_last, &a.ldd_last)) ||
        (rc = check_state(d_h0, nseq, mx.cols, &first, &a.ldd_h0)))
        return rc;
    if (bad_workspace(ws, ws_bytes, scan_workspace(mx.rows, mx.cols))) return DGC_EINVAL;
    if (mx.cols == 0 || nseq == 0) return DGC_OK;
    a.saved = const_cast<float*>(states);
    a.d_h0 = const_cast<float*>(first);
    a.x = mx.p;
    a.ldx = mx.ld;
    a.gate = mg.p;
    a.ldg = mg.ld;
    a.dy = my.p;
    a.lddy = my.ld;
    a.dx = md.p;
    a.lddx = md.ld;
    a.dgate = me.p;
    a.lddg = me.ld;
    a.offsets = offsets;
    a.nseq = (uint32_t)nseq;
    a.rows = (uint32_t)mx.rows;
    a.cols = (uint32_t)mx.cols;
    a.status = status;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const ScanLayout L = scan_layout(mx.rows, mx.cols, kBackRows);
    if ((uint64_t)L.tiles * L.chunks > 0x7FFFFFFFull) return DGC_EUNSUPPORTED;
    if ((rc = start_scan(a, L, ws, s))) return rc;
    const size_t two = 2 * mx.entry();
    const bool pair = mx.on(two) && mg.on(two) && my.on(two) && md.on(two) && me.on(two);
    const dim3 grid(L.tiles * L.chunks);
    return with_type(mx.dtype, [&](auto t) {
        using T = decltype(t);
        return launch_rows_kernel(pair ? k_scan_back<T, true, kBackRows / kWarps>
                                       : k_scan_back<T, false, kBackRows / kWarps>,
                                  grid, kThreads, s, a);
    });
}
