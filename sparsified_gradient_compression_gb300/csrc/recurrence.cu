// recurrence.cu -- a gated linear recurrence over packed sequences and its backward pass (sm_103a).
//
//   a = 1 / (1 + e^-gate);  h_t = a_t h_{t-1} + (1 - a_t) x_t;  y_t = h_t
//   u_t = a_t G_t;  G_t = dy_t + u_{t+1};  dx_t = G_t (1 - a_t)
//   dgate_t = G_t (h_{t-1} - x_t) a_t (1 - a_t)
//
// Columns are independent; rows are a scan. A step, and any run of steps, is an affine map of the
// state, h -> A h + B, so a run's map is known before the state that enters it. A block takes tiles
// of 64 columns by a chunk of rows, each of its 8 warps kS rows, two columns a lane:
//   1. each warp composes its rows' map; the last warp composes the warps' and publishes the
//      chunk's (A, B);
//   2. 16 or 32 chunks are a group: the warps collect the maps of the chunks ahead of this one in
//      its group, two or four each, and the state that enters the group, which the last chunk of
//      the group ahead publishes. (Which maps are joined, and how, is fixed, so the rounding is
//      too: results are the same bits on every run. A chain from chunk to chunk would cost its
//      latency for each.)
//   3. each warp walks its rows again from the state it enters with, and writes.
// Up to 128 rows are one chunk's: k_scan_few has no more than its block's exchange.
// The data is read once. Blocks stay: the next tile is on its way to shared memory as soon as the
// rows of this one are in registers, while the maps are exchanged and the results written. (One
// block a tile, with its loads at its beginning, took 279 us for 32768 x 2048.) Tiles go by a
// ticket, in order, so a block only waits for tiles that running blocks hold; waits are bounded all
// the same.
// A ticket is taken late: the further ahead, the less tiles are begun in the order in which they
// wait for one another (103 us; half a tile earlier 113, two tiles ahead 132). What lies between a
// tile's arrival and its map counts as much, since others wait for that: where sequences begin and
// end in it, and the state ahead of it, are looked up a tile ahead.
//
// Maps and states are published without flags: the workspace is filled with a bit pattern that no
// result has, and a reader waits until it has gone.
//
// A sequence's first row has no predecessor: its map is h -> B with B = a h0 + (1 - a) x, kept as
// A = kReset, so that nothing of what is ahead, infinities and NaNs among it, comes through.
//
// The backward pass is the same scan from the end (u_{t+1} -> u_t = a_t u_{t+1} + a_t dy_t). It
// needs h_{t-1}, which it walks again from the state ahead of each piece of 64 rows that the forward
// pass left.
#include <algorithm>

#include "rows.cuh"

namespace dgc {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCols = 64;        // of a tile
constexpr uint32_t kPiece = 64;  // rows between two saved states
constexpr uint32_t kFew = 128;   // rows of a call that one block a column tile does
constexpr float kReset = -1.0f;  // no run of steps has a negative A
constexpr uint32_t kNotYet = 0xFFFFFFFFu;  // a NaN that no arithmetic makes

struct ScanArgs {
    const void *x, *gate, *dy;
    void *y, *dx, *dgate;
    uint64_t ldx, ldg, lddy, ldy, lddx, lddg;
    const float *h0, *d_last;
    float *h_last, *d_h0, *saved;
    uint64_t ldh0, ldd_last, ldh_last, ldd_h0, lds;
    const int64_t* offsets;
    uint32_t nseq, rows, cols, tiles, tiles_inverse, chunks;
    // the workspace: a ticket, whether a wait gave up, the chunks' maps {A, A, B, B} and the groups'
    // entering states of a lane's two columns. ticket null: one chunk, nothing is shared.
    uint32_t *ticket, *abort;
    uint4* maps;
    uint2* states;
    uint32_t spin_limit, lost;  // lost: self-test, a chunk that publishes nothing
    int32_t* status;
};

// Two columns of a row: kPair whole, where the address allows it and both are there.
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

// a = 1 / (1 + e^-g) and 1 - a = e^-g / (1 + e^-g), neither by a subtraction; each is off by some
// 4 * 2^-24 of itself. The hardware's 2^p takes p = -g / ln 2 rounded; what that lost, r, is put back
// as e (1 + r). Gates are taken to [-86, 104]: 2^124 has a normal reciprocal, and 1 - a is 0 from
// 87.4 on. A shut gate thus lets 2^-124 of the state through; to make that nothing by a comparison for
// each gate took 105.2 us for 102.7 (32768 x 2048). A NaN stays one.
__device__ __forceinline__ void sigmoids(float2 g, float2& a, float2& keep) {
    float2 v, e;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(v.x) : "f"(-g.x), "f"(-104.0f));
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(v.y) : "f"(-g.y), "f"(-104.0f));
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(v.x) : "f"(v.x), "f"(86.0f));
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(v.y) : "f"(v.y), "f"(86.0f));
    const float2 p = mul2(v, both(1.44269504f));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(p.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(p.y));
    e = fma2(e, fma2(p, both(-0.69314718f), v), e);
    const float2 d = add2(both(1.0f), e);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(a.x) : "f"(d.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(a.y) : "f"(d.y));
    keep = mul2(e, a);
}

// h -> A h + B, two columns. A reset is one of both.
struct Map {
    float2 A, B;
    __device__ float2 operator()(float2 h) const {
        const float2 r = fma2(A, h, B);
        const bool reset = A.x < 0.0f;
        return {reset ? B.x : r.x, reset ? B.y : r.y};
    }
    // this one first, then q
    __device__ Map then(const Map& q) const {
        const float2 p = mul2(q.A, A);
        const bool reset = fminf(q.A.x, A.x) < 0.0f;
        return {{reset ? kReset : p.x, reset ? kReset : p.y}, q(B)};
    }
    // the same where neither has a reset
    __device__ Map plain_then(const Map& q) const { return {mul2(q.A, A), fma2(q.A, B, q.B)}; }
    __device__ float4 packed() const { return {A.x, A.y, B.x, B.y}; }
};
__device__ __forceinline__ Map map_of(const float4& v) { return {{v.x, v.y}, {v.z, v.w}}; }
__device__ __forceinline__ Map identity() { return {both(1.0f), both(0.0f)}; }

// An offset of the table as a row. Of a bad table it may be anything: then it is no row.
constexpr uint32_t kNoRow = 0xFFFFFFFFu;
__device__ __forceinline__ uint32_t offset_at(const ScanArgs& a, uint32_t i) {
    const int64_t off = a.offsets[i];
    return off >= 0 && off < (int64_t)kNoRow ? (uint32_t)off : kNoRow;
}
// Every ceil(n / 32)-th of a table of n offsets, one a lane: the first step of a search.
__device__ __forceinline__ uint32_t landmark(const ScanArgs& a) {
    const uint32_t n = a.nseq + 1, step = (n + 31) / 32;
    return offset_at(a, min(((threadIdx.x & 31) + 1) * step, n) - 1);
}
// Where sequences start and end in a warp's kS rows: bits, and the sequences in the arrays (the
// warp's own). mine: the lane's landmark.
template <int kS>
struct Marks {
    static_assert(kS <= 16, "two of 16 bits");
    uint32_t bits;
    __device__ uint32_t start() const { return bits & 0xFFFFu; }
    __device__ uint32_t end() const { return bits >> 16; }
    __device__ bool starts_at(int s) const { return bits >> s & 1; }
    __device__ bool ends_at(int s) const { return bits >> (16 + s) & 1; }
    __device__ Marks(const ScanArgs& a, uint32_t begin, uint32_t mine, int32_t* starts,
                     int32_t* ends) {
        const uint32_t lane = threadIdx.x & 31, n = a.nseq + 1, step = (n + 31) / 32;
        const uint32_t stop = begin + kS;
        bits = 0;
        __syncwarp();  // the arrays' readers of two tiles before
        uint32_t i0 = 0;
        if (step > 1) {
            const uint32_t less = __popc(__ballot_sync(kFull, mine < begin));
            i0 = min(less * step, n);
            if (step > 32) i0 = first_from(a.offsets, i0, min(step, n - i0),
                                            (int64_t)begin);
        }
        for (;;) {
            const uint32_t i = i0 + lane;
            const uint32_t off = i >= n ? kNoRow : step > 1 ? offset_at(a, i) : mine;
            const bool here = i < n && off >= begin && off <= stop;
            if (__any_sync(kFull, here)) {
                uint32_t b = 0;
                if (here) {
                    const uint32_t r = off - begin;
                    if (r < kS && i + 1 < n && offset_at(a, i + 1) > off) {
                        starts[r] = (int32_t)i;
                        b = 1u << r;
                    }
                    if (r > 0 && i > 0 && offset_at(a, i - 1) < off) {
                        ends[r - 1] = (int32_t)i - 1;
                        b |= 0x10000u << (r - 1);
                    }
                }
                bits |= __reduce_or_sync(kFull, b);
            }
            if (step == 1 || !__all_sync(kFull, off <= stop)) break;
            i0 += 32;
            // Sequences without rows share an offset: after 32 of them the others are passed by a
            // search, up to the last one. Other blocks wait for what comes behind this. (32 at a time,
            // a step for 100 of 4096 slots of 1024 columns, the others idle behind them, took 72 us
            // for 15, for 100 of 2^20 slots 25 ms.)
            const uint32_t top = __shfl_sync(kFull, off, 31);
            if (__all_sync(kFull, off == top))
                i0 = max(i0, first_from(a.offsets, i0, n - i0, (int64_t)top + 1) - 1);
        }
        __syncwarp();
    }
};

// What has no row: sequences of length 0 pass their state on; and the table's check. A tile's columns
// by `parts` blocks, of which this is one.
__device__ __forceinline__ void empty_sequences(const ScanArgs& a, uint32_t tile, uint32_t part,
                                                uint32_t parts, const float* from, uint64_t ld_from,
                                                float* to, uint64_t ld_to) {
    const int lane = threadIdx.x & 31;
    const uint32_t col = tile * kCols + 2 * lane, n = col < a.cols ? min(2u, a.cols - col) : 0;
    bool bad = false;
    for (uint32_t q0 = part * kThreads + (threadIdx.x & ~31u); q0 < a.nseq;
         q0 += parts * kThreads) {
        const uint32_t q = q0 + lane;
        const int64_t b = q < a.nseq ? a.offsets[q] : 0, e = q < a.nseq ? a.offsets[q + 1] : 1;
        bad |= q < a.nseq && (b > e || b < 0 || e > (int64_t)a.rows);
        uint32_t todo = to && to != from ? __ballot_sync(kFull, b == e) : 0;
        while (todo) {  // four at once, so that no store waits for one load alone
            uint32_t s[4];
            float2 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i, todo &= todo - 1) {
                s[i] = todo ? q0 + __ffs(todo) - 1 : a.nseq;
                v[i] = from && s[i] < a.nseq ? load_state(from, ld_from, s[i], col, n)
                                             : both(0.0f);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (s[i] < a.nseq) store_state(to, ld_to, s[i], col, n, v[i]);
        }
    }
    if (tile == 0 && bad) report(a.status, DGC_EINVAL);
}
// The same by all blocks, at their end: no block waits for it.
__device__ __forceinline__ void all_empty_sequences(const ScanArgs& a, const float* from,
                                                    uint64_t ld_from, float* to, uint64_t ld_to) {
    const uint32_t parts = max(1u, gridDim.x / a.tiles), part = blockIdx.x / a.tiles;
    if (part < parts)
        for (uint32_t tile = blockIdx.x % a.tiles; tile < a.tiles; tile += gridDim.x)
            empty_sequences(a, tile, part, parts, from, ld_from, to, ld_to);
}

// A tile: its chunk's place in the scan's direction, and its columns. order of chunks on: none.
struct Tile {
    uint32_t order, tile;
};
__device__ __forceinline__ Tile tile_of(const ScanArgs& a, uint32_t ticket) {
    // ticket / tiles, by the reciprocal rounded down: at most one short
    uint32_t order = __umulhi(ticket, a.tiles_inverse);
    if (ticket - order * a.tiles >= a.tiles) ++order;
    return {order, ticket - order * a.tiles};
}
__device__ __forceinline__ Tile first_tile(const ScanArgs& a, uint32_t* slot) {
    if (!a.ticket) return {blockIdx.x < a.tiles ? 0 : ~0u, blockIdx.x};
    if (threadIdx.x == 0) *slot = atomicAdd(a.ticket, 1u);
    __syncthreads();
    const Tile t = tile_of(a, *slot);
    __syncthreads();
    return t;
}

// What a warp has of a tile: its rows, how many of them there are, and its lane's columns.
struct Spot {
    uint32_t first, left, col, lane_col, n;
    __device__ Spot(const ScanArgs& a, uint32_t chunk, uint32_t tile, uint32_t rows, uint32_t s) {
        first = chunk * rows + (threadIdx.x >> 5) * s;
        left = first < a.rows ? a.rows - first : 0;
        col = tile * kCols;
        lane_col = col + 2 * (threadIdx.x & 31);
        n = lane_col < a.cols ? min(2u, a.cols - lane_col) : 0;
    }
};

// The states at the borders (bits) in a warp's rows, `which` the sequences. One is loaded ahead of the
// rows' arithmetic, more all at once behind it.
template <int kS>
struct Given {
    const float* m;
    uint64_t ld;
    const int32_t* which;
    uint32_t bits, col, n;
    float2 one;
    __device__ Given(const float* m, uint64_t ld, const int32_t* which, uint32_t bits,
                     const Spot& at)
        : m(m), ld(ld), which(which), bits(m ? bits : 0), col(at.lane_col), n(at.n) {
        one = both(0.0f);
        if (this->bits) one = load_state(m, ld, which[__ffs(this->bits) - 1], col, n);
    }
    // f(s, state) for each
    template <typename F>
    __device__ void each(F f) const {
        if (!bits) return;
        if ((bits & (bits - 1)) == 0) {
#pragma unroll
            for (int s = 0; s < kS; ++s)
                if (bits >> s & 1) f(s, one);
            return;
        }
        float2 v[kS];
#pragma unroll
        for (int s = 0; s < kS; ++s) {
            const bool here = bits >> s & 1;
            v[s] = load_state(m, ld, here ? which[s] : 0, col, here ? n : 0);
        }
#pragma unroll
        for (int s = 0; s < kS; ++s)
            if (bits >> s & 1) f(s, v[s]);
    }
};

// What the warps of a block tell one another about a tile. A tile has two barriers: what is written
// ahead of the first one is read between the two, what is written between them is read behind the
// second one and ahead of the next tile's first.
struct Board {
    float4 map[kWarps][32];    // the warps' maps, in the scan's direction
    float4 ahead[kWarps][32];  // the chunks' ahead of this one, each to an entry
    float2 state[32];          // that enters the group
    uint32_t next;             // ticket
    uint32_t fresh;            // a sequence begins with the chunk: nothing enters
};

__device__ __forceinline__ uint32_t not_kept(float f) {  // the bits, never kNotYet
    const uint32_t b = __float_as_uint(f);
    return b == kNotYet ? 0x7FFFFFFFu : b;
}
__device__ __forceinline__ void publish(uint4* p, const Map& m) {
    asm volatile("st.relaxed.gpu.global.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(p),
                 "r"(not_kept(m.A.x)), "r"(not_kept(m.A.y)), "r"(not_kept(m.B.x)),
                 "r"(not_kept(m.B.y))
                 : "memory");
}
__device__ __forceinline__ void publish(uint2* p, float2 h) {
    asm volatile("st.relaxed.gpu.global.v2.u32 [%0], {%1, %2};" ::"l"(p), "r"(not_kept(h.x)),
                 "r"(not_kept(h.y))
                 : "memory");
}
__device__ __forceinline__ uint4 look(const uint4* p) {
    uint4 v;
    asm volatile("ld.relaxed.gpu.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}
__device__ __forceinline__ uint2 look(const uint2* p) {
    uint2 v;
    asm volatile("ld.relaxed.gpu.global.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p)
                 : "memory");
    return v;
}
__device__ __forceinline__ bool there(const uint4& v) {
    return v.x != kNotYet && v.y != kNotYet && v.z != kNotYet && v.w != kNotYet;
}
__device__ __forceinline__ bool there(const uint2& v) { return v.x != kNotYet && v.y != kNotYet; }

// Whether a wait goes on, after so many polls. When one gives up, the others do too.
__device__ __forceinline__ bool wait_on(const ScanArgs& a, uint32_t polls) {
    if (polls <= a.spin_limit && ((polls & 63) != 63 || ld_relaxed_u32(a.abort) == 0)) return true;
    if ((threadIdx.x & 31) == 0) {
        report(a.status, DGC_ETIMEOUT);
        atomicExch(a.abort, 1u);
    }
    return false;
}

// Step 1's end, by all warps: `w` is the warp's place in the scan's direction, m its map (on the
// board), `order` the chunk's place, resets: whether a sequence begins in it. Returns the map of the
// warps ahead of this one; the last one publishes the chunk's.
__device__ __forceinline__ Map compose(const ScanArgs& a, const Board& b, uint32_t order,
                                       uint32_t tile, int w, const Map& m, bool resets) {
    const uint32_t lane = threadIdx.x & 31;
    Map before = identity();
    if (resets) {
#pragma unroll
        for (int i = 0; i < kWarps - 1; ++i)
            if (i < w) before = before.then(map_of(b.map[i][lane]));
    } else
#pragma unroll
        for (int i = 0; i < kWarps - 1; ++i)
            if (i < w) before = before.plain_then(map_of(b.map[i][lane]));
    if (a.ticket && w == kWarps - 1 && order != a.lost)
        publish(&a.maps[((uint64_t)order * a.tiles + tile) * 32 + lane], before.then(m));
    return before;
}

// Step 2: a warp collects the maps of kEach chunks, the last one also the state that enters the
// group (it has the fewest chunks to wait for). The first look is taken ahead of the next tile's
// copies, or it would queue behind them (2500 clocks for 900).
template <uint32_t kEach>
struct LookBack {
    const uint4* maps;
    const uint2* state;
    uint64_t step;
    uint32_t count;
    uint4 v[kEach];
    uint2 h;
    __device__ LookBack(const ScanArgs& a, uint32_t order, uint32_t tile, int w, bool fresh) {
        const uint32_t lane = threadIdx.x & 31;
        const uint32_t group = order / (kEach * kWarps), k = order % (kEach * kWarps);
        const uint32_t from = kEach * (uint32_t)w;
        count = 0;
        state = nullptr;
        h = make_uint2(0, 0);
        if (!a.ticket || fresh) return;
        if (k > from) count = min(kEach, k - from);
        step = (uint64_t)a.tiles * 32;
        maps = a.maps + ((uint64_t)order - k + from) * step + tile * 32 + lane;
        if (w == kWarps - 1 && group > 0) state = a.states + group * step + tile * 32 + lane;
        look_again();
    }
    __device__ void look_again() {
#pragma unroll
        for (uint32_t i = 0; i < kEach; ++i)
            if (i < count) v[i] = look(maps + i * step);
        if (state) h = look(state);
    }
    // A barrier has to follow.
    __device__ void finish(const ScanArgs& a, Board& b, int w) {
        const uint32_t lane = threadIdx.x & 31;
        for (uint32_t polls = 0;; ++polls) {
            bool ready = !state || there(h);
#pragma unroll
            for (uint32_t i = 0; i < kEach; ++i)
                if (i < count) ready = ready && there(v[i]);
            if (__all_sync(kFull, ready) || !wait_on(a, polls)) break;
            look_again();
        }
        Map all = identity();
#pragma unroll
        for (uint32_t i = 0; i < kEach; ++i)
            if (i < count)
                all = all.then({{__uint_as_float(v[i].x), __uint_as_float(v[i].y)},
                                {__uint_as_float(v[i].z), __uint_as_float(v[i].w)}});
        b.ahead[w][lane] = all.packed();  // without any: the identity
        if (w == kWarps - 1)
            b.state[lane] = {__uint_as_float(h.x), __uint_as_float(h.y)};
    }
};

// After the barrier: the state that enters the chunk. The last warp passes a group's on.
template <uint32_t kEach>
__device__ __forceinline__ float2 enter(const ScanArgs& a, const Board& b, uint32_t order,
                                        uint32_t tile, int w, const Map& before, const Map& m,
                                        bool fresh) {
    const uint32_t lane = threadIdx.x & 31;
    const uint32_t group = order / (kEach * kWarps), k = order % (kEach * kWarps);
    float2 h = {0.0f, 0.0f};
    if (!a.ticket) return h;
    if (!fresh) {
        h = b.state[lane];
#pragma unroll
        for (uint32_t i = 0; i < kWarps; ++i)
            if (kEach * i < k) h = map_of(b.ahead[i][lane])(h);
    }
    if (w == kWarps - 1 && k == kEach * kWarps - 1 && order + 1 < a.chunks && order != a.lost)
        publish(&a.states[((uint64_t)(group + 1) * a.tiles + tile) * 32 + lane], m(before(h)));
    return h;
}

__global__ void __launch_bounds__(256)
    k_scan_clear(uint32_t* control, uint4* words, uint64_t n) {
    grid_dep_wait();
    grid_dep_launch();
    if (blockIdx.x == 0 && threadIdx.x < 2) control[threadIdx.x] = 0;
    for (uint64_t i = (uint64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (uint64_t)gridDim.x * 256)
        words[i] = make_uint4(kNotYet, kNotYet, kNotYet, kNotYet);
}

// The operands' tiles in shared memory, each warp's rows for itself, by copies of kUnit bytes: 16
// where every operand's rows allow it, two entries, or (0) by loads and stores of single ones.
template <typename T, int kUnit, int kS, int kOperands>
struct Landing {
    using Word = std::conditional_t<sizeof(T) == 4, uint2, uint32_t>;  // a lane's two columns
    static constexpr uint32_t kRow = kCols * sizeof(T);
    static constexpr uint32_t kBytes = kOperands * kWarps * kS * kRow;
    Word* words;
    __device__ explicit Landing(void* ring) : words(static_cast<Word*>(ring)) {}
    __device__ Word* rows(int q) const {
        return words + (q * kWarps + (threadIdx.x >> 5)) * kS * 32;
    }
    // rows `first` to first + kS - 1 of m, of which `left` are there, columns from col on
    __device__ void fetch(int q, const void* m, uint64_t ld, uint64_t first, uint32_t left,
                          uint32_t col, uint32_t cols) const {
        const uint32_t lane = threadIdx.x & 31;
        const T* p = static_cast<const T*>(m) + first * ld + col;
        Word* to = rows(q);
        if constexpr (kUnit == 16) {
            constexpr uint32_t kLanes = kRow / 16, kStep = 32 / kLanes;  // of a row; rows a turn
            const uint32_t r = lane / kLanes, c = lane % kLanes * (16 / sizeof(T));
            const T* src = p + r * ld + c;
            uint4* dst = reinterpret_cast<uint4*>(to) + lane;
            const uint32_t n = cols - col > c ? min(cols - col - c, 16u / (uint32_t)sizeof(T)) : 0;
            if (left >= kS && cols - col >= kCols) {
#pragma unroll
                for (int i = 0; i < kS / (int)kStep; ++i, src += kStep * ld)
                    copy_async<16>(dst + i * 32, src, 16);
            } else {
#pragma unroll
                for (int i = 0; i < kS / (int)kStep; ++i, src += kStep * ld) {
                    const uint32_t here = r + i * kStep < left ? n : 0;
                    copy_async<16>(dst + i * 32, here ? src : m, here * sizeof(T));
                }
            }
        } else {
            p += 2 * lane;
            to += lane;
            const uint32_t n = cols - col > 2 * lane ? min(cols - col - 2 * lane, 2u) : 0;
            if constexpr (kUnit != 0) {
#pragma unroll
                for (int s = 0; s < kS; ++s) {
                    const uint32_t here = s < left ? n : 0;
                    copy_async<sizeof(Word)>(to + s * 32, here ? p + s * ld : m, here * sizeof(T));
                }
            } else {
                Packed<T, 2> v[kS];
#pragma unroll
                for (int s = 0; s < kS; ++s) v[s] = load_some<T, 2>(p + s * ld, s < left ? n : 0);
#pragma unroll
                for (int s = 0; s < kS; ++s) to[s * 32] = *reinterpret_cast<Word*>(v[s].w);
            }
        }
    }
    __device__ float2 get(int q, int s) const {
        Packed<T, 2> p;
        *reinterpret_cast<Word*>(p.w) = rows(q)[s * 32 + (threadIdx.x & 31)];
        return pair_of<T, 2>(p, 0);
    }
};

// --------------------------------------------------------------------------------- forward
// x and gate read once, y written once. 32768 x 2048 bf16: 103 us, 3.9 TB/s; binary32 178 us,
// 4.5 TB/s. Not bound by HBM but by
// a tile's steps one behind the other, by two blocks of 8 warps an SM (the rows in registers leave
// room for no more). Timing copies that left steps out: waits for maps 89 us, all of the look-back
// 84, the sigmoids too 76, the stores too 65. Less registers by computing the sigmoids twice 114; a
// tile's map published ahead of the wait of the one before it, both tiles' rows in registers, 139.
// Rows with a border among them take a way of their own; 16001 x 2048 fp16 takes 56 us for 1
// sequence, 57 for 37 and 62 for 200.
template <typename T, int kUnit, int kS, int kBlocks, uint32_t kEach>
__global__ void __launch_bounds__(kThreads, kBlocks) k_scan(const __grid_constant__ ScanArgs a) {
    constexpr int kRows = kWarps * kS;
    constexpr bool kPair = kUnit != 0;
    extern __shared__ uint4 ring[];
    __shared__ Board board;
    __shared__ int32_t starts_of[2][kWarps][kS], ends_of[2][kWarps][kS];
    const Landing<T, kUnit, kS, 2> land(ring);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_dep_wait();
    grid_dep_launch();
    Tile t = first_tile(a, &board.next);
    auto fetch = [&] {
        if (t.order < a.chunks) {
            const Spot at(a, t.order, t.tile, kRows, kS);
            land.fetch(0, a.gate, a.ldg, at.first, at.left, at.col, a.cols);
            land.fetch(1, a.x, a.ldx, at.first, at.left, at.col, a.cols);
        }
        copy_commit();
    };
    fetch();
    const uint32_t valid0 = offset_at(a, 0), valid1 = min(a.rows, offset_at(a, a.nseq));
    const uint32_t mine = landmark(a);
    uint32_t turn = 0;
    auto look_marks = [&](uint32_t order) {
        const Spot at(a, order, t.tile, kRows, kS);
        return Marks<kS>(a, at.first, mine, starts_of[turn & 1][warp], ends_of[turn & 1][warp]);
    };
    // (a block without a tile has come for the sequences without rows)
    Marks<kS> marks_next = look_marks(min(t.order, a.chunks - 1));
    while (t.order < a.chunks) {
        const uint32_t chunk = t.order, tile = t.tile;
        const Spot at(a, chunk, tile, kRows, kS);
        const Marks<kS> marks = marks_next;
        const uint32_t slot = turn++ & 1;
        copy_wait<0>();
        __syncwarp();
        // the next ticket; not ahead of the wait, which would wait for it too
        uint32_t more = 0xFFFFFFFFu;
        if (a.ticket && threadIdx.x == 0) more = atomicAdd(a.ticket, 1u);
        const Given<kS> given(a.h0, a.ldh0, starts_of[slot][warp], marks.start(), at);
        // rows as h -> A h + B
        float2 A[kS], B[kS];
#pragma unroll
        for (int s = 0; s < kS; ++s) {
            float2 keep;
            sigmoids(land.get(0, s), A[s], keep);
            B[s] = mul2(keep, land.get(1, s));
        }
        Map m = identity();
        if (marks.start()) {
            given.each([&](int s, float2 h) { B[s] = fma2(A[s], h, B[s]); });
#pragma unroll
            for (int s = 0; s < kS; ++s)
                if (marks.starts_at(s)) m.B = B[s];
                else m.B = fma2(A[s], m.B, B[s]);
            m.A = both(kReset);
        } else {
#pragma unroll
            for (int s = 0; s < kS; ++s) m = m.plain_then({A[s], B[s]});
        }
        board.map[warp][lane] = m.packed();
        if (threadIdx.x == 0) {
            board.fresh = marks.starts_at(0);
            board.next = more;
        }
        const bool resets = __syncthreads_or(marks.start() != 0);
        const Map before = compose(a, board, chunk, tile, warp, m, resets);
        const bool fresh = board.fresh;
        LookBack<kEach> back(a, chunk, tile, warp, fresh);
        t = tile_of(a, board.next);
        fetch();
        if (t.order < a.chunks) marks_next = look_marks(t.order);
        back.finish(a, board, warp);
        __syncthreads();
        float2 h = before(enter<kEach>(a, board, chunk, tile, warp, before, m, fresh));
        if (a.saved && at.first % kPiece == 0 && at.left)
            store_state(a.saved, a.lds, at.first / kPiece, at.lane_col, at.n, h);
        const bool whole = kPair && at.first >= valid0 && at.first + kS <= valid1 &&
                           at.col + kCols <= a.cols;
        T* y = static_cast<T*>(a.y) + at.first * a.ldy + at.lane_col;
        auto put = [&] {
            Packed<T, 2> p;
            set_pair<T, 2>(p, 0, h);
            store_packed<T, 2>(y, p);
            y += a.ldy;
        };
        if (whole && !marks.bits) {
#pragma unroll
            for (int s = 0; s < kS; ++s) {
                h = fma2(A[s], h, B[s]);
                put();
            }
        } else if (whole) {
#pragma unroll
            for (int s = 0; s < kS; ++s) {
                if (marks.starts_at(s)) h = B[s];
                else h = fma2(A[s], h, B[s]);
                put();
                if (marks.ends_at(s) && a.h_last)
                    store_state(a.h_last, a.ldh_last, ends_of[slot][warp][s], at.lane_col, 2, h);
            }
        } else {
#pragma unroll
            for (int s = 0; s < kS; ++s) {
                const uint32_t row = at.first + s;
                h = marks.starts_at(s) ? B[s] : fma2(A[s], h, B[s]);
                if (row >= valid0 && row < valid1)
                    store_two<T, kPair>(a.y, a.ldy, row, at.lane_col, at.n, h);
                if (a.h_last && marks.ends_at(s) && s < at.left)
                    store_state(a.h_last, a.ldh_last, ends_of[slot][warp][s], at.lane_col, at.n,
                                h);
            }
        }
    }
    copy_wait<0>();
    all_empty_sequences(a, a.h0, a.ldh0, a.h_last, a.ldh_last);
}

// Up to kWarps * kS rows: the first block of a column tile. For a step of a model that answers, a start and a
// round trip to memory.
template <typename T, bool kPair, int kS>
__global__ void __launch_bounds__(kThreads) k_scan_few(const __grid_constant__ ScanArgs a) {
    __shared__ float4 maps[kWarps][32];
    __shared__ int32_t starts_of[kWarps][kS], ends_of[kWarps][kS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int32_t *starts = starts_of[warp], *ends = ends_of[warp];
    grid_dep_wait();
    grid_dep_launch();
    if (blockIdx.y) {
        empty_sequences(a, blockIdx.x, blockIdx.y, gridDim.y, a.h0, a.ldh0, a.h_last, a.ldh_last);
        return;
    }
    const Spot at(a, 0, blockIdx.x, kWarps * kS, kS);
    const T* gate = static_cast<const T*>(a.gate) + (uint64_t)at.first * a.ldg + at.lane_col;
    const T* x = static_cast<const T*>(a.x) + (uint64_t)at.first * a.ldx + at.lane_col;
    Packed<T, 2> pg[kS], px[kS];
#pragma unroll
    for (int s = 0; s < kS; ++s) {
        pg[s] = load_piece<kPair, T, 2>(gate + s * a.ldg, s < at.left ? at.n : 0);
        px[s] = load_piece<kPair, T, 2>(x + s * a.ldx, s < at.left ? at.n : 0);
    }
    const uint32_t valid0 = offset_at(a, 0), valid1 = min(a.rows, offset_at(a, a.nseq));
    const uint32_t mine = landmark(a);
    const Marks<kS> marks(a, at.first, mine, starts, ends);
    float2 given[kS];
#pragma unroll
    for (int s = 0; s < kS; ++s) {
        const bool here = a.h0 && marks.starts_at(s);
        given[s] = load_state(a.h0, a.ldh0, here ? starts[s] : 0, at.lane_col, here ? at.n : 0);
    }
    empty_sequences(a, blockIdx.x, 0, gridDim.y, a.h0, a.ldh0, a.h_last, a.ldh_last);
    float2 A[kS], B[kS];
    Map m = identity();
#pragma unroll
    for (int s = 0; s < kS; ++s) {
        float2 keep;
        sigmoids(pair_of<T, 2>(pg[s], 0), A[s], keep);
        B[s] = mul2(keep, pair_of<T, 2>(px[s], 0));
        if (marks.starts_at(s)) {
            B[s] = fma2(A[s], given[s], B[s]);
            m = {both(kReset), B[s]};
        } else {
            m = m.then({A[s], B[s]});
        }
    }
    maps[warp][lane] = m.packed();
    const bool resets = __syncthreads_or(marks.start() != 0);
    float2 h = both(0.0f);
    for (int w = 0; w < warp; ++w) {
        const Map q = map_of(maps[w][lane]);
        h = resets ? q(h) : fma2(q.A, h, q.B);
    }
    if (a.saved && at.first % kPiece == 0 && at.left)
        store_state(a.saved, a.lds, at.first / kPiece, at.lane_col, at.n, h);
#pragma unroll
    for (int s = 0; s < kS; ++s) {
        const uint32_t row = at.first + s;
        h = marks.starts_at(s) ? B[s] : fma2(A[s], h, B[s]);
        if (row >= valid0 && row < valid1)
            store_two<T, kPair>(a.y, a.ldy, row, at.lane_col, at.n, h);
        if (a.h_last && marks.ends_at(s) && s < at.left)
            store_state(a.h_last, a.ldh_last, ends[s], at.lane_col, at.n, h);
    }
}

// -------------------------------------------------------------------------------- backward
// x, gate and dy read once, dx and dgate written once, the states of every 64th row read.
// 16001 x 2048 fp16 in 37 sequences: 103 us, 3.2 TB/s, bound as k_scan is (three walks over the rows).
// Both directions in binary32 223 us for 161. Rows off the boundary of two entries are copied entry by
// entry: 16001 x 2049 bf16 packed, both directions, 511 us.
template <typename T, int kUnit, int kS, int kBlocks, uint32_t kEach>
__global__ void __launch_bounds__(kThreads, kBlocks) k_scan_back(const __grid_constant__ ScanArgs a) {
    constexpr int kRows = kWarps * kS;
    constexpr bool kPair = kUnit != 0;
    static_assert(kRows == kPiece, "a chunk begins at its saved state");
    extern __shared__ uint4 ring[];
    __shared__ Board board;
    __shared__ float4 maps[kWarps][32];  // of h, as the board's are of u
    __shared__ int32_t starts_of[2][kWarps][kS], ends_of[2][kWarps][kS];
    const Landing<T, kUnit, kS, 3> land(ring);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, place = kWarps - 1 - warp;
    grid_dep_wait();
    grid_dep_launch();
    Tile t = first_tile(a, &board.next);
    float2 entering = both(0.0f);
    auto fetch = [&] {
        if (t.order < a.chunks) {
            const Spot at(a, a.chunks - 1 - t.order, t.tile, kRows, kS);
            land.fetch(0, a.gate, a.ldg, at.first, at.left, at.col, a.cols);
            land.fetch(1, a.x, a.ldx, at.first, at.left, at.col, a.cols);
            land.fetch(2, a.dy, a.lddy, at.first, at.left, at.col, a.cols);
            const uint32_t chunk = a.chunks - 1 - t.order;
            if (a.rows) entering = load_state(a.saved, a.lds, chunk, at.lane_col, at.n);
        }
        copy_commit();
    };
    fetch();
    const uint32_t valid0 = offset_at(a, 0), valid1 = min(a.rows, offset_at(a, a.nseq));
    const uint32_t mine = landmark(a);
    uint32_t turn = 0;
    auto look_marks = [&](uint32_t order) {
        const Spot at(a, a.chunks - 1 - order, t.tile, kRows, kS);
        return Marks<kS>(a, at.first, mine, starts_of[turn & 1][warp], ends_of[turn & 1][warp]);
    };
    // (a block without a tile has come for the sequences without rows)
    Marks<kS> marks_next = look_marks(min(t.order, a.chunks - 1));
    while (t.order < a.chunks) {
        const uint32_t order = t.order, tile = t.tile;
        const uint32_t chunk = a.chunks - 1 - order;
        const Spot at(a, chunk, tile, kRows, kS);
        float2 h = entering;
        const Marks<kS> marks = marks_next;
        const uint32_t slot = turn++ & 1;
        copy_wait<0>();
        __syncwarp();
        // the next ticket; not ahead of the wait, which would wait for it too
        uint32_t more = 0xFFFFFFFFu;
        if (a.ticket && threadIdx.x == 0) more = atomicAdd(a.ticket, 1u);
        const Given<kS> first(a.h0, a.ldh0, starts_of[slot][warp], marks.start(), at);
        const Given<kS> last(a.d_last, a.ldd_last, ends_of[slot][warp], marks.end(), at);
        float2 A[kS], keep[kS], q[kS], G[kS];  // q: (1-a) x, then (h_{t-1} - x) a (1 - a)
#pragma unroll
        for (int s = 0; s < kS; ++s) {
            sigmoids(land.get(0, s), A[s], keep[s]);
            q[s] = mul2(keep[s], land.get(1, s));
            G[s] = land.get(2, s);
        }
        last.each([&](int s, float2 g) { G[s] = add2(G[s], g); });
        // the rows' map of h, and from the end that of u
        Map m = identity(), u = identity();
        if (marks.bits) {
            float2 B[kS];
#pragma unroll
            for (int s = 0; s < kS; ++s) B[s] = q[s];
            first.each([&](int s, float2 h) { B[s] = fma2(A[s], h, B[s]); });
#pragma unroll
            for (int s = 0; s < kS; ++s) {
                if (marks.starts_at(s)) m.B = B[s];
                else m.B = fma2(A[s], m.B, B[s]);
                m.A = mul2(A[s], m.A);
            }
            u.A = m.A;
#pragma unroll
            for (int s = kS - 1; s >= 0; --s) {
                if (marks.ends_at(s)) u.B = mul2(A[s], G[s]);
                else u.B = mul2(A[s], add2(G[s], u.B));
            }
            if (marks.start()) m.A = both(kReset);
            if (marks.end()) u.A = both(kReset);
        } else {
#pragma unroll
            for (int s = 0; s < kS; ++s) m = m.plain_then({A[s], q[s]});
#pragma unroll
            for (int s = kS - 1; s >= 0; --s) u.B = mul2(A[s], add2(G[s], u.B));
            u.A = m.A;
        }
        maps[warp][lane] = m.packed();
        board.map[place][lane] = u.packed();
        if (threadIdx.x == kThreads - 1) board.fresh = marks.ends_at(kS - 1);
        if (threadIdx.x == 0) board.next = more;
        const bool resets = __syncthreads_or(marks.bits != 0);
        const Map behind = compose(a, board, order, tile, place, u, resets);
        const bool fresh = board.fresh;
        if (resets) {
#pragma unroll
            for (int w = 0; w < kWarps - 1; ++w)
                if (w < warp) h = map_of(maps[w][lane])(h);
        } else
#pragma unroll
            for (int w = 0; w < kWarps - 1; ++w)
                if (w < warp) {
                    const Map p = map_of(maps[w][lane]);
                    h = fma2(p.A, h, p.B);
                }
#pragma unroll
        for (int s = 0; s < kS; ++s) {
            if (marks.starts_at(s))
                h = a.h0 ? load_state(a.h0, a.ldh0, starts_of[slot][warp][s], at.lane_col, at.n)
                         : both(0.0f);
            const float2 x = land.get(1, s), b = q[s];
            q[s] = mul2(mul2(A[s], keep[s]), add2(h, {-x.x, -x.y}));
            h = fma2(A[s], h, b);
        }
        LookBack<kEach> back(a, order, tile, place, fresh);
        __syncwarp();
        t = tile_of(a, board.next);
        fetch();
        if (t.order < a.chunks) marks_next = look_marks(t.order);
        back.finish(a, board, place);
        __syncthreads();
        // u of the row behind
        float2 v = behind(enter<kEach>(a, board, order, tile, place, behind, u, fresh));
        const bool whole = kPair && at.first >= valid0 && at.first + kS <= valid1 &&
                           at.col + kCols <= a.cols;
        T* dx = static_cast<T*>(a.dx) + (at.first + kS - 1) * a.lddx + at.lane_col;
        T* dgate = static_cast<T*>(a.dgate) + (at.first + kS - 1) * a.lddg + at.lane_col;
        auto put = [&](int s) {
            const float2 g = add2(G[s], v);
            Packed<T, 2> p, r;
            set_pair<T, 2>(p, 0, mul2(g, keep[s]));
            set_pair<T, 2>(r, 0, mul2(g, q[s]));
            store_packed<T, 2>(dx, p);
            store_packed<T, 2>(dgate, r);
            v = mul2(A[s], g);
            dx -= a.lddx;
            dgate -= a.lddg;
        };
        if (whole && !marks.bits) {
#pragma unroll
            for (int s = kS - 1; s >= 0; --s) put(s);
        } else if (whole) {
#pragma unroll
            for (int s = kS - 1; s >= 0; --s) {
                if (marks.ends_at(s)) v = both(0.0f);
                put(s);
                if (marks.starts_at(s) && a.d_h0)
                    store_state(a.d_h0, a.ldd_h0, starts_of[slot][warp][s], at.lane_col, 2, v);
            }
        } else {
#pragma unroll
            for (int s = kS - 1; s >= 0; --s) {
                const uint32_t row = at.first + s;
                if (marks.ends_at(s)) v = both(0.0f);
                const float2 g = add2(G[s], v);
                if (row >= valid0 && row < valid1) {
                    store_two<T, kPair>(a.dx, a.lddx, row, at.lane_col, at.n, mul2(g, keep[s]));
                    store_two<T, kPair>(a.dgate, a.lddg, row, at.lane_col, at.n, mul2(g, q[s]));
                }
                v = mul2(A[s], g);
                if (a.d_h0 && marks.starts_at(s) && s < at.left)
                    store_state(a.d_h0, a.ldd_h0, starts_of[slot][warp][s], at.lane_col, at.n,
                                v);
            }
        }
    }
    copy_wait<0>();
    all_empty_sequences(a, a.d_last, a.ldd_last, a.d_h0, a.ldd_h0);
}

// ----------------------------------------------------------------------------------- host
// Rows of a warp, and blocks of an SM.
template <typename T>
struct Form {
    static constexpr int kS = sizeof(T) == 2 ? 16 : 8, kBlocks = 2;
    static constexpr int kBackS = kPiece / kWarps, kBackBlocks = 2;
};

// Columns from which on 16 chunks are a group (32768 x 2048: 5 us less), with two maps for a
// warp to collect. Below, where a tile of columns has most of the blocks to itself, 32: there the
// chain of groups counts more (16384 x 64: 10 us for 12).
constexpr uint64_t kWideCols = 8 * kCols;

struct ScanLayout {
    size_t maps, states, total;
    uint32_t chunks, groups, tiles;
};
ScanLayout scan_layout(uint64_t rows, uint64_t cols, uint32_t chunk_rows, uint32_t each) {
    ScanLayout L{};
    L.chunks = (uint32_t)std::max<uint64_t>(1, (rows + chunk_rows - 1) / chunk_rows);
    L.tiles = (uint32_t)((cols + kCols - 1) / kCols);
    L.groups = (L.chunks + each * kWarps - 1) / (each * kWarps);
    if (L.chunks == 1) return L;
    L.maps = 256;
    L.states = L.maps + (size_t)L.chunks * L.tiles * 32 * sizeof(uint4);
    L.total = (L.states + (size_t)L.groups * L.tiles * 32 * sizeof(uint2) + 255) & ~(size_t)255;
    return L;
}
// For the shortest chunks and groups that the calls use.
size_t scan_workspace(uint64_t rows, uint64_t cols) {
    return scan_layout(rows, cols, kPiece, 2).total;
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

// By how many blocks a column tile's sequences without rows are looked through.
uint64_t empty_parts(uint64_t nseq) { return umin64(64, (nseq + kThreads - 1) / kThreads); }

template <typename T, int kUnit, int kS, int kOperands, int kBlocks, uint32_t kEach>
int launch_scan(void (*kernel)(ScanArgs), ScanArgs a, void* ws, int sms, cudaStream_t s) {
    const ScanLayout L = scan_layout(a.rows, a.cols, kWarps * kS, kEach);
    if ((uint64_t)L.tiles * L.chunks > 0x7FFFFFFFull) return DGC_EUNSUPPORTED;
    a.tiles = L.tiles;
    a.tiles_inverse = (uint32_t)(0xFFFFFFFFull / L.tiles);
    a.chunks = L.chunks;
    if (!a.spin_limit) {
        a.spin_limit = kDefaultSpinLimit;
        a.lost = ~0u;
    }
    uint32_t blocks = L.tiles;
    if (L.chunks > 1) {
        char* w = static_cast<char*>(ws);
        a.ticket = reinterpret_cast<uint32_t*>(w);
        a.abort = a.ticket + 1;
        a.maps = reinterpret_cast<uint4*>(w + L.maps);
        a.states = reinterpret_cast<uint2*>(w + L.states);
        const uint64_t words = (L.total - L.maps) / sizeof(uint4);
        const int rc = launch_rows_kernel(k_scan_clear,
                                          dim3((unsigned)umin64((words + 1023) / 1024, 1024)), 256,
                                          s, a.ticket, a.maps, words);
        if (rc) return rc;
        blocks = (uint32_t)umin64((uint64_t)L.tiles * L.chunks, (uint64_t)sms * kBlocks);
    }
    // Few rows of many sequences: more blocks than tiles, for the states of those without rows (100 rows
    // and 2^20 of them, 16 columns, backward: 0.5 ms for 13).
    blocks = std::max(blocks,
                      (uint32_t)umin64(L.tiles * empty_parts(a.nseq), (uint64_t)sms * kBlocks));
    return launch_shared_kernel(kernel, dim3(blocks), kThreads,
                                Landing<T, kUnit, kS, kOperands>::kBytes, s, a);
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
    const int sms = dgc_internal_sm_count();
    if (sms <= 0) return DGC_ECUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const size_t two = 2 * mx.entry();
    const bool pair = mx.on(two) && mg.on(two) && my.on(two);
    const bool wide = pair && mx.on(16) && mg.on(16);
    return with_type(mx.dtype, [&](auto t) {
        using T = decltype(t);
        constexpr int kS = Form<T>::kS, kBlocks = Form<T>::kBlocks, kTwo = 2 * sizeof(T);
        if (mx.rows <= kFew) {
            auto few = a.rows <= kFew / 2
                           ? (pair ? k_scan_few<T, true, 8> : k_scan_few<T, false, 8>)
                           : (pair ? k_scan_few<T, true, 16> : k_scan_few<T, false, 16>);
            // blocks of their own for sequences without rows, where there are many: as the slots of
            // a model that answers
            return launch_rows_kernel(few,
                                      dim3((unsigned)((mx.cols + kCols - 1) / kCols),
                                           (unsigned)empty_parts(a.nseq)),
                                      kThreads, s, a);
        }
        // (rows off 16-byte boundaries: groups of 32 chunks, for one kernel less)
        if (wide && mx.cols >= kWideCols)
            return launch_scan<T, 16, kS, 2, kBlocks, 2>(
                k_scan<T, 16, kS, kBlocks, 2>, a, ws, sms, s);
        if (wide)
            return launch_scan<T, 16, kS, 2, kBlocks, 4>(
                k_scan<T, 16, kS, kBlocks, 4>, a, ws, sms, s);
        if (pair)
            return launch_scan<T, kTwo, kS, 2, kBlocks, 4>(
                k_scan<T, kTwo, kS, kBlocks, 4>, a, ws, sms, s);
        return launch_scan<T, 0, kS, 2, kBlocks, 4>(
            k_scan<T, 0, kS, kBlocks, 4>, a, ws, sms, s);
    });
}

int recurrence_backward(const dgc_matrix* dy, const dgc_matrix* x, const dgc_matrix* gate,
                        const int64_t* offsets, int32_t nseq, const dgc_matrix* h0,
                        const dgc_matrix* saved, const dgc_matrix* d_last, const dgc_matrix* dx,
                        const dgc_matrix* dgate, const dgc_matrix* d_h0, int32_t* status, void* ws,
                        size_t ws_bytes, dgc_stream_t stream, uint32_t test_spins) {
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
    if (test_spins) a.spin_limit = test_spins;
    const int sms = dgc_internal_sm_count();
    if (sms <= 0) return DGC_ECUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const size_t two = 2 * mx.entry();
    const bool pair = mx.on(two) && mg.on(two) && my.on(two) && md.on(two) && me.on(two);
    const bool wide = pair && mx.on(16) && mg.on(16) && my.on(16);
    return with_type(mx.dtype, [&](auto t) {
        using T = decltype(t);
        constexpr int kS = Form<T>::kBackS, kBlocks = Form<T>::kBackBlocks, kTwo = 2 * sizeof(T);
        // (rows off 16-byte boundaries: groups of 32 chunks, for one kernel less)
        if (wide && mx.cols >= kWideCols)
            return launch_scan<T, 16, kS, 3, kBlocks, 2>(
                k_scan_back<T, 16, kS, kBlocks, 2>, a, ws, sms, s);
        if (wide)
            return launch_scan<T, 16, kS, 3, kBlocks, 4>(
                k_scan_back<T, 16, kS, kBlocks, 4>, a, ws, sms, s);
        if (pair)
            return launch_scan<T, kTwo, kS, 3, kBlocks, 4>(
                k_scan_back<T, kTwo, kS, kBlocks, 4>, a, ws, sms, s);
        return launch_scan<T, 0, kS, 3, kBlocks, 4>(
            k_scan_back<T, 0, kS, kBlocks, 4>, a, ws, sms, s);
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
    return recurrence_backward(dy, x, gate, offsets, nseq, h0, saved, d_last, dx, dgate, d_h0,
                               status, ws, ws_bytes, stream, 0);
}

extern "C" int dgc_selftest_recurrence_backward_timeout(
    const dgc_matrix* dy, const dgc_matrix* x, const dgc_matrix* gate, const int64_t* offsets,
    int32_t nseq, const dgc_matrix* saved, const dgc_matrix* dx, const dgc_matrix* dgate,
    int32_t* status, void* ws, size_t ws_bytes, uint32_t spin_limit, dgc_stream_t stream) {
    if (spin_limit == 0 || spin_limit > kDefaultSpinLimit) return DGC_EINVAL;
    return recurrence_backward(dy, x, gate, offsets, nseq, nullptr, saved, nullptr, dx, dgate,
                               nullptr, status, ws, ws_bytes, stream, spin_limit);
}
