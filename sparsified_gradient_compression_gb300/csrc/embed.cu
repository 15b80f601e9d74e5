// embed.cu -- embedding lookup with scaling, and its gradient by sorted tokens (sm_103a).
//
//   out[t] = scale table[token[t]]
//   dtable[w] = scale sum of dy[t] over the t with token[t] = w, in the order of t; or added
//
//   k_embed        the lookup.
//   k_sort         a stable radix sort of (token, position), lowest digit first, digits of up to 9
//                  bits, by one cluster: up to 32768 tokens.
//   k_sort_count   for more: how often a block's tokens have each value of a digit;
//   k_sort_move    puts them in the digit's order, equal ones in theirs.
//   k_embed_sum    a warp sums the rows of 8 or 32 sorted tokens over some columns, and writes each
//                  word's sum once; other blocks zero the rows of words that are not met.
//   k_embed_join   joins the sums of words that are met more often than that, in order.
//
// No sum is made by atomic additions: the order of the additions is that of the positions within
// these tokens, and of these parts.
#include <algorithm>

#include "rows.cuh"

namespace dgc {
namespace {

constexpr int kThreads = 256;

struct Tokens {
    const void* p;
    int32_t wide;  // 64 bits
    __device__ int64_t operator[](uint64_t i) const {
        return wide ? static_cast<const int64_t*>(p)[i] : static_cast<const int32_t*>(p)[i];
    }
};

// --------------------------------------------------------------------------------- lookup
constexpr uint32_t kUnknown = 0xFFFFFFFFu;  // no word
// Pieces of 16 bytes of the result that a thread has under way, where 8 blocks are to be on an SM: more
// pieces take registers from other blocks (16384 x 2048 binary32: 33 us with 4 pieces, 31 with 3; to
// fp16 21.5 with 4, 19.7 with 2; 16384 x 4096 bf16 34.2 with 4, 32.5 with 3, although 12 bytes a
// thread are spilled for it).
template <typename S, typename D>
constexpr int kStepsOf = sizeof(S) > sizeof(D) ? 2 : 3;
struct EmbedArgs {
    const void* table;
    void* out;
    uint64_t ldt, ldo;
    Tokens tokens;
    PieceWalk walk;
    uint32_t cols, vocab;
    float scale;
    int32_t* status;
};

// Bound by HBM: the result is written once, each row of the table that is met is read from HBM
// once as far as L2 holds it. 16384 x 4096 bf16 from a table of 50000 rows: 32.5 us, 5.7 TB/s.
// What is lost is the start and two latencies in a row (the word, then its row). One short-lived
// block a tile: blocks that stay and look up the next tile's words ahead took 39 us at 6 an SM and
// 51 at 4, with the table's pieces copied to shared memory ahead 53.
template <typename S, typename D, bool kWide>
__global__ void __launch_bounds__(kThreads, kWide ? 8 : 1)
    k_embed(const __grid_constant__ EmbedArgs a) {
    constexpr int kSteps = kStepsOf<S, D>;
    constexpr int kN = 16 / sizeof(D);
    grid_dep_wait();
    grid_dep_launch();
    const S* table = static_cast<const S*>(a.table);
    D* out = static_cast<D*>(a.out);
    constexpr uint64_t kTile = kThreads * kSteps;
    for (uint64_t tile = blockIdx.x; tile * kTile < a.walk.total; tile += gridDim.x) {
        Pieces<kThreads, kSteps> at(a.walk, tile);
        const uint64_t first = tile * kTile + threadIdx.x;
        uint32_t row[kSteps], col[kSteps], left[kSteps], word[kSteps];
        Packed<S, kN> p[kSteps];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            row[i] = (uint32_t)at.row;
            col[i] = at.at * kN;
            left[i] = first + i * kThreads < a.walk.total ? a.cols - col[i] : 0;
            const int64_t w = left[i] ? a.tokens[row[i]] : 0;
            word[i] = w >= 0 && w < (int64_t)a.vocab ? (uint32_t)w : kUnknown;
            at.next(a.walk);
        }
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const bool known = word[i] != kUnknown;
            if (!known) report(a.status, DGC_EINVAL);
            p[i] = load_piece<kWide, S, kN, false>(
                table + (known ? (uint64_t)word[i] : 0) * a.ldt + col[i], known ? left[i] : 0);
        }
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            float f[kN];
            unpack<S, kN>(p[i], f);
#pragma unroll
            for (int j = 0; j < kN; ++j) f[j] *= a.scale;
            // an unknown word's row is 0 whatever the scale
            if (word[i] == kUnknown)
#pragma unroll
                for (int j = 0; j < kN; ++j) f[j] = 0.0f;
            store_piece<kWide, D, kN>(out + row[i] * a.ldo + col[i], pack<D, kN>(f), left[i]);
        }
    }
}

// ----------------------------------------------------------------------------------- sort
constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr uint32_t kSortRows = 8;                             // tokens of a lane, at most
constexpr uint32_t kSortTile = kSortThreads * kSortRows;      // of a block
constexpr int kDigits = 512;                                  // of up to 9 bits
constexpr uint32_t kSortCluster = 8;                          // blocks
constexpr uint32_t kSortMost = 256;                           // blocks of the launches for more

// A token on its way: its word in the upper half, its position below. Sorted, items rise.
using Item = uint64_t;

struct SortArgs {
    Tokens tokens;                 // the first pass's source
    Item *from, *to;               // the first pass writes from, the second one to, and so on
    uint32_t* counts;              // [block][digit]
    uint32_t n, per_block, rows;   // rows: of a lane in a tile; per_block: whole tiles
    uint32_t vocab, digit_bits, passes;
    int64_t padding;
    uint32_t* list_count;          // zeroed for k_embed_sum
    int32_t* status;
};

// Token i's item; `vocab` (behind all words) as the word of those without a gradient.
__device__ __forceinline__ Item sort_item(const SortArgs& a, const Item* from, uint32_t i) {
    if (from) return __ldcg(&from[i]);  // perhaps of another block of this launch
    const int64_t w = a.tokens[i];
    const bool known = w >= 0 && w < (int64_t)a.vocab;
    if (!known) report(a.status, DGC_EINVAL);
    return (Item)(known && w != a.padding ? (uint32_t)w : a.vocab) << 32 | i;
}
__device__ __forceinline__ uint32_t digit_of(Item v, uint32_t shift, uint32_t mask) {
    return (uint32_t)(v >> 32 >> shift) & mask;
}

// A block's tile of items in shared memory, a warp's rows * 32 of them in a row. Short loops: code
// that runs once waits for its instructions.
constexpr Item kNone = ~0ull;
struct SortTile {
    Item item[kSortTile];
    uint16_t rank[kSortTile];

    __device__ void load(const SortArgs& a, const Item* from, uint32_t first, uint32_t end) {
#pragma unroll 1
        for (uint32_t i = 0; i < a.rows; i += 4) {
            Item v[4];  // four loads under way: none waits for another one's way to shared memory
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j) {
                const uint32_t s = (i + j) * kSortThreads + threadIdx.x;
                v[j] = i + j < a.rows && first + s < end ? sort_item(a, from, first + s) : kNone;
            }
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j)
                if (i + j < a.rows) item[(i + j) * kSortThreads + threadIdx.x] = v[j];
        }
    }
    // Each token's place among its equals in the warp; count: how many of each digit it has.
    __device__ void ranks(const SortArgs& a, uint32_t shift, uint32_t mask, uint32_t* count) {
        rank_items(a, item, rank, shift, mask, count);
    }
    __device__ static void rank_items(const SortArgs& a, const Item* item, uint16_t* rank,
                                      uint32_t shift, uint32_t mask, uint32_t* count) {
        const uint32_t lane = threadIdx.x & 31, below = (1u << lane) - 1;
        uint32_t s = (threadIdx.x >> 5) * (32 * a.rows) + lane;
#pragma unroll 1
        for (uint32_t i = 0; i < a.rows; ++i, s += 32) {
            const Item v = item[s];
            const uint32_t d = v == kNone ? kDigits : digit_of(v, shift, mask);
            const unsigned same = __match_any_sync(kFull, d);
            const uint32_t r = d < kDigits ? count[d] : 0;
            __syncwarp();
            if (d < kDigits && (same & below) == 0) count[d] = r + __popc(same);
            rank[s] = (uint16_t)(r + __popc(same & below));
            __syncwarp();
        }
    }
    __device__ void store(const SortArgs& a, Item* to, uint32_t shift, uint32_t mask,
                          const uint32_t* place) const {
        uint32_t s = (threadIdx.x >> 5) * (32 * a.rows) + (threadIdx.x & 31);
#pragma unroll 1
        for (uint32_t i = 0; i < a.rows; ++i, s += 32) {
            const Item v = item[s];
            if (v != kNone) to[place[digit_of(v, shift, mask)] + rank[s]] = v;
        }
    }
};

__device__ __forceinline__ void clear_places(uint32_t (*place)[kDigits]) {
#pragma unroll 4
    for (int w = 0; w < kSortWarps; ++w) place[w][threadIdx.x] = 0;
}
// Where the thread's digit begins in the order: behind all smaller ones and those of the blocks
// before this one. count(b): block b's.
template <typename Count>
__device__ __forceinline__ uint32_t digit_begin(uint32_t blocks, uint32_t block, uint32_t* scan,
                                                Count count) {
    uint32_t before = 0, all = 0;
#pragma unroll 8
    for (uint32_t b = 0; b < blocks; ++b) {
        const uint32_t c = count(b);
        all += c;
        if (b < block) before += c;
    }
    uint32_t total;
    return block_excl_scan<kSortThreads>(all, scan, &total) + before;
}
// The thread's digit in each warp: counts become places, from `at` on. Returns the end.
__device__ __forceinline__ uint32_t warp_places(uint32_t (*place)[kDigits], uint32_t at) {
#pragma unroll 1
    for (int w = 0; w < kSortWarps; w += 8) {
        uint32_t c[8];  // read ahead of the writes, which might be to the same place for all the
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = place[w + i][threadIdx.x];  // compiler knows
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            place[w + i][threadIdx.x] = at;
            at += c[i];
        }
    }
    return at;
}
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of the same shared variable in block `rank` of the cluster.
__device__ __forceinline__ uint32_t in_block(const void* p, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr(p)), "r"(rank));
    return r;
}

// All passes by one cluster of up to 8 blocks, a tile each: the items stay in the blocks' shared
// memory and go from pass to pass to where they belong. Bound by latency: two passes of a few
// dependent steps each. 16384 tokens with cold caches 16 us, where two kernels a pass, with the
// items in L2, took 23.
struct ClusterTile {
    Item item[2][kSortTile];
    uint16_t rank[kSortTile];
    uint32_t own[kDigits];
};
__global__ void __launch_bounds__(kSortThreads) k_sort(const __grid_constant__ SortArgs a) {
    extern __shared__ uint4 shared[];
    ClusterTile& tile = *reinterpret_cast<ClusterTile*>(shared);
    __shared__ uint32_t place[kSortWarps][kDigits];
    __shared__ uint32_t scan[33];
    const int warp = threadIdx.x >> 5;
    grid_dep_wait();
    grid_dep_launch();
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.list_count = 0;
    const uint32_t mask = (1u << a.digit_bits) - 1, begin = blockIdx.x * a.per_block;
#pragma unroll 4
    for (uint32_t i = 0; i < a.rows; ++i) {
        const uint32_t s = i * kSortThreads + threadIdx.x;
        const Item v = begin + s < a.n ? sort_item(a, nullptr, begin + s) : kNone;
        tile.item[0][s] = v;
        if (v == kNone) tile.item[1][s] = v;
    }
    for (uint32_t pass = 0; pass < a.passes; ++pass) {
        const uint32_t shift = pass * a.digit_bits;
        const Item* item = tile.item[pass & 1];
        clear_places(place);
        __syncthreads();
        SortTile::rank_items(a, item, tile.rank, shift, mask, place[warp]);
        __syncthreads();
        uint32_t own = 0;
#pragma unroll 4
        for (int w = 0; w < kSortWarps; ++w) own += place[w][threadIdx.x];
        tile.own[threadIdx.x] = own;
        cluster_barrier();
        warp_places(place, digit_begin(gridDim.x, blockIdx.x, scan, [&](uint32_t b) {
                        uint32_t c;
                        asm volatile("ld.shared::cluster.u32 %0, [%1];"
                                     : "=r"(c)
                                     : "r"(in_block(&tile.own[threadIdx.x], b))
                                     : "memory");
                        return c;
                    }));
        __syncthreads();
        uint32_t s = warp * (32 * a.rows) + (threadIdx.x & 31);
#pragma unroll 1
        for (uint32_t i = 0; i < a.rows; ++i, s += 32) {
            const Item v = item[s];
            if (v == kNone) continue;
            const uint32_t to = place[warp][digit_of(v, shift, mask)] + tile.rank[s];
            if (pass + 1 == a.passes) {
                a.from[to] = v;
            } else {
                const uint32_t b = to / a.per_block;
                asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(
                                 in_block(&tile.item[~pass & 1][to - b * a.per_block], b)),
                             "l"(v)
                             : "memory");
            }
        }
        cluster_barrier();
    }
}

__global__ void __launch_bounds__(kSortThreads)
    k_sort_count(const __grid_constant__ SortArgs a, const Item* from, uint32_t shift) {
    __shared__ uint32_t count[kDigits];
    grid_dep_wait();
    grid_dep_launch();
    count[threadIdx.x] = 0;
    __syncthreads();
    const uint32_t mask = (1u << a.digit_bits) - 1;
    const uint32_t begin = blockIdx.x * a.per_block, end = min(a.n, begin + a.per_block);
    for (uint32_t i = begin + threadIdx.x; i < end; i += kSortThreads)
        atomicAdd(&count[digit_of(sort_item(a, from, i), shift, mask)], 1u);
    __syncthreads();
    a.counts[blockIdx.x * kDigits + threadIdx.x] = count[threadIdx.x];
}

// A block's tiles one behind the other.
__global__ void __launch_bounds__(kSortThreads)
    k_sort_move(const __grid_constant__ SortArgs a, const Item* from, Item* to, uint32_t shift) {
    extern __shared__ uint4 shared[];
    SortTile& tile = *reinterpret_cast<SortTile*>(shared);
    __shared__ uint32_t place[kSortWarps][kDigits];
    __shared__ uint32_t scan[33];
    const int warp = threadIdx.x >> 5;
    grid_dep_wait();
    grid_dep_launch();
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.list_count = 0;
    const uint32_t mask = (1u << a.digit_bits) - 1;
    const uint32_t begin = blockIdx.x * a.per_block, end = min(a.n, begin + a.per_block);
    uint32_t at = digit_begin(gridDim.x, blockIdx.x, scan, [&](uint32_t b) {
        return a.counts[b * kDigits + threadIdx.x];
    });
    for (uint32_t first = begin; first < end; first += a.rows * kSortThreads) {
        tile.load(a, from, first, end);
        clear_places(place);
        __syncthreads();
        tile.ranks(a, shift, mask, place[warp]);
        __syncthreads();
        at = warp_places(place, at);
        __syncthreads();
        tile.store(a, to, shift, mask, place[warp]);
        __syncthreads();
    }
}

// ------------------------------------------------------------------------------- gradient
constexpr uint32_t kZeroRows = 32, kZeroCols = 1024;  // of a unit of zeros

struct SumArgs {
    const Item* items;           // sorted
    uint32_t n, vocab, cols;
    const void* dy;
    uint64_t ldy;
    float* dtable;
    uint64_t ldt;
    float scale;
    int32_t accumulate;
    uint32_t tiles;              // of columns: a warp's
    uint32_t sum_blocks;         // the others zero
    uint32_t tokens;             // of a chunk
    float* part;                 // [chunk][2][ldp]: of words met more often, the sum in a chunk that
    uint64_t ldp;                // goes on from the last one, and in one that starts it
    uint32_t *list, *list_count; // chunks where such words start
};

__device__ __forceinline__ uint32_t trailing_ones(uint32_t x) { return ~x ? __ffs(~x) - 1 : 32; }

// kTokens (8 or 32) sorted tokens and what surrounds them, as bits: whether a token has its
// predecessor's word.
template <int kTokens>
struct Chunk {
    static constexpr uint32_t kMask = kTokens == 32 ? 0xFFFFFFFFu : (1u << kTokens) - 1;
    Item item, item_next;  // of this lane: 32 tokens, and (kTokens 32) the 32 behind
    uint32_t e0, e1, e2;   // bits of the tokens ahead, of the chunk, and of those behind
    uint32_t valid;        // how many of the chunk have a gradient
    __device__ Chunk(const SumArgs& a, uint32_t base) {
        const int lane = threadIdx.x & 31;
        // no two neighbours outside the list are alike
        auto at = [&](int64_t i) {
            return i >= 0 && i < (int64_t)a.n ? a.items[i]
                                              : (Item)(0x80000000u + ((uint32_t)i & 1)) << 32;
        };
        auto bits = [&](Item v, uint32_t last) {
            const uint32_t k = (uint32_t)(v >> 32);
            uint32_t p = __shfl_up_sync(kFull, k, 1);
            if (lane == 0) p = last;
            return __ballot_sync(kFull, k == p);
        };
        auto word = [&](Item v, int from) {
            return __shfl_sync(kFull, (uint32_t)(v >> 32), from);
        };
        if constexpr (kTokens == 32) {
            const Item before = at((int64_t)base - 32 + lane);
            item = at((int64_t)base + lane);
            item_next = at((int64_t)base + 32 + lane);
            e0 = bits(before, ~(uint32_t)(before >> 32));
            e1 = bits(item, word(before, 31));
            e2 = bits(item_next, word(item, 31));
            valid = __popc(__ballot_sync(kFull, (uint32_t)(item >> 32) < a.vocab));
        } else {
            item = at((int64_t)base - kTokens + lane);
            const uint32_t all = bits(item, ~(uint32_t)(item >> 32));
            e0 = all & kMask;
            e1 = all >> kTokens & kMask;
            e2 = all >> 2 * kTokens & kMask;
            const uint32_t known = __ballot_sync(kFull, (uint32_t)(item >> 32) < a.vocab);
            valid = __popc(known >> kTokens & kMask);
        }
    }
    // the e-th token from the chunk's first one on
    __device__ Item get(uint32_t e) const {
        if constexpr (kTokens == 32)
            return __shfl_sync(kFull, e < 32 ? item : item_next, e & 31);
        else
            return __shfl_sync(kFull, item, e + kTokens);
    }
};

// A lane's kN columns of a row. kWide: neighbours, all of them in the row or none, on a 16-byte
// boundary (8 for four 16-bit entries); else 32 apart. Columns behind the row's end are read as the
// last one's and not written, so that no load waits for a test.
template <int kN, bool kWide>
struct Cols {
    uint32_t at[kWide ? 1 : kN];
    uint32_t n;  // how many are the row's
    __device__ Cols(uint32_t tile, uint32_t cols) {
        const uint32_t lane = threadIdx.x & 31, first = tile * 32 * kN + (kWide ? lane * kN : lane);
        n = 0;
#pragma unroll
        for (int i = 0; i < (kWide ? 1 : kN); ++i) {
            n += first + 32 * i < cols;
            at[i] = min(first + 32 * i, cols - (kWide ? kN : 1));
        }
        if (kWide) n *= kN;
    }
    template <typename T>
    __device__ Packed<T, kN> load(const T* row) const {
        if constexpr (kWide) {
            return load_packed<T, kN>(row + at[0]);
        } else {
            Packed<T, kN> r;
#pragma unroll
            for (int i = 0; i < Packed<T, kN>::kWords; ++i) r.w[i] = 0;
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                const uint32_t one = load_packed<T, 1>(row + at[i]).w[0];
                if constexpr (sizeof(T) == 4) r.w[i] = one;
                else r.w[i / 2] |= one << (16 * (i & 1));
            }
            return r;
        }
    }
    __device__ void store(float* row, const float (&f)[kN]) const {
        if constexpr (kWide) {
            if (n) store_packed<float, kN>(row + at[0], pack<float, kN>(f));
        } else {
#pragma unroll
            for (int i = 0; i < kN; ++i)
                if ((uint32_t)i < n) __stcs(row + at[i], f[i]);
        }
    }
};

// Blocks an SM, at least: as many as there is room for without spilling, but for one form of float16.
// Off 16-byte boundaries, with chunks of 32 tokens written (16384 x 1001 into 32000 rows) and with chunks
// of 8 added (5001 x 1001 to 10000 rows, a tenth padding):
//   float16   72 us with 3 blocks, 80 with 2;  27.4 with 4 blocks (spilling 24 bytes a thread), 30.3 with 3
//   bfloat16  60 us with 2 blocks, 64 with 3 (spilling 64);  24.5 with 3 blocks, 26.2 with 4 (spilling 56)
template <typename T, int kTokens, int kN, bool kWide, bool kAdd>
constexpr int sum_blocks_of_sm() {
    constexpr bool spills = std::is_same_v<T, __nv_bfloat16> && !kWide;
    if (kTokens == 8) return kAdd && (sizeof(T) == 4 || spills) ? 3 : 4;
    return kN == 4 && !kAdd && sizeof(T) == 2 && !spills ? 3 : 2;
}

// Bound by HBM: dy read once, the table written once (read and written where it is added to).
// 16384 x 4096 bf16 into 50000 rows: 133 us, 7.2 TB/s; the sort ahead and the join behind are
// latency.
// A word met up to kTokens times is summed by the warp in whose chunk it starts; a longer run is cut
// at the chunks' borders. kN: a lane's columns.
template <typename T, int kTokens, int kN, bool kWide, bool kAdd>
__global__ void __launch_bounds__(kThreads, sum_blocks_of_sm<T, kTokens, kN, kWide, kAdd>())
    k_embed_sum(const __grid_constant__ SumArgs a) {
    // rows in flight (and of the table). More take so many registers that there are less warps: of 16
    // bytes (16384 x 4096 over 50000 words: 175 us for 162), and for 8 tokens, where blocks then come
    // in two turns and a bit (5001 x 1001, added: 33 us for 29)
    constexpr int kBatch = kN == 8 || kTokens == 8 ? 4 : 8;
    const int lane = threadIdx.x & 31;
    grid_dep_wait();
    grid_dep_launch();
    if (blockIdx.x >= a.sum_blocks) {
        const uint32_t col_units = (a.cols + kZeroCols - 1) / kZeroCols;
        const uint64_t units = (uint64_t)((a.vocab + kZeroRows - 1) / kZeroRows) * col_units;
        for (uint64_t u = blockIdx.x - a.sum_blocks; u < units; u += gridDim.x - a.sum_blocks) {
            const uint32_t row0 = (uint32_t)(u / col_units) * kZeroRows;
            const uint32_t tile = (uint32_t)(u % col_units) * (kThreads / 32) + (threadIdx.x >> 5);
            const Cols<4, kWide> cols(tile, a.cols);
            // is this lane's row met? The rows' stretch of the list first, then a row's
            const uint32_t row = row0 + lane;
            const uint32_t from = first_from(a.items, 0, a.n, (Item)row0 << 32);
            uint32_t lo = from, hi = first_from(a.items, from, a.n - from,
                                                (Item)(row0 + kZeroRows) << 32);
            const uint32_t stop = hi;
            while (lo < hi) {
                const uint32_t mid = (lo + hi) >> 1;
                if (a.items[mid] < (Item)row << 32) lo = mid + 1; else hi = mid;
            }
            const bool met = lo < stop && (uint32_t)(a.items[lo] >> 32) == row;
            uint32_t todo = __ballot_sync(kFull, !met && row < a.vocab);
            const float zero[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            for (; todo; todo &= todo - 1)
                cols.store(a.dtable + (row0 + __ffs(todo) - 1) * a.ldt, zero);
        }
        return;
    }
    const T* dy = static_cast<const T*>(a.dy);
    constexpr uint32_t kT = kTokens;
    const uint32_t chunks = (a.n + kT - 1) / kT;
    const uint64_t units = (uint64_t)chunks * a.tiles;
    for (uint64_t u = (uint64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); u < units;
         u += (uint64_t)a.sum_blocks * (kThreads / 32)) {
        const uint32_t chunk = (uint32_t)(u / a.tiles), tile = (uint32_t)(u % a.tiles);
        const Cols<kN, kWide> cols(tile, a.cols);
        const Chunk<kTokens> c(a, chunk * kT);
        // the run that the first token continues: how much of it is ahead and from here on
        const bool goes_on = c.e1 & 1;
        const uint32_t ahead =
            goes_on ? 1 + min(kT - 1, (uint32_t)__clz(~(c.e0 << (32 - kTokens)))) : 0;
        uint32_t head = 1 + trailing_ones(c.e1 >> 1);  // e1 >> 1 has one bit less
        if (head == kT) head += min(kT, trailing_ones(c.e2));
        const bool long_head = goes_on && ahead + head > kT;
        // the last run that starts here, and how far it goes
        const uint32_t begins = ~c.e1 & c.kMask;
        const uint32_t last = begins ? 31 - __clz(begins) : kT;
        const uint32_t behind = min(kT, trailing_ones(c.e2));
        const bool long_tail = begins && kT - last + behind > kT;
        const uint32_t begin = !goes_on || long_head ? 0 : head;
        uint32_t end = !begins || long_tail ? kT : kT + behind;
        if (c.valid < kT) end = min(end, c.valid);  // words without a gradient are the last ones
        if (long_tail && c.valid == kT && tile == 0 && lane == 0)
            a.list[atomicAdd(a.list_count, 1u)] = chunk;
        // which tokens end a run, and which of those runs are whole: from head on, ahead of last
        const uint64_t ends = ~(((uint64_t)c.e2 << kTokens | c.e1) >> 1);  // the last bit: 1
        const uint32_t whole_from = long_head ? head : 0, whole_to = long_tail ? last : 64;
        struct Batch {
            Packed<T, kN> p[kBatch];
            Packed<float, kN> old[kAdd ? kBatch : 1];
            float* row[kBatch];  // where the run's sum goes, at its end
        };
        auto load = [&](Batch& b, uint32_t e0) {
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const uint32_t e = min(e0 + i, end - 1);
                const Item item = c.get(e);
                const uint32_t word = (uint32_t)(item >> 32);
                b.p[i] = cols.load(dy + (uint64_t)(uint32_t)item * a.ldy);
                const bool stop = e0 + i < end && ((ends >> e & 1) || e + 1 == end);
                const bool whole = stop && e >= whole_from && e < whole_to;
                float* const to = whole ? a.dtable + (uint64_t)word * a.ldt
                                        : a.part + ((uint64_t)chunk * 2 + (e >= whole_from)) * a.ldp;
                b.row[i] = stop ? to : nullptr;
                if (kAdd) b.old[i] = cols.load(whole ? to : a.part);  // no test ahead of a load
            }
        };
        float acc[kN];
#pragma unroll
        for (int j = 0; j < kN; ++j) acc[j] = 0.0f;
        auto add = [&](const Batch& b, uint32_t e0) {
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const uint32_t e = e0 + i;
                if (e < end) {
                    float f[kN];
                    unpack<T, kN>(b.p[i], f);
#pragma unroll
                    for (int j = 0; j < kN; ++j) acc[j] += f[j];
                }
                if (b.row[i]) {
                    if (e >= whole_from && e < whole_to) {
                        float was[kN];
                        if (kAdd) unpack<float, kN>(b.old[kAdd ? i : 0], was);
#pragma unroll
                        for (int j = 0; j < kN; ++j)
                            acc[j] = kAdd ? fmaf(acc[j], a.scale, was[j]) : acc[j] * a.scale;
                    }
                    cols.store(b.row[i], acc);
#pragma unroll
                    for (int j = 0; j < kN; ++j) acc[j] = 0.0f;
                }
            }
        };
#pragma unroll 1
        for (uint32_t e0 = begin; e0 < end; e0 += kBatch) {
            Batch b;
            load(b, e0);
            add(b, e0);
        }
    }
}

// The parts of a long run, 128 columns by a block: each warp sums an eighth of them in order, the
// first warp adds the eight. Lanes' columns as in k_embed_sum.
template <bool kWide, bool kAdd>
__global__ void __launch_bounds__(kThreads) k_embed_join(const __grid_constant__ SumArgs a) {
    constexpr int kWarps = kThreads / 32;
    __shared__ float4 sm[kWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_dep_wait();
    grid_dep_launch();
    const uint32_t count = *a.list_count;
    const uint32_t tiles = (a.cols + 127) / 128;
    for (uint64_t u = blockIdx.x; u < (uint64_t)count * tiles; u += gridDim.x) {
        const uint32_t chunk = a.list[u / tiles], next = (chunk + 1) * a.tokens;
        const Cols<4, kWide> cols((uint32_t)(u % tiles), a.cols);
        const uint32_t word = (uint32_t)(a.items[next - 1] >> 32);
        float* out = a.dtable + (uint64_t)word * a.ldt;
        Packed<float, 4> old{};
        if (kAdd && warp == 0) old = cols.load(out);
        uint32_t parts = 1;  // and one for each chunk that begins in the run, 32 looked at at once
        for (uint32_t more = 32; more == 32; parts += more) {
            const uint64_t at = (uint64_t)(chunk + parts + lane) * a.tokens;
            more = trailing_ones(__ballot_sync(
                kFull, at < a.n && (uint32_t)(a.items[at < a.n ? at : 0] >> 32) == word));
        }
        const uint32_t share = (parts + kWarps - 1) / kWarps;
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        const uint32_t from = min(parts, warp * share), to = min(parts, from + share);
#pragma unroll 8
        for (uint32_t i = from; i < to; ++i) {  // the first part starts the run
            float v[4];
            unpack<float, 4>(cols.load(a.part + ((uint64_t)(chunk + i) * 2 + (i == 0)) * a.ldp), v);
#pragma unroll
            for (int j = 0; j < 4; ++j) s[j] += v[j];
        }
        sm[warp][lane] = make_float4(s[0], s[1], s[2], s[3]);
        __syncthreads();
        if (warp == 0) {
            for (int w = 1; w < kWarps; ++w) {
                const float4 v = sm[w][lane];
                s[0] += v.x;
                s[1] += v.y;
                s[2] += v.z;
                s[3] += v.w;
            }
            float was[4];
            unpack<float, 4>(old, was);
#pragma unroll
            for (int j = 0; j < 4; ++j) s[j] = kAdd ? fmaf(s[j], a.scale, was[j]) : s[j] * a.scale;
            cols.store(out, s);
        }
        __syncthreads();
    }
}

// ----------------------------------------------------------------------------------- host
struct BackwardLayout {
    uint32_t blocks, per_block, rows, passes, digit_bits;  // of the sort
    uint32_t tokens;                                       // of a chunk of the sums
    size_t items[2], counts, list, part, total;
    uint64_t ldp;
};
BackwardLayout backward_layout(uint64_t n, uint64_t vocab, uint64_t dim) {
    auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
    BackwardLayout L{};
    uint32_t bits = 1;
    while ((vocab >> bits) != 0) ++bits;  // keys 0 to vocab
    L.passes = (bits + 8) / 9;
    L.digit_bits = (bits + L.passes - 1) / L.passes;
    // A tile a block where a cluster sorts, over as many blocks as it may have (2048 tokens x 1024
    // columns: 17 us, with tiles of 2048 tokens 20); else whole tiles, as many as it takes.
    if (n <= kSortCluster * (uint64_t)kSortTile) {
        const uint64_t rows = (n + kSortThreads - 1) / kSortThreads;
        L.rows = (uint32_t)((rows + kSortCluster - 1) / kSortCluster);
        L.per_block = L.rows * kSortThreads;
    } else {
        const uint64_t tiles = (n + kSortTile - 1) / kSortTile;
        L.rows = kSortRows;
        L.per_block = (uint32_t)((tiles + kSortMost - 1) / kSortMost * kSortTile);
    }
    L.blocks = L.per_block ? (uint32_t)((n + L.per_block - 1) / L.per_block) : 0;
    size_t at = 0;
    for (int i = 0; i < 2; ++i) {
        L.items[i] = at;
        at = up(at + n * sizeof(Item));
    }
    L.counts = at;
    at = up(at + (size_t)kSortMost * kDigits * 4);
    // Chunks of 32 tokens; of 8 where that would leave 152 SMs less than 16 warps each: a warp's
    // rows are then all under way at once (5001 tokens x 1001 columns: 36 us for 52).
    L.tokens = (n + 31) / 32 * ((dim + 127) / 128) < 152 * 16 ? 8 : 32;
    const uint64_t chunks = (n + L.tokens - 1) / L.tokens;
    L.list = at;  // the count, then the chunks
    at = up(at + (chunks + 1) * 4);
    L.ldp = (dim + 3) & ~3ull;
    L.part = at;
    at = up(at + chunks * 2 * L.ldp * sizeof(float));
    L.total = at;
    return L;
}

template <typename T, int kTokens, int kN>
int launch_sums(SumArgs a, bool wide, int sms, cudaStream_t s) {
    a.tiles = (a.cols + 32 * kN - 1) / (32 * kN);
    const uint64_t chunks = (a.n + kTokens - 1) / kTokens;
    a.sum_blocks = (uint32_t)umin64((chunks * a.tiles + 7) / 8, 1u << 24);
    const uint64_t zeros = a.accumulate ? 0
                                        : ((uint64_t)a.vocab + kZeroRows - 1) / kZeroRows *
                                              ((a.cols + kZeroCols - 1) / kZeroCols);
    const dim3 grid(a.sum_blocks + (unsigned)umin64(zeros, 1u << 24));
    if (grid.x == 0) return DGC_OK;
    auto pick = [&] {
        if constexpr (kN == 8)  // wide
            return a.accumulate ? k_embed_sum<T, kTokens, kN, true, true>
                                : k_embed_sum<T, kTokens, kN, true, false>;
        else
            return a.accumulate ? (wide ? k_embed_sum<T, kTokens, kN, true, true>
                                        : k_embed_sum<T, kTokens, kN, false, true>)
                                : (wide ? k_embed_sum<T, kTokens, kN, true, false>
                                        : k_embed_sum<T, kTokens, kN, false, false>);
    };
    const int rc = launch_rows_kernel(pick(), grid, kThreads, s, a);
    // only a list of more tokens than a chunk's can hold a word more often
    if (rc || a.n <= kTokens) return rc;
    auto joiner = a.accumulate ? (wide ? k_embed_join<true, true> : k_embed_join<false, true>)
                               : (wide ? k_embed_join<true, false> : k_embed_join<false, false>);
    const uint64_t blocks = umin64((uint64_t)sms * 4, chunks * ((a.cols + 127) / 128));
    return launch_rows_kernel(joiner, dim3((unsigned)blocks), kThreads, s, a);
}

int launch_sort(const SortArgs& a, const BackwardLayout& L, cudaStream_t s) {
    if (L.blocks <= kSortCluster) {
        cudaLaunchConfig_t c{};
        c.gridDim = dim3(L.blocks);
        c.blockDim = dim3(kSortThreads);
        c.dynamicSmemBytes = sizeof(ClusterTile);
        c.stream = s;
        if (cudaFuncSetAttribute(k_sort, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 sizeof(ClusterTile)) != cudaSuccess) {
            cudaGetLastError();
            return DGC_ECUDA;
        }
        cudaLaunchAttribute at[2];
        at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[0].val.programmaticStreamSerializationAllowed = 1;
        at[1].id = cudaLaunchAttributeClusterDimension;
        at[1].val.clusterDim.x = L.blocks;
        at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
        c.attrs = at;
        c.numAttrs = 2;
        if (cudaLaunchKernelEx(&c, k_sort, a) != cudaSuccess) {
            cudaGetLastError();
            return DGC_ECUDA;
        }
        dgc_internal_count_launches(1);
        return DGC_OK;
    }
    const Item* from = nullptr;
    Item *to = a.from, *other = a.to;
    for (uint32_t pass = 0; pass < a.passes; ++pass) {
        const uint32_t shift = pass * a.digit_bits;
        int rc = launch_rows_kernel(k_sort_count, dim3(L.blocks), kSortThreads, s, a, from, shift);
        if (rc) return rc;
        rc = launch_shared_kernel(k_sort_move, dim3(L.blocks), kSortThreads, sizeof(SortTile), s, a,
                                  from, to, shift);
        if (rc) return rc;
        from = to;
        to = other;
        other = const_cast<Item*>(from);
    }
    return DGC_OK;
}

int check_tokens(const dgc_tensor* t, Tokens* out) {
    if (!t || (t->dtype != DGC_I32 && t->dtype != DGC_I64) || t->n < 0) return DGC_EINVAL;
    if (t->n > kMaxExtent) return DGC_EUNSUPPORTED;
    *out = Tokens{t->data, t->dtype == DGC_I64};
    return check_vector(t, (uint64_t)t->n, t->dtype);
}

template <typename S, typename D>
int launch_embed(const EmbedArgs& a, bool wide, cudaStream_t s) {
    constexpr int kTile = kThreads * kStepsOf<S, D>;
    const uint64_t tiles = (a.walk.total + kTile - 1) / kTile;
    const dim3 grid((unsigned)umin64(tiles, 1u << 30));
    return launch_rows_kernel(wide ? k_embed<S, D, true> : k_embed<S, D, false>, grid, kThreads, s,
                              a);
}

}  // namespace
}  // namespace dgc

using namespace dgc;

extern "C" int dgc_embed(const dgc_matrix* table, const dgc_tensor* tokens, float scale,
                         const dgc_matrix* out, int32_t* status, dgc_stream_t stream) {
    Rows mt, mo;
    EmbedArgs a{};
    int rc;
    if (!status) return DGC_EINVAL;
    if ((rc = check_rows(table, &mt, -1)) || (rc = check_tokens(tokens, &a.tokens)) ||
        (rc = check_rows(out, &mo, -1)))
        return rc;
    if (!mo.shaped((uint64_t)tokens->n, mt.cols)) return DGC_EINVAL;
    if (mo.rows == 0 || mo.cols == 0) return DGC_OK;
    a.table = mt.p;
    a.ldt = mt.ld;
    a.out = mo.p;
    a.ldo = mo.ld;
    a.cols = (uint32_t)mo.cols;
    a.vocab = (uint32_t)mt.rows;
    a.scale = scale;
    a.status = status;
    const uint32_t piece = (uint32_t)(16 / mo.entry());
    a.walk = piece_walk(mo.rows, (a.cols + piece - 1) / piece, kThreads);
    const bool wide = mo.on(16) && mt.on(umin64(16, piece * mt.entry()));
    return with_type(mt.dtype, [&](auto s) {
        return with_type(mo.dtype, [&](auto d) {
            return launch_embed<decltype(s), decltype(d)>(a, wide,
                                                          reinterpret_cast<cudaStream_t>(stream));
        });
    });
}

extern "C" int dgc_embed_backward_workspace(int64_t tokens, int64_t vocab, int64_t dim,
                                            size_t* bytes) {
    if (!bytes || tokens < 0 || vocab < 0 || dim < 0) return DGC_EINVAL;
    if (tokens > kMaxExtent || vocab > kMaxExtent || dim > kMaxExtent) return DGC_EUNSUPPORTED;
    *bytes = backward_layout((uint64_t)tokens, (uint64_t)vocab, (uint64_t)dim).total;
    return DGC_OK;
}

extern "C" int dgc_embed_backward(const dgc_tensor* tokens, const dgc_matrix* dy, float scale,
                                  int64_t padding, int32_t accumulate, const dgc_matrix* dtable,
                                  int32_t* status, void* ws, size_t ws_bytes, dgc_stream_t stream) {
    Rows my, mt;
    Tokens tok;
    int rc;
    if (!status || padding < -1) return DGC_EINVAL;
    if ((rc = check_tokens(tokens, &tok)) || (rc = check_rows(dy, &my, -1)) ||
        (rc = check_rows(dtable, &mt, DGC_F32)))
        return rc;
    if (!my.shaped((uint64_t)tokens->n, mt.cols)) return DGC_EINVAL;
    const uint32_t n = (uint32_t)my.rows;
    const BackwardLayout L = backward_layout(n, mt.rows, mt.cols);
    if (ws_bytes < L.total || !ws || ((uintptr_t)ws & 255u)) return DGC_EINVAL;
    if (mt.cols == 0 || (n == 0 && (accumulate || mt.rows == 0))) return DGC_OK;
    const int sms = dgc_internal_sm_count();
    if (sms <= 0) return DGC_ECUDA;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    char* w = static_cast<char*>(ws);
    auto words = [&](size_t at) { return reinterpret_cast<uint32_t*>(w + at); };

    SumArgs sum{};
    sum.list_count = words(L.list);
    sum.list = sum.list_count + 1;
    if (n) {
        SortArgs a{};
        a.tokens = tok;
        a.n = n;
        a.per_block = L.per_block;
        a.vocab = (uint32_t)mt.rows;
        a.padding = padding;
        a.counts = words(L.counts);
        a.status = status;
        a.digit_bits = L.digit_bits;
        a.passes = L.passes;
        a.list_count = sum.list_count;
        a.rows = L.rows;
        a.from = reinterpret_cast<Item*>(w + L.items[0]);
        a.to = reinterpret_cast<Item*>(w + L.items[1]);
        if ((rc = launch_sort(a, L, s))) return rc;
        // one cluster sorts into the first array, the launches take turns
        sum.items = L.blocks <= kSortCluster || (L.passes & 1) ? a.from : a.to;
    }
    sum.n = n;
    sum.vocab = (uint32_t)mt.rows;
    sum.cols = (uint32_t)mt.cols;
    sum.dy = my.p;
    sum.ldy = my.ld;
    sum.dtable = static_cast<float*>(mt.p);
    sum.ldt = mt.ld;
    sum.scale = scale;
    sum.accumulate = accumulate != 0;
    sum.part = reinterpret_cast<float*>(w + L.part);
    sum.ldp = L.ldp;
    const bool wide = my.on(16) && mt.on(16) && mt.cols % 4 == 0;
    sum.tokens = L.tokens;
    // eight columns a lane where that leaves the SMs 16 warps each: 16-byte loads of 16-bit entries
    const bool eight = my.dtype != DGC_F32 && wide && mt.cols % 8 == 0 && L.tokens == 32 &&
                       (uint64_t)((n + 31) / 32) * ((mt.cols + 255) / 256) >= (uint64_t)sms * 16;
    return with_type(my.dtype, [&](auto t) {
        using T = decltype(t);
        if constexpr (sizeof(T) == 2)
            if (eight) return launch_sums<T, 32, 8>(sum, wide, sms, s);
        return L.tokens == 8 ? launch_sums<T, 8, 4>(sum, wide, sms, s)
                             : launch_sums<T, 32, 4>(sum, wide, sms, s);
    });
}
