// embed.cu -- embedding lookup with scaling, and its gradient by sorted tokens (sm_103a).
//
//   out[t] = scale table[token[t]]
//   dtable[w] = scale sum of dy[t] over the t with token[t] = w, in the order of t; or added
//
//   k_embed        the lookup.
//   k_sort_count   how often a block's tokens have each value of a digit of up to 9 bits;
//   k_sort_move    puts (token, position) in the digit's order, equal ones in theirs: a stable
//                  radix sort, lowest digit first, two launches a digit (one for few tokens).
//   k_embed_sum    a warp sums the rows of 32 sorted tokens over 32 pieces of columns, and writes
//                  each word's sum once; other blocks zero the rows of words that are not met.
//   k_embed_join   joins the sums of words that are met more than 32 times, in order.
//
// No sum is made by atomic additions: the order of the additions is that of the positions within
// 32 sorted tokens, and of these parts.
#include <algorithm>

#include "rows.cuh"

namespace dgc {
namespace {

constexpr int kThreads = 256;
constexpr int kSteps = 4;

struct Tokens {
    const void* p;
    int32_t wide;  // 64 bits
    __device__ int64_t operator[](uint64_t i) const {
        return wide ? static_cast<const int64_t*>(p)[i] : static_cast<const int32_t*>(p)[i];
    }
};

// --------------------------------------------------------------------------------- lookup
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
// once as far as L2 holds it.
template <typename S, typename D, bool kWide>
__global__ void __launch_bounds__(kThreads) k_embed(const __grid_constant__ EmbedArgs a) {
    constexpr int kN = 16 / sizeof(D);
    grid_dep_wait();
    grid_dep_launch();
    const S* table = static_cast<const S*>(a.table);
    D* out = static_cast<D*>(a.out);
    constexpr uint64_t kTile = kThreads * kSteps;
    for (uint64_t tile = blockIdx.x; tile * kTile < a.walk.total; tile += gridDim.x) {
        Pieces<kThreads, kSteps> at(a.walk, tile);
        const uint64_t first = tile * kTile + threadIdx.x;
        uint64_t row[kSteps];
        uint32_t col[kSteps], left[kSteps];
        int64_t word[kSteps];
        Packed<S, kN> p[kSteps];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            row[i] = at.row;
            col[i] = at.at * kN;
            left[i] = first + i * kThreads < a.walk.total ? a.cols - col[i] : 0;
            word[i] = left[i] ? a.tokens[row[i]] : 0;
            at.next(a.walk);
        }
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const bool known = word[i] >= 0 && word[i] < (int64_t)a.vocab;
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
            const bool known = word[i] >= 0 && word[i] < (int64_t)a.vocab;
            if (!known)
#pragma unroll
                for (int j = 0; j < kN; ++j) f[j] = 0.0f;
            store_piece<kWide, D, kN>(out + row[i] * a.ldo + col[i], pack<D, kN>(f), left[i]);
        }
    }
}

// ----------------------------------------------------------------------------------- sort
constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kDigits = 512;          // of up to 9 bits
constexpr uint32_t kSortMost = 256;   // blocks
constexpr uint32_t kSortLeast = 4096; // tokens up to which one block sorts alone

struct SortArgs {
    Tokens tokens;                 // the first pass's source
    const uint32_t *key, *pos;     // the others'
    uint32_t *key_out, *pos_out;
    uint32_t* counts;              // [block][digit]
    uint32_t n, per_block;         // per_block: a multiple of kSortThreads
    uint32_t vocab, shift, mask;
    int64_t padding;
    uint32_t* list_count;          // zeroed for k_embed_sum
    int32_t first;
    int32_t* status;
};

// The key of token i: its word; `vocab` (behind all words) for those without a gradient.
__device__ __forceinline__ uint32_t sort_key(const SortArgs& a, uint32_t i, bool check) {
    if (!a.first) return a.key[i];
    const int64_t w = a.tokens[i];
    const bool known = w >= 0 && w < (int64_t)a.vocab;
    if (check && !known) report(a.status, DGC_EINVAL);
    return known && w != a.padding ? (uint32_t)w : a.vocab;
}

__global__ void __launch_bounds__(kSortThreads) k_sort_count(const __grid_constant__ SortArgs a) {
    __shared__ uint32_t count[kDigits];
    grid_dep_wait();
    grid_dep_launch();
    count[threadIdx.x] = 0;
    __syncthreads();
    const uint32_t begin = blockIdx.x * a.per_block, end = min(a.n, begin + a.per_block);
    for (uint32_t i = begin + threadIdx.x; i < end; i += kSortThreads)
        atomicAdd(&count[(sort_key(a, i, false) >> a.shift) & a.mask], 1u);
    __syncthreads();
    a.counts[blockIdx.x * kDigits + threadIdx.x] = count[threadIdx.x];
}

// A warp owns a run of the block's tokens. Counted once by warp and digit, summed up to where each
// warp's tokens of a digit begin, then walked again, 32 tokens at a time: a token's place among
// its equals is that of its lane.
__global__ void __launch_bounds__(kSortThreads) k_sort_move(const __grid_constant__ SortArgs a) {
    __shared__ uint32_t place[kSortWarps][kDigits];
    __shared__ uint32_t scan[33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_dep_wait();
    grid_dep_launch();
    if (a.list_count && blockIdx.x == 0 && threadIdx.x == 0) *a.list_count = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) place[w][threadIdx.x] = 0;
    __syncthreads();
    const uint32_t per_warp = a.per_block / kSortWarps;
    const uint32_t begin = min(a.n, blockIdx.x * a.per_block + warp * per_warp);
    const uint32_t end = min(a.n, begin + per_warp);
    for (uint32_t i = begin + lane; i < end; i += 32)
        atomicAdd(&place[warp][(sort_key(a, i, true) >> a.shift) & a.mask], 1u);
    __syncthreads();
    {
        const uint32_t d = threadIdx.x;
        uint32_t before = 0, own = 0, all = 0;  // in earlier blocks, in this one, everywhere
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) own += place[w][d];
        if (gridDim.x == 1) {
            all = own;
        } else {
#pragma unroll 8
            for (uint32_t b = 0; b < gridDim.x; ++b) {
                const uint32_t c = a.counts[b * kDigits + d];
                all += c;
                if (b < blockIdx.x) before += c;
            }
        }
        uint32_t total;
        uint32_t at = block_excl_scan<kSortThreads>(all, scan, &total) + before;
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) {
            const uint32_t c = place[w][d];
            place[w][d] = at;
            at += c;
        }
    }
    __syncthreads();
    for (uint32_t i0 = begin; i0 < end; i0 += 32) {
        const uint32_t i = i0 + lane;
        const bool in = i < end;
        const uint32_t key = in ? sort_key(a, i, false) : 0;
        const uint32_t d = in ? (key >> a.shift) & a.mask : kDigits;
        const unsigned same = __match_any_sync(kFull, d);
        const int leader = __ffs(same) - 1;
        uint32_t to = 0;
        if (in && lane == leader) {
            to = place[warp][d];
            place[warp][d] = to + __popc(same);
        }
        to = __shfl_sync(kFull, to, leader) + __popc(same & ((1u << lane) - 1));
        if (in) {
            a.key_out[to] = key;
            a.pos_out[to] = a.first ? i : a.pos[i];
        }
        __syncwarp();
    }
}

// ------------------------------------------------------------------------------- gradient
constexpr uint32_t kZeroRows = 32, kZeroCols = 1024;  // of a unit of zeros

struct SumArgs {
    const uint32_t *key, *pos;   // sorted
    uint32_t n, vocab, cols;
    const void* dy;
    uint64_t ldy;
    float* dtable;
    uint64_t ldt;
    float scale;
    int32_t accumulate;
    uint32_t tiles;              // of columns, a warp's 32 pieces each
    uint32_t sum_blocks;         // the others zero
    float* part;                 // [chunk][2][ldp]: of words met more than 32 times, the sum in a
    uint64_t ldp;                // chunk that goes on from the last one, and in one that starts it
    uint32_t *list, *list_count; // chunks where such words start
};

__device__ __forceinline__ uint32_t trailing_ones(uint32_t x) { return ~x ? __ffs(~x) - 1 : 32; }

// 32 sorted tokens and what surrounds them, as bits: whether a token has its predecessor's word.
struct Chunk {
    uint32_t key, key_next;  // of this lane, here and 32 tokens on
    uint32_t e0, e1, e2;     // bits of the 32 tokens ahead, of the chunk, and of the 32 behind
    __device__ Chunk(const SumArgs& a, uint32_t base) {
        const int lane = threadIdx.x & 31;
        // no two neighbours outside the list are alike
        auto at = [&](int64_t i) {
            return i >= 0 && i < (int64_t)a.n ? a.key[i] : 0x80000000u + ((uint32_t)i & 1);
        };
        const uint32_t before = at((int64_t)base - 32 + lane);
        key = at((int64_t)base + lane);
        key_next = at((int64_t)base + 32 + lane);
        auto bits = [&](uint32_t k, uint32_t last) {
            uint32_t p = __shfl_up_sync(kFull, k, 1);
            if (lane == 0) p = last;
            return __ballot_sync(kFull, k == p);
        };
        e0 = bits(before, ~before);
        e1 = bits(key, __shfl_sync(kFull, before, 31));
        e2 = bits(key_next, __shfl_sync(kFull, key, 31));
    }
};

// One row of sums to the table, or (scaled later) to a part.
template <bool kWide, bool kAdd, int kN>
__device__ __forceinline__ void write_sums(float* p, const float (&acc)[kN], float scale,
                                           const float (&old)[kN], uint32_t left) {
    float f[kN];
#pragma unroll
    for (int j = 0; j < kN; ++j) f[j] = kAdd ? fmaf(acc[j], scale, old[j]) : acc[j] * scale;
    store_piece<kWide, float, kN>(p, pack<float, kN>(f), left);
}

// Bound by HBM: dy read once, the table written once (read and written where it is added to).
// A word met up to 32 times is summed by the warp in whose chunk it starts; a longer run is cut at
// the chunks' borders.
template <typename T, bool kWide, bool kWideTable, bool kAdd>
__global__ void __launch_bounds__(kThreads) k_embed_sum(const __grid_constant__ SumArgs a) {
    constexpr int kN = 16 / sizeof(T);
    constexpr int kBatch = kAdd ? 4 : 8;  // rows in flight (and as many rows of the table)
    const int lane = threadIdx.x & 31;
    grid_dep_wait();
    grid_dep_launch();
    if (blockIdx.x >= a.sum_blocks) {
        const uint32_t col_units = (a.cols + kZeroCols - 1) / kZeroCols;
        const uint64_t units = (uint64_t)((a.vocab + kZeroRows - 1) / kZeroRows) * col_units;
        for (uint64_t u = blockIdx.x - a.sum_blocks; u < units; u += gridDim.x - a.sum_blocks) {
            const uint32_t row0 = (uint32_t)(u / col_units) * kZeroRows;
            const uint32_t col = (uint32_t)(u % col_units) * kZeroCols + threadIdx.x * 4;
            const uint32_t left = col < a.cols ? a.cols - col : 0;
            // is this lane's row met?
            const uint32_t row = row0 + lane;
            uint32_t lo = 0, hi = a.n;
            while (lo < hi) {
                const uint32_t mid = (lo + hi) >> 1;
                if (a.key[mid] < row) lo = mid + 1; else hi = mid;
            }
            const bool met = lo < a.n && a.key[lo] == row;
            uint32_t todo = __ballot_sync(kFull, !met && row < a.vocab);
            const float zero[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            for (; todo; todo &= todo - 1)
                store_piece<kWideTable, float, 4>(
                    a.dtable + (row0 + __ffs(todo) - 1) * a.ldt + col, pack<float, 4>(zero), left);
        }
        return;
    }
    const T* dy = static_cast<const T*>(a.dy);
    const uint32_t chunks = (a.n + 31) / 32;
    const uint64_t units = (uint64_t)chunks * a.tiles;
    for (uint64_t u = (uint64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); u < units;
         u += (uint64_t)a.sum_blocks * (kThreads / 32)) {
        const uint32_t chunk = (uint32_t)(u / a.tiles), tile = (uint32_t)(u % a.tiles);
        const uint32_t base = chunk * 32, col = (tile * 32 + lane) * kN;
        const uint32_t left = col < a.cols ? a.cols - col : 0;
        const Chunk c(a, base);
        const uint32_t pos = base + lane < a.n ? a.pos[base + lane] : 0;
        const uint32_t pos_next = base + 32 + lane < a.n ? a.pos[base + 32 + lane] : 0;
        const uint32_t valid = __popc(__ballot_sync(kFull, c.key < a.vocab));
        // the run that the first token continues: how much of it is ahead and from here on
        const bool goes_on = c.e1 & 1;
        const uint32_t ahead = goes_on ? 1 + min(31, __clz(~c.e0)) : 0;
        uint32_t head = 1 + trailing_ones(c.e1 >> 1);  // e1 >> 1 has 31 bits
        if (head == 32) head += trailing_ones(c.e2);
        const bool long_head = goes_on && ahead + head > 32;
        // the last run that starts here, and how far it goes
        const int last = ~c.e1 ? 31 - __clz(~c.e1) : -1;
        const uint32_t behind = trailing_ones(c.e2);
        const bool long_tail = last >= 0 && 32 - last + behind > 32;
        const uint32_t begin = !goes_on || long_head ? 0 : head;
        uint32_t end = last < 0 || long_tail ? 32 : 32 + behind;
        if (valid < 32) end = min(end, valid);  // words without a gradient are the last ones
        if (long_tail && valid == 32 && tile == 0 && lane == 0)
            a.list[atomicAdd(a.list_count, 1u)] = chunk;
        const uint64_t next_starts = ~(((uint64_t)c.e2 << 32 | c.e1) >> 1);  // bit 63: 1
        float acc[kN];
#pragma unroll
        for (int j = 0; j < kN; ++j) acc[j] = 0.0f;
        for (uint32_t e0 = begin; e0 < end; e0 += kBatch) {
            Packed<T, kN> p[kBatch];
            Packed<float, kN> old[kAdd ? kBatch : 1];
            uint32_t word[kBatch];
            uint32_t flush = 0;
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const uint32_t e = e0 + i;
                const uint32_t t = __shfl_sync(kFull, e < 32 ? pos : pos_next, e & 31);
                word[i] = __shfl_sync(kFull, e < 32 ? c.key : c.key_next, e & 31);
                const bool in = e < end;
                p[i] = load_piece<kWide, T, kN>(dy + (uint64_t)t * a.ldy + col, in ? left : 0);
                const bool ends = in && ((next_starts >> e & 1) || e + 1 == end);
                if (ends) flush |= 1u << i;
                if (kAdd) {
                    const bool whole = ends && !(long_head && e < head) &&
                                       !(long_tail && (int)e >= last);
                    old[i] = load_piece<kWideTable, float, kN>(
                        a.dtable + (uint64_t)word[i] * a.ldt + col, whole ? left : 0);
                }
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const uint32_t e = e0 + i;
                if (e >= end) break;
                float f[kN];
                unpack<T, kN>(p[i], f);
#pragma unroll
                for (int j = 0; j < kN; ++j) acc[j] += f[j];
                if (flush >> i & 1) {
                    float was[kN];
                    const bool to_head = long_head && e < head;
                    if (to_head || (long_tail && (int)e >= last)) {
                        float* q = a.part + ((uint64_t)chunk * 2 + (to_head ? 0 : 1)) * a.ldp + col;
                        store_piece<true, float, kN>(q, pack<float, kN>(acc), left);
                    } else {
                        if (kAdd) unpack<float, kN>(old[kAdd ? i : 0], was);
                        write_sums<kWideTable, kAdd, kN>(a.dtable + (uint64_t)word[i] * a.ldt + col,
                                                         acc, a.scale, was, left);
                    }
#pragma unroll
                    for (int j = 0; j < kN; ++j) acc[j] = 0.0f;
                }
            }
        }
    }
}

// The parts of a long run, 128 columns by a block: each warp sums an eighth of them in order, the
// first warp adds the eight.
template <bool kWideTable, bool kAdd>
__global__ void __launch_bounds__(kThreads) k_embed_join(const __grid_constant__ SumArgs a) {
    constexpr int kWarps = kThreads / 32;
    __shared__ float4 sm[kWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_dep_wait();
    grid_dep_launch();
    const uint32_t count = *a.list_count;
    const uint32_t tiles = (a.cols + 127) / 128;
    for (uint64_t u = blockIdx.x; u < (uint64_t)count * tiles; u += gridDim.x) {
        const uint32_t chunk = a.list[u / tiles], col = (uint32_t)(u % tiles) * 128 + lane * 4;
        const uint32_t left = col < a.cols ? a.cols - col : 0;
        const uint32_t word = a.key[chunk * 32 + 31];
        uint32_t lo = chunk * 32 + 32, hi = a.n;  // the run's end
        while (lo < hi) {
            const uint32_t mid = (lo + hi) >> 1;
            if (a.key[mid] <= word) lo = mid + 1; else hi = mid;
        }
        const uint32_t parts = (lo - 1) / 32 - chunk + 1, share = (parts + kWarps - 1) / kWarps;
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        const uint32_t from = min(parts, warp * share), to = min(parts, from + share);
        if (left)
#pragma unroll 8
            for (uint32_t i = from; i < to; ++i) {  // the first part starts the run
                const float4 v = __ldcs(reinterpret_cast<const float4*>(
                    a.part + ((uint64_t)(chunk + i) * 2 + (i == 0)) * a.ldp + col));
                s[0] += v.x;
                s[1] += v.y;
                s[2] += v.z;
                s[3] += v.w;
            }
        sm[warp][lane] = make_float4(s[0], s[1], s[2], s[3]);
        __syncthreads();
        if (warp == 0) {
            float old[4];
            float* out = a.dtable + (uint64_t)word * a.ldt + col;
            if (kAdd) unpack<float, 4>(load_piece<kWideTable, float, 4>(out, left), old);
            for (int w = 1; w < kWarps; ++w) {
                const float4 v = sm[w][lane];
                s[0] += v.x;
                s[1] += v.y;
                s[2] += v.z;
                s[3] += v.w;
            }
            write_sums<kWideTable, kAdd, 4>(out, s, a.scale, old, left);
        }
        __syncthreads();
    }
}

// ----------------------------------------------------------------------------------- host
struct BackwardLayout {
    uint32_t blocks, per_block, passes, digit_bits;
    size_t key[2], pos[2], counts, list, part, total;
    uint64_t ldp;
};
BackwardLayout backward_layout(uint64_t n, uint64_t vocab, uint64_t dim) {
    auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
    BackwardLayout L{};
    uint32_t bits = 1;
    while ((vocab >> bits) != 0) ++bits;  // keys 0 to vocab
    L.passes = (bits + 8) / 9;
    L.digit_bits = (bits + L.passes - 1) / L.passes;
    const uint64_t blocks =
        n <= kSortLeast ? 1 : std::min<uint64_t>(kSortMost, (n + 2047) / 2048);
    L.per_block = (uint32_t)(((n + blocks - 1) / blocks + kSortThreads - 1) / kSortThreads *
                             kSortThreads);
    L.blocks = L.per_block ? (uint32_t)((n + L.per_block - 1) / L.per_block) : 0;
    size_t at = 0;
    for (int i = 0; i < 2; ++i) {
        L.key[i] = at;
        at = up(at + n * 4);
        L.pos[i] = at;
        at = up(at + n * 4);
    }
    L.counts = at;
    at = up(at + (size_t)kSortMost * kDigits * 4);
    const uint64_t chunks = (n + 31) / 32;
    L.list = at;  // the count, then the chunks
    at = up(at + (chunks + 1) * 4);
    L.ldp = (dim + 3) & ~3ull;
    L.part = at;
    at = up(at + chunks * 2 * L.ldp * sizeof(float));
    L.total = at;
    return L;
}

template <typename T>
int launch_sums(const SumArgs& a, bool wide, bool wide_table, unsigned zero_blocks, unsigned join,
                cudaStream_t s) {
    auto pick = [&](auto w, auto wt, auto add) {
        return k_embed_sum<T, decltype(w)::value, decltype(wt)::value, decltype(add)::value>;
    };
    using Y = std::true_type;
    using N = std::false_type;
    auto kernel = a.accumulate
                      ? (wide ? (wide_table ? pick(Y{}, Y{}, Y{}) : pick(Y{}, N{}, Y{}))
                              : (wide_table ? pick(N{}, Y{}, Y{}) : pick(N{}, N{}, Y{})))
                      : (wide ? (wide_table ? pick(Y{}, Y{}, N{}) : pick(Y{}, N{}, N{}))
                              : (wide_table ? pick(N{}, Y{}, N{}) : pick(N{}, N{}, N{})));
    const int rc = launch_rows_kernel(kernel, dim3(a.sum_blocks + zero_blocks), kThreads, s, a);
    if (rc || !join) return rc;
    auto joiner = a.accumulate ? (wide_table ? k_embed_join<true, true> : k_embed_join<false, true>)
                               : (wide_table ? k_embed_join<true, false>
                                             : k_embed_join<false, false>);
    return launch_rows_kernel(joiner, dim3(join), kThreads, s, a);
}

int check_tokens(const dgc_tensor* t, Tokens* out) {
    if (!t || (t->dtype != DGC_I32 && t->dtype != DGC_I64) || t->n < 0) return DGC_EINVAL;
    if (t->n > kMaxExtent) return DGC_EUNSUPPORTED;
    *out = Tokens{t->data, t->dtype == DGC_I64};
    return check_vector(t, (uint64_t)t->n, t->dtype);
}

template <typename S, typename D>
int launch_embed(const EmbedArgs& a, bool wide, cudaStream_t s) {
    const uint64_t tiles = (a.walk.total + kThreads * kSteps - 1) / (kThreads * kSteps);
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
        for (uint32_t pass = 0; pass < L.passes; ++pass) {
            a.first = pass == 0;
            a.key = words(L.key[pass & 1]);
            a.pos = words(L.pos[pass & 1]);
            a.key_out = words(L.key[~pass & 1]);
            a.pos_out = words(L.pos[~pass & 1]);
            a.shift = pass * L.digit_bits;
            a.mask = (1u << L.digit_bits) - 1;
            a.list_count = pass + 1 == L.passes ? sum.list_count : nullptr;
            if (L.blocks > 1 &&
                (rc = launch_rows_kernel(k_sort_count, dim3(L.blocks), kSortThreads, s, a)))
                return rc;
            if ((rc = launch_rows_kernel(k_sort_move, dim3(L.blocks), kSortThreads, s, a)))
                return rc;
        }
        sum.key = a.key_out;
        sum.pos = a.pos_out;
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
    const uint32_t span = 32 * (uint32_t)(16 / my.entry());  // a warp's columns
    sum.tiles = (sum.cols + span - 1) / span;
    const uint64_t units = (uint64_t)((n + 31) / 32) * sum.tiles;
    sum.sum_blocks = (uint32_t)umin64((units + 7) / 8, 1u << 24);
    const uint64_t zeros = accumulate ? 0
                                      : ((mt.rows + kZeroRows - 1) / kZeroRows) *
                                            ((mt.cols + kZeroCols - 1) / kZeroCols);
    const unsigned zero_blocks = (unsigned)umin64(zeros, 1u << 24);
    // only a list of more than 32 tokens can hold a word more than 32 times
    const unsigned join = n > 32 ? (unsigned)umin64((uint64_t)sms * 2, (uint64_t)((n + 31) / 32) *
                                                                           ((mt.cols + 127) / 128))
                                 : 0;
    const bool wide = my.on(16), wide_table = mt.on(16);
    if (sum.sum_blocks + zero_blocks == 0) return DGC_OK;
    return with_type(my.dtype, [&](auto t) {
        return launch_sums<decltype(t)>(sum, wide, wide_table, zero_blocks, join, s);
    });
}
