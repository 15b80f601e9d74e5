// norm.cu -- layer norm and its backward pass (sm_103a).
//
//   mean, rstd = 1 / sqrt(var + eps) of a row; xhat = (x - mean) rstd
//   y  = xhat gamma + beta
//   g  = dy gamma;  dx = rstd (g - avg(g) - xhat avg(g xhat)) + residual
//   dgamma = sum over rows of dy xhat, dbeta = sum over rows of dy; written, or added
//
//   k_norm         a row by 1 to 16 warps, held in registers: one read, one write (k_norm_any: rows
//                  off 16-byte boundaries).
//   k_norm_long    rows of more than 8192 entries: a block a row, read three times.
//   k_norm_back    persistent blocks: dx of a row after the other by 1 to 16 warps, and the
//                  block's own sums of the two weights' gradients in registers, written at the end
//                  (k_norm_back_any: rows off 16-byte boundaries).
//   k_norm_sums, k_norm_columns   the same for longer rows, in two kernels.
//   k_norm_join    adds the blocks' sums in order.
//
// Everything is binary32. A row's mean m is rounded, so x - m is off by the same amount in every
// column; the average c of x - m (the differences are exact next to the mean) is taken out again:
// the variance is avg((x-m)^2) - c^2 and xhat (x - m - c) rstd. Without it, a row whose mean is 2^12
// times its deviation would lose a dozen bits. So any m near the mean will do, and a warp takes its
// own columns' mean: the warps that share a row meet at one barrier.
#include <algorithm>

#include "rows.cuh"

namespace dgc {
namespace {

constexpr int kMaxWarps = 16;

// Whether the group's warps have come here. A warp alone needs no barrier but its own.
template <int kShare>
__device__ __forceinline__ void group_sync(int bar) {
    if (kShare > 1)
        asm volatile("bar.sync %0, %1;" ::"r"(bar), "n"(kShare * 32) : "memory");
    else
        __syncwarp();
}

// Sum over kShare neighbouring lanes (a power of two); all get the same bits.
template <int kShare>
__device__ __forceinline__ float share_sum(float x) {
#pragma unroll
    for (int o = 1; o < kShare; o <<= 1) x += __shfl_xor_sync(kFull, x, o);
    return x;
}

// Sums over the lanes of the kShare warps that share a row, in a fixed order. sm: kN * kShare floats
// of this row's group, for this call alone (two calls on the same room have another call on other
// room between them). bar: the group's barrier.
template <int kShare, int kN>
__device__ __forceinline__ void row_sums(float (&s)[kN], int warp, int bar, float* sm) {
#pragma unroll
    for (int i = 0; i < kN; ++i) s[i] = warp_sum(s[i]);
    if (kShare == 1) return;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int i = 0; i < kN; ++i) sm[i * kShare + warp] = s[i];
    group_sync<kShare>(bar);
    // a lane a warp's sums, added over the lanes
#pragma unroll
    for (int i = 0; i < kN; ++i) s[i] = sm[i * kShare + (threadIdx.x & (kShare - 1))];
#pragma unroll
    for (int i = 0; i < kN; ++i) s[i] = share_sum<kShare>(s[i]);
}

// kN weights of a row of which `left` are left; wide: their array starts on a 16-byte boundary.
template <int kN>
__device__ __forceinline__ void load_weights(const float* p, uint32_t left, bool wide,
                                             float (&f)[kN]) {
    if (kN > 1 && wide)
        unpack<float, kN>(load_piece<true, float, kN, false>(p, left), f);
    else
        unpack<float, kN>(load_some<float, kN, false>(p, left), f);
}

struct NormArgs {
    const void* x;
    void* y;
    uint64_t ldx, ldy, rows;
    uint32_t cols;
    const float *gamma, *beta;
    int32_t wide_weights;
    float eps, inv_cols;
    float *mean, *rstd;
};

// The reciprocal deviation. A NaN stays one.
__device__ __forceinline__ float rstd_of(float var, float eps) {
    if (var < 0.0f) var = 0.0f;
    return __frsqrt_rn(var + eps);
}

// A lane's columns in the kernels that hold a row in registers, and their longest row.
constexpr int kC = 16;
constexpr uint32_t kLongest = kC * 32 * kMaxWarps;

// A warp's place: kShare warps share a row, the block's warps are so many groups. kN: entries of a
// piece.
template <int kShare, int kN>
struct Place {
    static constexpr int kV = kC / kN;  // a lane's pieces
    int lane, group, warp, groups;
    __device__ Place() {
        const int all = threadIdx.x >> 5;
        lane = threadIdx.x & 31;
        group = all / kShare;
        warp = all % kShare;
        groups = (int)(blockDim.x >> 5) / kShare;
    }
    // the first column of this lane's v-th piece
    __device__ uint32_t col(int v) const { return ((v * kShare + warp) * 32 + lane) * kN; }
    // how many columns of the row are this warp's
    __device__ uint32_t columns(uint32_t cols) const {
        uint32_t n = 0;
        for (int v = 0; v < kV; ++v) {
            const uint32_t first = (v * kShare + warp) * 32 * kN;
            n += first < cols ? min(cols - first, 32u * kN) : 0;
        }
        return n;
    }
};

// A lane's columns as pairs, kPairs of them a unit: a piece, or two pieces of one entry (kN 1).
template <typename T, int kN>
struct Lane {
    static constexpr int kPairs = kN == 1 ? 1 : kN / 2, kUnits = kC / 2 / kPairs;
    template <typename Load>
    __device__ static void read(int u, float2* f, Load load) {
        if constexpr (kN == 1) {
            float a[1], b[1];
            unpack<T, 1>(load(2 * u), a);
            unpack<T, 1>(load(2 * u + 1), b);
            f[0] = {a[0], b[0]};
        } else {
            const Packed<T, kN> p = load(u);
#pragma unroll
            for (int j = 0; j < kPairs; ++j) f[j] = pair_of<T, kN>(p, j);
        }
    }
    template <bool kFull, int kShare>
    __device__ static void write(int u, T* row, const Place<kShare, kN>& at, uint32_t cols,
                                 const float2* f) {
        if constexpr (kN == 1) {
            const float one[1] = {f[0].x}, two[1] = {f[0].y};
            store_some<T, 1>(row + at.col(2 * u), pack<T, 1>(one), at.col(2 * u) < cols);
            store_some<T, 1>(row + at.col(2 * u + 1), pack<T, 1>(two), at.col(2 * u + 1) < cols);
        } else {
            const uint32_t col = at.col(u);
            Packed<T, kN> p;
#pragma unroll
            for (int j = 0; j < kPairs; ++j) set_pair<T, kN>(p, j, f[j]);
            if (kFull)
                store_packed<T, kN>(row + col, p);
            else
                store_piece<true, T, kN>(row + col, p, col < cols ? cols - col : 0);
        }
    }
    template <typename Load>
    __device__ static void read_all(float2 (&f)[kC / 2], Load load) {
#pragma unroll
        for (int u = 0; u < kUnits; ++u) read(u, f + u * kPairs, load);
    }
};
// The column of a lane's i-th pair's first or second entry.
template <int kShare, int kN>
__device__ __forceinline__ uint32_t pair_col(const Place<kShare, kN>& at, int i, int second) {
    return kN == 1 ? at.col(2 * i + second) : at.col(2 * i / kN) + 2 * i % kN + second;
}

// Mean, deviation and result of a row that the group's lanes hold. kFull: every piece is whole.
// share: 1 / columns, the warp's.
// Each warp takes its columns' deviations from its own mean m_w; m_w - m_0 =: o_w moves them to
// those from the first warp's: the row's mean is m_0 + c, c = avg(d) + sum n_w o_w / n.
template <typename T, int kShare, int kN, bool kFull, typename Load>
__device__ __forceinline__ void norm_row(const NormArgs& a, const Place<kShare, kN>& at,
                                         uint64_t row, const float2 (&gamma)[kC / 2],
                                         const float2 (&beta)[kC / 2], float columns, float share,
                                         float4* sm, Load load) {
    float2 f[kC / 2], s = both(0.0f);
    using Cols = Lane<T, kN>;
    Cols::read_all(f, load);
#pragma unroll
    for (int i = 0; i < kC / 2; ++i) s = add2(s, f[i]);
    const float mean = warp_sum(s.x + s.y) * share;
    float2 q0 = both(0.0f), q1 = both(0.0f);
#pragma unroll
    for (int i = 0; i < kC / 2; ++i) {
        f[i] = add2(f[i], both(-mean));
        if (!kFull) {
            if (pair_col(at, i, 0) >= a.cols) f[i].x = 0.0f;
            if (pair_col(at, i, 1) >= a.cols) f[i].y = 0.0f;
        }
        q0 = add2(q0, f[i]);
        q1 = fma2(f[i], f[i], q1);
    }
    float sum = warp_sum(q0.x + q0.y), squares = warp_sum(q1.x + q1.y), first = mean;
    if (kShare > 1) {
        if (at.lane == 0) sm[at.warp] = make_float4(mean, sum, squares, columns);
        group_sync<kShare>(1 + at.group);
        first = sm[0].x;
        const float4 p = sm[at.lane & (kShare - 1)];
        const float o = p.w > 0.0f ? p.x - first : 0.0f;
        sum = fmaf(p.w, o, p.y);
        squares = share_sum<kShare>(fmaf(o, sum + p.y, p.z));  // d^2 + 2 o d + o^2, its columns'
        sum = share_sum<kShare>(sum);
    }
    const float c = sum * a.inv_cols;
    const float rstd = rstd_of(fmaf(squares, a.inv_cols, -c * c), a.eps);
    if (a.mean && at.warp == 0 && at.lane == 0) {
        a.mean[row] = first + c;
        a.rstd[row] = rstd;
    }
    const float2 shift = both(((mean - first) - c) * rstd);
#pragma unroll
    for (int i = 0; i < kC / 2; ++i)
        f[i] = fma2(fma2(f[i], both(rstd), shift), gamma[i], beta[i]);
#pragma unroll
    for (int u = 0; u < Cols::kUnits; ++u)
        Cols::template write<kFull>(u, static_cast<T*>(a.y) + row * a.ldy, at, a.cols,
                                    f + u * Cols::kPairs);
}

template <int kShare, int kN>
__device__ __forceinline__ void load_row_weights(const float* p, const Place<kShare, kN>& at,
                                                 uint32_t cols, bool wide, float2 (&f)[kC / 2]) {
    float t[kC / kN][kN];
#pragma unroll
    for (int v = 0; v < kC / kN; ++v) {
        const uint32_t col = at.col(v);
        load_weights<kN>(p + col, p && col < cols ? cols - col : 0, wide, t[v]);
    }
#pragma unroll
    for (int i = 0; i < kC / 2; ++i)
        f[i] = {t[2 * i / kN][2 * i % kN], t[(2 * i + 1) / kN][(2 * i + 1) % kN]};
}

// A ring of rows in shared memory: every lane's own pieces of kOperands matrices.
template <typename T, int kShare, int kOperands, int kStages>
struct RowRing {
    static constexpr int kN = 16 / sizeof(T), kV = kC / kN;
    static constexpr int kThreads = 32 * (kShare > 8 ? kShare : 8);
    static constexpr size_t kBytes = (size_t)kStages * kOperands * kV * kThreads * 16;
    uint4* words;
    __device__ uint4* at(int stage, int q, int v) const {
        return words + ((stage * kOperands + q) * kV + v) * kThreads + threadIdx.x;
    }
    __device__ Packed<T, kN> get(int stage, int q, int v) const {
        const uint4 w = *at(stage, q, v);
        return {{w.x, w.y, w.z, w.w}};
    }
    template <bool kFull>
    __device__ void fetch(int stage, int q, const T* row, const Place<kShare, kN>& place,
                          uint32_t cols) const {
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const uint32_t col = place.col(v);
            const uint32_t n = kFull ? kN : col < cols ? min(cols - col, (uint32_t)kN) : 0;
            copy_async<16>(at(stage, q, v), n ? row + col : row, n * sizeof(T));
        }
    }
};

// Bound by HBM: 16384 x 4096 bf16 44 us, 6.1 TB/s, with instructions issued in 60% of the clocks.
// The next rows are on their way to shared memory while one is computed, each lane's columns to a
// place of its own, so that no barrier but the sums' is needed and no register holds them. (Loads
// to registers, one row at a time: 111 us.)
template <typename T, int kShare, int kStages>
__global__ void __launch_bounds__(kShare > 8 ? 32 * kShare : 256, kShare > 8 ? 1 : 3)
    k_norm(const __grid_constant__ NormArgs a) {
    using Ring = RowRing<T, kShare, 1, kStages>;
    constexpr int kN = Ring::kN;
    extern __shared__ uint4 words[];
    __shared__ float4 sm[2][kMaxWarps];
    const Place<kShare, kN> at;
    const Ring ring{words};
    grid_dep_wait();
    grid_dep_launch();
    float2 gamma[kC / 2], beta[kC / 2];
    load_row_weights(a.gamma, at, a.cols, a.wide_weights, gamma);
    load_row_weights(a.beta, at, a.cols, a.wide_weights, beta);
    const uint64_t step = (uint64_t)gridDim.x * at.groups;
    uint64_t row = (uint64_t)blockIdx.x * at.groups + at.group;
    const float columns = (float)at.columns(a.cols);
    const float share = columns > 0.0f ? 1.0f / columns : 0.0f;
    auto rows = [&](auto full) {
        uint64_t ahead = row;  // the next row to fetch
        auto fetch = [&](int stage) {
            if (ahead < a.rows)
                ring.template fetch<decltype(full)::value>(
                    stage, 0, static_cast<const T*>(a.x) + ahead * a.ldx, at, a.cols);
            copy_commit();
            ahead += step;
        };
#pragma unroll
        for (int i = 0; i + 1 < kStages; ++i) fetch(i);
        int turn = 0;
        for (int stage = 0; row < a.rows; row += step, turn ^= 1) {
            fetch(stage == 0 ? kStages - 1 : stage - 1);
            copy_wait<kStages - 1>();
            norm_row<T, kShare, kN, decltype(full)::value>(
                a, at, row, gamma, beta, columns, share, &sm[turn][at.group * kShare],
                [&](int v) { return ring.get(stage, 0, v); });
            stage = stage + 1 == kStages ? 0 : stage + 1;
        }
    };
    if (at.col(Ring::kV - 1) - at.lane * kN + 32 * kN <= a.cols)
        rows(std::true_type{});
    else
        rows(std::false_type{});
    copy_wait<0>();
}

// Rows off 16-byte boundaries, entry by entry: 16384 x 4097 bf16 packed 468 us.
template <typename T, int kShare>
__global__ void __launch_bounds__(kShare > 8 ? 32 * kShare : 256)
    k_norm_any(const __grid_constant__ NormArgs a) {
    __shared__ float4 sm[2][kMaxWarps];
    const Place<kShare, 1> at;
    grid_dep_wait();
    grid_dep_launch();
    float2 gamma[kC / 2], beta[kC / 2];
    load_row_weights(a.gamma, at, a.cols, false, gamma);
    load_row_weights(a.beta, at, a.cols, false, beta);
    const float columns = (float)at.columns(a.cols);
    const float share = columns > 0.0f ? 1.0f / columns : 0.0f;
    int turn = 0;
    for (uint64_t row = (uint64_t)blockIdx.x * at.groups + at.group; row < a.rows;
         row += (uint64_t)gridDim.x * at.groups, turn ^= 1) {
        const T* x = static_cast<const T*>(a.x) + row * a.ldx;
        Packed<T, 1> p[kC];
#pragma unroll
        for (int v = 0; v < kC; ++v) {
            const uint32_t col = at.col(v);
            p[v] = load_some<T, 1>(x + col, col < a.cols ? 1 : 0);
        }
        norm_row<T, kShare, 1, false>(a, at, row, gamma, beta, columns, share,
                                      &sm[turn][at.group * kShare], [&](int v) { return p[v]; });
    }
}

constexpr int kLongThreads = 512;
constexpr int kLongWarps = kLongThreads / 32;

// A column of a row, read again (from L2, as far as the row stays there).
template <typename T>
__device__ __forceinline__ float entry(const T* p, uint32_t i) {
    return Num<T>::up(p[i]);
}

// 16384 x 12288 bf16: 259 us, 3.1 TB/s, bound by single entries' loads, three of each.
template <typename T>
__global__ void __launch_bounds__(kLongThreads) k_norm_long(const __grid_constant__ NormArgs a) {
    __shared__ float sm[2][2 * kLongWarps];
    const int warp = threadIdx.x >> 5;
    grid_dep_wait();
    grid_dep_launch();
    for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + row * a.ldx;
        T* y = static_cast<T*>(a.y) + row * a.ldy;
        float s[1] = {0.0f};
#pragma unroll 8
        for (uint32_t i = threadIdx.x; i < a.cols; i += kLongThreads) s[0] += entry(x, i);
        row_sums<kLongWarps>(s, warp, 1, sm[0]);
        const float mean = s[0] * a.inv_cols;
        float q[2] = {0.0f, 0.0f};
#pragma unroll 8
        for (uint32_t i = threadIdx.x; i < a.cols; i += kLongThreads) {
            const float d = entry(x, i) - mean;
            q[0] += d;
            q[1] = fmaf(d, d, q[1]);
        }
        row_sums<kLongWarps>(q, warp, 1, sm[1]);
        const float c = q[0] * a.inv_cols, rstd = rstd_of(fmaf(q[1], a.inv_cols, -c * c), a.eps);
        if (a.mean && threadIdx.x == 0) {
            a.mean[row] = mean + c;
            a.rstd[row] = rstd;
        }
#pragma unroll 4
        for (uint32_t i = threadIdx.x; i < a.cols; i += kLongThreads) {
            const float h = (entry(x, i) - mean - c) * rstd;
            y[i] = Num<T>::down(a.beta ? fmaf(h, a.gamma[i], a.beta[i]) : h * a.gamma[i]);
        }
    }
}

// ------------------------------------------------------------------------------- backward
constexpr uint32_t kMaxParts = 304;    // blocks that keep sums of their own (2 for each of 152 SMs)

struct NormBackArgs {
    const void *dy, *x, *residual;
    void* dx;
    uint64_t lddy, ldx, ldr, lddx, rows;
    uint32_t cols;
    float inv_cols;
    const float *gamma, *mean, *rstd;
    int32_t wide_weights;
    float* part;                   // [block][2][cols]: dgamma's and dbeta's
    uint32_t parts;
    float *dgamma, *dbeta;
    int32_t accumulate;
    float* row_sums;               // k_norm_sums: three a row
};

// What a row's sums make of it: dx = dy gamma p - x' q - o for x' = x - mean, and xhat = (x' - c) p.
struct RowBack {
    float c, p, q, o;
    __device__ RowBack(const float (&s)[3], float rstd, float inv_n) : p(rstd) {
        c = s[0] * inv_n;                                    // avg(x')
        const float m1 = s[1] * inv_n;                       // avg(g)
        const float m2 = rstd * ((s[2] - c * s[1]) * inv_n); // avg(g xhat)
        q = rstd * rstd * m2;
        o = fmaf(-c, q, rstd * m1);
    }
};

// dx of a row that the group's lanes hold, and its part of the weights' gradients. kFull: every piece
// is whole.
template <typename T, int kShare, int kN, bool kFull, typename Load>
__device__ __forceinline__ void back_row(const NormBackArgs& a, const Place<kShare, kN>& at,
                                         uint64_t row, const float2 (&gamma)[kC / 2],
                                         float2 (&dg)[kC / 2], float2 (&db)[kC / 2], float mean,
                                         float rstd, float* sm, Load load) {
    float2 d[kC / 2], dy[kC / 2], s0 = both(0.0f), s1 = both(0.0f), s2 = both(0.0f);
    using Cols = Lane<T, kN>;
    Cols::read_all(d, [&](int v) { return load(0, v); });
    Cols::read_all(dy, [&](int v) { return load(1, v); });
#pragma unroll
    for (int i = 0; i < kC / 2; ++i) {
        d[i] = add2(d[i], both(-mean));
        if (!kFull) {
            if (pair_col(at, i, 0) >= a.cols) d[i].x = 0.0f;
            if (pair_col(at, i, 1) >= a.cols) d[i].y = 0.0f;
        }
        const float2 g = mul2(dy[i], gamma[i]);
        s0 = add2(s0, d[i]);
        s1 = add2(s1, g);
        s2 = fma2(g, d[i], s2);
    }
    float s[3] = {s0.x + s0.y, s1.x + s1.y, s2.x + s2.y};
    row_sums<kShare>(s, at.warp, 1 + at.group, sm);
    const RowBack b(s, rstd, a.inv_cols);
    const float2 p = both(b.p), q = both(-b.q), o = both(-b.o), cp = both(-b.c * b.p);
    T* dx = static_cast<T*>(a.dx) + row * a.lddx;
#pragma unroll
    for (int u = 0; u < Cols::kUnits; ++u) {
        float2 t[Cols::kPairs], r[Cols::kPairs];
        if (a.residual) Cols::read(u, r, [&](int v) { return load(2, v); });
#pragma unroll
        for (int j = 0; j < Cols::kPairs; ++j) {
            const int i = u * Cols::kPairs + j;
            t[j] = fma2(mul2(dy[i], gamma[i]), p, fma2(d[i], q, o));
            if (a.residual) t[j] = add2(t[j], r[j]);
            dg[i] = fma2(dy[i], fma2(d[i], p, cp), dg[i]);
            db[i] = add2(db[i], dy[i]);
        }
        Cols::template write<kFull>(u, dx, at, a.cols, t);
    }
}

// The groups' sums of the weights' gradients, in order, then the block's into its part.
template <int kShare, int kN>
__device__ __forceinline__ void write_part(const NormBackArgs& a, const Place<kShare, kN>& at,
                                           float2 (&dg)[kC / 2], float2 (&db)[kC / 2],
                                           float2* fold) {
    if (!a.dgamma && !a.dbeta) return;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        for (int g = 1; g < at.groups; ++g) {
            __syncthreads();
            if (at.group == g)
#pragma unroll
                for (int i = 0; i < kC / 2; ++i)
                    fold[(at.warp * kC / 2 + i) * 32 + at.lane] = q ? db[i] : dg[i];
            __syncthreads();
            if (at.group == 0)
#pragma unroll
                for (int i = 0; i < kC / 2; ++i) {
                    float2& s = q ? db[i] : dg[i];
                    s = add2(s, fold[(at.warp * kC / 2 + i) * 32 + at.lane]);
                }
        }
        if (at.group == 0) {
            float* out = a.part + ((uint64_t)blockIdx.x * 2 + q) * a.cols;
#pragma unroll
            for (int i = 0; i < kC / 2; ++i) {
                const uint32_t col0 = pair_col(at, i, 0);
                const uint32_t col1 = pair_col(at, i, 1);
                if (col0 < a.cols) out[col0] = q ? db[i].x : dg[i].x;
                if (col1 < a.cols) out[col1] = q ? db[i].y : dg[i].y;
            }
        }
    }
}

// Bound by HBM: 16384 x 4096 bf16 with a residual 93 us with the join, 5.8 TB/s (binary32 165 us, 6.5
// TB/s). As k_norm: the next rows of the three operands are on their way to shared memory. Two blocks an
// SM leave 128 registers: 16-bit types spill 56 to 76 bytes a thread, binary32 8 to 20. One block an SM
// spills nothing and has half the rows under way: 96.5 us for 94, but 49 for 51 with 16384 x 2048 and 47
// for 57 with 65536 x 512.
template <typename T, int kShare, int kStages>
__global__ void __launch_bounds__(kShare > 8 ? 32 * kShare : 256, kShare > 8 ? 1 : 2)
    k_norm_back(const __grid_constant__ NormBackArgs a) {
    using Ring = RowRing<T, kShare, 3, kStages>;
    constexpr int kN = Ring::kN;
    extern __shared__ uint4 words[];  // the ring, then the groups' sums
    __shared__ float sm[2][3 * kMaxWarps];
    const Place<kShare, kN> at;
    const Ring ring{words};
    grid_dep_wait();
    grid_dep_launch();
    float2 dg[kC / 2], db[kC / 2], gamma[kC / 2];
    load_row_weights(a.gamma, at, a.cols, a.wide_weights, gamma);
#pragma unroll
    for (int i = 0; i < kC / 2; ++i) dg[i] = db[i] = both(0.0f);
    const uint64_t step = (uint64_t)gridDim.x * at.groups;
    uint64_t row = (uint64_t)blockIdx.x * at.groups + at.group;
    auto rows = [&](auto full) {
        constexpr bool kFull = decltype(full)::value;
        uint64_t ahead = row;  // the next row to fetch
        auto fetch = [&](int stage) {
            if (ahead < a.rows) {
                ring.template fetch<kFull>(stage, 0, static_cast<const T*>(a.x) + ahead * a.ldx, at,
                                           a.cols);
                ring.template fetch<kFull>(stage, 1, static_cast<const T*>(a.dy) + ahead * a.lddy,
                                           at, a.cols);
                if (a.residual)
                    ring.template fetch<kFull>(
                        stage, 2, static_cast<const T*>(a.residual) + ahead * a.ldr, at, a.cols);
            }
            copy_commit();
            ahead += step;
        };
#pragma unroll
        for (int i = 0; i + 1 < kStages; ++i) fetch(i);
        float mean = 0.0f, rstd = 0.0f;
        int turn = 0, of = 32;
        for (int stage = 0; row < a.rows; row += step, turn ^= 1) {
            fetch(stage == 0 ? kStages - 1 : stage - 1);
            // the statistics of 32 rows at a time, a lane a row's: a load for each row, even one
            // row ahead, held the copies up (16384 x 4096: 129 us for 101)
            if (of == 32) {
                of = 0;
                const uint64_t mine = row + at.lane * step;
                mean = mine < a.rows ? a.mean[mine] : 0.0f;
                rstd = mine < a.rows ? a.rstd[mine] : 0.0f;
            }
            copy_wait<kStages - 1>();
            back_row<T, kShare, kN, kFull>(
                a, at, row, gamma, dg, db, __shfl_sync(dgc::kFull, mean, of),
                __shfl_sync(dgc::kFull, rstd, of), &sm[turn][3 * at.group * kShare],
                [&](int q, int v) { return ring.get(stage, q, v); });
            ++of;
            stage = stage + 1 == kStages ? 0 : stage + 1;
        }
    };
    if (at.col(Ring::kV - 1) - at.lane * kN + 32 * kN <= a.cols)
        rows(std::true_type{});
    else
        rows(std::false_type{});
    copy_wait<0>();
    write_part(a, at, dg, db, reinterpret_cast<float2*>(words));
}

// Rows off 16-byte boundaries, entry by entry: 16384 x 4097 bf16 packed with a residual 525 us.
template <typename T, int kShare>
__global__ void __launch_bounds__(kShare > 8 ? 32 * kShare : 256, 1)
    k_norm_back_any(const __grid_constant__ NormBackArgs a) {
    __shared__ float2 fold[8 * 32 * kC / 2];
    __shared__ float sm[2][3 * kMaxWarps];
    const Place<kShare, 1> at;
    grid_dep_wait();
    grid_dep_launch();
    float2 dg[kC / 2], db[kC / 2], gamma[kC / 2];
    load_row_weights(a.gamma, at, a.cols, false, gamma);
#pragma unroll
    for (int i = 0; i < kC / 2; ++i) dg[i] = db[i] = both(0.0f);
    int turn = 0;
    for (uint64_t row = (uint64_t)blockIdx.x * at.groups + at.group; row < a.rows;
         row += (uint64_t)gridDim.x * at.groups, turn ^= 1) {
        const T* p[3] = {static_cast<const T*>(a.x) + row * a.ldx,
                         static_cast<const T*>(a.dy) + row * a.lddy,
                         static_cast<const T*>(a.residual) + row * a.ldr};
        Packed<T, 1> w[2][kC];
#pragma unroll
        for (int v = 0; v < kC; ++v) {
            const uint32_t col = at.col(v);
            w[0][v] = load_some<T, 1>(p[0] + col, col < a.cols ? 1 : 0);
            w[1][v] = load_some<T, 1>(p[1] + col, col < a.cols ? 1 : 0);
        }
        back_row<T, kShare, 1, false>(a, at, row, gamma, dg, db, a.mean[row], a.rstd[row],
                                      &sm[turn][3 * at.group * kShare], [&](int q, int v) {
                                          if (q < 2) return w[q & 1][v];
                                          const uint32_t col = at.col(v);
                                          return load_some<T, 1>(p[2] + col, col < a.cols ? 1 : 0);
                                      });
    }
    write_part(a, at, dg, db, fold);
}

// Longer rows: the three sums of every row, then strips of rows by column. 16384 x 12288 bf16 with a
// residual 1314 us, 1.2 TB/s: single entries, x and dy read twice, and a row's coefficients computed anew
// for every column.
template <typename T>
__global__ void __launch_bounds__(kLongThreads) k_norm_sums(const __grid_constant__ NormBackArgs a) {
    __shared__ float sm[2][3 * kLongWarps];
    grid_dep_wait();
    grid_dep_launch();
    int turn = 0;
    for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
        const T* x = static_cast<const T*>(a.x) + row * a.ldx;
        const T* dy = static_cast<const T*>(a.dy) + row * a.lddy;
        const float mean = a.mean[row];
        float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll 4
        for (uint32_t i = threadIdx.x; i < a.cols; i += kLongThreads) {
            const float d = entry(x, i) - mean, g = entry(dy, i) * a.gamma[i];
            s[0] += d;
            s[1] += g;
            s[2] = fmaf(g, d, s[2]);
        }
        row_sums<kLongWarps>(s, threadIdx.x >> 5, 1, sm[turn]);
        if (threadIdx.x < 3) a.row_sums[row * 3 + threadIdx.x] = s[threadIdx.x];
    }
}

// blockIdx.x: 256 columns; blockIdx.y: a strip of rows, and its part.
template <typename T>
__global__ void __launch_bounds__(256) k_norm_columns(const __grid_constant__ NormBackArgs a) {
    grid_dep_wait();
    grid_dep_launch();
    const uint32_t col = blockIdx.x * 256 + threadIdx.x;
    if (col >= a.cols) return;
    const uint64_t share = (a.rows + a.parts - 1) / a.parts;
    const uint64_t begin = blockIdx.y * share, end = umin64(a.rows, begin + share);
    const float gamma = a.gamma[col];
    const T* x = static_cast<const T*>(a.x) + col;
    const T* dy = static_cast<const T*>(a.dy) + col;
    const T* r = static_cast<const T*>(a.residual) + col;
    T* dx = static_cast<T*>(a.dx) + col;
    float dg = 0.0f, db = 0.0f;
#pragma unroll 4
    for (uint64_t row = begin; row < end; ++row) {
        const float s[3] = {a.row_sums[row * 3], a.row_sums[row * 3 + 1], a.row_sums[row * 3 + 2]};
        const RowBack b(s, a.rstd[row], a.inv_cols);
        const float y = Num<T>::up(dy[row * a.lddy]);
        const float d = Num<T>::up(x[row * a.ldx]) - a.mean[row];
        float t = fmaf(y * gamma, b.p, -fmaf(d, b.q, b.o));
        if (a.residual) t += Num<T>::up(r[row * a.ldr]);
        dx[row * a.lddx] = Num<T>::down(t);
        dg = fmaf(y, (d - b.c) * b.p, dg);
        db += y;
    }
    a.part[(uint64_t)blockIdx.y * 2 * a.cols + col] = dg;
    a.part[((uint64_t)blockIdx.y * 2 + 1) * a.cols + col] = db;
}

// 32 columns of dgamma or dbeta a block: each of 32 warps adds every 32nd part, the first one theirs.
// Latency: the parts come from L2 (16384 x 4096: 304 of them; fewer warps cost 7 us more).
constexpr int kJoinWarps = 32;
__global__ void __launch_bounds__(32 * kJoinWarps) k_norm_join(const __grid_constant__ NormBackArgs a) {
    __shared__ float sm[kJoinWarps][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_dep_wait();
    grid_dep_launch();
    float* out = blockIdx.y ? a.dbeta : a.dgamma;
    if (!out) return;
    const uint32_t col = blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (col < a.cols)
#pragma unroll 10
        for (uint32_t p = warp; p < a.parts; p += kJoinWarps)
            s += a.part[((uint64_t)p * 2 + blockIdx.y) * a.cols + col];
    sm[warp][lane] = s;
    __syncthreads();
    s = warp_sum(sm[lane][warp]);  // of this block's column `warp`
    const uint32_t mine = blockIdx.x * 32 + warp;
    if (lane == 0 && mine < a.cols) out[mine] = a.accumulate ? out[mine] + s : s;
}

// ----------------------------------------------------------------------------------- host
// f with the number of warps that share a row of `cols` columns: f(std::integral_constant).
template <typename F>
int with_share(uint64_t cols, F f) {
    if (cols <= 32 * kC) return f(std::integral_constant<int, 1>{});
    if (cols <= 64 * kC) return f(std::integral_constant<int, 2>{});
    if (cols <= 128 * kC) return f(std::integral_constant<int, 4>{});
    if (cols <= 256 * kC) return f(std::integral_constant<int, 8>{});
    return f(std::integral_constant<int, kMaxWarps>{});
}

template <typename T>
int launch_norm(const NormArgs& a, bool wide, int sms, cudaStream_t s) {
    if (a.cols > kLongest)
        return launch_rows_kernel(k_norm_long<T>, dim3((unsigned)umin64(a.rows, 1u << 24)),
                                  kLongThreads, s, a);
    return with_share(a.cols, [&](auto share) {
        constexpr int kShare = decltype(share)::value, kStages = sizeof(T) == 2 ? 4 : 3;
        using Ring = RowRing<T, kShare, 1, kStages>;
        const uint64_t rows = Ring::kThreads / 32 / kShare, groups = (a.rows + rows - 1) / rows;
        if (!wide)
            return launch_rows_kernel(k_norm_any<T, kShare>, dim3((unsigned)groups),
                                      Ring::kThreads, s, a);
        const dim3 grid((unsigned)umin64(groups, (uint64_t)sms * (kShare > 8 ? 1 : 3)));
        return launch_shared_kernel(k_norm<T, kShare, kStages>, grid, Ring::kThreads, Ring::kBytes,
                                    s, a);
    });
}

uint64_t back_parts(uint64_t rows, uint64_t cols) {
    return cols > kLongest ? std::min<uint64_t>(64, (rows + 31) / 32) : kMaxParts;
}
size_t back_workspace(uint64_t rows, uint64_t cols) {
    const size_t part = back_parts(rows, cols) * 2 * cols * sizeof(float);
    return ((part + 255) & ~(size_t)255) + (cols > kLongest ? rows * 3 * sizeof(float) : 0);
}

template <typename T>
int launch_back(NormBackArgs a, bool wide, int sms, cudaStream_t s) {
    int rc;
    if (a.cols > kLongest) {
        a.parts = (uint32_t)back_parts(a.rows, a.cols);
        a.row_sums = a.part + ((a.parts * 2ull * a.cols + 63) & ~63ull);
        if ((rc = launch_rows_kernel(k_norm_sums<T>, dim3((unsigned)umin64(a.rows, 1u << 24)),
                                     kLongThreads, s, a)))
            return rc;
        if ((rc = launch_rows_kernel(k_norm_columns<T>, dim3((a.cols + 255) / 256, a.parts), 256, s,
                                     a)))
            return rc;
    } else {
        rc = with_share(a.cols, [&](auto share) {
            constexpr int kShare = decltype(share)::value, kStages = sizeof(T) == 2 ? 3 : 2;
            using Ring = RowRing<T, kShare, 3, kStages>;
            const uint64_t groups = Ring::kThreads / 32 / kShare;
            const uint64_t most =
                std::min<uint64_t>(kMaxParts, (uint64_t)sms * (kShare > 8 ? 1 : 2));
            a.parts = (uint32_t)umin64((a.rows + groups - 1) / groups, most);
            return wide ? launch_shared_kernel(k_norm_back<T, kShare, kStages>, dim3(a.parts),
                                               Ring::kThreads, Ring::kBytes, s, a)
                        : launch_rows_kernel(k_norm_back_any<T, kShare>, dim3(a.parts),
                                             Ring::kThreads, s, a);
        });
        if (rc) return rc;
    }
    if (!a.dgamma && !a.dbeta) return DGC_OK;
    return launch_rows_kernel(k_norm_join, dim3((a.cols + 31) / 32, 2), 32 * kJoinWarps, s,
                              a);
}

__global__ void __launch_bounds__(256) k_norm_zero(float* dgamma, float* dbeta, uint32_t cols) {
    grid_dep_wait();
    grid_dep_launch();
    const uint32_t col = blockIdx.x * 256 + threadIdx.x;
    if (col >= cols) return;
    if (dgamma) dgamma[col] = 0.0f;
    if (dbeta) dbeta[col] = 0.0f;
}

}  // namespace
}  // namespace dgc

using namespace dgc;

static bool on16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

extern "C" int dgc_layer_norm(const dgc_matrix* x, const dgc_tensor* gamma, const dgc_tensor* beta,
                              float eps, const dgc_matrix* y, float* mean, float* rstd,
                              dgc_stream_t stream) {
    Rows mx, my;
    int rc;
    if (!x || !(eps > 0.0f && eps <= 3.4028234e38f) || (mean == nullptr) != (rstd == nullptr) ||
        (((uintptr_t)mean | (uintptr_t)rstd) & 3u))
        return DGC_EINVAL;
    if ((rc = check_rows(x, &mx, -1)) || (rc = check_rows(y, &my, mx.dtype))) return rc;
    if (!my.shaped(mx.rows, mx.cols)) return DGC_EINVAL;
    if ((rc = check_vector(gamma, mx.cols, DGC_F32))) return rc;
    if (beta && (rc = check_vector(beta, mx.cols, DGC_F32))) return rc;
    if (mx.rows == 0 || mx.cols == 0) return DGC_OK;
    NormArgs a{};
    a.x = mx.p;
    a.ldx = mx.ld;
    a.y = my.p;
    a.ldy = my.ld;
    a.rows = mx.rows;
    a.cols = (uint32_t)mx.cols;
    a.inv_cols = 1.0f / (float)mx.cols;
    a.gamma = static_cast<const float*>(gamma->data);
    a.beta = beta ? static_cast<const float*>(beta->data) : nullptr;
    a.eps = eps;
    a.mean = mean;
    a.rstd = rstd;
    a.wide_weights = on16(a.gamma) && on16(a.beta);
    const bool wide = mx.on(16) && my.on(16);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int sms = dgc_internal_sm_count();
    if (sms <= 0) return DGC_ECUDA;
    return with_type(mx.dtype, [&](auto t) { return launch_norm<decltype(t)>(a, wide, sms, s); });
}

extern "C" int dgc_layer_norm_backward_workspace(int64_t rows, int64_t cols, size_t* bytes) {
    if (!bytes || rows < 0 || cols < 0) return DGC_EINVAL;
    if (rows > kMaxExtent || cols > kMaxExtent) return DGC_EUNSUPPORTED;
    *bytes = back_workspace((uint64_t)rows, (uint64_t)cols);
    return DGC_OK;
}

extern "C" int dgc_layer_norm_backward(const dgc_matrix* dy, const dgc_matrix* x,
                                       const dgc_tensor* gamma, const float* mean,
                                       const float* rstd, const dgc_matrix* residual,
                                       const dgc_matrix* dx, const dgc_tensor* dgamma,
                                       const dgc_tensor* dbeta, int32_t accumulate, void* ws,
                                       size_t ws_bytes, dgc_stream_t stream) {
    Rows my, mx, mr, md;
    int rc;
    if (!dy) return DGC_EINVAL;
    if ((rc = check_rows(dy, &my, -1)) || (rc = check_rows(x, &mx, my.dtype)) ||
        (rc = check_rows(dx, &md, my.dtype)))
        return rc;
    if (residual && (rc = check_rows(residual, &mr, my.dtype))) return rc;
    const uint64_t rows = my.rows, cols = my.cols;
    if (!mx.shaped(rows, cols) || !md.shaped(rows, cols) || (residual && !mr.shaped(rows, cols)))
        return DGC_EINVAL;
    if ((rc = check_vector(gamma, cols, DGC_F32))) return rc;
    if (dgamma && (rc = check_vector(dgamma, cols, DGC_F32))) return rc;
    if (dbeta && (rc = check_vector(dbeta, cols, DGC_F32))) return rc;
    if (rows && (!mean || !rstd || (((uintptr_t)mean | (uintptr_t)rstd) & 3u))) return DGC_EINVAL;
    const size_t need = back_workspace(rows, cols);
    if (ws_bytes < need || (need && (!ws || ((uintptr_t)ws & 255u)))) return DGC_EINVAL;
    if (cols == 0) return DGC_OK;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    NormBackArgs a{};
    a.dgamma = dgamma ? static_cast<float*>(dgamma->data) : nullptr;
    a.dbeta = dbeta ? static_cast<float*>(dbeta->data) : nullptr;
    if (rows == 0) {
        if (accumulate || (!a.dgamma && !a.dbeta)) return DGC_OK;
        return launch_rows_kernel(k_norm_zero, dim3((unsigned)((cols + 255) / 256)), 256, s,
                                  a.dgamma, a.dbeta, (uint32_t)cols);
    }
    const int sms = dgc_internal_sm_count();
    if (sms <= 0) return DGC_ECUDA;
    a.dy = my.p;
    a.lddy = my.ld;
    a.x = mx.p;
    a.ldx = mx.ld;
    if (residual) {
        a.residual = mr.p;
        a.ldr = mr.ld;
    }
    a.dx = md.p;
    a.lddx = md.ld;
    a.rows = rows;
    a.cols = (uint32_t)cols;
    a.inv_cols = 1.0f / (float)cols;
    a.gamma = static_cast<const float*>(gamma->data);
    a.mean = mean;
    a.rstd = rstd;
    a.part = static_cast<float*>(ws);
    a.accumulate = accumulate != 0;
    a.wide_weights = on16(a.gamma);
    const bool wide = my.on(16) && mx.on(16) && md.on(16) && (!residual || mr.on(16));
    return with_type(my.dtype, [&](auto t) { return launch_back<decltype(t)>(a, wide, sms, s); });
}
