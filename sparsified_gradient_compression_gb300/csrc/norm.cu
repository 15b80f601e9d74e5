// norm.cu -- layer norm and its backward pass (sm_103a).
//
//   mean, rstd = 1 / sqrt(var + eps) of a row; xhat = (x - mean) rstd
//   y  = xhat gamma + beta
//   g  = dy gamma;  dx = rstd (g - avg(g) - xhat avg(g xhat)) + residual
//   dgamma = sum over rows of dy xhat, dbeta = sum over rows of dy; written, or added
//
//   k_norm         a row by 1 to 16 warps, held in registers: one read, one write.
//   k_norm_long    rows that are too long for that: a block a row, read three times.
//   k_norm_back    persistent blocks: dx of a row after the other by 1 to 16 warps, and the
//                  block's own sums of the two columns' gradients in registers, written at the end.
//   k_norm_sums, k_norm_columns   the same for longer rows, in two kernels.
//   k_norm_join    adds the blocks' sums in order.
//
// Everything is binary32. A row's mean m is rounded, so x - m is off by the same amount in every
// column; the average c of x - m (the differences are exact next to the mean) is taken out again:
// the variance is avg((x-m)^2) - c^2 and xhat (x - m - c) rstd. Without it, a row whose mean is 2^12
// times its deviation would lose a dozen bits.
#include <algorithm>

#include "rows.cuh"

namespace dgc {
namespace {

constexpr int kMaxWarps = 16;

// Sums over the lanes of the `warps` warps that share a row (a power of two), in a fixed order.
// sm: room for kN * warps floats of this row's group, for this call alone (two calls on the same
// room have another call on other room between them). bar: the group's barrier.
template <int kN>
__device__ __forceinline__ void row_sums(float (&s)[kN], int warps, int warp, int bar, float* sm) {
#pragma unroll
    for (int i = 0; i < kN; ++i) s[i] = warp_sum(s[i]);
    if (warps == 1) return;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int i = 0; i < kN; ++i) sm[warp * kN + i] = s[i];
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(warps * 32) : "memory");
#pragma unroll
    for (int i = 0; i < kN; ++i) s[i] = sm[i];
    for (int w = 1; w < warps; ++w)
#pragma unroll
        for (int i = 0; i < kN; ++i) s[i] += sm[w * kN + i];
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
    uint32_t cols, warps;  // warps that share a row
    const float *gamma, *beta;
    int32_t wide_weights;
    float eps;
    float *mean, *rstd;
};

// The reciprocal deviation. A NaN stays one.
__device__ __forceinline__ float rstd_of(float squares, float c, float n, float eps) {
    float var = squares / n - c * c;
    if (var < 0.0f) var = 0.0f;
    return __frsqrt_rn(var + eps);
}

// Bound by HBM. kC: a lane's columns, in pieces of 16 bytes (kWide) or single entries.
template <typename T, bool kWide, int kC>
__global__ void __launch_bounds__(32 * kMaxWarps) k_norm(const __grid_constant__ NormArgs a) {
    constexpr int kN = kWide ? 16 / sizeof(T) : 1, kV = kC / kN;
    __shared__ float sm[2][2 * kMaxWarps];
    const int lane = threadIdx.x & 31, all = threadIdx.x >> 5;
    const int group = all / a.warps, warp = all % a.warps, groups = (blockDim.x >> 5) / a.warps;
    grid_dep_wait();
    grid_dep_launch();
    const float n = (float)a.cols;
    for (uint64_t row = (uint64_t)blockIdx.x * groups + group; row < a.rows;
         row += (uint64_t)gridDim.x * groups) {
        const T* x = static_cast<const T*>(a.x) + row * a.ldx;
        Packed<T, kN> p[kV];
        float f[kC];
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const uint32_t col = ((v * a.warps + warp) * 32 + lane) * kN;
            p[v] = load_piece<kWide, T, kN>(x + col, col < a.cols ? a.cols - col : 0);
        }
        float s[1] = {0.0f};
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            float t[kN];
            unpack<T, kN>(p[v], t);
#pragma unroll
            for (int j = 0; j < kN; ++j) {
                f[v * kN + j] = t[j];
                s[0] += t[j];
            }
        }
        row_sums(s, a.warps, warp, 1 + group, &sm[0][group * a.warps]);
        const float mean = s[0] / n;
        float q[2] = {0.0f, 0.0f};
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const uint32_t col = ((v * a.warps + warp) * 32 + lane) * kN;
#pragma unroll
            for (int j = 0; j < kN; ++j) {
                float& d = f[v * kN + j];
                d = col + j < a.cols ? d - mean : 0.0f;
                q[0] += d;
                q[1] = fmaf(d, d, q[1]);
            }
        }
        row_sums(q, a.warps, warp, 1 + group, &sm[1][2 * group * a.warps]);
        const float c = q[0] / n, rstd = rstd_of(q[1], c, n, a.eps);
        if (a.mean && warp == 0 && lane == 0) {
            a.mean[row] = mean + c;
            a.rstd[row] = rstd;
        }
        T* y = static_cast<T*>(a.y) + row * a.ldy;
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const uint32_t col = ((v * a.warps + warp) * 32 + lane) * kN;
            const uint32_t left = col < a.cols ? a.cols - col : 0;
            float g[kN], b[kN], t[kN];
            load_weights<kN>(a.gamma + col, left, a.wide_weights, g);
            if (a.beta) load_weights<kN>(a.beta + col, left, a.wide_weights, b);
#pragma unroll
            for (int j = 0; j < kN; ++j) {
                const float h = (f[v * kN + j] - c) * rstd;
                t[j] = a.beta ? fmaf(h, g[j], b[j]) : h * g[j];
            }
            store_piece<kWide, T, kN>(y + col, pack<T, kN>(t), left);
        }
    }
}

constexpr int kLongThreads = 512;
constexpr int kLongWarps = kLongThreads / 32;

// A column of a row, read again (from L2, as far as the row stays there).
template <typename T>
__device__ __forceinline__ float entry(const T* p, uint32_t i) {
    return Num<T>::up(p[i]);
}

template <typename T>
__global__ void __launch_bounds__(kLongThreads) k_norm_long(const __grid_constant__ NormArgs a) {
    __shared__ float sm[2][2 * kLongWarps];
    const int warp = threadIdx.x >> 5;
    grid_dep_wait();
    grid_dep_launch();
    const float n = (float)a.cols;
    for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + row * a.ldx;
        T* y = static_cast<T*>(a.y) + row * a.ldy;
        float s[1] = {0.0f};
#pragma unroll 8
        for (uint32_t i = threadIdx.x; i < a.cols; i += kLongThreads) s[0] += entry(x, i);
        row_sums(s, kLongWarps, warp, 1, sm[0]);
        const float mean = s[0] / n;
        float q[2] = {0.0f, 0.0f};
#pragma unroll 8
        for (uint32_t i = threadIdx.x; i < a.cols; i += kLongThreads) {
            const float d = entry(x, i) - mean;
            q[0] += d;
            q[1] = fmaf(d, d, q[1]);
        }
        row_sums(q, kLongWarps, warp, 1, sm[1]);
        const float c = q[0] / n, rstd = rstd_of(q[1], c, n, a.eps);
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
constexpr int kBackCols = 16;          // a lane's columns in k_norm_back
constexpr uint32_t kBackLongest = kBackCols * 32 * kMaxWarps;

struct NormBackArgs {
    const void *dy, *x, *residual;
    void* dx;
    uint64_t lddy, ldx, ldr, lddx, rows;
    uint32_t cols, warps;
    const float *gamma, *mean, *rstd;
    int32_t wide_weights;
    float* part;                   // [block][2][cols]: dgamma's and dbeta's
    uint32_t parts;
    float *dgamma, *dbeta;
    int32_t accumulate;
    float* row_sums;               // k_norm_sums: three a row
};

// What a row's sums make of it.
struct RowBack {
    float c, rstd, m1, m2;
    __device__ RowBack(const float (&s)[3], float rstd_, float n) : rstd(rstd_) {
        c = s[0] / n;                                // avg(x - mean)
        m1 = s[1] / n;                               // avg(g)
        m2 = rstd * ((s[2] - c * s[1]) / n);         // avg(g xhat)
    }
};

// Bound by HBM. The rows' loads do not wait for one another: with 16-bit entries the next row's are
// under way while a row's sums are exchanged.
template <typename T, bool kWide>
__global__ void __launch_bounds__(32 * kMaxWarps, 1)
    k_norm_back(const __grid_constant__ NormBackArgs a) {
    constexpr int kC = kBackCols, kN = kWide ? 16 / sizeof(T) : 1, kV = kC / kN;
    constexpr bool kAhead = sizeof(T) == 2;
    __shared__ float sm[2][3 * kMaxWarps];
    __shared__ float fold[8 * 32 * kC];  // groups * warps <= 8 where there are several groups
    const int lane = threadIdx.x & 31, all = threadIdx.x >> 5;
    const int group = all / a.warps, warp = all % a.warps, groups = (blockDim.x >> 5) / a.warps;
    grid_dep_wait();
    grid_dep_launch();
    const float n = (float)a.cols;
    const uint64_t step = (uint64_t)gridDim.x * groups;
    float dg[kC], db[kC], gamma[kC];
#pragma unroll
    for (int v = 0; v < kV; ++v) {
        const uint32_t col = ((v * a.warps + warp) * 32 + lane) * kN;
        float g[kN];
        load_weights<kN>(a.gamma + col, col < a.cols ? a.cols - col : 0, a.wide_weights, g);
#pragma unroll
        for (int j = 0; j < kN; ++j) {
            gamma[v * kN + j] = g[j];
            dg[v * kN + j] = db[v * kN + j] = 0.0f;
        }
    }
    struct Row {
        Packed<T, kN> x[kV], dy[kV], r[kV];
        float mean, rstd;
    };
    auto load = [&](Row& w, uint64_t row) {
        w.mean = a.mean[row];
        w.rstd = a.rstd[row];
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const uint32_t col = ((v * a.warps + warp) * 32 + lane) * kN;
            const uint32_t left = col < a.cols ? a.cols - col : 0;
            w.x[v] = load_piece<kWide, T, kN>(
                static_cast<const T*>(a.x) + row * a.ldx + col, left);
            w.dy[v] = load_piece<kWide, T, kN>(
                static_cast<const T*>(a.dy) + row * a.lddy + col, left);
            if (a.residual)
                w.r[v] = load_piece<kWide, T, kN>(
                    static_cast<const T*>(a.residual) + row * a.ldr + col, left);
        }
    };
    uint64_t row = (uint64_t)blockIdx.x * groups + group;
    Row next;
    if (kAhead && row < a.rows) load(next, row);
    for (int turn = 0; row < a.rows; row += step, turn ^= 1) {
        Row w;
        if (kAhead) {
            w = next;
            if (row + step < a.rows) load(next, row + step);
        } else {
            load(w, row);
        }
        float d[kC], dy[kC];
        float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const uint32_t col = ((v * a.warps + warp) * 32 + lane) * kN;
            float tx[kN], ty[kN];
            unpack<T, kN>(w.x[v], tx);
            unpack<T, kN>(w.dy[v], ty);
#pragma unroll
            for (int j = 0; j < kN; ++j) {
                const int i = v * kN + j;
                d[i] = col + j < a.cols ? tx[j] - w.mean : 0.0f;
                dy[i] = ty[j];
                const float g = ty[j] * gamma[i];
                s[0] += d[i];
                s[1] += g;
                s[2] = fmaf(g, d[i], s[2]);
            }
        }
        row_sums(s, a.warps, warp, 1 + group, &sm[turn][3 * group * a.warps]);
        const RowBack b(s, w.rstd, n);
        T* dx = static_cast<T*>(a.dx) + row * a.lddx;
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const uint32_t col = ((v * a.warps + warp) * 32 + lane) * kN;
            float t[kN], r[kN];
            if (a.residual) unpack<T, kN>(w.r[v], r);
#pragma unroll
            for (int j = 0; j < kN; ++j) {
                const int i = v * kN + j;
                const float h = (d[i] - b.c) * b.rstd;
                t[j] = b.rstd * (fmaf(dy[i], gamma[i], -b.m1) - h * b.m2);
                if (a.residual) t[j] += r[j];
                dg[i] = fmaf(dy[i], h, dg[i]);
                db[i] += dy[i];
            }
            store_piece<kWide, T, kN>(dx + col, pack<T, kN>(t), col < a.cols ? a.cols - col : 0);
        }
    }
    if (!a.dgamma && !a.dbeta) return;
    // the groups' sums, in order, then the block's into its part
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        if (groups > 1) {
            __syncthreads();
            for (int g = 1; g < groups; ++g) {
                if (group == g)
#pragma unroll
                    for (int i = 0; i < kC; ++i)
                        fold[(warp * kC + i) * 32 + lane] = q ? db[i] : dg[i];
                __syncthreads();
                if (group == 0)
#pragma unroll
                    for (int i = 0; i < kC; ++i)
                        (q ? db[i] : dg[i]) += fold[(warp * kC + i) * 32 + lane];
                __syncthreads();
            }
        }
        if (group == 0) {
            float* out = a.part + ((uint64_t)blockIdx.x * 2 + q) * a.cols;
#pragma unroll
            for (int v = 0; v < kV; ++v) {
                const uint32_t col = ((v * a.warps + warp) * 32 + lane) * kN;
#pragma unroll
                for (int j = 0; j < kN; ++j)
                    if (col + j < a.cols) out[col + j] = q ? db[v * kN + j] : dg[v * kN + j];
            }
        }
    }
}

// Longer rows: the three sums of every row, then strips of rows by column.
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
        row_sums(s, kLongWarps, threadIdx.x >> 5, 1, sm[turn]);
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
    const float gamma = a.gamma[col], n = (float)a.cols;
    const T* x = static_cast<const T*>(a.x) + col;
    const T* dy = static_cast<const T*>(a.dy) + col;
    const T* r = static_cast<const T*>(a.residual) + col;
    T* dx = static_cast<T*>(a.dx) + col;
    float dg = 0.0f, db = 0.0f;
#pragma unroll 4
    for (uint64_t row = begin; row < end; ++row) {
        const float s[3] = {a.row_sums[row * 3], a.row_sums[row * 3 + 1], a.row_sums[row * 3 + 2]};
        const RowBack b(s, a.rstd[row], n);
        const float y = Num<T>::up(dy[row * a.lddy]);
        const float h = (Num<T>::up(x[row * a.ldx]) - a.mean[row] - b.c) * b.rstd;
        float t = b.rstd * (fmaf(y, gamma, -b.m1) - h * b.m2);
        if (a.residual) t += Num<T>::up(r[row * a.ldr]);
        dx[row * a.lddx] = Num<T>::down(t);
        dg = fmaf(y, h, dg);
        db += y;
    }
    a.part[(uint64_t)blockIdx.y * 2 * a.cols + col] = dg;
    a.part[((uint64_t)blockIdx.y * 2 + 1) * a.cols + col] = db;
}

// 32 columns of dgamma or dbeta a block: each warp adds every eighth part, the first one the eight.
__global__ void __launch_bounds__(256) k_norm_join(const __grid_constant__ NormBackArgs a) {
    __shared__ float sm[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_dep_wait();
    grid_dep_launch();
    const uint32_t col = blockIdx.x * 32 + lane;
    float* out = blockIdx.y ? a.dbeta : a.dgamma;
    if (!out) return;
    float s = 0.0f;
    if (col < a.cols)
#pragma unroll 8
        for (uint32_t p = warp; p < a.parts; p += 8)
            s += a.part[((uint64_t)p * 2 + blockIdx.y) * a.cols + col];
    sm[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && col < a.cols) {
        for (int w = 1; w < 8; ++w) s += sm[w][lane];
        out[col] = a.accumulate ? out[col] + s : s;
    }
}

// ----------------------------------------------------------------------------------- host
// Warps that share a row of `cols` columns, kC a lane.
uint32_t warps_for(uint64_t cols, uint32_t per_lane) {
    uint32_t w = 1;
    while ((uint64_t)w * 32 * per_lane < cols) w *= 2;
    return w;
}

template <typename T, bool kWide>
int launch_norm(NormArgs a, cudaStream_t s) {
    const uint32_t per_lane = a.cols <= 256 ? 8 : a.cols <= 4096 ? 16 : 32;
    a.warps = warps_for(a.cols, per_lane);
    if (a.warps > kMaxWarps)
        return launch_rows_kernel(k_norm_long<T>, dim3((unsigned)umin64(a.rows, 1u << 24)),
                                  kLongThreads, s, a);
    const unsigned block = std::max(8u, a.warps);
    const uint64_t rows = block / a.warps;
    const dim3 grid((unsigned)((a.rows + rows - 1) / rows));
    auto kernel = per_lane == 8    ? k_norm<T, kWide, 8>
                  : per_lane == 16 ? k_norm<T, kWide, 16>
                                   : k_norm<T, kWide, 32>;
    return launch_rows_kernel(kernel, grid, block * 32, s, a);
}

uint64_t back_parts(uint64_t rows, uint64_t cols) {
    return cols > kBackLongest ? std::min<uint64_t>(64, (rows + 31) / 32) : kMaxParts;
}
size_t back_workspace(uint64_t rows, uint64_t cols) {
    const size_t part = back_parts(rows, cols) * 2 * cols * sizeof(float);
    return ((part + 255) & ~(size_t)255) + (cols > kBackLongest ? rows * 3 * sizeof(float) : 0);
}

template <typename T>
int launch_back(NormBackArgs a, bool wide, int sms, cudaStream_t s) {
    int rc;
    if (a.cols > kBackLongest) {
        a.parts = (uint32_t)back_parts(a.rows, a.cols);
        a.row_sums = a.part + ((a.parts * 2ull * a.cols + 63) & ~63ull);
        if ((rc = launch_rows_kernel(k_norm_sums<T>, dim3((unsigned)umin64(a.rows, 1u << 24)),
                                     kLongThreads, s, a)))
            return rc;
        if ((rc = launch_rows_kernel(k_norm_columns<T>, dim3((a.cols + 255) / 256, a.parts), 256, s,
                                     a)))
            return rc;
    } else {
        a.warps = warps_for(a.cols, kBackCols);
        const unsigned block = std::max(8u, a.warps), groups = block / a.warps;
        const uint64_t most = std::min<uint64_t>(kMaxParts, (uint64_t)sms * (block > 8 ? 1 : 2));
        a.parts = (uint32_t)umin64((a.rows + groups - 1) / groups, most);
        if ((rc = launch_rows_kernel(wide ? k_norm_back<T, true> : k_norm_back<T, false>,
                                     dim3(a.parts), block * 32, s, a)))
            return rc;
    }
    if (!a.dgamma && !a.dbeta) return DGC_OK;
    return launch_rows_kernel(k_norm_join, dim3((a.cols + 31) / 32, 2), 256, s, a);
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
    a.gamma = static_cast<const float*>(gamma->data);
    a.beta = beta ? static_cast<const float*>(beta->data) : nullptr;
    a.eps = eps;
    a.mean = mean;
    a.rstd = rstd;
    a.wide_weights = on16(a.gamma) && on16(a.beta);
    const bool wide = mx.on(16) && my.on(16);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return with_type(mx.dtype, [&](auto t) {
        using T = decltype(t);
        return wide ? launch_norm<T, true>(a, s) : launch_norm<T, false>(a, s);
    });
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
    a.gamma = static_cast<const float*>(gamma->data);
    a.mean = mean;
    a.rstd = rstd;
    a.part = static_cast<float*>(ws);
    a.accumulate = accumulate != 0;
    a.wide_weights = on16(a.gamma);
    const bool wide = my.on(16) && mx.on(16) && md.on(16) && (!residual || mr.on(16));
    return with_type(my.dtype, [&](auto t) { return launch_back<decltype(t)>(a, wide, sms, s); });
}
