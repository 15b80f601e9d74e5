// dropout.cu -- dropout with a mask that is computed where it is needed and never stored (sm_103a).
//
//   key  = mix64(seed + G (1 + *step))              mix64: SplitMix64's output function, G its
//   word = mix64(key + G (row ceil(cols/4) + col/4 + 1))                               increment
//   kept where bits 16 (col % 4) .. + 15 of the word >= threshold = floor(65536 p + 1/2)
//   out  = [residual +] (kept ? x 65536 / (65536 - threshold) : 0)
//
// The generator is counter-based: an entry's bits depend on its row and column alone, not on
// strides, types or the launch. The backward pass is the same call on the gradient.
#include "rows.cuh"

namespace dgc {
namespace {

constexpr int kThreads = 256;
constexpr int kSteps = 4;  // pieces of 16 bytes a thread has in flight

struct DropArgs {
    const void *x, *residual;
    void* out;
    uint64_t ldx, ldr, ldo;
    PieceWalk walk;
    uint32_t cols, words;
    uint64_t seed;
    const uint64_t* step;
    uint32_t threshold;
    float scale;
};

// Bound by HBM: 8192 x 11264 bf16 with a residual 81 us, 6.8 TB/s, as fast as a plain copy. A word
// of the generator costs some 20 instructions and serves four entries; instructions are issued in
// 64% of the clocks (with 32 bits an entry, 16-bit types would be bound by them).
template <typename T, bool kResidual, bool kWide>
__global__ void __launch_bounds__(kThreads) k_dropout(const __grid_constant__ DropArgs a) {
    constexpr int kN = 16 / sizeof(T);
    grid_dep_wait();
    grid_dep_launch();
    const uint64_t key = mix64(a.seed + kGolden * (1 + (a.step ? *a.step : 0)));
    const T* x = static_cast<const T*>(a.x);
    const T* r = static_cast<const T*>(a.residual);
    T* out = static_cast<T*>(a.out);
    constexpr uint64_t kTile = kThreads * kSteps;
    for (uint64_t tile = blockIdx.x; tile * kTile < a.walk.total; tile += gridDim.x) {
        Pieces<kThreads, kSteps> at(a.walk, tile);
        const uint64_t first = tile * kTile + threadIdx.x;
        uint64_t row[kSteps];
        uint32_t col[kSteps], left[kSteps];
        Packed<T, kN> px[kSteps], pr[kSteps];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            row[i] = at.row;
            col[i] = at.at * kN;
            left[i] = first + i * kThreads < a.walk.total ? a.cols - col[i] : 0;
            px[i] = load_piece<kWide, T, kN>(x + row[i] * a.ldx + col[i], left[i]);
            if (kResidual) pr[i] = load_piece<kWide, T, kN>(r + row[i] * a.ldr + col[i], left[i]);
            at.next(a.walk);
        }
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            float f[kN], g[kN];
            unpack<T, kN>(px[i], f);
            if (kResidual) unpack<T, kN>(pr[i], g);
            uint64_t z = key + kGolden * (row[i] * a.words + (col[i] >> 2) + 1);
#pragma unroll
            for (int j = 0; j < kN; j += 4, z += kGolden) {
                const uint64_t w = mix64(z);
                const uint32_t lo = (uint32_t)w, hi = (uint32_t)(w >> 32);
                const uint32_t bits[4] = {lo & 0xFFFFu, lo >> 16, hi & 0xFFFFu, hi >> 16};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const bool kept = bits[k] >= a.threshold;
                    if (kResidual)
                        f[j + k] = kept ? fmaf(f[j + k], a.scale, g[j + k]) : g[j + k];
                    else
                        f[j + k] = kept ? f[j + k] * a.scale : 0.0f;
                }
            }
            store_piece<kWide, T, kN>(out + row[i] * a.ldo + col[i], pack<T, kN>(f), left[i]);
        }
    }
}

template <typename T>
int launch(const DropArgs& a, bool wide, cudaStream_t s) {
    const uint64_t tiles = (a.walk.total + kThreads * kSteps - 1) / (kThreads * kSteps);
    const dim3 grid((unsigned)umin64(tiles, 1u << 30));
    auto kernel = a.residual ? (wide ? k_dropout<T, true, true> : k_dropout<T, true, false>)
                             : (wide ? k_dropout<T, false, true> : k_dropout<T, false, false>);
    return launch_rows_kernel(kernel, grid, kThreads, s, a);
}

}  // namespace
}  // namespace dgc

using namespace dgc;

extern "C" int dgc_dropout(const dgc_matrix* x, const dgc_matrix* residual, double p, uint64_t seed,
                           const uint64_t* step, const dgc_matrix* out, dgc_stream_t stream) {
    Rows mx, mr, mo;
    int rc;
    if (!x || !(p >= 0.0 && p <= 1.0) || ((uintptr_t)step & 7u)) return DGC_EINVAL;
    if ((rc = check_rows(x, &mx, -1)) || (rc = check_rows(out, &mo, mx.dtype))) return rc;
    if (residual && (rc = check_rows(residual, &mr, mx.dtype))) return rc;
    if (!mo.shaped(mx.rows, mx.cols) || (residual && !mr.shaped(mx.rows, mx.cols)))
        return DGC_EINVAL;
    if (mx.rows == 0 || mx.cols == 0) return DGC_OK;
    DropArgs a{};
    a.x = mx.p;
    a.ldx = mx.ld;
    if (residual) {
        a.residual = mr.p;
        a.ldr = mr.ld;
    }
    a.out = mo.p;
    a.ldo = mo.ld;
    a.cols = (uint32_t)mx.cols;
    a.words = (a.cols + 3) / 4;
    const uint32_t piece = (uint32_t)(16 / mx.entry());
    a.walk = piece_walk(mx.rows, (a.cols + piece - 1) / piece, kThreads);
    a.seed = seed;
    a.step = step;
    a.threshold = (uint32_t)(p * 65536.0 + 0.5);
    a.scale = a.threshold < 65536 ? (float)(65536.0 / (65536 - a.threshold)) : 0.0f;
    const bool wide = mx.on(16) && mo.on(16) && (!residual || mr.on(16));
    return with_type(mx.dtype, [&](auto t) {
        return launch<decltype(t)>(a, wide, reinterpret_cast<cudaStream_t>(stream));
    });
}
