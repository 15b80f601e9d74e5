// ffn.cu -- the gated feed-forward block and its backward pass (sm_103a): five matrix products
// with what surrounds them in their epilogues, on the tensor cores.
//
//   x [M,D], w_gate, w_up [F,D], w_down [D,F]; act one of SiLU, GELU (erf or tanh), ReLU
//   gate          G = x Wg^T, U = x Wu^T, H = act(G) o U     one accumulator tile holds both
//   down          y = H Wd^T + r
//   down_backward dH = dy Wd; dG = dH o U o act'(G), dU = dH o act(G)     dH is never stored
//   gate_backward dx = dG Wg + dU Wu + r                     one sum over both products
//   weight_grad   dW = dy^T x, binary32, or dW += dy^T x
//
// Three routes. Forward products of one or two tokens are read by warps that stream the weights
// (k_rows); products with an operand, or an input of the epilogue, whose rows lie off 16-byte
// boundaries go to the ordinary cores (k_any); all others, of each of the five kinds, are k_ffn's.
//
// k_ffn: a persistent block per SM computes 128-row output tiles:
// warp 0 brings the operands' 64-deep slices by TMA into a ring of shared-memory stages, warp 1
// issues tcgen05.mma on them into one of two accumulators in tensor memory, warps 2-9 empty the
// other one: tcgen05.ld, the epilogue's arithmetic in binary32, one rounding, and a TMA store
// from shared memory. Operands whose long axis is the sum's (x, H, dy, dG, dU and the weights of
// the forward pass) are read along it ("K-major"); the others (the weights of the backward pass,
// both operands of the weight gradient) are read across it, in place: no transposed copy is made.
//
// Every wait is bounded: a block whose wait runs out reports DGC_ETIMEOUT, waits (bounded) for
// the copies it has in flight, frees its tensor memory and returns.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "dgc_device.cuh"

namespace dgc {
namespace {

enum Kind { kGate = 0, kDown = 1, kDownBwd = 2, kGateBwd = 3, kWGrad = 4 };

constexpr int kEpilogueWarps = 8;
constexpr int kFfnThreads = 64 + 32 * kEpilogueWarps;  // 10 warps: up to 168 registers a thread
constexpr int kBlockM = 128;
constexpr int kBlockK = 64;                    // 128 bytes of 16-bit entries: the swizzle's span
constexpr uint32_t kStageA = kBlockM * kBlockK * 2;
constexpr int kMaxStages = 8;
// The weight gradient's long sums leave the tensor cores every 12 slices (768 tokens) and are added
// up in registers, rounded to nearest: the tensor cores' own accumulation cuts bits off, which
// over 8192 tokens in one go took 9e-6 of the gradient's norm. Measured so, as a share of its norm:
// 7.3e-7 over 768 tokens, 7.2e-7 over 8192, 1.0e-6 over 2^20 (products of one sign: 1.5e-6; the
// additions' own share grows as the root of the tokens, 2.6e-6 at 2^24). A product in binary32 took
// 2e-7 over 768 tokens and 1.4e-6 over 2^20. Costs 2% at 8192 tokens x 11264 x 4096.
constexpr uint32_t kSumSlices = 12;

constexpr uint32_t kSmemLimit = 232448;        // 227 KB
constexpr uint32_t kFfnWaitLimit = 1u << 23;   // probes of a wait, and its time: the longest sum
constexpr uint64_t kFfnWaitNs = 2000000000;    // takes far less
constexpr uint32_t kSleepNs = 20000;
constexpr int64_t kMaxExtent = 1 << 24;

struct FfnArgs {
    CUtensorMap a0, a1, b0, b1;       // operands; a1, b1: the second product's, or B's up half
    CUtensorMap in0, in1;             // residual; gate and up
    CUtensorMap out0, out1, out2;
    uint32_t m, n;                    // the output's extents
    uint32_t kb0, kb;                 // 64-deep slices of the first product, of both
    uint32_t tiles_m, tiles_n, tiles; // tiles = tiles_m * tiles_n * splits
    uint32_t group;                   // row tiles that are walked together
    uint32_t kb_split;                // slices of one part of a split sum
    uint32_t splits;                  // ... and its parts, where a cluster's blocks sum them
    uint32_t split_rows;              // weight gradient: rows of the workspace between parts
    uint32_t bn, stages, a_rows, stage_bytes, load_bytes;
    uint32_t idesc, tmem_cols;
    int32_t act, half, residual, accumulate;
    // The results as plain matrices. TMA writes whole 16-byte pieces: where the last piece of a
    // row is not all the matrix's own (ragged), the columns of the last box are stored one by
    // one, and every column where TMA cannot address the rows at all (unaligned).
    void* out[3];
    uint64_t ld[3];
    int32_t ragged, unaligned;
    uint32_t lost;                    // self-test: a slice whose copies are left out
    uint64_t wait_ns;
    int32_t* status;
};

// ------------------------------------------------------------------- tensor-core PTX
// kCg: blocks that compute a tile together. With 2, `bar` is an address in the cluster's window:
// the barrier of the pair's first block counts the bytes of both.
template <int kCg>
__device__ __forceinline__ void tma_load(void* dst, const CUtensorMap* map, int32_t x, int32_t y,
                                         uint32_t bar) {
    if (kCg == 1)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3}], [%4];"
            ::"r"(smem_addr(dst)), "l"(map), "r"(x), "r"(y), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global"
            ".mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
            ::"r"(smem_addr(dst)), "l"(map), "r"(x), "r"(y), "r"(bar)
            : "memory");
}
__device__ __forceinline__ void tma_store(const CUtensorMap* map, const void* src, int32_t x,
                                          int32_t y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];"
                 ::"l"(map), "r"(x), "r"(y), "r"(smem_addr(src))
                 : "memory");
}
__device__ __forceinline__ void tma_add(const CUtensorMap* map, const void* src, int32_t x,
                                        int32_t y) {
    asm volatile(
        "cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.bulk_group [%0, {%1, %2}], [%3];"
        ::"l"(map), "r"(x), "r"(y), "r"(smem_addr(src))
        : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
template <int kN>
__device__ __forceinline__ void bulk_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kN) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// The address of the same shared variable in block `rank` of the cluster.
__device__ __forceinline__ uint32_t peer_addr(uint32_t p, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(p), "r"(rank));
    return r;
}
__device__ __forceinline__ uint32_t peer_addr(const void* p, uint32_t rank) {
    return peer_addr(smem_addr(p), rank);
}
__device__ __forceinline__ float4 ld_peer(uint32_t at) {
    float4 r;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(r.x), "=f"(r.y), "=f"(r.z), "=f"(r.w)
                 : "r"(at)
                 : "memory");
    return r;
}
__device__ __forceinline__ void mbar_arrive_peer(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
                 : "memory");
}
// Probes that may put the thread to sleep for up to `ns` while the phase is not complete.
template <bool kCluster>
__device__ __forceinline__ bool mbar_sleep_wait(uint64_t* bar, uint32_t parity, uint32_t ns) {
    uint32_t ok;
    if (kCluster)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_addr(bar)), "r"(parity), "r"(ns)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_addr(bar)), "r"(parity), "r"(ns)
            : "memory");
    return ok != 0;
}
__device__ __forceinline__ uint64_t global_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
// One lane of a converged warp. Under this predicate the compiler knows that one lane issues, and
// keeps operands in uniform registers; under a test of the lane's number it does not.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xFFFFFFFF;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
template <int kCg>
__device__ __forceinline__ void tmem_alloc(uint32_t* slot, uint32_t cols) {
    if (kCg == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_addr(slot)), "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_addr(slot)), "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
}
template <int kCg>
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
    if (kCg == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols)
                     : "memory");
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols)
                     : "memory");
}
template <int kCg>
__device__ __forceinline__ void mma_16bit(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          bool add) {
    if (kCg == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.u32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
            ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.u32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
            ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
            : "memory");
}
// Arrives at `bar` (of the pair's blocks, whose bits `mask` has) when the products issued so far
// are done.
template <int kCg>
__device__ __forceinline__ void mma_commit(uint64_t* bar, uint16_t mask) {
    if (kCg == 1)
        asm volatile(
            "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
            ::"r"(smem_addr(bar))
            : "memory");
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster"
            ".multicast::cluster.b64 [%0], %1;"
            ::"r"(smem_addr(bar)), "h"(mask)
            : "memory");
}
__device__ __forceinline__ void tmem_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// 32 columns of this warp's 32 rows: lane i gets row i.
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_load16(uint32_t addr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_wait_load() {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// Shared-memory operand descriptor, 128-byte swizzle. K-major: rows of 128 bytes (64 entries of
// the sum), 8 rows a swizzle atom, atoms 1024 bytes apart. Across the sum: slices of 64 rows (one
// per step of the sum) of 128 bytes (64 entries of the operand's own axis); 8 steps are 1024
// bytes apart, the next 64 entries of the own axis one slice (8192 bytes) further.
template <bool kAcross>
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
    constexpr uint64_t lead = kAcross ? 8192 >> 4 : 1, stride = 1024 >> 4;
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | (lead << 16) | (stride << 32) | (1ull << 46) |
           (2ull << 61);
}

// ----------------------------------------------------------------------- activations
// Values and slopes in binary32, followed by a rounding to 16 bits (2^-11 at the finest). The
// epilogue of a wide tile is bound by these instructions, so exponentials and reciprocals are the
// hardware's (relative errors about 2^-22, and |x| 2^-24 from the exponent's rounding).
struct ActValue {
    float value, slope;
};
__device__ __forceinline__ float exp_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
    return r;
}
__device__ __forceinline__ float reciprocal(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// The reciprocal flushes what is below 2^-126, which a sigmoid is from x = -87.3 on while g times it
// is not: it is taken 2^8 times larger. Below -88.7, where e^-x leaves binary32, the result is 0
// (g times it would be under 2.7e-37).
__device__ __forceinline__ float sigmoid(float x) {
    return 0x1p-8f * reciprocal(fmaf(exp_fast(-x), 0x1p-8f, 0x1p-8f));
}

// The normal distribution function: erfc(z) = t exp(-z^2 + p(t)), t = 1 / (1 + z/2), z >= 0, with
// the Chebyshev fit p of Press, Flannery, Teukolsky and Vetterling (Numerical Recipes, section 6.2:
// relative error below 1.2e-7 everywhere; in binary32 4e-6 up to |g| = 6, from the exponent's
// rounding). 1 + erf would lose its digits where it cancels, 1e-3 of the value already at -4; the
// library's normcdff took 2 us more of a call over 777 x 1001 x 2721. 0 below g = -12.9, where the
// exponential leaves the normal range (g times it would be under 1.5e-38).
__device__ __forceinline__ float normal_cdf(float g) {
    const float z = fabsf(g) * 0.7071067811865476f, t = reciprocal(fmaf(0.5f, z, 1.0f));
    float p = fmaf(t, 0.17087277f, -0.82215223f);
    p = fmaf(t, p, 1.48851587f);
    p = fmaf(t, p, -1.13520398f);
    p = fmaf(t, p, 0.27886807f);
    p = fmaf(t, p, -0.18628806f);
    p = fmaf(t, p, 0.09678418f);
    p = fmaf(t, p, 0.37409196f);
    p = fmaf(t, p, 1.00002368f);
    p = fmaf(t, p, -1.26551223f);
    const float c = 0.5f * t * exp_fast(fmaf(-z, z, p));
    return g < 0.0f ? c : 1.0f - c;
}

constexpr float kGeluC = 0.7978845608028654f;   // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

template <int kAct>
__device__ __forceinline__ float act_value(float g) {
    if (kAct == DGC_ACT_SILU) return g * sigmoid(g);
    if (kAct == DGC_ACT_GELU) return g * normal_cdf(g);
    if (kAct == DGC_ACT_GELU_TANH)  // (1 + tanh z) / 2 = sigmoid(2 z)
        return g * sigmoid(2.0f * kGeluC * g * fmaf(kGeluA * g, g, 1.0f));
    return g <= 0.0f ? 0.0f : g;
}
template <int kAct>
__device__ __forceinline__ ActValue act_both(float g) {
    ActValue r;
    if (kAct == DGC_ACT_SILU) {
        const float s = sigmoid(g);
        r.value = g * s;
        r.slope = fmaf(r.value, 1.0f - s, s);
    } else if (kAct == DGC_ACT_GELU) {
        const float p = normal_cdf(g);
        r.value = g * p;
        r.slope = fmaf(g * 0.3989422804014327f, exp_fast(-0.5f * g * g), p);
    } else if (kAct == DGC_ACT_GELU_TANH) {
        // Beyond 16 the sigmoid is 0 or 1 to the last bit: a square held there keeps the slope's
        // polynomial finite, where 0 * inf would make a NaN of gates from 1.9e19 on.
        const float g2 = fminf(g * g, 256.0f);
        const float s = sigmoid(2.0f * kGeluC * g * fmaf(kGeluA, g2, 1.0f));
        r.value = g * s;
        r.slope = fmaf(r.value * (1.0f - s), 2.0f * kGeluC * fmaf(3.0f * kGeluA, g2, 1.0f), s);
    } else {
        r.value = g <= 0.0f ? 0.0f : g;
        r.slope = g > 0.0f ? 1.0f : 0.0f;
    }
    return r;
}

template <bool kHalf>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
    if (kHalf) {
        const __half2 h = __floats2half2_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __nv_bfloat162 b = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&b);
}
template <bool kHalf>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if (kHalf) return __half22float2(*reinterpret_cast<const __half2*>(&w));
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
}

// --------------------------------------------------------------------------- the kernel
struct FfnShared {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t in_full[kEpilogueWarps][2];
    uint64_t drain;
    uint32_t tmem;
    volatile uint32_t abort;
};

// At most kFfnWaitLimit probes and about a.wait_ns.
template <bool kCluster = false>
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, FfnShared* sh,
                                         const FfnArgs& a) {
    if (mbar_sleep_wait<kCluster>(bar, parity, kSleepNs)) return true;
    const uint64_t begin = global_ns();
    for (uint32_t i = 0; i < kFfnWaitLimit; ++i) {
        if (mbar_sleep_wait<kCluster>(bar, parity, kSleepNs)) return true;
        if (sh->abort) return false;
        if (global_ns() - begin > a.wait_ns) break;
    }
    report(a.status, DGC_ETIMEOUT);
    sh->abort = 1;
    return false;
}
// For the way out of a block that gave up, and for its last commit: no report, its own limit.
__device__ __forceinline__ void wait_quietly(uint64_t* bar, uint32_t parity) {
    const uint64_t begin = global_ns();
    for (uint32_t i = 0; i < (1u << 20); ++i)
        if (mbar_test_wait(bar, parity) || global_ns() - begin > 50000000) return;
}

struct Tile {
    uint32_t mt, nt, split;
};
// Tiles in groups of `group` row tiles, columns outside, rows inside: the tiles that run at the
// same time share few operand slices, which stay in L2.
__device__ __forceinline__ Tile tile_at(const FfnArgs& a, uint32_t t) {
    Tile r;
    const uint32_t per = a.tiles_m * a.tiles_n;
    r.split = t / per;
    t -= r.split * per;
    const uint32_t g = t / (a.group * a.tiles_n);
    const uint32_t first = g * a.group;
    const uint32_t rows = min(a.group, a.tiles_m - first);
    t -= first * a.tiles_n;
    r.nt = t / rows;
    r.mt = first + (t - r.nt * rows);
    return r;
}
__device__ __forceinline__ void k_range(const FfnArgs& a, uint32_t split, uint32_t* k0,
                                        uint32_t* k1) {
    *k0 = min(a.kb, split * a.kb_split);
    *k1 = min(a.kb, *k0 + a.kb_split);
}

template <int kKind>
struct Epilogue {
    static constexpr int kIn = kKind == kDownBwd ? 2 : (kKind == kDown || kKind == kGateBwd) ? 1 : 0;
    static constexpr int kOut = kKind == kGate ? 3 : kKind == kDownBwd ? 2 : 1;
    static constexpr int kBufs = kOut > kIn ? kOut : kIn;       // 32 x 32 boxes of one set
    static constexpr uint32_t kBox = kKind == kWGrad ? 4096 : 2048;
    // sets: one is written while the others' stores leave and their loads arrive
    static constexpr int kSets = kKind == kGate || kKind == kWGrad ? 1 : 2;
    static constexpr uint32_t kWarpBytes = kSets * kBufs * kBox;
    static constexpr uint32_t kBytes = kWarpBytes * kEpilogueWarps;
};

// A chunk's 32 rows x 32 columns, a row a lane: v (and u) from the accumulator, the inputs from the
// staging boxes i0, i1, the results into o0.. in their place, 16 bytes at a time in the swizzled
// order of a TMA box.
template <int kKind, int kAct, bool kHalf>
__device__ __forceinline__ void chunk_16bit(const uint32_t (&v)[32], const uint32_t (&u)[32],
                                            bool residual, char* b0, char* b1, char* b2, int lane) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const uint32_t at = lane * 64 + ((p ^ ((lane >> 1) & 3)) << 4);
        uint32_t o0[4], o1[4], o2[4];
        uint4 q = make_uint4(0, 0, 0, 0), w = q;
        if (kKind == kDownBwd || ((kKind == kDown || kKind == kGateBwd) && residual))
            q = *reinterpret_cast<const uint4*>(b0 + at);
        if (kKind == kDownBwd) w = *reinterpret_cast<const uint4*>(b1 + at);
        const uint32_t i0[4] = {q.x, q.y, q.z, q.w}, i1[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float v0 = __uint_as_float(v[8 * p + 2 * j]);
            const float v1 = __uint_as_float(v[8 * p + 2 * j + 1]);
            if (kKind == kGate) {
                const float u0 = __uint_as_float(u[8 * p + 2 * j]);
                const float u1 = __uint_as_float(u[8 * p + 2 * j + 1]);
                o0[j] = pack2<kHalf>(act_value<kAct>(v0) * u0, act_value<kAct>(v1) * u1);
                o1[j] = pack2<kHalf>(v0, v1);
                o2[j] = pack2<kHalf>(u0, u1);
            } else if (kKind == kDownBwd) {
                const float2 g = unpack2<kHalf>(i0[j]), x = unpack2<kHalf>(i1[j]);
                const ActValue f0 = act_both<kAct>(g.x), f1 = act_both<kAct>(g.y);
                o0[j] = pack2<kHalf>(v0 * x.x * f0.slope, v1 * x.y * f1.slope);
                o1[j] = pack2<kHalf>(v0 * f0.value, v1 * f1.value);
            } else {
                const float2 r = unpack2<kHalf>(i0[j]);
                o0[j] = residual ? pack2<kHalf>(v0 + r.x, v1 + r.y) : pack2<kHalf>(v0, v1);
            }
        }
        *reinterpret_cast<uint4*>(b0 + at) = make_uint4(o0[0], o0[1], o0[2], o0[3]);
        if (kKind == kGate || kKind == kDownBwd)
            *reinterpret_cast<uint4*>(b1 + at) = make_uint4(o1[0], o1[1], o1[2], o1[3]);
        if (kKind == kGate)
            *reinterpret_cast<uint4*>(b2 + at) = make_uint4(o2[0], o2[1], o2[2], o2[3]);
    }
}

// A split sum's parts: a chunk of this block's accumulator into its shared memory, and the same
// chunk of all blocks of the cluster added up in the parts' order. Four columns of the 32 rows are
// 512 consecutive bytes, one access of a warp here and from another block.
__device__ __forceinline__ void put_part(char* parts, uint32_t chunk, const uint32_t (&v)[32],
                                         bool empty, int lane) {
    char* to = parts + chunk * 4096 + lane * 16;
#pragma unroll
    for (int p = 0; p < 8; ++p)
        *reinterpret_cast<uint4*>(to + p * 512) =
            empty ? make_uint4(0, 0, 0, 0)
                  : make_uint4(v[4 * p], v[4 * p + 1], v[4 * p + 2], v[4 * p + 3]);
}
template <int kCg>
__device__ __forceinline__ void add_parts(const char* parts, uint32_t chunk, uint32_t splits,
                                          uint32_t row_rank, uint32_t (&r)[32], int lane) {
    const uint32_t at = smem_addr(parts) + chunk * 4096 + lane * 16;
#pragma unroll
    for (int i = 0; i < 32; ++i) r[i] = 0;
#pragma unroll 2
    for (uint32_t q = 0; q < splits; ++q) {
        const uint32_t from = peer_addr(at, q * kCg + row_rank);
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            const float4 w = ld_peer(from + p * 512);
            r[4 * p] = __float_as_uint(__uint_as_float(r[4 * p]) + w.x);
            r[4 * p + 1] = __float_as_uint(__uint_as_float(r[4 * p + 1]) + w.y);
            r[4 * p + 2] = __float_as_uint(__uint_as_float(r[4 * p + 2]) + w.z);
            r[4 * p + 3] = __float_as_uint(__uint_as_float(r[4 * p + 3]) + w.w);
        }
    }
}

// One chunk out of registers: the epilogue's arithmetic into the set's boxes, and their stores.
template <int kKind, int kAct>
__device__ __forceinline__ void finish_chunk(const FfnArgs& a, const uint32_t (&v)[32],
                                             const uint32_t (&u)[32], bool has_in, char* set,
                                             uint32_t x, uint32_t y, uint32_t split, int lane) {
    using E = Epilogue<kKind>;
    auto buf = [&](int i) { return set + i * E::kBox; };
    if (kKind == kWGrad) {
#pragma unroll
        for (int p = 0; p < 8; ++p)
            *reinterpret_cast<uint4*>(buf(0) + lane * 128 + ((p ^ (lane & 7)) << 4)) =
                make_uint4(v[4 * p], v[4 * p + 1], v[4 * p + 2], v[4 * p + 3]);
    } else if (a.half) {
        chunk_16bit<kKind, kAct, true>(v, u, has_in, buf(0), buf(E::kBufs > 1), buf(E::kBufs - 1),
                                       lane);
    } else {
        chunk_16bit<kKind, kAct, false>(v, u, has_in, buf(0), buf(E::kBufs > 1), buf(E::kBufs - 1),
                                        lane);
    }
    if (a.unaligned || (a.ragged && x + 32 > a.n)) {
        // a row of up to 32 columns per step, one column a lane
        __syncwarp();
        const uint32_t rows = min(32u, a.m - y);
        const int outs = kKind == kGate ? (a.residual ? 3 : 1) : E::kOut;
        if (x + lane < a.n)
            for (uint32_t r = 0; r < rows; ++r)
                for (int i = 0; i < outs; ++i) {
                    const uint64_t to = (uint64_t)(y + r) * a.ld[i] + x + lane;
                    if (kKind == kWGrad) {
                        const float f = *reinterpret_cast<const float*>(
                            buf(0) + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4);
                        float* d = static_cast<float*>(a.out[0]) + to;
                        *d = a.accumulate ? *d + f : f;
                    } else {
                        static_cast<uint16_t*>(a.out[i])[to] = *reinterpret_cast<const uint16_t*>(
                            buf(i) + r * 64 + (((lane >> 3) ^ ((r >> 1) & 3)) << 4) +
                            (lane & 7) * 2);
                    }
                }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) bulk_commit();  // an empty group: the sets are counted by groups
        return;
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
        if (kKind == kWGrad) {
            if (a.accumulate)
                tma_add(&a.out0, buf(0), x, y + split * a.split_rows);
            else
                tma_store(&a.out0, buf(0), x, y + split * a.split_rows);
        } else {
            tma_store(&a.out0, buf(0), x, y);
            if (kKind == kDownBwd) tma_store(&a.out1, buf(1), x, y);
            if (kKind == kGate && a.residual) {  // gate and up are wanted
                tma_store(&a.out1, buf(1), x, y);
                tma_store(&a.out2, buf(2), x, y);
            }
        }
        bulk_commit();
    }
}

// Warps 2-9: two for each quarter of the accumulator's rows (the quarter a warp may read is its
// number modulo 4), taking every other chunk of 32 columns. With kSplit the blocks of a cluster
// have summed a part of the tile's products each: every block puts its accumulator into its own
// shared memory (the stages, which are empty by then), and after a barrier each of them adds up,
// in the order of the parts, the chunks that fall to it.
template <int kKind, int kCg, bool kSplit, int kAct>
__device__ __forceinline__ void epilogue(const FfnArgs& a, FfnShared* sh, char* parts,
                                         char* staging, uint32_t tmem, uint32_t rank) {
    using E = Epilogue<kKind>;
    const int warp = (threadIdx.x >> 5) - 2, lane = threadIdx.x & 31;
    const uint32_t quarter = (threadIdx.x >> 5) & 3;
    char* mine = staging + warp * E::kWarpBytes;
    auto set_at = [&](uint32_t n) { return mine + (n % E::kSets) * E::kBufs * E::kBox; };
    const uint32_t out_cols = kKind == kGate ? a.bn / 2 : a.bn;  // columns of one tile's output
    const uint32_t chunks = out_cols / 32;
    const uint32_t row_rank = rank % kCg, part = rank / kCg, lead = rank - row_rank;
    const uint32_t first_chunk = (kSplit ? 2 * part : 0) + (warp >> 2);
    const uint32_t chunk_step = kSplit ? 2 * a.splits : 2;
    const bool has_in = E::kIn > 0 && (kKind == kDownBwd || a.residual);
    const uint32_t first_tile = kSplit ? blockIdx.x / (a.splits * kCg) : blockIdx.x / kCg;
    const uint32_t tile_step = kSplit ? a.tiles : gridDim.x / kCg;
    const uint32_t row_in_tile = row_rank * kBlockM + quarter * 32;
    const uint32_t acc_empty = kCg == 1 ? 0 : peer_addr(sh->acc_empty, lead);

    // The loads of one chunk's inputs; chunks outside the output have none.
    uint32_t load_tile = first_tile, load_chunk = first_chunk, load_n = 0;
    auto issue_load = [&]() {  // lane 0: the next chunk's inputs, if there is one left
        while (load_tile < a.tiles) {
            const Tile t = tile_at(a, load_tile);
            const uint32_t y = t.mt * kBlockM * kCg + row_in_tile;
            const uint32_t x = t.nt * out_cols + load_chunk * 32;
            if (y >= a.m || x >= a.n || load_chunk >= chunks) {  // none left in this tile
                load_chunk = first_chunk;
                load_tile += tile_step;
                continue;
            }
            char* set = set_at(load_n);
            uint64_t* bar = &sh->in_full[warp][load_n % E::kSets];
            mbar_arrive_expect_tx(bar, 2048u * E::kIn);
            tma_load<1>(set, &a.in0, x, y, smem_addr(bar));
            if (E::kIn > 1) tma_load<1>(set + E::kBox, &a.in1, x, y, smem_addr(bar));
            ++load_n;
            load_chunk += chunk_step;
            return;
        }
    };
    if (has_in && lane == 0)
        for (int i = 0; i < E::kSets - 1; ++i) issue_load();

    uint32_t done = 0;  // chunks this warp has finished
    uint32_t it = 0;
    bool ok = true;
    // Makes the set of the next chunk ready for its results (and its inputs).
    auto ready = [&]() {
        if (has_in) {
            // the store before this one has left its set: the next inputs go there
            if (lane == 0) {
                bulk_wait_read<0>();
                issue_load();
            }
            __syncwarp();
            ok = __all_sync(kFull, wait_bar(&sh->in_full[warp][done % E::kSets],
                                            (done / E::kSets) & 1, sh, a));
        } else {
            // the last store from this set has left it
            if (lane == 0) bulk_wait_read<E::kSets - 1>();
            __syncwarp();
        }
        return ok;
    };
    uint32_t v[32], u[32];
    for (uint32_t ti = first_tile; ti < a.tiles && ok; ti += tile_step, ++it) {
        const Tile t = tile_at(a, ti);
        const uint32_t acc = it & 1, y = t.mt * kBlockM * kCg + row_in_tile;
        uint32_t k0, k1;
        k_range(a, kSplit ? part : t.split, &k0, &k1);
        ok = __all_sync(kFull, wait_bar(&sh->acc_full[acc], (it >> 1) & 1, sh, a));
        tmem_fence_after();
        const uint32_t src = tmem + acc * a.bn + (quarter * 32 << 16);
        if (kSplit) {
            for (uint32_t c = warp >> 2; c < a.bn / 32 && ok; c += 2) {
                tmem_load32(src + c * 32, v);
                tmem_wait_load();
                put_part(parts, c * 4 + quarter, v, k0 >= k1, lane);
            }
            __syncwarp();
            cluster_sync();
            for (uint32_t c = first_chunk; c < chunks && y < a.m && ok; c += chunk_step) {
                const uint32_t x = t.nt * out_cols + c * 32;
                if (x >= a.n) break;
                add_parts<kCg>(parts, c * 4 + quarter, a.splits, row_rank, v, lane);
                if (kKind == kGate)
                    add_parts<kCg>(parts, (c + chunks) * 4 + quarter, a.splits, row_rank, u, lane);
                if (!ready()) break;
                finish_chunk<kKind, kAct>(a, v, u, has_in, set_at(done), x, y, 0, lane);
                ++done;
            }
            break;
        }
        if (!ok) break;
        for (uint32_t c = first_chunk; c < chunks && y < a.m; c += 2) {
            const uint32_t x = t.nt * out_cols + c * 32;
            if (x >= a.n) break;
            tmem_load32(src + c * 32, v);
            if (kKind == kGate) tmem_load32(src + out_cols + c * 32, u);
            if (!ready()) break;
            tmem_wait_load();
            if (k0 >= k1) {  // an empty sum: the accumulator was never written
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = u[i] = 0;
            }
            finish_chunk<kKind, kAct>(a, v, u, has_in, set_at(done), x, y, t.split, lane);
            ++done;
        }
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) {
            if (kCg == 1)
                mbar_arrive(&sh->acc_empty[acc]);
            else
                mbar_arrive_peer(acc_empty + acc * 8);
        }
    }
    if (lane == 0) {
        // inputs still on their way to a block that gave up
        if (!ok && has_in)
            for (uint32_t i = done; i < load_n; ++i)
                wait_quietly(&sh->in_full[warp][i % E::kSets], (i / E::kSets) & 1);
        bulk_wait_read<0>();  // the block's shared memory may go
    }
}

// The weight gradient's: every kSumSlices slices the accumulator is added to this warp's sums in
// registers (up to four chunks), which are the tile's result at its end. 128 of the 168 registers
// hold sums; 20 to 36 bytes a thread are spilled.
template <int kCg, bool kSplit>
__device__ __forceinline__ void epilogue_sums(const FfnArgs& a, FfnShared* sh, char* parts,
                                              char* staging, uint32_t tmem, uint32_t rank) {
    using E = Epilogue<kWGrad>;
    const int warp = (threadIdx.x >> 5) - 2, lane = threadIdx.x & 31;
    const uint32_t quarter = (threadIdx.x >> 5) & 3, half = warp >> 2;
    char* box = staging + warp * E::kWarpBytes;
    const uint32_t row_rank = rank % kCg, part = rank / kCg, lead = rank - row_rank;
    const uint32_t chunks = a.bn / 32;
    const uint32_t first_tile = kSplit ? blockIdx.x / (a.splits * kCg) : blockIdx.x / kCg;
    const uint32_t tile_step = kSplit ? a.tiles : gridDim.x / kCg;
    const uint32_t acc_empty = kCg == 1 ? 0 : peer_addr(sh->acc_empty, lead);
    uint32_t it = 0;
    bool ok = true;
    auto finish = [&](const Tile& t, uint32_t c, const uint32_t (&v)[32]) {
        const uint32_t y = (t.mt * kCg + row_rank) * kBlockM + quarter * 32;
        const uint32_t x = t.nt * a.bn + c * 32;
        if (y >= a.m || x >= a.n) return;
        if (lane == 0) bulk_wait_read<0>();  // the last store has left the box
        __syncwarp();
        finish_chunk<kWGrad, DGC_ACT_RELU>(a, v, v, false, box, x, y, t.split, lane);
    };
    for (uint32_t ti = first_tile; ti < a.tiles && ok; ti += tile_step) {
        const Tile t = tile_at(a, ti);
        uint32_t k0, k1;
        k_range(a, kSplit ? part : t.split, &k0, &k1);
        uint32_t sum[4][32];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 32; ++j) sum[i][j] = 0;
        for (uint32_t kb = k0; kb < k1; kb += kSumSlices, ++it) {
            const uint32_t acc = it & 1;
            ok = __all_sync(kFull, wait_bar(&sh->acc_full[acc], (it >> 1) & 1, sh, a));
            if (!ok) break;
            tmem_fence_after();
            const uint32_t src = tmem + acc * a.bn + (quarter * 32 << 16);
            // 16 columns at a time, the next ones on their way while these are added (128 registers
            // hold the sums)
            uint32_t v[2][16];
            if (half < chunks) tmem_load16(src + half * 32, v[0]);
#pragma unroll
            for (int h = 0; h < 8; ++h) {
                if (half + 2 * (h / 2) >= chunks) break;
                tmem_wait_load();
                const uint32_t next = half + 2 * ((h + 1) / 2);
                if (h < 7 && next < chunks)
                    tmem_load16(src + next * 32 + ((h + 1) & 1) * 16, v[(h + 1) & 1]);
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    uint32_t& r = sum[h / 2][(h & 1) * 16 + j];
                    r = __float_as_uint(__uint_as_float(r) + __uint_as_float(v[h & 1][j]));
                }
            }
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (kCg == 1)
                    mbar_arrive(&sh->acc_empty[acc]);
                else
                    mbar_arrive_peer(acc_empty + acc * 8);
            }
        }
        if (kSplit) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (half + 2 * i < chunks)
                    put_part(parts, (half + 2 * i) * 4 + quarter, sum[i], false, lane);
            __syncwarp();
            cluster_sync();
            for (uint32_t c = 2 * part + half; c < chunks && ok; c += 2 * a.splits) {
                add_parts<kCg>(parts, c * 4 + quarter, a.splits, row_rank, sum[0], lane);
                finish(t, c, sum[0]);
            }
            break;
        }
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (half + 2 * i < chunks) finish(t, half + 2 * i, sum[i]);
    }
    if (lane == 0) bulk_wait_read<0>();  // the block's shared memory may go
}

// The product of one kind. Bound by the tensor cores where the tiles are 256 x 256 and fill the
// GPU: 8192 x 4096 x 11264 bf16 gate 850-880 us (1.72-1.78 PFLOP/s), down and gate backward 1.7,
// weight gradient 1.62, at the 1.4 kW cap and 1.55-1.6 GHz, where the vendor's library takes 839 us
// for the gate's products alone. Below that by the operands' way from L2 (about 68 bytes a clock and
// SM) and, under about 20 us, by the start, the first loads and the last epilogue (1 + 1 + 2-4 us).
// Ten warps, one block an SM: the stages take what shared memory the epilogue leaves.
template <int kKind, int kCg, bool kSplit>
__global__ void __launch_bounds__(kFfnThreads, 1) k_ffn(const __grid_constant__ FfnArgs a) {
    constexpr bool kAcrossA = kKind == kWGrad;
    constexpr bool kAcrossB = kKind == kDownBwd || kKind == kGateBwd || kKind == kWGrad;
    extern __shared__ char dyn[];
    __shared__ FfnShared shared;
    FfnShared* sh = &shared;
    char* base = dyn + ((1024u - (smem_addr(dyn) & 1023u)) & 1023u);
    char* staging = base + a.stages * a.stage_bytes;
    const int warp = threadIdx.x >> 5;
    // A cluster is `splits` blocks or pairs: which part of the sum, and which rows of the pair's
    // tile, are this block's. lead: the pair's first block, which issues its products.
    const uint32_t rank = kCg == 2 || kSplit ? cluster_rank() : 0;
    const uint32_t row_rank = rank % kCg, part = rank / kCg, lead = rank - row_rank;
    const uint32_t first_tile = kSplit ? blockIdx.x / (a.splits * kCg) : blockIdx.x / kCg;
    const uint32_t tile_step = kSplit ? a.tiles : gridDim.x / kCg;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(&sh->full[i], 1);
            mbar_init(&sh->empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh->acc_full[i], 1);
            mbar_init(&sh->acc_empty[i], kEpilogueWarps * kCg);
        }
        for (int w = 0; w < kEpilogueWarps; ++w)
            for (int i = 0; i < 2; ++i) mbar_init(&sh->in_full[w][i], 1);
        mbar_init(&sh->drain, 1);
        mbar_init_fence();
        sh->abort = 0;
    }
    if (warp == 1) tmem_alloc<kCg>(&sh->tmem, a.tmem_cols);
    if (threadIdx.x == 64) {
        prefetch_map(&a.a0);
        prefetch_map(&a.b0);
        if (kKind == kGate || kKind == kGateBwd) prefetch_map(&a.b1);
        if (kKind == kGateBwd) prefetch_map(&a.a1);
    }
    tmem_fence_before();
    __syncthreads();
    if (kCg == 2) cluster_sync();
    tmem_fence_after();
    const uint32_t tmem = sh->tmem;
    // a dependent launch: all of the above may run while the kernel ahead ends
    grid_dep_wait();
    grid_dep_launch();

    // One elected lane of warps 0 and 1 works.
    if (warp == 0 && elect_one()) {
        const uint32_t cols = a.bn / kCg;  // of B, loaded by this block
        const uint32_t full = kCg == 1 ? smem_addr(sh->full) : peer_addr(sh->full, lead);
        const uint32_t stages = a.stages, stage_bytes = a.stage_bytes;
        uint32_t n = 0;  // stages filled so far
        uint32_t s = 0, phase = 1;
        bool ok = true;
        for (uint32_t ti = first_tile; ti < a.tiles && ok; ti += tile_step) {
            const Tile t = tile_at(a, ti);
            const int32_t row = (t.mt * kCg + row_rank) * kBlockM;
            const int32_t col = t.nt * a.bn + row_rank * cols;
            uint32_t k0, k1;
            k_range(a, kSplit ? part : t.split, &k0, &k1);
            for (uint32_t kb = k0; kb < k1; ++kb, ++n) {
                ok = wait_bar(&sh->empty[s], phase, sh, a);
                if (!ok) break;
                if (kb != a.lost) {
                    char* sa = base + s * stage_bytes;
                    char* sb = sa + kStageA;
                    const uint32_t bar = full + s * 8;
                    if (row_rank == 0) mbar_arrive_expect_tx(&sh->full[s], a.load_bytes);
                    const bool second = kKind == kGateBwd && kb >= a.kb0;
                    const int32_t k = (int32_t)(second ? kb - a.kb0 : kb) * kBlockK;
                    const CUtensorMap* ma = second ? &a.a1 : &a.a0;
                    const CUtensorMap* mb = second ? &a.b1 : &a.b0;
                    if (kAcrossA) {
                        tma_load<kCg>(sa, ma, row, k, bar);
                        tma_load<kCg>(sa + 8192, ma, row + 64, k, bar);
                    } else {
                        tma_load<kCg>(sa, ma, k, row, bar);
                    }
                    if (kAcrossB) {
                        for (uint32_t c = 0; c < cols / 64; ++c)
                            tma_load<kCg>(sb + c * 8192, mb, col + c * 64, k, bar);
                    } else if (kKind == kGate) {
                        // gate rows, then up rows; of a pair, one block brings each
                        const int32_t f = t.nt * (a.bn / 2);
                        if (kCg == 1) {
                            tma_load<kCg>(sb, &a.b0, k, f, bar);
                            tma_load<kCg>(sb + a.bn / 2 * 128, &a.b1, k, f, bar);
                        } else {
                            tma_load<kCg>(sb, row_rank == 0 ? &a.b0 : &a.b1, k, f, bar);
                        }
                    } else {
                        tma_load<kCg>(sb, mb, k, col, bar);
                    }
                }
                if (++s == stages) s = 0, phase ^= 1;
            }
        }
        if (!ok || sh->abort)  // copies in flight to a block that gives up
            for (uint32_t i = n > stages ? n - stages : 0; i < n; ++i) {
                if (row_rank == 0)
                    wait_quietly(&sh->full[i % stages], (i / stages) & 1);
                else
                    wait_quietly(&sh->empty[i % stages], (i / stages) & 1);
            }
    } else if (warp == 1 && row_rank == 0 && elect_one()) {
        const uint32_t stages = a.stages, stage_bytes = a.stage_bytes, idesc = a.idesc;
        const uint16_t mask = (uint16_t)(3u << lead);
        const uint64_t da0 = operand_desc<kAcrossA>(smem_addr(base));
        const uint64_t db0 = operand_desc<kAcrossB>(smem_addr(base) + kStageA);
        uint32_t s = 0, phase = 0, it = 0;
        bool ok = true;
        for (uint32_t ti = first_tile; ti < a.tiles && ok; ti += tile_step) {
            const Tile t = tile_at(a, ti);
            uint32_t kb, k1;
            k_range(a, kSplit ? part : t.split, &kb, &k1);
            if (kKind == kWGrad && kb >= k1) continue;  // its epilogue waits for no empty sum
            do {
                const uint32_t acc = it & 1;
                const uint32_t k0 = kb, end = kKind == kWGrad ? min(k1, kb + kSumSlices) : k1;
                ok = wait_bar<kCg == 2>(&sh->acc_empty[acc], ((it >> 1) & 1) ^ 1, sh, a);
                if (!ok) break;
                tmem_fence_after();
                const uint32_t d = tmem + acc * a.bn;
                for (; kb < end; ++kb) {
                    ok = wait_bar(&sh->full[s], phase, sh, a);
                    if (!ok) break;
                    tmem_fence_after();
                    const uint64_t da = da0 + (s * stage_bytes >> 4);
                    const uint64_t db = db0 + (s * stage_bytes >> 4);
#pragma unroll
                    for (int k = 0; k < kBlockK / 16; ++k)  // 16 of the sum: 32 bytes, or 16 rows
                        mma_16bit<kCg>(d, da + k * (kAcrossA ? 2048 >> 4 : 2),
                                       db + k * (kAcrossB ? 2048 >> 4 : 2), idesc,
                                       kb > k0 || k > 0);
                    mma_commit<kCg>(&sh->empty[s], mask);
                    if (++s == stages) s = 0, phase ^= 1;
                }
                if (!ok) break;
                mma_commit<kCg>(&sh->acc_full[acc], mask);
                ++it;
            } while (kb < k1);
        }
        mma_commit<kCg>(&sh->drain, mask);  // what was issued is done before the end
        wait_quietly(&sh->drain, 0);
    } else if (warp >= 2) {
        if (kKind == kWGrad)
            epilogue_sums<kCg, kSplit>(a, sh, base, staging, tmem, rank);
        else if (kKind != kGate && kKind != kDownBwd)
            epilogue<kKind, kCg, kSplit, DGC_ACT_RELU>(a, sh, base, staging, tmem, rank);
        else if (a.act == DGC_ACT_SILU)
            epilogue<kKind, kCg, kSplit, DGC_ACT_SILU>(a, sh, base, staging, tmem, rank);
        else if (a.act == DGC_ACT_GELU)
            epilogue<kKind, kCg, kSplit, DGC_ACT_GELU>(a, sh, base, staging, tmem, rank);
        else if (a.act == DGC_ACT_GELU_TANH)
            epilogue<kKind, kCg, kSplit, DGC_ACT_GELU_TANH>(a, sh, base, staging, tmem, rank);
        else
            epilogue<kKind, kCg, kSplit, DGC_ACT_RELU>(a, sh, base, staging, tmem, rank);
    }
    __syncwarp();
    if (kSplit && warp < 2) cluster_sync();  // the epilogue's warps pass theirs between their steps
    tmem_fence_before();
    __syncthreads();
    // the pair's last commit has arrived here before this block's shared memory goes
    if (kCg == 2 && row_rank == 1 && threadIdx.x == 32) wait_quietly(&sh->drain, 0);
    __syncthreads();
    if (kCg == 2 || kSplit) cluster_sync();
    tmem_fence_after();
    if (warp == 1) tmem_free<kCg>(tmem, a.tmem_cols);
}

// ------------------------------------------------------------------------- a few tokens
// The forward products of one or two tokens: the weights' bytes are all there is to it. A warp (or
// 2, 4, 8 of a block, which split the sum) reads two weight rows -- gate: a column's gate and up
// rows; down: two columns' rows -- with 16-byte loads, 4 in flight of each, past L1; the tokens'
// rows stay in L1. The tensor cores would read the same bytes behind a pipeline's start, a tile's
// barriers and a cluster's sum: one token x 1024 x 4096 5.0 + 7.0 us (gate, down; here 3.7 + 2.8),
// x 4096 x 11264 40 + 15.6 us (here 29.1 + 13.9, the weights at the copy rate 27.6 + 13.8). From
// three tokens on they are ahead. Rows off 16-byte boundaries are read entry by entry (1023 x 4095:
// 22 + 14 us).
constexpr uint32_t kFewTokens = 2;
constexpr int kRowsWarps = 8;

struct RowsArgs {
    const uint16_t *x, *w0, *w1, *residual;
    uint64_t ldx, ldw0, ldw1, ldr;
    uint32_t n, k;
    int32_t log_split, act;
    uint16_t* out[3];
    uint64_t ld[3];
};

__device__ __forceinline__ uint4 load_stream(const uint16_t* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
template <bool kHalf>
__device__ __forceinline__ float dot8(uint4 a, uint4 b, float s) {
    const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 p = unpack2<kHalf>(x[i]), q = unpack2<kHalf>(y[i]);
        s = fmaf(p.y, q.y, fmaf(p.x, q.x, s));
    }
    return s;
}
__device__ __forceinline__ float act_at(int act, float g) {
    if (act == DGC_ACT_SILU) return act_value<DGC_ACT_SILU>(g);
    if (act == DGC_ACT_GELU) return act_value<DGC_ACT_GELU>(g);
    if (act == DGC_ACT_GELU_TANH) return act_value<DGC_ACT_GELU_TANH>(g);
    return act_value<DGC_ACT_RELU>(g);
}

__device__ __forceinline__ ActValue act_both_at(int act, float g) {
    if (act == DGC_ACT_SILU) return act_both<DGC_ACT_SILU>(g);
    if (act == DGC_ACT_GELU) return act_both<DGC_ACT_GELU>(g);
    if (act == DGC_ACT_GELU_TANH) return act_both<DGC_ACT_GELU_TANH>(g);
    return act_both<DGC_ACT_RELU>(g);
}

template <int kKind, bool kHalf, int kM, bool kAligned>
__global__ void __launch_bounds__(32 * kRowsWarps) k_rows(const __grid_constant__ RowsArgs a) {
    constexpr int kW = 2;    // weight rows of a warp
    constexpr int kFly = 4;  // loads in flight of each
    constexpr int kCols = kKind == kGate ? 1 : 2;
    __shared__ float part_sum[kRowsWarps][kW * kM];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t splits = 1u << a.log_split, part = warp & (splits - 1);
    const uint32_t col = ((blockIdx.x * kRowsWarps + warp) >> a.log_split) * kCols;
    grid_dep_wait();
    grid_dep_launch();
    float sum[kW][kM];
#pragma unroll
    for (int i = 0; i < kW; ++i)
#pragma unroll
        for (int m = 0; m < kM; ++m) sum[i][m] = 0.0f;
    if (col < a.n) {
        // down's second column, or the first again where there is none
        const uint16_t* w[2] = {a.w0 + col * a.ldw0,
                                kKind == kGate ? a.w1 + col * a.ldw1
                                               : a.w0 + min(col + 1, a.n - 1) * a.ldw0};
        // rows off 16-byte boundaries: entry by entry
        const uint32_t first = (uint32_t)((uint64_t)a.k * part >> a.log_split);
        const uint32_t end = (uint32_t)((uint64_t)a.k * (part + 1) >> a.log_split);
        for (uint32_t k = first + lane; !kAligned && k < end; k += 32 * 2 * kFly) {
            uint16_t q[kW][2 * kFly];
#pragma unroll
            for (int u = 0; u < 2 * kFly; ++u)
#pragma unroll
                for (int i = 0; i < kW; ++i) q[i][u] = k + 32 * u < end ? w[i][k + 32 * u] : 0;
#pragma unroll
            for (int u = 0; u < 2 * kFly; ++u) {
                if (k + 32 * u >= end) break;
#pragma unroll
                for (int m = 0; m < kM; ++m) {
                    const float t = unpack2<kHalf>(a.x[m * a.ldx + k + 32 * u]).x;
#pragma unroll
                    for (int i = 0; i < kW; ++i)
                        sum[i][m] = fmaf(unpack2<kHalf>(q[i][u]).x, t, sum[i][m]);
                }
            }
        }
        const uint32_t vecs = kAligned ? a.k / 8 : 0;
        const uint32_t v0 = (uint32_t)((uint64_t)vecs * part >> a.log_split);
        const uint32_t v1 = (uint32_t)((uint64_t)vecs * (part + 1) >> a.log_split);
        for (uint32_t v = v0 + lane; v < v1; v += 32 * kFly) {
            uint4 q[kW][kFly];
#pragma unroll
            for (int u = 0; u < kFly; ++u)
#pragma unroll
                for (int i = 0; i < kW; ++i)
                    q[i][u] = v + 32 * u < v1 ? load_stream(w[i] + (uint64_t)(v + 32 * u) * 8)
                                              : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int u = 0; u < kFly; ++u) {
                if (v + 32 * u >= v1) break;
#pragma unroll
                for (int m = 0; m < kM; ++m) {
                    const uint4 t = *reinterpret_cast<const uint4*>(
                        a.x + m * a.ldx + (uint64_t)(v + 32 * u) * 8);
#pragma unroll
                    for (int i = 0; i < kW; ++i) sum[i][m] = dot8<kHalf>(q[i][u], t, sum[i][m]);
                }
            }
        }
        const uint32_t at = vecs * 8 + lane;  // the last few of the sum
        if (kAligned && part == splits - 1 && at < a.k)
#pragma unroll
            for (int m = 0; m < kM; ++m)
#pragma unroll
                for (int i = 0; i < kW; ++i)
                    sum[i][m] = fmaf(unpack2<kHalf>(w[i][at]).x,
                                     unpack2<kHalf>(a.x[m * a.ldx + at]).x, sum[i][m]);
    }
#pragma unroll
    for (int i = 0; i < kW; ++i)
#pragma unroll
        for (int m = 0; m < kM; ++m) sum[i][m] = warp_sum(sum[i][m]);
    if (splits > 1) {
        if (lane == 0)
#pragma unroll
            for (int i = 0; i < kW; ++i)
#pragma unroll
                for (int m = 0; m < kM; ++m) part_sum[warp][i * kM + m] = sum[i][m];
        __syncthreads();
        if (part != 0) return;
        for (uint32_t p = 1; p < splits; ++p)
#pragma unroll
            for (int i = 0; i < kW; ++i)
#pragma unroll
                for (int m = 0; m < kM; ++m) sum[i][m] += part_sum[warp + p][i * kM + m];
    }
    if (col >= a.n) return;
    auto put = [&](int i, int m, uint32_t c, float x) {
        if (a.out[i]) a.out[i][m * a.ld[i] + c] = (uint16_t)pack2<kHalf>(x, 0.0f);
    };
#pragma unroll
    for (int m = 0; m < kM; ++m) {
        if (kKind == kGate) {
            if (lane != m) continue;
            put(0, m, col, act_at(a.act, sum[0][m]) * sum[1][m]);
            put(1, m, col, sum[0][m]);
            put(2, m, col, sum[1][m]);
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (lane != 2 * m + i || col + i >= a.n) continue;
                float x = sum[i][m];
                if (a.residual) x += unpack2<kHalf>(a.residual[m * a.ldr + col + i]).x;
                put(0, m, col + i, x);
            }
        }
    }
}

// ---------------------------------------------------------------- rows off 16-byte boundaries
// The five products for operands that neither TMA nor 16-byte loads can address (an odd number of
// contiguous columns, a slice that starts anywhere): tiles of 128 x 128 (gate: 128 x 64, twice) in
// binary32 on the ordinary cores, 8 x 8 results a thread, 16 of the sum at a time through shared
// memory, in partial sums of 768 as above. Bound by the multiply-adds: 31-44 TFLOP/s at 4096 x 2047 x
// 4095, the five kinds.
struct AnyArgs {
    const uint16_t *a[2], *b[2], *b_up;
    uint64_t lda[2], ldb[2], ldb_up;
    uint32_t k[2];
    uint32_t m, n;
    int32_t act, residual, accumulate;
    const uint16_t *in0, *in1;
    uint64_t ld_in0, ld_in1;
    void* out[3];
    uint64_t ld[3];
};
constexpr int kAnyM = 128, kAnyK = 16, kAnyPad = 4;
template <int kKind>
constexpr int kAnyN = kKind == kGate ? 64 : 128;

template <int kKind, bool kHalf>
__global__ void __launch_bounds__(256) k_any(const __grid_constant__ AnyArgs a) {
    constexpr bool kAcrossA = kKind == kWGrad;
    constexpr bool kAcrossB = kKind == kDownBwd || kKind == kGateBwd || kKind == kWGrad;
    constexpr int kN = kAnyN<kKind>, kTn = kN / 16, kSets = kKind == kGate ? 2 : 1;
    constexpr int kProducts = kKind == kGateBwd ? 2 : 1;
    __shared__ __align__(16) float sa[kAnyK][kAnyM + kAnyPad];
    __shared__ __align__(16) float sb[kSets][kAnyK][kN + kAnyPad];
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    grid_dep_wait();
    grid_dep_launch();
    const uint32_t col0 = blockIdx.x * kN;
    for (uint32_t tile = blockIdx.y; tile * kAnyM < a.m; tile += gridDim.y) {
        const uint32_t row0 = tile * kAnyM;
        float sum[kSets][8][kTn], part[kSets][8][kTn];
#pragma unroll
        for (int s = 0; s < kSets; ++s)
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int j = 0; j < kTn; ++j) sum[s][i][j] = part[s][i][j] = 0.0f;
        // entry (own, k) of an operand, 0 outside of it
        auto at = [](const uint16_t* p, uint64_t ld, bool across, uint32_t own, uint32_t owns,
                     uint32_t k, uint32_t ks) {
            return own < owns && k < ks ? p[across ? k * ld + own : own * ld + k] : (uint16_t)0;
        };
        constexpr int kLa = kAnyM * kAnyK / 256, kLb = kN * kAnyK / 256;  // a thread's loads
        uint16_t ra[kLa], rb[kSets][kLb];
        // neighbouring threads take neighbouring entries in memory
        auto load = [&](int q, uint32_t k0) {
#pragma unroll
            for (int i = 0; i < kLa; ++i) {
                const int e = tid + 256 * i;
                ra[i] = at(a.a[q], a.lda[q], kAcrossA, row0 + (kAcrossA ? e % kAnyM : e / kAnyK), a.m,
                           k0 + (kAcrossA ? e / kAnyM : e % kAnyK), a.k[q]);
            }
#pragma unroll
            for (int i = 0; i < kLb; ++i) {
                const int e = tid + 256 * i;
                const uint32_t n = col0 + (kAcrossB ? e % kN : e / kAnyK);
                const uint32_t k = k0 + (kAcrossB ? e / kN : e % kAnyK);
                rb[0][i] = at(a.b[q], a.ldb[q], kAcrossB, n, a.n, k, a.k[q]);
                if (kKind == kGate) rb[kSets - 1][i] = at(a.b_up, a.ldb_up, false, n, a.n, k, a.k[q]);
            }
        };
        for (int q = 0; q < kProducts; ++q) {
            load(q, 0);
            for (uint32_t k0 = 0; k0 < a.k[q]; k0 += kAnyK) {
#pragma unroll
                for (int i = 0; i < kLa; ++i) {
                    const int e = tid + 256 * i;
                    sa[kAcrossA ? e / kAnyM : e % kAnyK][kAcrossA ? e % kAnyM : e / kAnyK] =
                        unpack2<kHalf>(ra[i]).x;
                }
#pragma unroll
                for (int i = 0; i < kLb; ++i) {
                    const int e = tid + 256 * i;
#pragma unroll
                    for (int s = 0; s < kSets; ++s)
                        sb[s][kAcrossB ? e / kN : e % kAnyK][kAcrossB ? e % kN : e / kAnyK] =
                            unpack2<kHalf>(rb[s][i]).x;
                }
                __syncthreads();
                if (k0 + kAnyK < a.k[q]) load(q, k0 + kAnyK);  // on their way during the products
#pragma unroll
                for (int k = 0; k < kAnyK; ++k) {
                    float x[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = sa[k][ty * 8 + i];
#pragma unroll
                    for (int s = 0; s < kSets; ++s)
#pragma unroll
                        for (int j = 0; j < kTn; ++j) {
                            const float y = sb[s][k][tx * kTn + j];
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                part[s][i][j] = fmaf(x[i], y, part[s][i][j]);
                        }
                }
                __syncthreads();
                if (k0 / kAnyK % (kSumSlices * kBlockK / kAnyK) ==
                        kSumSlices * kBlockK / kAnyK - 1 || k0 + kAnyK >= a.k[q]) {
#pragma unroll
                    for (int s = 0; s < kSets; ++s)
#pragma unroll
                        for (int i = 0; i < 8; ++i)
#pragma unroll
                            for (int j = 0; j < kTn; ++j) {
                                sum[s][i][j] += part[s][i][j];
                                part[s][i][j] = 0.0f;
                            }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t y = row0 + ty * 8 + i;
            if (y >= a.m) continue;
#pragma unroll
            for (int j = 0; j < kTn; ++j) {
                const uint32_t x = col0 + tx * kTn + j;
                if (x >= a.n) continue;
                const float v = sum[0][i][j];
                auto put = [&](int o, float f) {
                    if (a.out[o])
                        static_cast<uint16_t*>(a.out[o])[y * a.ld[o] + x] =
                            (uint16_t)pack2<kHalf>(f, 0.0f);
                };
                if (kKind == kWGrad) {
                    float* d = static_cast<float*>(a.out[0]) + y * a.ld[0] + x;
                    *d = a.accumulate ? *d + v : v;
                } else if (kKind == kGate) {
                    const float u = sum[kSets - 1][i][j];
                    put(0, act_at(a.act, v) * u);
                    put(1, v);
                    put(2, u);
                } else if (kKind == kDownBwd) {
                    const float g = unpack2<kHalf>(a.in0[y * a.ld_in0 + x]).x;
                    const float u = unpack2<kHalf>(a.in1[y * a.ld_in1 + x]).x;
                    const ActValue f = act_both_at(a.act, g);
                    put(0, v * u * f.slope);
                    put(1, v * f.value);
                } else {
                    put(0, a.residual ? v + unpack2<kHalf>(a.in0[y * a.ld_in0 + x]).x : v);
                }
            }
        }
    }
}

// The parts of a weight gradient, added in order: dW = (dW +) sum over s of part_s. Reads what the
// products have just left in L2: 4 parts of 1024 x 1024 in about 5 us.
__global__ void __launch_bounds__(256) k_wgrad_join(const float* part, uint64_t part_ld,
                                                    uint64_t split_stride, uint32_t splits,
                                                    float* dw, uint64_t ld, uint32_t rows,
                                                    uint32_t cols, int accumulate) {
    const uint32_t x = blockIdx.x * 256 + threadIdx.x;
    grid_dep_wait();
    if (x >= cols) return;
    for (uint32_t y = blockIdx.y; y < rows; y += gridDim.y) {
        const float* p = part + (uint64_t)y * part_ld + x;
        float s = 0.0f;
        for (uint32_t i = 0; i < splits; ++i) s += p[i * split_stride];
        float* d = dw + (uint64_t)y * ld + x;
        *d = accumulate ? *d + s : s;
    }
}

// Empty sums over no rows at all: dW = 0.
__global__ void __launch_bounds__(256) k_wgrad_zero(float* dw, uint64_t ld, uint32_t rows,
                                                    uint32_t cols) {
    const uint32_t x = blockIdx.x * 256 + threadIdx.x;
    if (x >= cols) return;
    for (uint32_t y = blockIdx.y; y < rows; y += gridDim.y) dw[(uint64_t)y * ld + x] = 0.0f;
}

// ----------------------------------------------------------------------------------- host
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static EncodeFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            p = nullptr;
        }
        return reinterpret_cast<EncodeFn>(p);
    }();
    return fn;
}

struct Mat {  // a checked matrix
    void* p;
    uint64_t rows, cols, ld;
    int32_t dtype;
    // whether TMA can address its rows
    bool aligned() const {
        return rows == 0 || cols == 0 || (((uintptr_t)p & 15u) == 0 && (ld & 7) == 0);
    }
};
bool aligned(const Mat* m) { return !m || m->aligned(); }

// A matrix argument of 16-bit entries.
int check_matrix(const dgc_matrix* m, Mat* out, int32_t dtype) {
    if (!m || m->rows < 0 || m->cols < 0 || m->reserved != 0) return DGC_EINVAL;
    if (m->dtype != DGC_F16 && m->dtype != DGC_BF16) return DGC_EINVAL;
    if (dtype >= 0 && m->dtype != dtype) return DGC_EINVAL;
    if (m->rows > kMaxExtent || m->cols > kMaxExtent) return DGC_EUNSUPPORTED;
    *out = Mat{m->data, (uint64_t)m->rows, (uint64_t)m->cols, (uint64_t)m->ld, m->dtype};
    if (m->rows == 0 || m->cols == 0) return DGC_OK;
    if (!m->data || ((uintptr_t)m->data & 1u)) return DGC_EINVAL;
    if (m->rows == 1) {
        out->ld = ((uint64_t)m->cols + 7) & ~7ull;
        return DGC_OK;
    }
    if (m->ld < m->cols) return DGC_EINVAL;
    if (m->ld > (1ll << 36)) return DGC_EUNSUPPORTED;
    return DGC_OK;
}
bool shaped(const Mat& m, uint64_t rows, uint64_t cols) { return m.rows == rows && m.cols == cols; }

// A box of bc x br entries of a matrix; bytes of a box row: 64 or 128, which is the swizzle too.
int make_map(CUtensorMap* map, const Mat& m, uint32_t bc, uint32_t br) {
    EncodeFn fn = encode_fn();
    if (!fn) return DGC_ECUDA;
    const uint32_t es = m.dtype == DGC_F32 ? 4 : 2;
    const cuuint64_t dims[2] = {m.cols, m.rows};
    const cuuint64_t strides[1] = {m.ld * es};
    const cuuint32_t box[2] = {bc, br}, step[2] = {1, 1};
    const CUtensorMapDataType type = m.dtype == DGC_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                     : m.dtype == DGC_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                          : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    auto encode = [&] {
        return fn(map, type, 2, m.p, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  bc * es == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    };
    CUresult r = encode();
    if (r == CUDA_ERROR_INVALID_CONTEXT) {
        // A driver call, in a thread whose first CUDA call this is: the runtime makes the device's
        // context the thread's own at the first of its calls that needs one.
        cudaFuncAttributes at;
        if (cudaFuncGetAttributes(&at, k_wgrad_zero) != cudaSuccess) cudaGetLastError();
        r = encode();
    }
    return r == CUDA_SUCCESS ? DGC_OK : DGC_ECUDA;
}

uint32_t ceil_div(uint64_t a, uint64_t b) { return (uint32_t)((a + b - 1) / b); }

template <int kKind, int kCg, bool kSplit>
bool raise_smem() {
    return cudaFuncSetAttribute(k_ffn<kKind, kCg, kSplit>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)(kSmemLimit - 1024)) == cudaSuccess;
}
template <int kKind>
bool raise_smem_all() {
    return raise_smem<kKind, 1, false>() && raise_smem<kKind, 1, true>() &&
           raise_smem<kKind, 2, false>() && raise_smem<kKind, 2, true>();
}
// How many clusters of so many blocks the GPU holds at once, by the cluster's size. Those of a GPU
// with all its 152 SMs are what a plan goes by where it must not depend on the device.
struct Slots {
    int of[9];
};
constexpr Slots kFullSlots = {{0, 152, 76, 46, 36, 28, 23, 15, 15}};

// The shared-memory limit of every form of the kernel, the slots and the driver's entry point, once
// per device, by the first call that has work, whichever route it takes: the header promises that a
// capture after it only enqueues. First calls may come from several threads.
int ffn_device(const Slots** slots) {
    static std::atomic<bool> known[128];
    static std::mutex first;
    static Slots table[128];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return DGC_ECUDA;
    *slots = &table[dev];
    if (known[dev].load(std::memory_order_acquire)) return DGC_OK;
    std::lock_guard<std::mutex> lock(first);
    if (known[dev].load(std::memory_order_relaxed)) return DGC_OK;
    encode_fn();
    bool ok = raise_smem_all<kGate>() && raise_smem_all<kDown>() && raise_smem_all<kDownBwd>() &&
              raise_smem_all<kGateBwd>() && raise_smem_all<kWGrad>();
    for (unsigned size = 1; ok && size <= 8; ++size) {
        cudaLaunchConfig_t c{};
        c.gridDim = dim3(size * 256);
        c.blockDim = dim3(kFfnThreads);
        c.dynamicSmemBytes = kSmemLimit - 2048;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = size;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        c.attrs = at;
        c.numAttrs = 1;
        ok = cudaOccupancyMaxActiveClusters(&table[dev].of[size], k_ffn<kDown, 1, true>, &c) ==
                 cudaSuccess &&
             table[dev].of[1] > 0;
    }
    if (!ok) {
        cudaGetLastError();
        return DGC_ECUDA;
    }
    known[dev].store(true, std::memory_order_release);
    return DGC_OK;
}

template <int kKind, int kCg, bool kSplit>
int launch_ffn(FfnArgs& a, int32_t dtype, int sms, cudaStream_t s) {
    if (a.wait_ns == 0) {
        a.wait_ns = kFfnWaitNs;
        a.lost = ~0u;
    }
    constexpr bool kAcrossA = kKind == kWGrad;
    constexpr bool kAcrossB = kKind == kDownBwd || kKind == kGateBwd || kKind == kWGrad;
    a.stage_bytes = kStageA + a.bn / kCg * 128;
    constexpr uint32_t staging = Epilogue<kKind>::kBytes;
    a.stages = std::min<uint32_t>(kMaxStages, (kSmemLimit - 2048 - staging) / a.stage_bytes);
    a.load_bytes = (kAcrossA ? kBlockM : a.a_rows) * 128 * kCg + a.bn * 128;
    a.tmem_cols = 2 * a.bn;  // a power of two, 64 at least
    a.half = dtype == DGC_F16;
    const uint32_t type = dtype == DGC_F16 ? 0 : 1;
    a.idesc = (1u << 4) | (type << 7) | (type << 10) | ((uint32_t)kAcrossA << 15) |
              ((uint32_t)kAcrossB << 16) | ((a.bn >> 3) << 17) | ((kBlockM * kCg >> 4) << 24);
    a.group = 16 / kCg;
    const uint32_t smem = a.stages * a.stage_bytes + staging + 1024;
    const uint32_t cluster = kSplit ? a.splits * kCg : kCg;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(kSplit ? a.tiles * cluster
                            : std::min<uint32_t>(a.tiles, (uint32_t)sms / kCg) * kCg);
    c.blockDim = dim3(kFfnThreads);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    c.attrs = at;
    c.numAttrs = cluster > 1 ? 2 : 1;
    if (cudaLaunchKernelEx(&c, k_ffn<kKind, kCg, kSplit>, a) != cudaSuccess) {
        cudaGetLastError();
        return DGC_ECUDA;
    }
    dgc_internal_count_launches(1);
    return DGC_OK;
}

// How a product is cut: pairs of blocks or single ones, the tile's columns, the parts of its sum.
struct Plan {
    bool pairs;
    uint32_t bn, splits;
    uint64_t cost;
};
// A product as the model below sees it.
struct Shape {
    uint64_t m, n;
    uint32_t kb, halves, narrowest;
    uint32_t a_rows;    // rows of A that a tile loads
    uint32_t epilogue;  // clocks per column of a tile
};
// The cheapest of the shapes that the kernel has, in SM clocks, by a model that was fitted to the
// times of every shape on 279 products (3 to 8192 rows, 64 to 11264 columns, more than half of them
// odd; its choices take 0.9% longer than the best ones). A tile's slice of 64 costs the tensor
// cores 2.2 bn (2 bn by count), the way from L2 a clock per 68 of its operand bytes, the issuing
// loop 300: the largest counts; a pair's agreement adds 22, and a lone block's 256-column tile,
// whose stages are the fewest, a quarter. A tile's epilogue costs `epilogue` bn and 1200; the last
// one's shows in full, the others hide behind the sums, or the sums behind them. A split sum pays
// for its cluster's start and barriers, and for moving the parts; in more than one wave it was
// never worth that.
uint64_t slice_cost(const Shape& p, uint32_t bn, uint32_t cg) {
    const uint64_t bytes = (p.a_rows + bn / cg) * 128;
    uint64_t cost = std::max<uint64_t>({300, bn * 11 / 5, bytes / 68});
    if (cg == 2) return cost + 22;
    return bn == 256 && p.a_rows > 64 ? cost + cost / 4 : cost;
}
Plan choose_plan(const Shape& p, const Slots& slots) {
    constexpr uint32_t kCluster[9] = {0, 0, 10, 19, 15, 0, 23, 0, 24};  // tenths of a pair's start
    Plan best{false, 256, 1, ~0ull};
    for (int pairs = 1; pairs >= 0; --pairs) {
        if (pairs && p.m <= kBlockM) continue;
        const uint32_t cg = pairs ? 2 : 1;
        for (uint32_t bn = 256; bn >= (pairs ? std::max(128u, p.narrowest) : p.narrowest); bn /= 2) {
            const uint64_t slice = slice_cost(p, bn, cg);
            const uint64_t tiles =
                (uint64_t)ceil_div(p.m, kBlockM * cg) * ceil_div(p.n, bn / p.halves);
            for (uint32_t splits = 1; splits <= 4 && (splits == 1 || splits * 4 <= p.kb); ++splits) {
                const uint32_t cluster = splits * cg;
                const uint64_t held = (uint64_t)std::max(1, slots.of[cluster]);
                const uint64_t waves = (tiles + held - 1) / held;
                if (splits > 1 && waves > 1) continue;
                const uint64_t tile = (p.kb + splits - 1) / splits * slice;
                uint64_t cost = waves * std::max<uint64_t>(tile, p.epilogue * bn + 1200) +
                                p.epilogue * bn / splits;
                if (pairs) cost += 770;
                if (splits > 1) cost += kCluster[cluster] * (3100 + bn * 6 / 5) / 10;
                if (cost < best.cost) best = Plan{pairs != 0, bn, splits, cost};
            }
        }
    }
    return best;
}

template <int kKind>
int launch_plan(FfnArgs& a, const Plan& p, int32_t dtype, int sms, cudaStream_t s) {
    a.splits = p.splits;
    a.kb_split = ceil_div(a.kb, p.splits);
    if (p.splits > 1)
        return p.pairs ? launch_ffn<kKind, 2, true>(a, dtype, sms, s)
                       : launch_ffn<kKind, 1, true>(a, dtype, sms, s);
    return p.pairs ? launch_ffn<kKind, 2, false>(a, dtype, sms, s)
                   : launch_ffn<kKind, 1, false>(a, dtype, sms, s);
}

// A product along rows: A [m, k] K-major, against B [n, k] K-major or [k, n] across.
struct Product {
    const Mat *a, *b;
};

template <int kKind, bool kHalf, bool kAligned>
int launch_rows(const RowsArgs& a, uint32_t m, unsigned grid, cudaStream_t s) {
    auto kernel = m == 1 ? k_rows<kKind, kHalf, 1, kAligned> : k_rows<kKind, kHalf, 2, kAligned>;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(grid);
    c.blockDim = dim3(32 * kRowsWarps);
    c.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    c.attrs = at;
    c.numAttrs = 1;
    if (cudaLaunchKernelEx(&c, kernel, a) != cudaSuccess) {
        cudaGetLastError();
        return DGC_ECUDA;
    }
    dgc_internal_count_launches(1);
    return DGC_OK;
}

template <int kKind>
int launch_any(const AnyArgs& a, int32_t dtype, cudaStream_t s) {
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(ceil_div(a.n, kAnyN<kKind>),
                     std::min<uint32_t>(ceil_div(a.m, kAnyM), 65535));
    c.blockDim = dim3(256);
    c.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    c.attrs = at;
    c.numAttrs = 1;
    const cudaError_t e = dtype == DGC_F16 ? cudaLaunchKernelEx(&c, k_any<kKind, true>, a)
                                           : cudaLaunchKernelEx(&c, k_any<kKind, false>, a);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return DGC_ECUDA;
    }
    dgc_internal_count_launches(1);
    return DGC_OK;
}

// The products of up to kFewTokens tokens, with enough warps to a sum that the SMs have 16 each.
template <int kKind>
int few_tokens(const Mat& x, const Mat& w0, const Mat* w1, const Mat* residual,
               const Mat* const (&outs)[3], int32_t act, int sms, cudaStream_t s) {
    RowsArgs a{};
    a.x = static_cast<const uint16_t*>(x.p);
    a.ldx = x.ld;
    a.w0 = static_cast<const uint16_t*>(w0.p);
    a.ldw0 = w0.ld;
    if (w1) {
        a.w1 = static_cast<const uint16_t*>(w1->p);
        a.ldw1 = w1->ld;
    }
    if (residual) {
        a.residual = static_cast<const uint16_t*>(residual->p);
        a.ldr = residual->ld;
    }
    for (int i = 0; i < 3; ++i)
        if (outs[i]) {
            a.out[i] = static_cast<uint16_t*>(outs[i]->p);
            a.ld[i] = outs[i]->ld;
        }
    a.n = (uint32_t)w0.rows;
    a.k = (uint32_t)w0.cols;
    a.act = act;
    const uint64_t warps = kKind == kGate ? a.n : ceil_div(a.n, 2);
    while (a.log_split < 3 && (warps << a.log_split) < (uint64_t)sms * 16) ++a.log_split;
    const unsigned grid = ceil_div(warps << a.log_split, kRowsWarps);
    const uint32_t m = (uint32_t)x.rows;
    if (x.aligned() && w0.aligned() && aligned(w1))
        return x.dtype == DGC_F16 ? launch_rows<kKind, true, true>(a, m, grid, s)
                                  : launch_rows<kKind, false, true>(a, m, grid, s);
    return x.dtype == DGC_F16 ? launch_rows<kKind, true, false>(a, m, grid, s)
                              : launch_rows<kKind, false, false>(a, m, grid, s);
}

template <int kKind>
int rows_product(Product p0, const Product* p1, const Mat* b_up, const Mat* in0, const Mat* in1,
                 const Mat* out0, const Mat* out1, const Mat* out2, int32_t act, int32_t* status,
                 dgc_stream_t stream, uint32_t test_wait_ms = 0) {
    constexpr bool kAcrossB = kKind == kDownBwd || kKind == kGateBwd;
    const int sms = dgc_internal_sm_count();
    if (sms <= 0) return DGC_ECUDA;
    const Slots* slots;
    int rc = ffn_device(&slots);
    if (rc) return rc;
    const Mat* const outs[3] = {out0, out1, out2};
    if constexpr (kKind == kGate || kKind == kDown)
        if (out0->rows <= kFewTokens && !test_wait_ms)
            return few_tokens<kKind>(*p0.a, *p0.b, b_up, in0, outs, act, sms,
                                     reinterpret_cast<cudaStream_t>(stream));
    if (!p0.a->aligned() || !p0.b->aligned() || !aligned(b_up) || !aligned(in0) || !aligned(in1) ||
        (p1 && (!p1->a->aligned() || !p1->b->aligned()))) {
        AnyArgs a{};
        const Product* products[2] = {&p0, p1};
        for (int i = 0; i < (p1 ? 2 : 1); ++i) {
            a.a[i] = static_cast<const uint16_t*>(products[i]->a->p);
            a.lda[i] = products[i]->a->ld;
            a.b[i] = static_cast<const uint16_t*>(products[i]->b->p);
            a.ldb[i] = products[i]->b->ld;
            a.k[i] = (uint32_t)products[i]->a->cols;
        }
        if (b_up) {
            a.b_up = static_cast<const uint16_t*>(b_up->p);
            a.ldb_up = b_up->ld;
        }
        if (in0) {
            a.in0 = static_cast<const uint16_t*>(in0->p);
            a.ld_in0 = in0->ld;
        }
        if (in1) {
            a.in1 = static_cast<const uint16_t*>(in1->p);
            a.ld_in1 = in1->ld;
        }
        for (int i = 0; i < 3; ++i)
            if (outs[i]) {
                a.out[i] = outs[i]->p;
                a.ld[i] = outs[i]->ld;
            }
        a.m = (uint32_t)out0->rows;
        a.n = (uint32_t)out0->cols;
        a.act = act;
        a.residual = in0 != nullptr;
        return launch_any<kKind>(a, out0->dtype, reinterpret_cast<cudaStream_t>(stream));
    }
    FfnArgs a{};
    if (test_wait_ms) {  // the self-test: the second slice never arrives
        a.wait_ns = test_wait_ms * 1000000ull;
        a.lost = 1;
    }
    a.m = (uint32_t)out0->rows;
    a.n = (uint32_t)out0->cols;
    constexpr uint32_t halves = kKind == kGate ? 2 : 1;
    a.kb0 = ceil_div(p0.a->cols, kBlockK);
    a.kb = a.kb0 + (p1 ? ceil_div(p1->a->cols, kBlockK) : 0);
    a.a_rows = std::min<uint32_t>(kBlockM, (a.m + 7) & ~7u);
    const Plan plan = choose_plan(
        Shape{a.m, a.n, a.kb, halves, kKind == kDown ? 32u : 64u, a.a_rows,
              kKind == kDownBwd ? 23u : kKind == kGate ? 17u : kKind == kDown ? 14u : 12u},
        *slots);
    const bool pairs = plan.pairs;
    a.bn = plan.bn;
    a.tiles_m = ceil_div(a.m, pairs ? 2 * kBlockM : kBlockM);
    a.tiles_n = ceil_div(a.n, a.bn / halves);
    if ((uint64_t)a.tiles_m * a.tiles_n > 0x3FFFFFFFull) return DGC_EUNSUPPORTED;
    a.tiles = a.tiles_m * a.tiles_n;
    a.act = act;
    a.status = status;
    auto operand = [&](CUtensorMap* map, const Mat& m, uint32_t bc, uint32_t br) {
        if (!rc && m.rows && m.cols) rc = make_map(map, m, bc, br);
    };
    auto b_map = [&](CUtensorMap* map, const Mat& m) {
        if (kAcrossB)
            operand(map, m, 64, kBlockK);
        else
            operand(map, m, kBlockK, a.bn / (pairs ? 2 : halves));
    };
    operand(&a.a0, *p0.a, kBlockK, a.a_rows);
    b_map(&a.b0, *p0.b);
    if (b_up) b_map(&a.b1, *b_up);
    if (p1) {
        operand(&a.a1, *p1->a, kBlockK, a.a_rows);
        b_map(&a.b1, *p1->b);
    }
    for (int i = 0; i < 3; ++i)
        if (outs[i]) {
            a.out[i] = outs[i]->p;
            a.ld[i] = outs[i]->ld;
        }
    a.ragged = (a.n & 7) != 0;
    a.unaligned = !out0->aligned() || !aligned(out1) || !aligned(out2);
    if (!a.unaligned) {
        operand(&a.out0, *out0, 32, 32);
        if (out1) operand(&a.out1, *out1, 32, 32);
        if (out2) operand(&a.out2, *out2, 32, 32);
    }
    if (in0) operand(&a.in0, *in0, 32, 32);
    if (in1) operand(&a.in1, *in1, 32, 32);
    if (rc) return rc;
    a.residual = kKind == kGate ? out1 != nullptr : in0 != nullptr;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return launch_plan<kKind>(a, plan, out0->dtype, sms, s);
}

bool bad_act(int32_t act) { return act < DGC_ACT_SILU || act > DGC_ACT_RELU; }

// A weight gradient's cut. Where the weight is small and the tokens are many, the sum is cut into
// parts whose results go to the workspace and are added in order by k_wgrad_join: on the narrowest
// tiles where even clusters would leave most SMs idle, or on the widest, which need the fewest
// operand bytes, where that is cheaper than the best cut without (the join: a read and a write of
// every part and 3000 clocks; 65536 tokens x 512 x 512 34.8 us, by clusters 52.8; 32768 x 1024 x
// 1024 49 and 54). By sizes alone, for 152 SMs, so that the workspace can be asked for without a
// device.
struct WgradPlan {
    Plan cut;
    uint32_t parts;
};
WgradPlan wgrad_plan(uint64_t rows, uint64_t cols, uint64_t tokens) {
    const uint64_t sms = kFullSlots.of[1], pairs = kFullSlots.of[2];
    const uint32_t kb = ceil_div(tokens, kBlockK);
    const uint64_t narrow = (uint64_t)ceil_div(rows, kBlockM) * ceil_div(cols, 64);
    const uint64_t wide = (uint64_t)ceil_div(rows, 256) * ceil_div(cols, 256);
    if (narrow && narrow <= 16 && kb >= 64)
        return {Plan{false, 64, 1, 0}, (uint32_t)std::min<uint64_t>(sms / narrow, kb / 8)};
    const Shape shape{rows, cols, kb, 1, 64, kBlockM, 15};
    WgradPlan best{choose_plan(shape, kFullSlots), 1};
    for (uint32_t parts = 2; wide && rows > kBlockM && wide * parts <= pairs && parts * 32 <= kb;
         ++parts) {
        const uint64_t cost = ceil_div(kb, parts) * slice_cost(shape, 256, 2) + 15 * 256 + 770 + 3000 +
                              rows * cols * 8 * (parts + 1) / 2600;
        if (cost < best.cut.cost) best = {Plan{true, 256, 1, cost}, parts};
    }
    return best;
}
uint64_t wgrad_workspace(uint64_t rows, uint64_t cols, uint64_t tokens) {
    const WgradPlan p = wgrad_plan(rows, cols, tokens);
    if (p.parts < 2) return 0;
    const uint64_t tile = p.cut.pairs ? 2 * kBlockM : kBlockM;
    return p.parts * (ceil_div(rows, tile) * tile) * ((cols + 3) & ~3ull) * sizeof(float);
}

}  // namespace
}  // namespace dgc

using namespace dgc;

extern "C" int dgc_ffn_gate(const dgc_matrix* x, const dgc_matrix* w_gate, const dgc_matrix* w_up,
                            int32_t act, const dgc_matrix* hidden, const dgc_matrix* gate,
                            const dgc_matrix* up, int32_t* status, dgc_stream_t stream) {
    Mat mx, mg, mu, mh, og, ou;
    int rc;
    if (!x || !status || bad_act(act) || (gate == nullptr) != (up == nullptr)) return DGC_EINVAL;
    if ((rc = check_matrix(x, &mx, -1)) || (rc = check_matrix(w_gate, &mg, mx.dtype)) ||
        (rc = check_matrix(w_up, &mu, mx.dtype)) || (rc = check_matrix(hidden, &mh, mx.dtype)))
        return rc;
    if (gate && ((rc = check_matrix(gate, &og, mx.dtype)) || (rc = check_matrix(up, &ou, mx.dtype))))
        return rc;
    const uint64_t m = mx.rows, d = mx.cols, f = mg.rows;
    if (!shaped(mg, f, d) || !shaped(mu, f, d) || !shaped(mh, m, f)) return DGC_EINVAL;
    if (gate && (!shaped(og, m, f) || !shaped(ou, m, f))) return DGC_EINVAL;
    if (m == 0 || f == 0) return DGC_OK;
    return rows_product<kGate>({&mx, &mg}, nullptr, &mu, nullptr, nullptr, &mh,
                               gate ? &og : nullptr, gate ? &ou : nullptr, act, status, stream);
}

static int ffn_down(const dgc_matrix* hidden, const dgc_matrix* w_down, const dgc_matrix* residual,
                    const dgc_matrix* y, int32_t* status, dgc_stream_t stream,
                    uint32_t test_wait_ms) {
    Mat mh, mw, mr, my;
    int rc;
    if (!hidden || !status) return DGC_EINVAL;
    if ((rc = check_matrix(hidden, &mh, -1)) || (rc = check_matrix(w_down, &mw, mh.dtype)) ||
        (rc = check_matrix(y, &my, mh.dtype)))
        return rc;
    if (residual && (rc = check_matrix(residual, &mr, mh.dtype))) return rc;
    const uint64_t m = mh.rows, f = mh.cols, d = mw.rows;
    if (!shaped(mw, d, f) || !shaped(my, m, d)) return DGC_EINVAL;
    if (residual && !shaped(mr, m, d)) return DGC_EINVAL;
    if (m == 0 || d == 0) return DGC_OK;
    return rows_product<kDown>({&mh, &mw}, nullptr, nullptr, residual ? &mr : nullptr, nullptr, &my,
                               nullptr, nullptr, 0, status, stream, test_wait_ms);
}

extern "C" int dgc_ffn_down(const dgc_matrix* hidden, const dgc_matrix* w_down,
                            const dgc_matrix* residual, const dgc_matrix* y, int32_t* status,
                            dgc_stream_t stream) {
    return ffn_down(hidden, w_down, residual, y, status, stream, 0);
}

extern "C" int dgc_selftest_ffn_timeout(const dgc_matrix* hidden, const dgc_matrix* w_down,
                                        const dgc_matrix* y, int32_t* status, uint32_t wait_ms,
                                        dgc_stream_t stream) {
    if (wait_ms == 0 || wait_ms > 1000) return DGC_EINVAL;
    return ffn_down(hidden, w_down, nullptr, y, status, stream, wait_ms);
}

extern "C" int dgc_ffn_down_backward(const dgc_matrix* dy, const dgc_matrix* w_down,
                                     const dgc_matrix* gate, const dgc_matrix* up, int32_t act,
                                     const dgc_matrix* d_gate, const dgc_matrix* d_up,
                                     int32_t* status, dgc_stream_t stream) {
    Mat my, mw, mg, mu, og, ou;
    int rc;
    if (!dy || !status || bad_act(act)) return DGC_EINVAL;
    if ((rc = check_matrix(dy, &my, -1)) || (rc = check_matrix(w_down, &mw, my.dtype)) ||
        (rc = check_matrix(gate, &mg, my.dtype)) || (rc = check_matrix(up, &mu, my.dtype)) ||
        (rc = check_matrix(d_gate, &og, my.dtype)) || (rc = check_matrix(d_up, &ou, my.dtype)))
        return rc;
    const uint64_t m = my.rows, d = my.cols, f = mw.cols;
    if (!shaped(mw, d, f) || !shaped(mg, m, f) || !shaped(mu, m, f) || !shaped(og, m, f) ||
        !shaped(ou, m, f))
        return DGC_EINVAL;
    if (m == 0 || f == 0) return DGC_OK;
    return rows_product<kDownBwd>({&my, &mw}, nullptr, nullptr, &mg, &mu, &og, &ou, nullptr, act,
                                  status, stream);
}

extern "C" int dgc_ffn_gate_backward(const dgc_matrix* d_gate, const dgc_matrix* d_up,
                                     const dgc_matrix* w_gate, const dgc_matrix* w_up,
                                     const dgc_matrix* residual, const dgc_matrix* dx,
                                     int32_t* status, dgc_stream_t stream) {
    Mat ag, au, mg, mu, mr, mx;
    int rc;
    if (!d_gate || !status) return DGC_EINVAL;
    if ((rc = check_matrix(d_gate, &ag, -1)) || (rc = check_matrix(d_up, &au, ag.dtype)) ||
        (rc = check_matrix(w_gate, &mg, ag.dtype)) || (rc = check_matrix(w_up, &mu, ag.dtype)) ||
        (rc = check_matrix(dx, &mx, ag.dtype)))
        return rc;
    if (residual && (rc = check_matrix(residual, &mr, ag.dtype))) return rc;
    const uint64_t m = ag.rows, f = ag.cols, d = mg.cols;
    if (!shaped(au, m, f) || !shaped(mg, f, d) || !shaped(mu, f, d) || !shaped(mx, m, d))
        return DGC_EINVAL;
    if (residual && !shaped(mr, m, d)) return DGC_EINVAL;
    if (m == 0 || d == 0) return DGC_OK;
    const Product second{&au, &mu};
    return rows_product<kGateBwd>({&ag, &mg}, &second, nullptr, residual ? &mr : nullptr, nullptr,
                                  &mx, nullptr, nullptr, 0, status, stream);
}

extern "C" int dgc_ffn_weight_grad_workspace(int64_t rows, int64_t cols, int64_t tokens,
                                             size_t* bytes) {
    if (!bytes || rows < 0 || cols < 0 || tokens < 0) return DGC_EINVAL;
    if (rows > kMaxExtent || cols > kMaxExtent || tokens > kMaxExtent) return DGC_EUNSUPPORTED;
    *bytes = (size_t)wgrad_workspace((uint64_t)rows, (uint64_t)cols, (uint64_t)tokens);
    return DGC_OK;
}

extern "C" int dgc_ffn_weight_grad(const dgc_matrix* dy, const dgc_matrix* x, int32_t accumulate,
                                   const dgc_matrix* dw, int32_t* status, void* ws,
                                   size_t ws_bytes, dgc_stream_t stream) {
    Mat my, mx;
    int rc;
    if (!dy || !dw || !status) return DGC_EINVAL;
    if ((rc = check_matrix(dy, &my, -1)) || (rc = check_matrix(x, &mx, my.dtype))) return rc;
    if (dw->rows < 0 || dw->cols < 0 || dw->reserved != 0 || dw->dtype != DGC_F32) return DGC_EINVAL;
    if (mx.rows != my.rows || (uint64_t)dw->rows != my.cols || (uint64_t)dw->cols != mx.cols)
        return DGC_EINVAL;
    if (dw->rows == 0 || dw->cols == 0) return DGC_OK;
    if (!dw->data || ((uintptr_t)dw->data & 3u) || (dw->rows > 1 && dw->ld < dw->cols))
        return DGC_EINVAL;
    if (dw->rows > 1 && dw->ld > (1ll << 36)) return DGC_EUNSUPPORTED;
    const uint64_t rows = my.cols, cols = mx.cols, tokens = my.rows;
    const uint64_t need = wgrad_workspace(rows, cols, tokens);
    if (ws_bytes < need || (need && (!ws || ((uintptr_t)ws & 255u)))) return DGC_EINVAL;
    const int sms = dgc_internal_sm_count();
    if (sms <= 0) return DGC_ECUDA;
    const Slots* slots;  // the plan does not go by them
    if ((rc = ffn_device(&slots))) return rc;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    auto launched = [] {
        if (cudaPeekAtLastError() != cudaSuccess) {
            cudaGetLastError();
            return (int)DGC_ECUDA;
        }
        dgc_internal_count_launches(1);
        return (int)DGC_OK;
    };
    const Mat out{dw->data, rows, cols, rows == 1 ? (cols + 3) & ~3ull : (uint64_t)dw->ld, DGC_F32};
    const dim3 grid2(ceil_div(cols, 256), (unsigned)std::min<uint64_t>(rows, 4096));
    if (tokens == 0) {
        if (accumulate) return DGC_OK;
        k_wgrad_zero<<<grid2, 256, 0, s>>>((float*)out.p, out.ld, (uint32_t)rows, (uint32_t)cols);
        return launched();
    }
    if (!my.aligned() || !mx.aligned()) {
        AnyArgs a{};
        a.a[0] = static_cast<const uint16_t*>(my.p);
        a.lda[0] = my.ld;
        a.b[0] = static_cast<const uint16_t*>(mx.p);
        a.ldb[0] = mx.ld;
        a.k[0] = (uint32_t)tokens;
        a.m = (uint32_t)rows;
        a.n = (uint32_t)cols;
        a.accumulate = accumulate != 0;
        a.out[0] = out.p;
        a.ld[0] = out.ld;
        return launch_any<kWGrad>(a, my.dtype, s);
    }
    FfnArgs a{};
    a.m = (uint32_t)rows;
    a.n = (uint32_t)cols;
    a.a_rows = kBlockM;
    a.kb0 = a.kb = ceil_div(tokens, kBlockK);
    a.status = status;
    if ((rc = make_map(&a.a0, my, 64, kBlockK)) || (rc = make_map(&a.b0, mx, 64, kBlockK))) return rc;
    const WgradPlan wp = wgrad_plan(rows, cols, tokens);
    const Plan plan = wp.cut;
    const uint32_t parts = wp.parts;
    a.bn = plan.bn;
    const uint32_t tile_rows = plan.pairs ? 2 * kBlockM : kBlockM;
    a.tiles_m = ceil_div(rows, tile_rows);
    a.tiles_n = ceil_div(cols, a.bn);
    if ((uint64_t)a.tiles_m * a.tiles_n > 0x3FFFFFFFull) return DGC_EUNSUPPORTED;
    if (parts > 1) {
        a.kb_split = ceil_div(a.kb, parts);
        const uint32_t used = ceil_div(a.kb, a.kb_split);
        a.tiles = a.tiles_m * a.tiles_n * used;
        a.split_rows = a.tiles_m * tile_rows;
        const Mat part{ws, (uint64_t)a.split_rows * used, cols, (cols + 3) & ~3ull, DGC_F32};
        if ((rc = make_map(&a.out0, part, 32, 32))) return rc;
        rc = plan.pairs ? launch_ffn<kWGrad, 2, false>(a, my.dtype, sms, s)
                        : launch_ffn<kWGrad, 1, false>(a, my.dtype, sms, s);
        if (rc) return rc;
        cudaLaunchConfig_t c{};
        c.gridDim = grid2;
        c.blockDim = dim3(256);
        c.stream = s;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[0].val.programmaticStreamSerializationAllowed = 1;
        c.attrs = at;
        c.numAttrs = 1;
        cudaLaunchKernelEx(&c, k_wgrad_join, (const float*)ws, part.ld, part.ld * a.split_rows, used,
                           (float*)out.p, out.ld, (uint32_t)rows, (uint32_t)cols, (int)accumulate);
        return launched();
    }
    a.tiles = a.tiles_m * a.tiles_n;
    a.accumulate = accumulate != 0;
    a.out[0] = out.p;
    a.ld[0] = out.ld;
    a.ragged = (cols & 3) != 0;
    a.unaligned = ((uintptr_t)out.p & 15u) || (out.ld & 3u);
    if (!a.unaligned && (rc = make_map(&a.out0, out, 32, 32))) return rc;
    return launch_plan<kWGrad>(a, plan, my.dtype, sms, s);
}
