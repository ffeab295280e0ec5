// moe_tc.cu -- the experts' products for many rows, on the tensor cores:
//   h[p] = act(x[t] Wg[e]^T) * (x[t] Wu[e]^T)   for each slot p = (t, j), e = indices[p]
//   y[t] = sum_j weights[t, j] (h[t, j] Wd[e]^T)
//
// Kernels of one call:
//   1. prep      slots ordered by expert (stable), x copied into that order,
//                each expert's rows cut into chunks of at most `cap` rows;
//   2. gate/up   grouped product with the gated activation in its epilogue;
//   3. down      grouped product, one fp32 row per slot;
//   4. combine   a token's rows added in slot order with their weights and
//                rounded once.
// Both products are moe_tc_kernel.  Everything lies in the caller's workspace.
//
// The product.  D[n, m] (+)= W~[n, k] x[m, k]: 128 weight rows are the MMA's M,
// up to 192 activation rows its N, k runs in blocks of 64.  The packed weight is
// dequantized on chip into tensor memory (operand A); the activations are
// operand B in shared memory.  The first product's 128 rows are 64 gate and 64
// up rows, placed so that the two rows of a feature are 16 lanes apart in one
// warp: the epilogue exchanges halves by shuffle and writes h once.
//
// Order of k.  One 32-bit word holds codes 0..7; masks and shifts give codes e
// and e + 4 in the two halves of a register, so a block's elements enter the
// MMA in the order 0 4 1 5 2 6 3 7 of every eight.  The sum does not depend on
// it: x is copied, and h written, in the same order.
//
// E2M1 to 16 bits.  Sign, exponent and mantissa bits of a code land in a
// register half as a number 2^-126 (bf16) or 2^-14 (f16) times its value,
// subnormals included, and one packed multiply by X 2^126 (X 2^14) gives
// X * element exactly.  Scales for which that factor leaves the type's range
// take the element values in fp32 instead.
//
// Roles (one CTA per SM, 25 warps, persistent over chunk x 128-row tiles; the
// roles that everything waits for have the lowest warp numbers):
//   0-3    epilogue;
//   4      issues the MMAs, by one lane;
//   5, 6   TMA of packed tiles (gate and up, or the down tile), 256 k at a time,
//          and of their scales (and biases), a window of 16 bytes a row;
//   7      TMA of activation tiles;
//   8-23   dequantize, four groups of four warps, each one or two blocks of a
//          packed tile;
//   24     scale windows by asynchronous copies of 32 bytes a row, where a row of
//          scales is not made of whole 16 bytes (300 rows x 3 of 10 experts 4160
//          x 4160 mxfp4: 160 us, 255 with loads of 2 bytes).
// Three rings: packed tiles and windows, activation tiles, and dequantized
// blocks in tensor memory.  A barrier's hand-over costs its waiter 150 cycles
// and more even when it need not wait, an MMA 40 and a TMA 200 cycles of their
// thread, whatever their sizes: so a packed tile is 256 elements wide, an
// activation tile comes in one box as high as the chunk needs (heights in
// kHeights), and k-blocks reach the MMA thread in units of 4 (of 2 with tall
// chunks, whose accumulators leave less tensor memory).
//
// Rounding.  The MMA's operands are 16 bits: h is rounded to the activations'
// type, and so is an affine weight s q + b; E2M1 weights are exact while X times
// the element is a normal value.  (Two 16-bit pieces per value would keep them,
// at twice the MMAs and twice the tensor memory; the library's GEMM rounds
// weights alike.)  The accumulators, and the rows that the combine adds, are fp32.
//
// Bound: with few rows per expert the dequantize warps' instructions (about 3
// per element), with many rows the tensor cores and, on short contractions, the
// epilogue.  Single cold calls: 2048 rows, 8 experts 4096 x 14336, 2 each, nvfp4:
// gate/up 645 us, down 416 us (1.36e15 operations a second; back to back, at the
// power limit, the whole call takes 1293 us, 1.1e15); 512 rows: 230 and 165 us.
// Two CTAs sharing an activation tile (MMAs of 256 rows) measured 741 and 446, 292
// and 200 us where one measured 777 and 465, 273 and 191: the hand-overs between
// the two cost what the halved copies save.
#include <cuda.h>

#include <algorithm>

#include "moe.cuh"
#include "mx.cuh"
#include "ptx_sm100.cuh"
#include "tcgen05.cuh"

namespace qmm {
namespace {

constexpr int kGroups = 4;
constexpr int kDqWarps = 4 * kGroups;
constexpr int kMmaWarp = 4;               // after the epilogue's 0..3
constexpr int kWWarp = kMmaWarp + 1;      // 5, 6
constexpr int kBWarp = kWWarp + 2;        // 7
constexpr int kDqWarp = kBWarp + 1;       // 8..23: a multiple of 4, warp % 4 is the tensor memory quarter
constexpr int kSWarp = kDqWarp + kDqWarps;  // 24
constexpr int kThreads = 32 * (kSWarp + 1);
constexpr int kBM = 128, kBK = 64;
constexpr int kStageK = kBK * kGroups;    // k per packed stage
constexpr int kPBytes = kBM * kStageK / 2;  // 16 KB
constexpr int kRing = 8;                  // hand-over barriers (more than units in flight)
constexpr int kBarBytes = 1024;           // barriers and the tensor-memory address
constexpr int kMaxCap = 192;              // activation rows of a tile at most
constexpr int kNumHeights = 6;
constexpr int kHeights[kNumHeights] = {16, 32, 64, 96, 128, 192};

// Chunks of at most CAP rows: two accumulators of CAP columns leave room for NU
// units of U dequantized k-blocks (32 columns each) in tensor memory; SB units
// of activations lie in shared memory.  A dequantize group takes BPG blocks per
// hand-over: two where the units are four blocks (32 rows x 8 of 64 experts: 84
// us against 92 with one and 94 with four), one where two units of two are all
// there is (2048 rows x 2 of 8: 1087 us against 1185 with two).
template <int CAP>
struct TileCfg {
    static constexpr int U = CAP <= 64 ? 4 : 2;
    static constexpr int NU = (512 - 2 * CAP) / (32 * U);
    static constexpr int BPG = CAP <= 64 ? 2 : 1;  // blocks of a stage per dequantize group
    static constexpr int SB = 3;
    static constexpr int BBytes = CAP * 128 * U;
};

struct MoeHeader {
    int num_chunks;
};

struct MoePlan {
    size_t hdr, chunks, pos, x, h, parts, total;
    int64_t max_chunks;
};

struct ActMaps {
    CUtensorMap m[kNumHeights];
};

// Per weight matrix: packed codes, and where whole 16-byte windows allow it
// scales and biases.
struct WeightMaps {
    CUtensorMap w[2], s[2], b[2];
};

struct TcParams {
    const void *scales[2], *biases[2];
    void *out;                // h [R / 64][rows][64] T, or parts [slots][R] fp32, both in sorted order
    int64_t row_bytes_sb;     // bytes of one row of scales
    int rows;                 // slots
    int R, KB, gs_log, n_tiles;
    int SP;                   // packed stages
    int win;                  // bytes of a row's scale window: 16 (by TMA) or 32
    int64_t bytes_sb;         // bytes of all scales of a stack
    int act;
    const MoeHeader *hdr;
    const int4 *chunks;       // {expert, first sorted row, rows, box (box_of)}
    int *err;
};

// ---------------------------------------------------------------------------
// Dequantization: one word (8 codes) -> 4 registers (e, e + 4).
// ---------------------------------------------------------------------------
template <typename T> struct Half2;
template <> struct Half2<__nv_bfloat16> {
    using V = __nv_bfloat162;
    static constexpr uint32_t MAGIC = 0x43004300u;  // 128.0, 128.0
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        const V v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    static __device__ __forceinline__ uint32_t off() { return MAGIC; }
};
template <> struct Half2<__half> {
    using V = __half2;
    static constexpr uint32_t MAGIC = 0x64006400u;  // 1024.0, 1024.0
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
        const V v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    static __device__ __forceinline__ uint32_t off() { return MAGIC; }
};
template <typename T>
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
    using V = typename Half2<T>::V;
    const V r = __hmul2(*reinterpret_cast<const V *>(&a), *reinterpret_cast<const V *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}
template <typename T>
__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b) {
    using V = typename Half2<T>::V;
    const V r = __hsub2(*reinterpret_cast<const V *>(&a), *reinterpret_cast<const V *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}
template <typename T>
__device__ __forceinline__ uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
    using V = typename Half2<T>::V;
    const V r = __hfma2(*reinterpret_cast<const V *>(&a), *reinterpret_cast<const V *>(&b),
                        *reinterpret_cast<const V *>(&c));
    return *reinterpret_cast<const uint32_t *>(&r);
}

__device__ __forceinline__ uint32_t mad(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("mad.lo.u32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

// Codes e and e + 4 of w as 2^-126 (bf16) or 2^-14 (f16) times their values.
// A multiplication moves bits on the FMA pipe, which is idle here, while
// shifts would go to the integer pipe that the masks already fill.  bf16: a
// nibble times 2^12 + 2^6 puts its sign at bit 15 and its magnitude at bits
// 6..8 (the two copies do not overlap, the rest is masked off).  f16, whose
// copies would overlap: sign and magnitude apart.
template <typename T>
__device__ __forceinline__ void e2m1_place(uint32_t w, uint32_t (&r)[4]) {
    const uint32_t u = w >> 8;
    if constexpr (std::is_same<T, __half>::value) {
        r[0] = mad(w & 0x00070007u, 512u, (w & 0x00080008u) * 4096u);
        r[1] = mad(w & 0x00700070u, 32u, (w & 0x00800080u) * 256u);
        r[2] = mad(u & 0x00070007u, 512u, (u & 0x00080008u) * 4096u);
        r[3] = mad(u & 0x00700070u, 32u, (u & 0x00800080u) * 256u);
    } else {
        constexpr uint32_t M = 0x81C081C0u;
        r[0] = mad(w & 0x000F000Fu, 4160u, 0u) & M;
        r[1] = mad(w & 0x00F000F0u, 260u, 0u) & M;
        r[2] = mad(u & 0x000F000Fu, 4160u, 0u) & M;
        r[3] = mad(u & 0x00F000F0u, 260u, 0u) & M;
    }
}

// The packed factor X 2^126 (bf16) or X 2^14 (f16) of a scale byte in range.
template <typename T, int MODE>
__device__ __forceinline__ bool scale_in_range(uint32_t s) {
    if constexpr (MODE == QMM_MODE_NVFP4) return (s & 0x7Fu) < 0x48u;  // |X| < 4
    else return s <= 128u;                                             // X <= 2
}
template <typename T, int MODE>
__device__ __forceinline__ uint32_t scale_factor(uint32_t s) {
    if constexpr (MODE == QMM_MODE_NVFP4) {
        const float x = mxf::scale_value<MODE>(s);
        const float f = std::is_same<T, __half>::value ? x * 16384.f : x * 8.507059173e37f;  // 2^14, 2^126
        return Half2<T>::pack(f, f);
    } else if constexpr (std::is_same<T, __half>::value) {
        // 2^(s - 113): normal from s = 99, subnormal down to s = 89, then 0
        // (where X * element is below half of f16's smallest value).
        const uint32_t b = s >= 99u ? (s - 98u) << 10 : (s >= 89u ? 1u << (s - 89u) : 0u);
        return b * 0x00010001u;
    } else {
        return (s + 126u) * 0x00800080u;  // exponent field s + 126 in both halves
    }
}

// Affine codes e and e + 4 of w as 2^-129 (bf16) or 2^-20 (f16) times their
// values: bits 4..7 of a register half, subnormals and the smallest normals, lie
// on one line.
__device__ __forceinline__ void affine_place(uint32_t w, uint32_t (&r)[4]) {
    const uint32_t u = w >> 8;
    r[0] = mad(w & 0x000F000Fu, 16u, 0u);
    r[1] = w & 0x00F000F0u;
    r[2] = mad(u & 0x000F000Fu, 16u, 0u);
    r[3] = u & 0x00F000F0u;
}

// A block of 64 elements: w[8] codes -> v[32].  sb: the block's scale bytes
// (affine: the scales, and bb the biases, of its two halves).
template <typename T, int MODE>
__device__ __forceinline__ void dequant_block(const uint32_t (&w)[8], uint32_t sb, uint32_t bb,
                                              uint32_t (&v)[32]) {
    if constexpr (MODE == QMM_MODE_AFFINE) {
        // s q + b, rounded once, as (2^-129 q) (2^129 s) + b while 2^129 s (f16:
        // 2^20 s) is in range, else from q itself (11 instructions per word instead
        // of 15: 5 rows x 4 of 16 experts 2048 x 2048 f16 54 -> 50 us).
        constexpr bool F16 = std::is_same<T, __half>::value;
        constexpr uint32_t kMag = 0x7FFF7FFFu, kLimit = F16 ? 0x2BFFu : 0x3EFFu;  // below 2^-4, 2^-1
        const uint32_t m = sb & kMag;
        if ((m & 0xFFFFu) <= kLimit && (m >> 16) <= kLimit) {
            // 2^129 = 2^127 4, 2^20 = 2^15 32
            const uint32_t up = mul2<T>(mul2<T>(sb, F16 ? 0x78007800u : 0x7F007F00u), F16 ? 0x50005000u : 0x40804080u);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t s2 = __byte_perm(up, up, i < 4 ? 0x1010 : 0x3232);
                const uint32_t b2 = __byte_perm(bb, bb, i < 4 ? 0x1010 : 0x3232);
                uint32_t r[4];
                affine_place(w[i], r);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[4 * i + e] = fma2<T>(r[e], s2, b2);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t s2 = __byte_perm(sb, sb, i < 4 ? 0x1010 : 0x3232);
                const uint32_t b2 = __byte_perm(bb, bb, i < 4 ? 0x1010 : 0x3232);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t t = ((w[i] >> (4 * e)) & 0x000F000Fu) | Half2<T>::MAGIC;
                    v[4 * i + e] = fma2<T>(sub2<T>(t, Half2<T>::off()), s2, b2);
                }
            }
        }
    } else {
        constexpr int NG = MODE == QMM_MODE_NVFP4 ? 4 : 2;  // groups per block
        bool fast = true;
#pragma unroll
        for (int g = 0; g < NG; ++g) fast = fast && scale_in_range<T, MODE>((sb >> (8 * g)) & 0xFFu);
        if (fast) {
#pragma unroll
            for (int g = 0; g < NG; ++g) {
                const uint32_t f = scale_factor<T, MODE>((sb >> (8 * g)) & 0xFFu);
#pragma unroll
                for (int i = g * 8 / NG; i < (g + 1) * 8 / NG; ++i) {
                    uint32_t r[4];
                    e2m1_place<T>(w[i], r);
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[4 * i + e] = mul2<T>(r[e], f);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float x = mxf::scale_value<MODE>((sb >> (8 * (i * NG / 8))) & 0xFFu);
                float f[8];
                mxf::elements<MODE>(w[i], f);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[4 * i + e] = Half2<T>::pack(x * f[e], x * f[e + 4]);
            }
        }
    }
}

// Gated activation for a value that is rounded to 16 bits next: the fast
// exponential and division stay within 2^-16 of the value (2 + 1.2 |z| units of
// 2^-23, |z| < 88), below that rounding.
template <int ACT>
__device__ __forceinline__ float gate_fast(float g) {
    float z = g;
    if constexpr (ACT != QMM_ACT_SILU) z = 1.5957691216057308f * (g + 0.044715f * g * g * g);
    return __fdividef(g, 1.f + __expf(-z));
}

// 16 bytes, of which the first n are read and the rest are zero.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t n) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
// Arrive on bar once this thread's cp.async so far have landed (counted among
// the barrier's arrivals).
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// Bounded wait for a barrier phase.  The polls come first: the clock and the
// limit, a read of global memory that costs as much as a block's work, are
// looked at only once a wait has gone on for long.  On timeout the device error
// word is set and the caller carries on in bounds.
__device__ __forceinline__ void wait_phase(uint32_t bar, uint32_t parity, int *err) {
    if (ptx::mbar_test(bar, parity)) return;
#pragma unroll 1
    for (int i = 0; i < 16; ++i)
        if (ptx::mbar_try_wait(bar, parity)) return;
    ptx::mbar_wait<true>(bar, parity, err);
}

struct Ring {
    int slot = 0;
    uint32_t phase = 0;
    bool wrapped = false;
    __device__ void next(int n) {
        if (++slot == n) {
            slot = 0;
            phase ^= 1;
            wrapped = true;
        }
    }
};

template <typename T, int MODE, bool GLU, int CAP, int WIN>
__global__ void __launch_bounds__(kThreads, 1)
moe_tc_kernel(const __grid_constant__ WeightMaps maps,
              const __grid_constant__ ActMaps map_b, const __grid_constant__ TcParams p) {
    constexpr bool AFF = MODE == QMM_MODE_AFFINE;
    constexpr int NW = AFF ? 2 : 1;             // windows per stage: scales (and biases)
    constexpr int NM = GLU ? 2 : 1;             // packed boxes per stage
    constexpr uint32_t TMEM_COLS = 512;
    constexpr bool kF16 = std::is_same<T, __half>::value;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *gbase = smem_raw + (base - raw);
    using Cfg = TileCfg<CAP>;
    constexpr int U = Cfg::U, BPG = Cfg::BPG, SB = Cfg::SB, BB = Cfg::BBytes;
    constexpr uint32_t NU = Cfg::NU;
    constexpr int win_bytes = kBM * WIN;  // scale windows of a stage (and as many of biases)
    const int SP = p.SP;
    // Barriers first, then the rings: activations, packed tiles, windows.
    const uint32_t bars = base, b0 = base + kBarBytes, p0 = b0 + SB * BB, s0 = p0 + SP * kPBytes;
    // full_p, empty_p: packed stages.  Unit n of k-blocks (counted over all of
    // the CTA's tiles) is handed over on ready[n % kRing]: four dequantize warps
    // per k-block and the activation tile's bytes; its MMAs complete
    // done[n % kRing], which frees slot n % NU of A and activation stage n % SB.
    const uint32_t full_p = bars, empty_p = full_p + 8 * SP, ready = empty_p + 8 * SP, done = ready + 8 * kRing;
    const uint32_t acc_full = done + 8 * kRing, acc_empty = acc_full + 16, fin = acc_empty + 16;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(gbase + (fin + 8 - base));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < SP; ++i) {
            ptx::mbar_init(full_p + 8 * i, NM + (WIN == 16 ? 0 : 32));
            ptx::mbar_init(empty_p + 8 * i, kDqWarps / BPG);
        }
        for (int i = 0; i < kRing; ++i) {
            ptx::mbar_init(ready + 8 * i, 4 * U / BPG + 1);
            ptx::mbar_init(done + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(acc_full + 8 * i, 1);
            ptx::mbar_init(acc_empty + 8 * i, 4);
        }
        ptx::mbar_init(fin, 1);
        ptx::fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(ptx::smem_addr(tmem_slot), TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // What the preceding kernels wrote (chunks, activations) is read from here on.
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int KB = p.KB, KS = (KB + kGroups - 1) / kGroups, KU = (KB + U - 1) / U;
    const int num_tiles = p.hdr->num_chunks * p.n_tiles;
    const uint32_t a_col0 = 2u * CAP;

    if (warp >= kDqWarp && warp < kSWarp) {
        // ------------------------- dequantize -------------------------
        const int g = (warp - kDqWarp) >> 2, q = warp & 3;
        const int row = GLU ? 16 * q + (lane & 15) + ((lane & 16) << 2) : 32 * q + lane;
        const uint8_t *prow = gbase + (p0 - base) + row * (kStageK / 2);
        const uint8_t *swin = gbase + (s0 - base) + row * WIN;
        uint32_t shift = 0;           // where the row's window begins in its 32 bytes
        const uint32_t dst = tmem + ((uint32_t)(32 * q) << 16) + a_col0;
        // A group takes BPG blocks, from b0k on, of every BPG-th stage.
        const int b0k = BPG * g % kGroups;
        uint32_t c = 0;               // units of the tiles before
        Ring ps;
        int st = g * BPG / kGroups;
        for (int i = 0; i < st; ++i) ps.next(SP);
        for (int tile = blockIdx.x; tile < num_tiles; tile += gridDim.x, st -= KS, c += KU) {
            if constexpr (WIN != 16) {
                const uint32_t n = (tile % p.n_tiles) * (kBM / NM) + (GLU ? row & 63 : row);
                shift = ((uint32_t)p.chunks[tile / p.n_tiles].x * p.R + n) * (uint32_t)p.row_bytes_sb & 15u;
            }
            for (; st < KS; st += BPG) {
                wait_phase(full_p + 8 * ps.slot, ps.phase, p.err);
                const uint8_t *src = prow + ps.slot * kPBytes;
                const uint8_t *sw = swin + ps.slot * (NW * win_bytes) + shift;
                const int kb0 = st * kGroups + b0k;
                const uint32_t n = c + kb0 / U;
                const uint32_t dn = dst + 32u * U * (n % NU) + 32u * (kb0 % U);
#pragma unroll
                for (int j = 0; j < BPG; ++j) {
                    const int kb = kb0 + j;
                    uint32_t v[32];
                    if (kb < KB) {
                        uint32_t w[8], sb = 0, bb = 0;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint4 u = *reinterpret_cast<const uint4 *>(src + (((2 * (b0k + j) + i) ^ (row & 7)) << 4));
                            w[4 * i] = u.x;
                            w[4 * i + 1] = u.y;
                            w[4 * i + 2] = u.z;
                            w[4 * i + 3] = u.w;
                        }
                        if constexpr (AFF) {
                            // first group of each half, as halves of a word
                            const int o0 = (((kb * kBK) >> p.gs_log) * 2) & 15;
                            const int o1 = (((kb * kBK + 32) >> p.gs_log) * 2) & 15;
                            sb = *reinterpret_cast<const uint16_t *>(sw + o0) |
                                 ((uint32_t)*reinterpret_cast<const uint16_t *>(sw + o1) << 16);
                            bb = *reinterpret_cast<const uint16_t *>(sw + win_bytes + o0) |
                                 ((uint32_t)*reinterpret_cast<const uint16_t *>(sw + win_bytes + o1) << 16);
                        } else if constexpr (MODE == QMM_MODE_NVFP4) {
                            sb = *reinterpret_cast<const uint32_t *>(sw + ((4 * kb) & 15));
                        } else {
                            sb = *reinterpret_cast<const uint16_t *>(sw + ((2 * kb) & 15));
                        }
                        dequant_block<T, MODE>(w, sb, bb, v);
                    }
                    if (j == BPG - 1) {
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(empty_p + 8 * ps.slot);
                    }
                    if (j == 0 && kb0 / U < KU && n >= NU) {
                        wait_phase(done + 8 * ((n - NU) % kRing), ((n - NU) / kRing) & 1, p.err);
                        tc_fence_after();
                    }
                    if (kb < KB) tmem_st32(dn + 32u * j, v);
                }
                if (kb0 / U < KU) {  // blocks missing from a tile's last unit count as there
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(ready + 8 * (n % kRing));
                }
#pragma unroll
                for (int i = 0; i < BPG; ++i) ps.next(SP);
            }
        }
    } else if (warp < kMmaWarp) {
        // ------------------------- epilogue -------------------------
        const int q = warp & 3;
        int i = 0;
        for (int tile = blockIdx.x; tile < num_tiles; tile += gridDim.x, ++i) {
            const int acc = i & 1, use = i >> 1;
            const int4 ch = p.chunks[tile / p.n_tiles];
            const int nt = tile % p.n_tiles;
            wait_phase(acc_full + 8 * acc, use & 1, p.err);
            tc_fence_after();
            const int nj = (ch.z + 31) / 32;
            for (int j = 0; j < nj; ++j) {
                uint32_t v[32];
                tmem_ld32(tmem + ((uint32_t)(32 * q) << 16) + acc * CAP + 32 * j, v);
                tmem_ld_wait();
                if (j == nj - 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(acc_empty + 8 * acc);
                }
                if constexpr (GLU) {
                    // Lanes 0-15 hold gate features 16 q + lane, lanes 16-31 the
                    // up values of the same features: the lower lanes take
                    // columns 0-15, the upper ones 16-31.
                    const bool upper = lane >= 16;
                    const int f = 16 * q + (lane & 15);
                    const int pos = (f & ~7) | ((f & 3) << 1) | ((f >> 2) & 1);
                    const int m0 = 32 * j + (upper ? 16 : 0), left = ch.z - m0;
                    T *h = static_cast<T *>(p.out) + ((int64_t)nt * p.rows + ch.y + m0) * kBK + pos;
                    auto finish = [&](auto act) {
#pragma unroll
                        for (int cc = 0; cc < 16; ++cc) {
                            const float lo = __uint_as_float(v[cc]), hi = __uint_as_float(v[cc + 16]);
                            const float own = upper ? hi : lo;
                            const float got = __shfl_xor_sync(0xffffffffu, upper ? lo : hi, 16);
                            const float r = gate_fast<decltype(act)::value>(upper ? got : own) * (upper ? own : got);
                            if (cc < left) h[cc * kBK] = Dt<T>::from_f(r);
                        }
                    };
                    if (p.act == QMM_ACT_SILU) finish(std::integral_constant<int, QMM_ACT_SILU>());
                    else finish(std::integral_constant<int, QMM_ACT_GELU_TANH>());
                } else {
                    const int n = nt * kBM + 32 * q + lane;
                    const int left = n < p.R ? ch.z - 32 * j : 0;
                    float *parts = static_cast<float *>(p.out) + (int64_t)(ch.y + 32 * j) * p.R + n;
#pragma unroll
                    for (int cc = 0; cc < 32; ++cc, parts += p.R)
                        if (cc < left) *parts = __uint_as_float(v[cc]);
                }
            }
        }
    } else if (warp == kMmaWarp) {
        // ------------------------- MMA issuer -------------------------
        // One elected lane runs the whole loop: with the loop shared by the warp
        // and only the waits and issues under the election, the commit of a tile
        // that had waited long for its accumulator went to the other
        // accumulator's barrier.
        if (elect_one()) {
            // Ring positions as running addresses: few instructions per unit,
            // which this one thread issues one after the other.
            const uint64_t desc0 = sw128_desc(b0);
            const uint32_t dhi = (uint32_t)(desc0 >> 32);
            constexpr uint32_t kStepB = BB >> 4, kEndB = kStepB * SB, kStepA = 32 * U, kEndA = kStepA * NU;
            uint32_t bar = ready, parity = 0, aoff = 0, boff = 0;
            int i = 0;
            for (int tile = blockIdx.x; tile < num_tiles; tile += gridDim.x, ++i) {
                const int acc = i & 1, use = i >> 1;
                const int4 ch = p.chunks[tile / p.n_tiles];
                const uint32_t idesc = make_idesc(kF16, kBM, (ch.z + 15) & ~15);
                const uint32_t zstep = (uint32_t)(ch.w >> 8) * 128u >> 4;  // descriptor step of one k-block
                if (i >= 2) wait_phase(acc_empty + 8 * acc, (use + 1) & 1, p.err);
                tc_fence_after();
                const uint32_t d = tmem + acc * CAP;
                uint32_t more = 0;  // whether the accumulator holds something
                for (int left = KB; left > 0; left -= U) {
                    wait_phase(bar, parity, p.err);
                    tc_fence_after();
                    uint32_t lo = (uint32_t)desc0 + boff;
                    const uint32_t ta = tmem + a_col0 + aoff;
                    auto block = [&](uint32_t a, uint32_t l) {
                        auto desc = [&](uint32_t v) { return (uint64_t)dhi << 32 | v; };
                        tc_mma_ts(d, a, desc(l), idesc, more);
                        more = 1;
                        tc_mma_ts(d, a + 8, desc(l + 2), idesc, 1);
                        tc_mma_ts(d, a + 16, desc(l + 4), idesc, 1);
                        tc_mma_ts(d, a + 24, desc(l + 6), idesc, 1);
                    };
                    if (left >= U) {
#pragma unroll
                        for (int u = 0; u < U; ++u, lo += zstep) block(ta + 32 * u, lo);
                    } else {
#pragma unroll 1
                        for (int u = 0; u < left; ++u, lo += zstep) block(ta + 32 * u, lo);
                    }
                    tc_commit(bar + 8 * kRing);  // done, behind ready
                    bar += 8;
                    if (bar == done) bar = ready, parity ^= 1;
                    aoff += kStepA;
                    if (aoff == kEndA) aoff = 0;
                    boff += kStepB;
                    if (boff == kEndB) boff = 0;
                }
                tc_commit(acc_full + 8 * acc);
            }
            // Every MMA has completed before tensor memory is freed.
            tc_commit(fin);
            ptx::mbar_drain(fin, 0, p.err);
        }
        __syncwarp();
    } else if (warp < kBWarp) {
        // ------------------------- packed tiles -------------------------
        const int m = warp - kWWarp;
        if (lane == 0 && m < NM) {
            const CUtensorMap *map = &maps.w[m];
            constexpr uint32_t bytes = kPBytes / NM, sbytes = kBM * 16 / NM;
            constexpr int ES = AFF ? 2 : 1;
            const bool windows = WIN == 16;
            const uint32_t total = bytes + (windows ? NW * sbytes : 0u);
            Ring ps;
            int n = 0;
            for (int tile = blockIdx.x; tile < num_tiles; tile += gridDim.x) {
                const int4 ch = p.chunks[tile / p.n_tiles];
                const int r0 = ch.x * p.R + (tile % p.n_tiles) * (kBM / NM);
                for (int st = 0; st < KS; ++st, ++n, ps.next(SP)) {
                    if (ps.wrapped) wait_phase(empty_p + 8 * ps.slot, ps.phase ^ 1, p.err);
                    ptx::mbar_arrive_expect_tx(full_p + 8 * ps.slot, total);
                    tma_load_2d(p0 + ps.slot * kPBytes + m * bytes, map, st * (kStageK / 8), r0,
                                full_p + 8 * ps.slot);
                    if (windows) {
                        const int at = (((st * kStageK) >> p.gs_log) * ES & ~15) / ES;
                        const uint32_t win = s0 + ps.slot * (NW * win_bytes) + m * sbytes;
                        tma_load_2d(win, &maps.s[m], at, r0, full_p + 8 * ps.slot);
                        if constexpr (AFF) tma_load_2d(win + win_bytes, &maps.b[m], at, r0, full_p + 8 * ps.slot);
                    }
                }
            }
            for (int k = max(0, n - SP); k < n; ++k) ptx::mbar_drain(full_p + 8 * (k % SP), (k / SP) & 1, p.err);
        }
    } else if (warp == kBWarp) {
        // ------------------------- activation tiles -------------------------
        if (lane == 0) {
            // the activations were written by ordinary stores of earlier kernels
            asm volatile("fence.proxy.async.global;" ::: "memory");
            uint32_t n = 0;
            int slot = 0;
            for (int tile = blockIdx.x; tile < num_tiles; tile += gridDim.x) {
                const int4 ch = p.chunks[tile / p.n_tiles];
                const CUtensorMap *map = &map_b.m[ch.w & 255];
                const uint32_t bytes = (uint32_t)(ch.w >> 8) * 128u * U;
                for (int ku = 0; ku < KU; ++ku, ++n) {
                    if (n >= (uint32_t)SB) wait_phase(done + 8 * ((n - SB) % kRing), ((n - SB) / kRing) & 1, p.err);
                    ptx::mbar_arrive_expect_tx(ready + 8 * (n % kRing), bytes);
                    tma_load_3d(b0 + slot * BB, map, 0, ch.y, U * ku, ready + 8 * (n % kRing));
                    if (++slot == SB) slot = 0;
                }
            }
            for (uint32_t k = n < (uint32_t)SB ? 0 : n - SB; k < n; ++k)
                ptx::mbar_drain(ready + 8 * (k % kRing), (k / kRing) & 1, p.err);
        }
    } else if (WIN != 16) {
        // ------------------------- scale windows -------------------------
        // Rows of scales that are not whole 16 bytes begin anywhere: the two
        // aligned 16-byte pieces that hold a row's window (the stack's first
        // byte is aligned), nothing past the stack's end.
        constexpr int ES = AFF ? 2 : 1;
        Ring ps;
        for (int tile = blockIdx.x; tile < num_tiles; tile += gridDim.x) {
            const int4 ch = p.chunks[tile / p.n_tiles];
            const int nt = tile % p.n_tiles;
            int64_t off[4];  // row's first byte, or past the end: not read
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = lane + 32 * i;
                const int n = GLU ? nt * (kBM / 2) + (r & 63) : nt * kBM + r;
                off[i] = n < p.R ? ((int64_t)ch.x * p.R + n) * p.row_bytes_sb : p.bytes_sb;
            }
            for (int st = 0; st < KS; ++st, ps.next(SP)) {
                if (ps.wrapped) wait_phase(empty_p + 8 * ps.slot, ps.phase ^ 1, p.err);
                const uint32_t win = s0 + ps.slot * (NW * win_bytes) + lane * 32;
                const int64_t at = (((int64_t)st * kStageK) >> p.gs_log) * ES & ~15;  // window's first byte
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int64_t from = (off[i] + at) & ~(int64_t)15;
#pragma unroll
                    for (int w = 0; w < NW; ++w) {
                        const uint8_t *src = static_cast<const uint8_t *>(w == 0 ? p.scales[GLU ? i >> 1 : 0]
                                                                                : p.biases[GLU ? i >> 1 : 0]) + from;
                        const uint32_t d = win + w * win_bytes + i * 1024;
                        const int64_t left = p.bytes_sb - from;
                        if (left > 0) cp_async16(d, src, (uint32_t)min(left, (int64_t)16));
                        if (left > 16) cp_async16(d + 16, src + 16, (uint32_t)min(left - 16, (int64_t)16));
                    }
                }
                cp_async_arrive(full_p + 8 * ps.slot);
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

// ---------------------------------------------------------------------------
// Preparation: slots sorted by expert, chunks, the copy of x.
// ---------------------------------------------------------------------------
constexpr int kPrepThreads = 512, kPrepWarps = kPrepThreads / 32;
constexpr int kPrepSeg = 8192;  // slots of a CTA at most

struct PrepParams {
    const int32_t *indices;
    const uint4 *x;
    uint4 *xs;
    int slots, E, cap, seg, top_k, vec;  // vec: 16-byte units of a row of x
    MoeHeader *hdr;
    int4 *chunks;
    int32_t *pos;             // sorted row of each slot, -1 without an expert
    int *err;
};

// Exclusive prefix sum of a[0..L) in place, a[L] the total; by the whole block.
__device__ void scan_counts(int *a, int L, int *tmp) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
    const int per = (L + blockDim.x - 1) / blockDim.x;
    const int lo = min(L, tid * per), hi = min(L, lo + per);
    int mine = 0;
    for (int i = lo; i < hi; ++i) mine += a[i];
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) tmp[warp] = incl;
    __syncthreads();
    int before = 0, total = 0;
    for (int w = 0; w < nw; ++w) {
        if (w < warp) before += tmp[w];
        total += tmp[w];
    }
    int run = before + incl - mine;
    for (int i = lo; i < hi; ++i) {
        const int t = a[i];
        a[i] = run;
        run += t;
    }
    __syncthreads();
    if (tid == 0) a[L] = total;
    __syncthreads();
}

// Lowest box that holds `rows` rows: its index in kHeights and, above 8 bits, its height.
__device__ __forceinline__ int box_of(int rows) {
    if (rows <= 16) return 0 | 16 << 8;
    if (rows <= 32) return 1 | 32 << 8;
    if (rows <= 64) return 2 | 64 << 8;
    if (rows <= 96) return 3 | 96 << 8;
    if (rows <= 128) return 4 | 128 << 8;
    return 5 | 192 << 8;
}

// Each CTA counts every slot's expert for itself (the indices are small and
// come from L2; 32768 slots of 64 experts, copied rows of 4 KB: 39 us for the
// kernel, 90 with lanes of the same expert matched before they add).  That gives
// it, without a second kernel, where the slots of its own stretch go: the
// experts' first rows, plus the same expert's slots in earlier stretches, plus
// the rank within its own.  It then copies their rows of x there, every eight
// elements in the order 0 4 1 5 2 6 3 7.  The first CTA also cuts each expert's
// rows into near-equal chunks of whole 16 rows, at most cap.  Counts are
// integers, and ranks follow the slots' order, so the result does not depend on
// timing.
__global__ void __launch_bounds__(kPrepThreads) moe_prep_kernel(const PrepParams p) {
    extern __shared__ int sm[];
    __shared__ int tmp[kPrepWarps];
    const int E = p.E;
    int *first = sm, *before = first + E + 2, *nch = before + E + 1;
    int *dst = nch + E + 1;  // sorted row of each slot of the stretch, -1 without an expert
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i < 2 * E + 3; i += kPrepThreads) sm[i] = 0;
    __syncthreads();
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int lo = blockIdx.x * p.seg, hi = min(p.slots, lo + p.seg);
    // Slots per expert, before the stretch and from it on.
    constexpr int U = 8;  // loads in flight per thread
    for (int b0 = tid; b0 < p.slots; b0 += U * kPrepThreads) {
        int key[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = b0 + u * kPrepThreads;
            key[u] = i < p.slots ? p.indices[i] : -1;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = b0 + u * kPrepThreads;
            if (i >= p.slots) break;
            if (key[u] < 0 || key[u] >= E) {
                if (key[u] != -1 && blockIdx.x == 0) record_device_error(p.err, QMM_ERR_INDEX);
                key[u] = E;
            }
            atomicAdd(i < lo ? &before[key[u]] : &first[key[u]], 1);
        }
    }
    __syncthreads();
    for (int i = tid; i <= E; i += kPrepThreads) first[i] += before[i];
    __syncthreads();
    scan_counts(first, E + 1, tmp);
    if (warp == 0) {
        const unsigned lt = (1u << lane) - 1u;
        for (int b = lo; b < hi; b += 32) {
            const int i = b + lane;
            int key = -1 - lane;
            if (i < hi) {
                const int e = moe_expert(p.indices, i, E, nullptr);
                key = e < 0 ? E : e;
            }
            const unsigned same = __match_any_sync(0xffffffffu, key);
            int pos = 0;
            if (key >= 0) pos = first[key] + before[key] + __popc(same & lt);
            __syncwarp();
            if (key >= 0) {
                if (lane == __ffs(same) - 1) before[key] += __popc(same);
                dst[i - lo] = p.pos[i] = key < E ? pos : -1;
            }
            __syncwarp();
        }
    }
    __syncthreads();
    for (int j = warp; j < hi - lo; j += kPrepWarps) {
        const int r = dst[j];
        if (r < 0) continue;
        const uint4 *src = p.x + (int64_t)((lo + j) / p.top_k) * p.vec;
        uint4 *out = p.xs + (int64_t)r * p.vec;
#pragma unroll 4
        for (int v = lane; v < p.vec; v += 32) {
            const uint4 a = __ldg(src + v);
            out[v] =
                make_uint4(__byte_perm(a.x, a.z, 0x5410), __byte_perm(a.x, a.z, 0x7632),
                           __byte_perm(a.y, a.w, 0x5410), __byte_perm(a.y, a.w, 0x7632));
        }
    }
    if (blockIdx.x != 0) return;
    auto size_of = [&](int rows) {
        const int n = (rows + p.cap - 1) / p.cap;
        return min(p.cap, ((rows + n - 1) / n + 15) & ~15);
    };
    for (int k = tid; k < E; k += kPrepThreads) {
        const int rows = first[k + 1] - first[k];
        nch[k] = rows ? (rows + size_of(rows) - 1) / size_of(rows) : 0;
    }
    __syncthreads();
    scan_counts(nch, E, tmp);
    for (int k = tid; k < E; k += kPrepThreads) {
        const int rows = first[k + 1] - first[k];
        if (rows == 0) continue;
        const int size = size_of(rows);
        for (int j = 0; j * size < rows; ++j) {
            const int n = min(size, rows - j * size);
            p.chunks[nch[k] + j] = make_int4(k, first[k] + j * size, n, box_of(n));
        }
    }
    if (tid == 0) p.hdr->num_chunks = nch[E];
}

// y[t] = sum over slots in order of weight * part, rounded once.
template <typename T, int VEC>
__global__ void __launch_bounds__(256) moe_combine_kernel(const float *parts, const int32_t *pos,
                                                          const float *weights, T *y, int64_t total, int N,
                                                          int top_k) {
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();
    const int nv = N / VEC;
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
        const int64_t t = i / nv;
        const int n = (int)(i - t * nv) * VEC;
        float acc[VEC];
#pragma unroll
        for (int c = 0; c < VEC; ++c) acc[c] = 0.f;
        constexpr int U = 4;  // rows in flight
        for (int j0 = 0; j0 < top_k; j0 += U) {
            float v[U][VEC], w[U];
            bool ok[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t slot = t * top_k + j0 + u;
                const int row = j0 + u < top_k ? pos[slot] : -1;
                ok[u] = row >= 0;
                if (!ok[u]) continue;
                w[u] = weights[slot];
                const float *src = parts + (int64_t)row * N + n;
                if constexpr (VEC == 4) {
                    const float4 f = __ldcs(reinterpret_cast<const float4 *>(src));
                    v[u][0] = f.x, v[u][1] = f.y, v[u][2] = f.z, v[u][3] = f.w;
                } else {
                    v[u][0] = *src;
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int c = 0; c < VEC; ++c)
                    if (ok[u]) acc[c] = __fmaf_rn(w[u], v[u][c], acc[c]);
        }
        if constexpr (VEC == 4) {
            *reinterpret_cast<uint2 *>(y + t * N + n) =
                make_uint2(Half2<T>::pack(acc[0], acc[1]), Half2<T>::pack(acc[2], acc[3]));
        } else {
            y[t * N + n] = Dt<T>::from_f(acc[0]);
        }
    }
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

MoePlan plan_of(const ExpertsArgs &a) {
    MoePlan w{};
    const int64_t P = a.T * a.top_k;
    w.max_chunks = a.n_experts + (P + 15) / 16 + 1;
    size_t off = 256;
    w.chunks = off;
    off += up256((size_t)w.max_chunks * sizeof(int4));
    w.pos = off;
    off += up256((size_t)P * 4);
    w.x = off;
    off += up256((size_t)P * (size_t)a.K * 2);
    w.h = off;
    off += up256((size_t)P * (size_t)a.I * 2);
    w.parts = off;
    off += up256((size_t)P * (size_t)a.N * 4);
    w.total = off;
    return w;
}

template <auto KERN, typename... Args>
cudaError_t launch_chained(dim3 grid, int threads, size_t smem, cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, KERN, args...);
    if (e != cudaSuccess) return e;
    count_launches(1);
    return cudaGetLastError();
}

// Rows per chunk at most: an expert's rows mostly fit one narrow chunk when
// there are few of them, and the rings hold more packed stages then.
int chunk_cap(int64_t slots, int64_t E) { return slots <= 32 * E ? 64 : kMaxCap; }

constexpr size_t kSmemMax = 227 * 1024;
constexpr size_t kSmemFixed = 1024 + kBarBytes;  // alignment; barriers

// Packed stages that fit beside the activations, p_bytes each with their windows.
template <int CAP>
constexpr int packed_stages(size_t p_bytes) {
    return (int)std::min<size_t>(8, (kSmemMax - kSmemFixed - (size_t)TileCfg<CAP>::SB * TileCfg<CAP>::BBytes) / p_bytes);
}

template <typename T, int MODE, bool GLU, int CAP, int WIN>
cudaError_t launch_product(int grid, size_t smem, cudaStream_t s, const WeightMaps &mw, const ActMaps &mb, const TcParams &p) {
    // A group that visits every BPG-th stage waits for the parity of stage s in
    // a ring slot whose last stage, s - SP, it did not take itself: were that one
    // still on its way, the wait would pass on the phase before it.  The group's
    // stage before, s - BPG, waited for the MMAs of unit s - BPG - NU (a unit is a
    // stage here), so that stages up to that one have arrived.
    using Cfg = TileCfg<CAP>;
    constexpr int SP = packed_stages<CAP>(kPBytes + (MODE == QMM_MODE_AFFINE ? 2 : 1) * kBM * WIN);
    static_assert(SP >= 2 && (Cfg::BPG == 1 || (Cfg::U == kGroups && SP >= Cfg::NU + Cfg::BPG)), "packed ring too short");
    auto kern = moe_tc_kernel<T, MODE, GLU, CAP, WIN>;
    struct Tag;
    const cudaError_t e = configure_once<Tag>(kSmemMax, [&]() {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemMax);
    });
    if (e != cudaSuccess) return e;
    return launch_chained<moe_tc_kernel<T, MODE, GLU, CAP, WIN>>(dim3(grid), kThreads, smem, s, mw, mb, p);
}

template <typename T, int MODE, bool GLU, int CAP>
cudaError_t run_product(const ExpertsArgs &a, const MoePlan &w, cudaStream_t s) {
    using Cfg = TileCfg<CAP>;
    uint8_t *ws = static_cast<uint8_t *>(a.ws);
    const int64_t P = a.T * a.top_k, C = GLU ? a.K : a.I, R = GLU ? a.I : a.N;
    constexpr int NM = GLU ? 2 : 1, NW = MODE == QMM_MODE_AFFINE ? 2 : 1;
    constexpr int ES = MODE == QMM_MODE_AFFINE ? 2 : 1;
    const ExpertWeight *ew[2] = {GLU ? &a.gate : &a.down, GLU ? &a.up : &a.down};
    TcParams p{};
    p.row_bytes_sb = C / a.group_size * ES;
    p.win = p.row_bytes_sb % 16 == 0 ? 16 : 32;
    p.bytes_sb = a.n_experts * R * p.row_bytes_sb;
    WeightMaps mw{};
    const uint64_t rows = (uint64_t)(a.n_experts * R);
    const CUtensorMapDataType st = ES == 2 ? CU_TENSOR_MAP_DATA_TYPE_UINT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8;
    for (int m = 0; m < NM; ++m) {
        auto window = [&](CUtensorMap *map, const void *ptr) {
            return make_map_2d(map, st, ptr, (uint64_t)(C / a.group_size), rows, (uint64_t)p.row_bytes_sb, 16 / ES,
                               kBM / NM, CU_TENSOR_MAP_SWIZZLE_NONE);
        };
        if (!make_map_2d(&mw.w[m], CU_TENSOR_MAP_DATA_TYPE_UINT32, ew[m]->wq, (uint64_t)C / 8, rows, (uint64_t)C / 2,
                         kStageK / 8, kBM / NM, CU_TENSOR_MAP_SWIZZLE_128B))
            return cudaErrorInvalidValue;
        if (p.win == 16 &&
            (!window(&mw.s[m], ew[m]->scales) || (NW == 2 && !window(&mw.b[m], ew[m]->biases))))
            return cudaErrorInvalidValue;
    }
    ActMaps mb;
    const uint64_t dims[3] = {64, (uint64_t)P, (uint64_t)C / 64};
    // x rows as they are ([slots][K], k-blocks 128 bytes apart); h by k-blocks
    const uint64_t strides[2] = {GLU ? (uint64_t)C * 2 : 128, GLU ? 128 : (uint64_t)P * 128};
    for (int i = 0; i < kNumHeights && kHeights[i] <= CAP; ++i) {
        const uint32_t box[3] = {64, (uint32_t)kHeights[i], (uint32_t)Cfg::U};
        if (!make_map(&mb.m[i], std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                               : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                      3, ws + (GLU ? w.x : w.h), dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
            return cudaErrorInvalidValue;
    }
    for (int m = 0; m < 2; ++m) {
        p.scales[m] = ew[m]->scales;
        p.biases[m] = ew[m]->biases;
    }
    p.out = ws + (GLU ? w.h : w.parts);
    p.rows = (int)P;
    p.R = (int)R;
    p.KB = (int)(C / kBK);
    p.gs_log = a.group_size == 16 ? 4 : (a.group_size == 32 ? 5 : (a.group_size == 64 ? 6 : 7));
    p.n_tiles = (int)((R + kBM / NM - 1) / (kBM / NM));
    const size_t p_bytes = kPBytes + NW * kBM * p.win;
    p.SP = packed_stages<CAP>(p_bytes);
    const size_t smem = kSmemFixed + (size_t)Cfg::SB * Cfg::BBytes + p.SP * p_bytes;
    p.act = a.act;
    p.hdr = reinterpret_cast<const MoeHeader *>(ws + w.hdr);
    p.chunks = reinterpret_cast<const int4 *>(ws + w.chunks);
    p.err = device_error_word();
    const int64_t most = std::min<int64_t>(w.max_chunks, std::min<int64_t>(P, a.n_experts) + P / 16) * p.n_tiles;
    const int grid = (int)std::min<int64_t>(std::max<int64_t>(most, 1), num_sms());
    return p.win == 16 ? launch_product<T, MODE, GLU, CAP, 16>(grid, smem, s, mw, mb, p)
                       : launch_product<T, MODE, GLU, CAP, 32>(grid, smem, s, mw, mb, p);
}

template <typename T, int MODE>
cudaError_t run_tc(const ExpertsArgs &a, cudaStream_t s) {
    const MoePlan w = plan_of(a);
    uint8_t *ws = static_cast<uint8_t *>(a.ws);
    const int64_t P = a.T * a.top_k;
    const int cap = chunk_cap(P, a.n_experts);
    MoeHeader *hdr = reinterpret_cast<MoeHeader *>(ws + w.hdr);
    int32_t *pos = reinterpret_cast<int32_t *>(ws + w.pos);

    PrepParams pp{};
    pp.indices = a.indices;
    pp.x = static_cast<const uint4 *>(a.x);
    pp.xs = reinterpret_cast<uint4 *>(ws + w.x);
    pp.slots = (int)P;
    pp.E = (int)a.n_experts;
    pp.cap = cap;
    pp.top_k = a.top_k;
    pp.vec = (int)(a.K / 8);
    pp.hdr = hdr;
    pp.chunks = reinterpret_cast<int4 *>(ws + w.chunks);
    pp.pos = pos;
    pp.err = device_error_word();
    // Two CTAs per SM, unless their stretches would be shorter than a warp's
    // share of rows or longer than shared memory holds.
    pp.seg = (int)std::min<int64_t>(kPrepSeg, std::max<int64_t>(8, (P + 2 * num_sms() - 1) / (2 * num_sms())));
    const size_t smem = (size_t)(3 * pp.E + 4 + pp.seg) * sizeof(int);  // 46 KB at most
    cudaError_t e = launch_chained<moe_prep_kernel>(dim3((unsigned)((P + pp.seg - 1) / pp.seg)), kPrepThreads, smem, s, pp);
    if (e != cudaSuccess) return e;
    if (cap <= 64) {
        if ((e = run_product<T, MODE, true, 64>(a, w, s)) != cudaSuccess) return e;
        if ((e = run_product<T, MODE, false, 64>(a, w, s)) != cudaSuccess) return e;
    } else {
        if ((e = run_product<T, MODE, true, kMaxCap>(a, w, s)) != cudaSuccess) return e;
        if ((e = run_product<T, MODE, false, kMaxCap>(a, w, s)) != cudaSuccess) return e;
    }

    const float *parts = reinterpret_cast<const float *>(ws + w.parts);
    const bool vec4 = a.N % 4 == 0;
    const int64_t total = a.T * (a.N / (vec4 ? 4 : 1));
    const int cgrid = (int)std::min<int64_t>((total + 255) / 256, (int64_t)num_sms() * 8);
    T *y = static_cast<T *>(a.y);
    if (vec4)
        return launch_chained<moe_combine_kernel<T, 4>>(dim3(cgrid), 256, 0, s, parts, pos, a.weights, y, total,
                              (int)a.N, a.top_k);
    return launch_chained<moe_combine_kernel<T, 1>>(dim3(cgrid), 256, 0, s, parts, pos, a.weights, y, total,
                          (int)a.N, a.top_k);
}

template <typename T>
cudaError_t run_tc_mode(const ExpertsArgs &a, cudaStream_t s) {
    switch (a.mode) {
    case QMM_MODE_AFFINE: return run_tc<T, QMM_MODE_AFFINE>(a, s);
    case QMM_MODE_MXFP4: return run_tc<T, QMM_MODE_MXFP4>(a, s);
    default: return run_tc<T, QMM_MODE_NVFP4>(a, s);
    }
}

}  // namespace

bool moe_tc_supported() { return encode_fn() != nullptr; }

size_t moe_tc_workspace(const ExpertsArgs &a) { return plan_of(a).total; }

cudaError_t launch_moe_tc(qmm_dtype dt, const ExpertsArgs &a, cudaStream_t s) {
    return dt == QMM_BF16 ? run_tc_mode<__nv_bfloat16>(a, s) : run_tc_mode<__half>(a, s);
}

}  // namespace qmm
