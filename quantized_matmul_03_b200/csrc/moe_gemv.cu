// moe_gemv.cu -- the experts' products for few rows (single tokens, small
// decode batches):
//   h[p] = act(x[t] Wg[e]^T) * (x[t] Wu[e]^T)   for each slot p = (t, j), e = indices[p]
//   y[t] = sum_j weights[t, j] (h[t, j] Wd[e]^T)
// in two kernels, both of one shape: CTA c owns a range of output rows of
// every expert; a unit is (slot, stretch of 1024 contraction elements); a warp
// takes a unit, holds its 32 activations per lane in registers, and streams the
// unit's piece of each of the CTA's rows (512 contiguous bytes of codes) past
// them.  The pieces of a row meet in shared memory and are added in a fixed
// order, so that results repeat bit for bit; the second kernel also adds a
// token's slots there, weighted, and rounds once.
//
// Arithmetic.  32 activations are held as 16-bit integers over a common power
// of two (error at most 2^-14 of the largest of the 32, or 2^-127: finer than the
// rounding of that one to a 16-bit type; DP2A takes two of them per instruction),
// codes are small integers, and DP2A sums their products exactly: 4-bit affine
// codes as they are, E2M1 codes doubled (an integer in [-12, 12]) and offset by 64,
// which -64 sum(x_int) takes out again.  The integer sum is scaled by the group's
// scale in fp32.  Between the kernels h stays in fp32.
//
// Every code is read once per slot.  Two forms of each kernel: weights streamed
// through shared memory by bulk copies (moe_stream_kernel), and, for shapes that
// those cannot take, loaded 16 bytes per lane with two batches of eight loads in
// flight per warp (moe_gemv_kernel).  One token, 2 of 8 experts 4096 x 14336
// mxfp4, 187 MB: 56 us per call back to back (3.3 TB/s; 69 us with plain loads),
// a single cold call 65 us; 8 of 64 experts 2048 x 1024 nvfp4, 28 MB: 24 us cold.
// Bound: the two launches with their ring's first and last stages, and between
// them the consumer warps' instructions.
#include "moe.cuh"
#include "mx.cuh"
#include "ptx_sm100.cuh"

namespace qmm {
namespace {

constexpr int kSeg = 1024;     // contraction elements of a unit: 32 lanes x 32 codes
constexpr int kMaxWarps = 16;
constexpr int kLoads = 8;      // 16-byte code loads per lane and batch
constexpr int kPartBytes = 96 * 1024;  // partial sums of a CTA at most

struct GemvParams {
    const void *x;         // first kernel: [T, K]; second: h [P, I] fp32
    ExpertWeight w[2];     // gate and up, or down twice
    const int32_t *indices;
    const float *weights;
    void *out;             // h [P, I] fp32, or y [T, N]
    int P, top_k, E;
    int64_t C, R;          // contraction length, output rows of an expert
    int rows_cta, S, units, unit_warps, row_splits;
    int gs_log, act;
    int *err;
};

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ int dp2a_lo(int xa, uint32_t b, int c) {
    int d;
    asm("dp2a.lo.s32.u32 %0, %1, %2, %3;" : "=r"(d) : "r"(xa), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ int dp2a_hi(int xa, uint32_t b, int c) {
    int d;
    asm("dp2a.hi.s32.u32 %0, %1, %2, %3;" : "=r"(d) : "r"(xa), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint4 ld_stream(const void *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// Value of an E8M0 byte without branches: 2^(s - 127), for s = 0 the subnormal
// 2^-127, for s = 255 NaN (the infinity's bits with one mantissa bit set).
__device__ __forceinline__ float e8m0(uint32_t s) {
    return __uint_as_float(max((s << 23) | (((s + 1u) << 14) & 0x00400000u), 0x00400000u));
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}

// Constants of the E2M1 decoding, held in registers (as literals they were set
// up again before every permutation, or turned a multiplication back into an
// instruction of the integer pipe).
struct E2m1Table {
    uint32_t pa, pb;   // 64 + 2 e of codes 0..7, a byte each
    uint32_t na, nb;   // 64 - 2 e
    uint32_t one;
    __device__ __forceinline__ void set() {
        asm volatile("mov.u32 %0, 0x43424140;" : "=r"(pa));
        asm volatile("mov.u32 %0, 0x4C484644;" : "=r"(pb));
        asm volatile("mov.u32 %0, 0x3D3E3F40;" : "=r"(na));
        asm volatile("mov.u32 %0, 0x34383A3C;" : "=r"(nb));
        asm volatile("mov.u32 %0, 1;" : "=r"(one));
    }
};
__device__ __forceinline__ uint32_t mad(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("mad.lo.u32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

// Eight E2M1 codes as unsigned bytes 64 + 2 e, four per word: a byte
// permutation of the first table by the raw nibbles gives the byte of every
// non-negative code and 0 for a negative one (selector bit 3 asks for the sign
// of a table byte), of the second by the nibbles with their sign bits flipped
// the converse.  The integer pipe is the kernel's busiest: their sum goes to the
// multiply pipe (one token, 2 of 8 experts 4096 x 14336, single cold calls: 63 us,
// 65.5 with integer additions).
__device__ __forceinline__ void e2m1_bytes(const E2m1Table &t, uint32_t w, uint32_t &lo, uint32_t &hi) {
    const uint32_t n = w ^ 0x88888888u;
    lo = mad(prmt(t.pa, t.pb, w), t.one, prmt(t.na, t.nb, n));
    hi = mad(prmt(t.pa, t.pb, w >> 16), t.one, prmt(t.na, t.nb, n >> 16));
}

// A lane's 32 activations: pairs of 16-bit integers in the order in which DP2A
// meets the codes, their scale 2^-sh, and the sums that the bias (affine) or
// the offset of the codes (E2M1; two groups for nvfp4) needs.
struct Slice {
    int x[16];
    float unit;      // 2^-sh (E2M1: half of it, the codes being doubled); NaN if any activation is infinite or NaN
    float xsum;      // affine: sum of the activations
    int off[2];      // E2M1: -64 * sum of the integers of each half
    E2m1Table e2m1;
};

// Element of half h (0, 1) of pair k within a word of eight codes.  Affine
// words split into two planes of four bytes (even and odd codes).
template <int MODE>
__host__ __device__ constexpr int pair_elem(int k, int h) {
    return MODE == QMM_MODE_AFFINE ? (k & 1) * 4 + h * 2 + (k >> 1) : 2 * k + h;
}

template <typename X>
__device__ __forceinline__ void load_slice(const X *x, bool ok, float (&f)[32]) {
    if constexpr (sizeof(X) == 4) {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            const float4 r = ok ? *reinterpret_cast<const float4 *>(x + 4 * c) : make_float4(0, 0, 0, 0);
            f[4 * c] = r.x;
            f[4 * c + 1] = r.y;
            f[4 * c + 2] = r.z;
            f[4 * c + 3] = r.w;
        }
    } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint4 r = ok ? *reinterpret_cast<const uint4 *>(x + 8 * c) : make_uint4(0, 0, 0, 0);
            const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const X lo = *reinterpret_cast<const X *>(&w[q]);
                const X hi = *(reinterpret_cast<const X *>(&w[q]) + 1);
                f[8 * c + 2 * q] = Dt<X>::to_f(lo);
                f[8 * c + 2 * q + 1] = Dt<X>::to_f(hi);
            }
        }
    }
}

template <int MODE>
__device__ __forceinline__ void make_slice(const float (&f)[32], Slice &s) {
    if constexpr (MODE != QMM_MODE_AFFINE) s.e2m1.set();
    uint32_t mb = 0;  // largest |x| by bit pattern (infinities and NaN largest)
#pragma unroll
    for (int i = 0; i < 32; ++i) mb = max(mb, __float_as_uint(f[i]) & 0x7FFFFFFFu);
    // largest < 2^ex; x 2^sh < 2^14 with sh = 14 - ex, kept where 2^sh and
    // 2^-sh are normal floats.
    const int ex = (int)(mb >> 23) - 126;
    const int sh = min(126, max(-126, 14 - ex));
    const float up = __uint_as_float((uint32_t)(127 + sh) << 23);
    s.unit = mb >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : __uint_as_float((uint32_t)(127 - sh) << 23);
    // rint(x 2^sh) by adding 1.5 * 2^23: the sum's low 16 bits are the
    // integer's two's complement, and sums of the words give sums of the
    // integers once the offsets are taken out.
    uint32_t sum[2] = {0u, 0u};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t a = __float_as_uint(__fmaf_rn(f[8 * w + pair_elem<MODE>(k, 0)], up, 12582912.0f));
            const uint32_t b = __float_as_uint(__fmaf_rn(f[8 * w + pair_elem<MODE>(k, 1)], up, 12582912.0f));
            s.x[4 * w + k] = (int)__byte_perm(a, b, 0x5410);
            sum[w >> 1] += a + b;
        }
    }
    const int s0 = (int)(sum[0] - 16u * 0x4B400000u), s1 = (int)(sum[1] - 16u * 0x4B400000u);
    s.xsum = s.unit * (float)(s0 + s1);
    if constexpr (MODE != QMM_MODE_AFFINE) s.unit *= 0.5f;
    if constexpr (MODE == QMM_MODE_NVFP4) {
        s.off[0] = -64 * s0;
        s.off[1] = -64 * s1;
    } else {
        s.off[0] = -64 * (s0 + s1);
        s.off[1] = 0;
    }
}

// The slice's product with 32 codes of one weight row; sb: the raw scale bits
// (mxfp4: one byte; nvfp4: two bytes; affine: scale | bias << 16).
template <typename T, int MODE>
__device__ __forceinline__ float dot_slice(const Slice &s, const uint4 &w, uint32_t sb) {
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
    if constexpr (MODE == QMM_MODE_AFFINE) {
        int a0 = 0, a1 = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t p0 = ws[i] & 0x0F0F0F0Fu, p1 = (ws[i] >> 4) & 0x0F0F0F0Fu;
            a0 = dp2a_lo(s.x[4 * i], p0, a0);
            a1 = dp2a_hi(s.x[4 * i + 1], p0, a1);
            a0 = dp2a_lo(s.x[4 * i + 2], p1, a0);
            a1 = dp2a_hi(s.x[4 * i + 3], p1, a1);
        }
        const uint16_t sh = (uint16_t)sb, bh = (uint16_t)(sb >> 16);
        const float sc = Dt<T>::to_f(*reinterpret_cast<const T *>(&sh));
        const float bi = Dt<T>::to_f(*reinterpret_cast<const T *>(&bh));
        // (scale * 2^-sh) first: the integer sum times 2^-sh alone could leave
        // the fp32 range for activations near the top of bf16's.
        return __fmaf_rn(sc * s.unit, (float)(a0 + a1), bi * s.xsum);
    } else {
        constexpr bool NV = MODE == QMM_MODE_NVFP4;
        int a0 = s.off[0], a1 = 0, b0 = s.off[1], b1 = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t lo, hi;
            e2m1_bytes(s.e2m1, ws[i], lo, hi);
            int &c0 = (NV && i >= 2) ? b0 : a0;
            int &c1 = (NV && i >= 2) ? b1 : a1;
            c0 = dp2a_lo(s.x[4 * i], lo, c0);
            c1 = dp2a_hi(s.x[4 * i + 1], lo, c1);
            c0 = dp2a_lo(s.x[4 * i + 2], hi, c0);
            c1 = dp2a_hi(s.x[4 * i + 3], hi, c1);
        }
        if constexpr (NV) {
            const uint32_t h = mxf::e4m3x2_to_h2(sb, 0);
            const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&h));
            return __fmaf_rn(x.y * s.unit, (float)(b0 + b1), (x.x * s.unit) * (float)(a0 + a1));
        } else {
            return (e8m0(sb) * s.unit) * (float)(a0 + a1);
        }
    }
}

// Sum of each v[0..8) over the 32 lanes; lane l returns the total of v[l % 8].
__device__ __forceinline__ float reduce8(float (&v)[8], int lane) {
#pragma unroll
    for (int s = 4; s >= 1; s >>= 1) {
        const bool upper = (lane & s) != 0;
#pragma unroll
        for (int j = 0; j < s; ++j) {
            const float send = upper ? v[j] : v[j + s];
            const float keep = upper ? v[j + s] : v[j];
            v[j] = keep + __shfl_xor_sync(0xffffffffu, send, s);
        }
    }
    float r = v[0];
    r += __shfl_xor_sync(0xffffffffu, r, 8);
    r += __shfl_xor_sync(0xffffffffu, r, 16);
    return r;
}

// From the partial sums of a CTA's rows: h, or the tokens' outputs.
template <typename T, bool GLU>
__device__ __forceinline__ void finish_rows(const GemvParams &p, const float *part, int64_t r0, int nr) {
    if constexpr (GLU) {
        float *h = static_cast<float *>(p.out);
        for (int i = threadIdx.x; i < p.P * nr; i += blockDim.x) {
            const int slot = i / nr, r = i - slot * nr;
            if (moe_expert(p.indices, slot, p.E, nullptr) < 0) continue;
            float g = 0.f, up = 0.f;
            for (int s = 0; s < p.S; ++s) {
                const float *q = part + ((int64_t)(slot * p.S + s) * p.rows_cta + r) * 2;
                g += q[0];
                up += q[1];
            }
            h[(int64_t)slot * p.R + r0 + r] = moe_gate(g, p.act) * up;
        }
    } else {
        const int T_ = p.P / p.top_k;
        for (int i = threadIdx.x; i < T_ * nr; i += blockDim.x) {
            const int t = i / nr, r = i - t * nr;
            float acc = 0.f;
            for (int j = 0; j < p.top_k; ++j) {
                const int slot = t * p.top_k + j;
                if (moe_expert(p.indices, slot, p.E, nullptr) < 0) continue;
                float d = 0.f;
                for (int s = 0; s < p.S; ++s) d += part[(int64_t)(slot * p.S + s) * p.rows_cta + r];
                acc = __fmaf_rn(__ldg(p.weights + slot), d, acc);
            }
            static_cast<T *>(p.out)[(int64_t)t * p.R + r0 + r] = Dt<T>::from_f(acc);
        }
    }
}

// X: type of the activations (T, or float for h).  GLU: the first kernel.
template <typename T, typename X, int MODE, bool GLU>
__global__ void __launch_bounds__(32 * kMaxWarps, 1) moe_gemv_kernel(const GemvParams p) {
    constexpr int NM = GLU ? 2 : 1;       // matrices a row is taken from
    constexpr int RB = kLoads / NM;       // rows per batch
    extern __shared__ float part[];       // [unit][row][NM]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t r0 = (int64_t)blockIdx.x * p.rows_cta;
    const int nr = (int)min((int64_t)p.rows_cta, p.R - r0);
    const int uw = warp % p.unit_warps, rw = warp / p.unit_warps;
    const int per = (nr + p.row_splits - 1) / p.row_splits;
    const int ra = min(nr, rw * per), rb = min(nr, ra + per);
    const int64_t row_bytes = p.C / 2;
    const int64_t gpr = p.C >> p.gs_log;
    ptx::grid_dependency_wait();
    ptx::grid_launch_dependents();

    for (int u = uw; u < p.units; u += p.unit_warps) {
        const int slot = u / p.S, seg = u - slot * p.S;
        const int e = moe_expert(p.indices, slot, p.E, blockIdx.x == 0 && lane == 0 ? p.err : nullptr);
        if (e < 0) continue;
        const int64_t k0 = (int64_t)seg * kSeg + lane * 32;
        const bool ok = k0 < p.C;
        const uint8_t *wbase[NM];
        const uint8_t *sbase[NM], *bbase[NM];
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            const int64_t row = (int64_t)e * p.R + r0;
            wbase[m] = reinterpret_cast<const uint8_t *>(p.w[m].wq) + row * row_bytes + k0 / 2;
            const int64_t g = row * gpr + (k0 >> p.gs_log);
            constexpr int SB = MODE == QMM_MODE_AFFINE ? 2 : 1;
            sbase[m] = static_cast<const uint8_t *>(p.w[m].scales) + SB * g;
            bbase[m] = MODE == QMM_MODE_AFFINE ? static_cast<const uint8_t *>(p.w[m].biases) + SB * g : nullptr;
        }
        uint4 wv[2][kLoads];
        uint32_t sv[2][kLoads];
        auto fetch = [&](int r, uint4 (&w)[kLoads], uint32_t (&s)[kLoads]) {
#pragma unroll
            for (int j = 0; j < RB; ++j) {
#pragma unroll
                for (int m = 0; m < NM; ++m) {
                    const int i = j * NM + m;
                    w[i] = make_uint4(0, 0, 0, 0);
                    s[i] = 0;
                    if (ok && r + j < rb) {
                        w[i] = ld_stream(wbase[m] + (int64_t)(r + j) * row_bytes);
                        if constexpr (MODE == QMM_MODE_AFFINE) {
                            const int64_t o = (int64_t)(r + j) * gpr * 2;
                            s[i] = (uint32_t)__ldg(reinterpret_cast<const uint16_t *>(sbase[m] + o)) |
                                   ((uint32_t)__ldg(reinterpret_cast<const uint16_t *>(bbase[m] + o)) << 16);
                        } else if constexpr (MODE == QMM_MODE_NVFP4) {
                            s[i] = __ldg(reinterpret_cast<const uint16_t *>(sbase[m] + (int64_t)(r + j) * gpr));
                        } else {
                            s[i] = __ldg(sbase[m] + (int64_t)(r + j) * gpr);
                        }
                    }
                }
            }
        };
        if (ra < rb) fetch(ra, wv[0], sv[0]);
        Slice sl;
        {
            float f[32];
            const int64_t xr = GLU ? slot / p.top_k : slot;
            load_slice<X>(static_cast<const X *>(p.x) + xr * p.C + k0, ok, f);
            make_slice<MODE>(f, sl);
        }
        auto use = [&](int r, const uint4 (&w)[kLoads], const uint32_t (&s)[kLoads]) {
            float v[kLoads];
#pragma unroll
            for (int i = 0; i < kLoads; ++i) v[i] = dot_slice<T, MODE>(sl, w[i], s[i]);  // (0 where !ok)
            const float t = reduce8(v, lane);
            if (lane < kLoads && r + lane / NM < rb)
                part[((int64_t)u * p.rows_cta + r) * NM + lane] = t;
        };
        for (int r = ra; r < rb; r += 2 * RB) {
            if (r + RB < rb) fetch(r + RB, wv[1], sv[1]);
            use(r, wv[0], sv[0]);
            if (r + RB < rb) {
                if (r + 2 * RB < rb) fetch(r + 2 * RB, wv[0], sv[0]);
                use(r + RB, wv[1], sv[1]);
            }
        }
    }
    __syncthreads();
    finish_rows<T, GLU>(p, part, r0, nr);
}

// ---------------------------------------------------------------------------
// The streaming form: the same units and arithmetic, with the weights brought
// in by bulk copies.  CTA c's rows of a slot's expert are one contiguous
// stretch of codes and one of scales; a producer warp streams them, a few rows
// of every slot of a round at a time, through a ring of stages in shared memory,
// so that the copies in flight depend on neither registers nor the warps'
// progress.  A round is as many slots as 16 consumer warps have units for; with
// few units a stage's rows are split among them.  The second kernel starts its
// copies before the first has finished: it waits only with its activations.
// ---------------------------------------------------------------------------
struct StreamParams {
    GemvParams g;
    int slots_round, rounds, rows_stage, stages, stage_bytes;
    int row_bytes, sb_bytes;  // of one row: codes; scales (or biases)
};

template <typename T, typename X, int MODE, bool GLU>
__global__ void __launch_bounds__(32 * (kMaxWarps + 1), 1) moe_stream_kernel(const StreamParams sp) {
    constexpr int NM = GLU ? 2 : 1;
    constexpr bool AFF = MODE == QMM_MODE_AFFINE;
    constexpr int NA = AFF ? 3 : 2;       // arrays per matrix: codes, scales (, biases)
    constexpr int RB = kLoads / NM;       // rows of a warp per stage at most
    extern __shared__ __align__(128) uint8_t sm[];
    const GemvParams &p = sp.g;
    const int D = sp.stages;
    const uint32_t full = ptx::smem_addr(sm), empty = full + 8 * D;
    uint8_t *ring = sm + 128;
    float *part = reinterpret_cast<float *>(ring + (size_t)D * sp.stage_bytes);  // [slot][seg][row][NM]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t r0 = (int64_t)blockIdx.x * p.rows_cta;
    const int nr = (int)min((int64_t)p.rows_cta, p.R - r0);
    const int nst = (nr + sp.rows_stage - 1) / sp.rows_stage;  // stages of a round
    // Bytes of one slot and matrix in a stage: codes, scales, biases of rows_stage rows.
    const int mat_bytes = sp.rows_stage * (sp.row_bytes + (NA - 1) * sp.sb_bytes);
    if (threadIdx.x == 0) {
        for (int i = 0; i < D; ++i) {
            ptx::mbar_init(full + 8 * i, 1);
            ptx::mbar_init(empty + 8 * i, kMaxWarps);
        }
        ptx::fence_mbar_init();
    }
    __syncthreads();
    // The first kernel allows the second one only once everything before itself
    // is complete; the second may therefore read indices and weights at once.
    if (GLU) {
        ptx::grid_dependency_wait();
        ptx::grid_launch_dependents();
    }
    if (warp == 0) {
        // ---------------- producer ----------------
        int n = 0;
        for (int rd = 0; rd < sp.rounds; ++rd) {
            const int first = rd * sp.slots_round, count = min(sp.slots_round, p.P - first);
            const int copies = count * NM * NA;
            for (int st = 0; st < nst; ++st, ++n) {
                const int slot_ = n % D;
                const int rows = min(sp.rows_stage, nr - st * sp.rows_stage);
                if (n >= D) ptx::mbar_wait(empty + 8 * slot_, ((n / D) - 1) & 1, p.err);
                __syncwarp();
                uint32_t bytes = 0;
                for (int j = lane; j < count; j += 32)
                    if (moe_expert(p.indices, first + j, p.E, nullptr) >= 0)
                        bytes += (uint32_t)(NM * rows * (sp.row_bytes + (NA - 1) * sp.sb_bytes));
                bytes = __reduce_add_sync(0xffffffffu, bytes);
                if (lane == 0) ptx::mbar_arrive_expect_tx(full + 8 * slot_, bytes);
                __syncwarp();
                for (int c = lane; c < copies; c += 32) {
                    const int a = c % NA, m = c / NA % NM, j = c / (NA * NM);
                    const int e = moe_expert(p.indices, first + j, p.E, nullptr);
                    if (e < 0) continue;
                    const int64_t row = (int64_t)e * p.R + r0 + (int64_t)st * sp.rows_stage;
                    const uint8_t *src = a == 0 ? reinterpret_cast<const uint8_t *>(p.w[m].wq) + row * sp.row_bytes
                                                : static_cast<const uint8_t *>(a == 1 ? p.w[m].scales : p.w[m].biases) +
                                                      row * sp.sb_bytes;
                    uint8_t *dst = ring + (size_t)slot_ * sp.stage_bytes + (j * NM + m) * mat_bytes +
                                   (a == 0 ? 0 : sp.rows_stage * (sp.row_bytes + (a - 1) * sp.sb_bytes));
                    ptx::bulk_g2s(ptx::smem_addr(dst), src, (uint32_t)(rows * (a == 0 ? sp.row_bytes : sp.sb_bytes)),
                                  full + 8 * slot_);
                }
            }
        }
        // No copy may land after the CTA has left.
        if (lane == 0)
            for (int k = max(0, n - D); k < n; ++k) ptx::mbar_drain(full + 8 * (k % D), (k / D) & 1, p.err);
    } else {
        // ---------------- consumers ----------------
        if (!GLU) ptx::grid_dependency_wait();  // h
        const int u = warp - 1, per_split = sp.slots_round * p.S;
        const int split = u / per_split, j = u % per_split / p.S, seg = u % p.S;
        const int64_t k0 = (int64_t)seg * kSeg + lane * 32;
        const bool in = split < p.row_splits && k0 < p.C;
        const int koff = in ? (int)(k0 / 2) : 0;
        const int goff = in ? (int)(k0 >> p.gs_log) * (AFF ? 2 : 1) : 0;
        int n = 0;
        for (int rd = 0; rd < sp.rounds; ++rd) {
            const int slot = rd * sp.slots_round + j;
            const int e = split < p.row_splits && slot < p.P
                              ? moe_expert(p.indices, slot, p.E, GLU && blockIdx.x == 0 && lane == 0 ? p.err : nullptr)
                              : -1;
            Slice sl;
            if (e >= 0) {
                float f[32];
                const int64_t xr = GLU ? slot / p.top_k : slot;
                load_slice<X>(static_cast<const X *>(p.x) + xr * p.C + k0, in, f);
                make_slice<MODE>(f, sl);
            }
            for (int st = 0; st < nst; ++st, ++n) {
                const int slot_ = n % D;
                const int rows = min(sp.rows_stage, nr - st * sp.rows_stage);
                const int per = (rows + p.row_splits - 1) / p.row_splits;
                const int ra = min(rows, split * per), rb = min(rows, ra + per);
                ptx::mbar_wait(full + 8 * slot_, (n / D) & 1, p.err);
                if (e >= 0) {
                    const uint32_t at0 = ptx::smem_addr(ring) + slot_ * sp.stage_bytes + j * NM * mat_bytes;
                    float *out = part + ((slot * p.S + seg) * p.rows_cta + st * sp.rows_stage) * NM;
                    for (int r = ra; r < rb; r += RB) {
                        // (a batch past the split's end repeats its last row, whose sums are dropped)
                        uint32_t cw = at0 + r * sp.row_bytes + koff;
                        uint32_t cs = at0 + sp.rows_stage * sp.row_bytes + r * sp.sb_bytes + goff;
                        float v[kLoads];
#pragma unroll
                        for (int i = 0; i < RB; ++i) {
#pragma unroll
                            for (int m = 0; m < NM; ++m) {
                                const uint4 w = lds128(cw + m * mat_bytes);
                                uint32_t sb;
                                if constexpr (AFF)
                                    sb = lds16(cs + m * mat_bytes) |
                                         (lds16(cs + m * mat_bytes + sp.rows_stage * sp.sb_bytes) << 16);
                                else if constexpr (MODE == QMM_MODE_NVFP4)
                                    sb = lds16(cs + m * mat_bytes);
                                else
                                    sb = lds8(cs + m * mat_bytes);
                                v[i * NM + m] = dot_slice<T, MODE>(sl, w, sb);
                            }
                            if (r + i + 1 < rb) {
                                cw += sp.row_bytes;
                                cs += sp.sb_bytes;
                            }
                        }
                        const float t = reduce8(v, lane);
                        if (lane < kLoads && r + lane / NM < rb) out[r * NM + lane] = t;
                    }
                }
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(empty + 8 * slot_);
            }
        }
    }
    __syncthreads();
    finish_rows<T, GLU>(p, part, r0, nr);
}

// Shape of the streaming form for one product, or false where it does not
// apply: contractions past 16 segments, or scale rows that a bulk copy cannot
// take (not in whole 16-byte units).
template <int MODE, bool GLU>
bool plan_stream(StreamParams &sp, size_t &smem) {
    constexpr int NM = GLU ? 2 : 1, NA = MODE == QMM_MODE_AFFINE ? 3 : 2, ES = MODE == QMM_MODE_AFFINE ? 2 : 1;
    GemvParams &p = sp.g;
    p.S = (int)((p.C + kSeg - 1) / kSeg);
    const int64_t sb = (p.C >> p.gs_log) * ES;
    if (p.S > kMaxWarps || sb % 16 != 0) return false;
    sp.row_bytes = (int)(p.C / 2);
    sp.sb_bytes = (int)sb;
    sp.slots_round = std::min(p.P, kMaxWarps / p.S);
    sp.rounds = (p.P + sp.slots_round - 1) / sp.slots_round;
    p.row_splits = kMaxWarps / (sp.slots_round * p.S);
    p.units = p.P * p.S;
    // Partial sums of at most 32 KB; the ring takes what is left of 220 KB.
    constexpr int64_t kPart = 32 * 1024, kRing = 220 * 1024 - kPart - 128;
    int64_t rows = (p.R + num_sms() - 1) / num_sms();
    rows = std::min<int64_t>(rows, kPart / ((int64_t)p.units * NM * 4));
    if (rows < 1) return false;
    p.rows_cta = (int)rows;
    const int64_t row_all = (int64_t)sp.slots_round * NM * (sp.row_bytes + (NA - 1) * sp.sb_bytes);
    int64_t rs = std::min<int64_t>(rows, (int64_t)(kLoads / NM) * p.row_splits);
    rs = std::min(rs, rows <= kRing / row_all ? rows : kRing / 3 / row_all);
    if (rs < 1) return false;
    sp.rows_stage = (int)rs;
    sp.stage_bytes = (int)(rs * row_all);
    sp.stages = (int)std::min<int64_t>(8, kRing / sp.stage_bytes);
    smem = 128 + (size_t)sp.stages * sp.stage_bytes + (size_t)p.units * rows * NM * 4;
    return true;
}

template <typename T, typename X, int MODE, bool GLU>
cudaError_t launch_half(GemvParams p, cudaStream_t s) {
    constexpr int NM = GLU ? 2 : 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    StreamParams sp{};
    sp.g = p;
    size_t ring = 0;
    if (plan_stream<MODE, GLU>(sp, ring)) {
        auto kern = moe_stream_kernel<T, X, MODE, GLU>;
        struct StreamTag;
        cudaError_t e = configure_once<StreamTag>((size_t)227 * 1024, [&]() {
            return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
        });
        if (e != cudaSuccess) return e;
        cfg.gridDim = dim3((unsigned)((p.R + sp.g.rows_cta - 1) / sp.g.rows_cta), 1, 1);
        cfg.blockDim = dim3(32 * (kMaxWarps + 1), 1, 1);
        cfg.dynamicSmemBytes = ring;
        e = cudaLaunchKernelEx(&cfg, kern, sp);
        if (e != cudaSuccess) return e;
        count_launches(1);
        return cudaGetLastError();
    }
    p.S = (int)((p.C + kSeg - 1) / kSeg);
    p.units = p.P * p.S;
    p.unit_warps = std::min(p.units, kMaxWarps);
    p.row_splits = kMaxWarps / p.unit_warps;
    int64_t rows = (p.R + num_sms() - 1) / num_sms();
    rows = std::min<int64_t>(rows, kPartBytes / ((int64_t)p.units * NM * 4));
    p.rows_cta = (int)rows;
    const size_t smem = (size_t)p.units * (size_t)rows * NM * 4;
    auto kern = moe_gemv_kernel<T, X, MODE, GLU>;
    struct Tag;
    cudaError_t e = configure_once<Tag>(smem, [&]() {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    });
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)((p.R + rows - 1) / rows), 1, 1);
    cfg.blockDim = dim3(32 * p.unit_warps * p.row_splits, 1, 1);
    cfg.dynamicSmemBytes = smem;
    e = cudaLaunchKernelEx(&cfg, kern, p);
    if (e != cudaSuccess) return e;
    count_launches(1);
    return cudaGetLastError();
}

template <typename T, int MODE>
cudaError_t run(const ExpertsArgs &a, cudaStream_t s) {
    GemvParams p{};
    p.indices = a.indices;
    p.weights = a.weights;
    p.P = (int)(a.T * a.top_k);
    p.top_k = a.top_k;
    p.E = (int)a.n_experts;
    p.gs_log = a.group_size == 16 ? 4 : (a.group_size == 32 ? 5 : (a.group_size == 64 ? 6 : 7));
    p.act = a.act;
    p.err = device_error_word();
    p.x = a.x;
    p.w[0] = a.gate;
    p.w[1] = a.up;
    p.out = a.ws;
    p.C = a.K;
    p.R = a.I;
    cudaError_t e = launch_half<T, T, MODE, true>(p, s);
    if (e != cudaSuccess) return e;
    p.x = a.ws;
    p.w[0] = p.w[1] = a.down;
    p.out = a.y;
    p.C = a.I;
    p.R = a.N;
    return launch_half<T, float, MODE, false>(p, s);
}

template <typename T>
cudaError_t run_mode(const ExpertsArgs &a, cudaStream_t s) {
    switch (a.mode) {
    case QMM_MODE_AFFINE: return run<T, QMM_MODE_AFFINE>(a, s);
    case QMM_MODE_MXFP4: return run<T, QMM_MODE_MXFP4>(a, s);
    default: return run<T, QMM_MODE_NVFP4>(a, s);
    }
}

// Tokens of one pass: about 64 slots, fewer for contractions so long that the
// partial sums of one row would pass a CTA's share of shared memory.
int64_t block_tokens(const ExpertsArgs &a) {
    const int64_t S = (std::max(a.K, a.I) + kSeg - 1) / kSeg;
    const int64_t slots = std::max<int64_t>(a.top_k, std::min<int64_t>(64, kPartBytes / (8 * S)));
    return std::max<int64_t>(1, slots / a.top_k);
}

}  // namespace

bool moe_gemv_supported(const ExpertsArgs &a) {
    return a.top_k * ((std::max(a.K, a.I) + kSeg - 1) / kSeg) * 8 <= kPartBytes;
}

size_t moe_gemv_workspace(const ExpertsArgs &a) {
    return (size_t)(std::min<int64_t>(a.T, block_tokens(a)) * a.top_k) * (size_t)a.I * 4;
}

cudaError_t launch_moe_gemv(qmm_dtype dt, const ExpertsArgs &a, cudaStream_t s) {
    const int64_t step = block_tokens(a);
    for (int64_t t = 0; t < a.T; t += step) {
        ExpertsArgs b = a;
        b.T = std::min(step, a.T - t);
        b.x = static_cast<const char *>(a.x) + t * a.K * 2;
        b.y = static_cast<char *>(a.y) + t * a.N * 2;
        b.indices = a.indices + t * a.top_k;
        b.weights = a.weights + t * a.top_k;
        const cudaError_t e = dt == QMM_BF16 ? run_mode<__nv_bfloat16>(b, s) : run_mode<__half>(b, s);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace qmm
