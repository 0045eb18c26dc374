// What the attention kernels for packed prompts and for trees share: one tile of the softmax on the
// tensor-core path, and the tensor maps of rows.
//
// A CTA has two lanes of 128 query rows, each with its own score, weight and output columns in tensor
// memory and a thread that issues its products:
//   S[row][key] = Q K^T (fp32, 128 columns) -> registers: running maximum, exp2, sum -> bf16 weights over
//   columns 0-31 and 64-95 of S -> O += P V with P read from tensor memory, V MN-major from shared memory.
// Eight warps serve a lane, two threads a row with 64 scores each: the same instructions as with one
// thread a row, at half the latency of a tile, and that is what bounds a lane: its next scores wait for
// this tile's weights, since S and P share their columns. The two threads' maxima meet in a barrier that
// carries one bit, "the maximum of some row has grown by more than 2^8": only then do they exchange them
// and rescale O. So weights are at most 2^8, and the sum stays fp32.
// The weights enter P V as bf16, the type that products with V want: off by 2^-9 relative on average, of
// both signs, while their sum is fp32.
//
// Tensor memory, columns: S/P of lane 0 and 1 at 0 and 128, O at 256 and 384.
#pragma once

#include <cudaTypedefs.h>

#include "evs_common.cuh"
#include "sm100_ptx.cuh"

namespace evs {
namespace attn {

using bf16 = __nv_bfloat16;

constexpr int KEYS = 128;                    // of a tile
constexpr int SOFT_WARPS = 16, AUX_WARPS = 4, THREADS = 32 * (SOFT_WARPS + AUX_WARPS);
constexpr float RESCALE_LOG2 = 8.f;
constexpr float LN2 = 0.6931471805599453f, LOG2E = 1.4426950408889634f;
// Registers of the launch's 640 x 96: 512 x 104 + 128 x 64
#define EVS_ATTN_SOFT_REGS "setmaxnreg.inc.sync.aligned.u32 104;"
#define EVS_ATTN_AUX_REGS "setmaxnreg.dec.sync.aligned.u32 64;"

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// Named barrier of the two warps that share 32 rows; true where any thread's pred is
__device__ __forceinline__ bool bar_any(int id, bool pred) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, %2, 64, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)pred), "r"(id)
        : "memory");
    return r != 0;
}

// A softmax thread: row `row` of lane `lane`, the columns of half `half`.
struct SoftThread {
    int lane, half, row, bar;            // bar: named barrier of its 64 threads
    uint32_t s_at, p_at, o_at;           // its scores, weights and output columns
    float* xch;                          // [128] of its lane, for what the two threads of a row exchange
    float m, l;                          // running maximum (log2 units), sum over its columns

    __device__ __forceinline__ void init(int warp, int ln, uint32_t tmem, float* exchange, int dh) {
        lane = warp >> 3;
        half = (warp >> 2) & 1;
        const int q4 = warp & 3;
        row = q4 * 32 + ln;
        bar = 1 + lane * 4 + q4;
        const uint32_t rows = tmem + ((uint32_t)(q4 * 32) << 16) + 0u;
        s_at = rows + (uint32_t)(lane * 128 + half * 64);
        p_at = s_at;
        o_at = rows + 256u + (uint32_t)(lane * 128 + half * (dh / 2));
        xch = exchange + lane * 128;
    }
    // One value of both threads of the row, by its first user (half 0) and then its second
    template <typename F> __device__ __forceinline__ float exchange(float mine, F both) {
        if (half == 1) xch[row] = mine;
        named_bar_sync(bar, 64);
        float r;
        if (half == 0) {
            r = both(mine, xch[row]);
            xch[row] = r;
        }
        named_bar_sync(bar, 64);
        if (half == 1) r = xch[row];
        return r;
    }
    __device__ __forceinline__ void begin() {
        m = -INFINITY;
        l = 0.f;
    }
    // The scores x (64 columns) of a tile become weights in tensor memory. first: O holds nothing yet;
    // pv_done(): waits until the products of the tile before are in O. false: that wait ran out.
    template <int DH, typename W>
    __device__ __forceinline__ bool tile(uint32_t (&x)[4][16], float sl, bool first, W pv_done) {
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int j = 0; j < 16; j += 2)
                mx[(j >> 1) & 3] = max3(mx[(j >> 1) & 3], __uint_as_float(x[c][j]), __uint_as_float(x[c][j + 1]));
        float mine = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl;
        auto grown = [&](float v) { return v > m + RESCALE_LOG2 || (m == -INFINITY && v > -INFINITY); };
        bool ok = true;
        if (bar_any(bar, grown(mine))) {
            mine = exchange(mine, [](float a, float b) { return fmaxf(a, b); });
            const bool move = grown(mine);
            if (!first) {
                ok = pv_done();
                tc_fence_after();
                const float f = move ? ex2_approx_ftz(m - mine) : 1.f;
                if (ok) {
#pragma unroll 1
                    for (int c = 0; c < DH / 32; ++c) {
                        uint32_t o[16];
                        tmem_ld16_issue(o_at + (uint32_t)(c * 16), o);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                        tmem_st16(o_at + (uint32_t)(c * 16), o);
                    }
                }
                l *= f;
            }
            if (move) m = mine;
        }
        const float mb = m == -INFINITY ? 0.f : m;       // only -inf scores so far: weights 0
        const uint64_t sl2 = pair(sl, sl), mb2 = pair(-mb, -mb);
        uint64_t sum0 = 0, sum1 = 0;                     // two fp32 each
#pragma unroll
        for (int c = 0; c < 2; ++c) {                    // 32 keys: 16 columns of weights
            uint32_t w[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const uint32_t* at = &x[2 * c + j / 8][(2 * j) & 15];
                float e0, e1;
                unpair(fma2(pair(__uint_as_float(at[0]), __uint_as_float(at[1])), sl2, mb2), e0, e1);
                e0 = ex2_approx_ftz(e0);
                e1 = ex2_approx_ftz(e1);
                if (j & 1) sum1 = add2(sum1, pair(e0, e1));
                else sum0 = add2(sum0, pair(e0, e1));
                w[j] = pack2(e0, e1);
            }
            tmem_st16(p_at + (uint32_t)(c * 16), w);
        }
        float l0, l1;
        unpair(add2(sum0, sum1), l0, l1);
        l += l0 + l1;
        return ok;
    }
    __device__ __forceinline__ void load(uint32_t (&x)[4][16]) const {
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld16_issue(s_at + (uint32_t)(c * 16), x[c]);
        tmem_wait_ld();
    }
};

// Keys behind the first n of a thread's 64: no weight
__device__ __forceinline__ void mask_from(uint32_t (&x)[4][16], int n) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int j = 0; j < 16; ++j)
            if (c * 16 + j >= n) x[c][j] = 0xff800000u;
}

// Clears the rows nv .. up to the end of its 16-row step of a V tile, by `threads` threads: they may hold
// anything, and the weight 0 of a key does not silence a NaN.
template <int DH> __device__ __forceinline__ void clear_rows(uint8_t* tile, int nv, int t, int threads) {
    const int rows = 16 - (nv & 15);
    for (int e = t; e < rows * (DH / 8); e += threads) {
        const int hf = e / (rows * 8), k = nv + (e - hf * rows * 8) / 8;
        *reinterpret_cast<uint4*>(tile + hf * KEYS * 128 + k * 128 + e % 8 * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
}

// Issue of O += P V over the first nv keys, by one thread. accumulate: O holds earlier tiles.
template <int DH>
__device__ __forceinline__ void issue_pv(uint32_t o_at, uint32_t s_at, uint64_t vd, int nv, bool accumulate) {
    constexpr uint32_t id = idesc_bf16_f32_bmn(128, DH);
    if (nv > KEYS - 16) {
#pragma unroll
        for (int kk = 0; kk < KEYS / 16; ++kk)
            tc_mma_f16_ta(o_at, s_at + (uint32_t)((kk >> 2) * 64 + (kk & 3) * 8), vd + (uint64_t)((kk * 16 * 128) >> 4), id,
                          (kk > 0 || accumulate) ? 1u : 0u);
    } else {
        for (int kk = 0; kk < (nv + 15) / 16; ++kk)
            tc_mma_f16_ta(o_at, s_at + (uint32_t)((kk >> 2) * 64 + (kk & 3) * 8), vd + (uint64_t)((kk * 16 * 128) >> 4), id,
                          (kk > 0 || accumulate) ? 1u : 0u);
    }
}
// Issue of S = Q K^T.
template <int DH> __device__ __forceinline__ void issue_scores(uint32_t s_at, uint64_t qd, uint64_t kd) {
    constexpr uint32_t id = idesc_bf16_f32(128, KEYS);
#pragma unroll
    for (int kk = 0; kk < DH / 16; ++kk) {
        const uint32_t off = (uint32_t)((kk >> 2) * KEYS * 128 + (kk & 3) * 32) >> 4;
        tc_mma_f16(s_at, qd + off, kd + off, id, kk > 0 ? 1u : 0u);
    }
}

// ---- host side ----------------------------------------------------------------------------------
inline size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

// Whether tensor maps describe rows of bf16 with these strides (elements; of a dimension of one: unused)
inline bool map_ok(const void* p, long long row, long long head, long long seq, bool heads, bool seqs) {
    return (uintptr_t)p % 16 == 0 && row % 8 == 0 && row > 0 && row < (1LL << 38) &&
           (!heads || (head % 8 == 0 && head > 0 && head < (1LL << 38))) &&
           (!seqs || (seq % 8 == 0 && seq > 0 && seq < (1LL << 38)));
}

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
        return nullptr;
    }();
    return fn;
}

// [seqs][heads][rows][dh] bf16, boxes of 128 rows x 64 columns; rows outside read as zero.
inline bool make_rows_map(CUtensorMap* m, const void* base, int dh, int rows, int heads, int seqs, int64_t row, int64_t head,
                          int64_t seq) {
    const auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)dh, (cuuint64_t)rows, (cuuint64_t)heads, (cuuint64_t)seqs};
    const cuuint64_t r2 = rows > 1 ? (cuuint64_t)row * 2 : (cuuint64_t)dh * 2;
    const cuuint64_t h2 = heads > 1 ? (cuuint64_t)head * 2 : r2, s2 = seqs > 1 ? (cuuint64_t)seq * 2 : h2;
    const cuuint64_t strides[3] = {r2, h2, s2};
    const cuuint32_t box[4] = {64, KEYS, 1, 1}, estr[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace attn
}  // namespace evs
