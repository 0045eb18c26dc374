// What the attention kernels for packed prompts and for trees share: one tile of the softmax on the
// tensor-core path, and the tensor maps of rows.
//
// A CTA has two lanes of 128 query rows, each with its own score, weight and output columns in tensor
// memory and two warps that issue its products, one for each kind (waits, issue and commits of both in one
// warp are as long as a tile takes):
//   S[row][key] = Q K^T (fp32) -> registers: running maximum, exp2, sum -> bf16 weights P in tensor memory
//   -> O += P V with P read from there, V MN-major from shared memory.
// A lane waits for neither product: the next tile's scores are computed while this one's weights are, and
// P V while the next one's are. Beside O a lane has three slots of columns (a, b, c), each as wide as half a
// tile's scores or all of its weights: S of an even tile lies in a and b and its P in a (its scores are in
// registers by then), S of an odd tile in b and c and its P in c. So S of a tile does not touch the weights
// of the one before, and touches those of the one before that only when their product is done. That sets the
// tile's width: 128 columns for heads of 128 are three slots of 40, 80 keys. For heads of 64, 192 columns would
// be 128 keys, but 96 is what fits a softmax thread's registers (619 us for 629 with 16384 tokens x 16 heads when
// it was chosen; 600 now). (With P over S, tiles of 128 keys and turns at the softmax: 1.58 ms for 32768 tokens x 8
// heads of 128; with a place of its own for P, but one only: 1.64; with this 1.62, of which the steps after it, products
// issued from uniform code by a warp for each kind and a ring of six slots, left 1.30.)
// Eight warps serve a lane, two threads a row with half of the scores each: their maxima meet in a barrier
// that carries one bit, "the maximum of some row has grown by more than 2^8": only then do they exchange
// them and rescale O. So weights are at most 2^8, and the sum stays fp32.
// The weights enter P V as bf16, the type that products with V want: off by 2^-9 relative on average, of
// both signs, while their sum is fp32.
#pragma once

#include <cudaTypedefs.h>

#include "evs_common.cuh"
#include "sm100_ptx.cuh"

namespace evs {
namespace attn {

using bf16 = __nv_bfloat16;

// A tile's keys; a lane's columns of tensor memory: where S and P of a tile are (by its parity), and O
constexpr int tile_keys(int dh) { return dh == 128 ? 80 : 96; }
constexpr uint32_t LANE_COLS = 256;
__host__ __device__ constexpr uint32_t s_col(int dh, uint32_t tile) { return (tile & 1u) * (uint32_t)(tile_keys(dh) / 2); }
__host__ __device__ constexpr uint32_t p_col(int dh, uint32_t tile) { return (tile & 1u) * (uint32_t)tile_keys(dh); }
constexpr uint32_t o_col(int dh) { return LANE_COLS - (uint32_t)dh; }
constexpr int tile_bytes(int dh) { return tile_keys(dh) * dh * 2; }
constexpr int Q_ROWS = 128;
// Slots of the ring of K and V tiles. At least three for each worker: who waits for a slot's next phase has to know
// that the one before is over (see the waits for full[]). More than six of 20 KB cost time: four a lane 232 us for
// 202 with three (41 nodes x 32 heads over 4 caches of 32768 rows), eight a pair 228 for 220 (packed prompts).
constexpr int ring_slots(int dh) { return dh == 128 ? 6 : 8; }
constexpr int SOFT_WARPS = 16, AUX_WARPS = 8, THREADS = 32 * (SOFT_WARPS + AUX_WARPS);
constexpr float RESCALE_LOG2 = 8.f;
constexpr float LN2 = 0.6931471805599453f, LOG2E = 1.4426950408889634f;
// Registers of the launch's 768 x 80: 512 x 96 + 256 x 48
#define EVS_ATTN_SOFT_REGS "setmaxnreg.inc.sync.aligned.u32 96;"
#define EVS_ATTN_AUX_REGS "setmaxnreg.dec.sync.aligned.u32 48;"

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

// Loads and stores of 32 lanes x 32 bits, N consecutive columns a lane, without the wait.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t* r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
        "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint32_t* r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3])
                 : "memory");
}

// A softmax thread: row `row` of lane `lane`, the columns of half `half`.
template <int DH> struct SoftThread {
    static constexpr int N = tile_keys(DH) / 2;   // its scores of a tile
    static_assert(N == 40 || N == 48, "loads and stores of a tile");
    int lane, half, row, bar;            // bar: named barrier of its 64 threads
    uint32_t s_at, p_at, o_at;           // its scores and weights of an even tile, its output columns
    float* xch;                          // [128] of its lane, for what the two threads of a row exchange
    float m, l;                          // running maximum (log2 units), sum over its columns

    __device__ __forceinline__ void init(int warp, int ln, uint32_t tmem, float* exchange) {
        lane = warp >> 3;
        half = (warp >> 2) & 1;
        const int q4 = warp & 3;
        row = q4 * 32 + ln;
        bar = 1 + lane * 4 + q4;
        const uint32_t at = tmem + ((uint32_t)(q4 * 32) << 16) + (uint32_t)lane * LANE_COLS;
        s_at = at + (uint32_t)(half * N);
        p_at = at + (uint32_t)(half * (N / 2));
        o_at = at + o_col(DH) + (uint32_t)(half * (DH / 2));
        xch = exchange + lane * 128;
    }
    // One value of both threads of the row
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
    // Scores of tile `tile` of the lane
    __device__ __forceinline__ void load(uint32_t (&x)[N], uint32_t tile) const {
        const uint32_t at = s_at + s_col(DH, tile);
        tmem_ld32(at, x);
        if constexpr (N == 40) tmem_ld8(at + 32, x + 32);
        else tmem_ld16_issue(at + 32, *reinterpret_cast<uint32_t(*)[16]>(x + 32));
        tmem_wait_ld();
    }
    // Scores behind the first n of the thread's: no weight
    static __device__ __forceinline__ void mask_from(uint32_t (&x)[N], int n) {
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (j >= n) x[j] = 0xff800000u;
    }
    // The scores x of tile `at` of the lane become weights in tensor memory. first: O holds nothing yet; before():
    // waits until the products of the tile before are in O.
    template <typename W> __device__ __forceinline__ void tile(uint32_t (&x)[N], float sl, uint32_t at, bool first, W before) {
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < N; j += 2)
            mx[(j >> 1) & 3] = max3(mx[(j >> 1) & 3], __uint_as_float(x[j]), __uint_as_float(x[j + 1]));
        float mine = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl;
        auto grown = [&](float v) { return v > m + RESCALE_LOG2 || (m == -INFINITY && v > -INFINITY); };
        if (bar_any(bar, grown(mine))) {                 // (also: both threads of a row have their scores)
            mine = exchange(mine, [](float a, float b) { return fmaxf(a, b); });
            const bool move = grown(mine);
            if (!first) {
                before();
                tc_fence_after();
                const float f = move ? ex2_approx_ftz(m - mine) : 1.f;
#pragma unroll 1
                for (int c = 0; c < DH / 32; ++c) {
                    uint32_t o[16];
                    tmem_ld16_issue(o_at + (uint32_t)(c * 16), o);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                    tmem_st16(o_at + (uint32_t)(c * 16), o);
                }
                l *= f;
            }
            if (move) m = mine;
        }
        const float mb = m == -INFINITY ? 0.f : m;       // only -inf scores so far: weights 0
        const uint64_t sl2 = pair(sl, sl), mb2 = pair(-mb, -mb);
        uint64_t sum0 = 0, sum1 = 0;                     // two fp32 each
        uint32_t w[N / 2];
        const uint32_t to = p_at + p_col(DH, at);
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
            float e0, e1;
            unpair(fma2(pair(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1])), sl2, mb2), e0, e1);
            e0 = ex2_approx_ftz(e0);
            e1 = ex2_approx_ftz(e1);
            if (j & 1) sum1 = add2(sum1, pair(e0, e1));
            else sum0 = add2(sum0, pair(e0, e1));
            w[j] = pack2(e0, e1);
            if (j == 15) tmem_st16(to, *reinterpret_cast<const uint32_t(*)[16]>(w));
        }
        tmem_st4(to + 16, w + 16);
        if constexpr (N == 48) tmem_st4(to + 20, w + 20);
        float l0, l1;
        unpair(add2(sum0, sum1), l0, l1);
        l += l0 + l1;
    }
};

// Slots of a ring that holds K0 V0 K1 V1 ..., as one who reads every other one goes through them
struct Cursor {
    int slot, slots;
    uint32_t phase;
    __device__ __forceinline__ Cursor(int first, int n) : slot(first), slots(n), phase(0) {}
    __device__ __forceinline__ void next() {
        slot += 2;
        if (slot >= slots) {
            slot -= slots;
            phase ^= 1u;
        }
    }
};

// Clears the rows nv .. up to the end of their 16-row step of a V tile, by a warp, ahead of its product: they may
// hold anything, and the weight 0 of a key does not silence a NaN. (Two lanes may both write these zeros.)
template <int DH> __device__ __forceinline__ void clear_rows(uint8_t* tile, int nv, int lane) {
    const int rows = 16 - (nv & 15);
#pragma unroll 1
    for (int e = lane; e < rows * (DH / 8); e += 32) {
        const int hf = e / (rows * 8), k = nv + (e - hf * rows * 8) / 8;
        *reinterpret_cast<uint4*>(tile + hf * tile_keys(DH) * 128 + k * 128 + e % 8 * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_proxy_async_smem();
    __syncwarp();
}

// V of keys that some rows of the tile do not read: the weight 0 does not silence what is not finite there. So warps
// that have nothing else to do look through such rows first, ahead of the weights, and where they find any clear
// those values; a CTA that has cleared any goes through its work once more at its end and adds them to the rows that
// do read them, where nothing else counts beside them.
// Any bf16 of these two that is not finite
__device__ __forceinline__ uint32_t not_finite2(uint32_t w) { return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }
// part: the warp's of `parts` that share the rows from .. to - 1
template <int DH> __device__ __forceinline__ bool scan_rows(const uint8_t* tile, int from, int to, int part, int parts, int lane) {
    uint32_t bad = 0;
#pragma unroll
    for (int hf = 0; hf < DH / 64; ++hf) {
        const uint8_t* at = tile + hf * tile_keys(DH) * 128 + (lane & 7) * 16;
#pragma unroll 2
        for (int k = from + part * 4 + (lane >> 3); k < to; k += parts * 4) {
            const uint4 x = *reinterpret_cast<const uint4*>(at + k * 128);
            bad |= not_finite2(x.x) | not_finite2(x.y) | not_finite2(x.z) | not_finite2(x.w);
        }
    }
    return __any_sync(0xffffffffu, bad != 0) != 0;
}
template <int DH> __device__ __forceinline__ void clear_values(uint8_t* tile, int from, int to, int part, int parts, int lane) {
#pragma unroll 1
    for (int e = lane; e < (to - from) * (DH / 2); e += 32) {
        const int k = from + e / (DH / 2), c = e % (DH / 2);
        if ((k - from) / 4 % parts != part) continue;
        uint32_t* x = reinterpret_cast<uint32_t*>(tile + (c >> 5) * tile_keys(DH) * 128 + k * 128 + (c & 31) * 4);
        const uint32_t bad = not_finite2(*x);
        if (bad) *x &= ~((bad >> 15 & 1u) * 0xffffu | (bad >> 31) * 0xffff0000u);
    }
    fence_proxy_async_smem();
    __syncwarp();
}
// The lane's columns (DH / 32 of them) of a row of V, what is finite as 0; true where any lane's is not.
template <int DH> __device__ __forceinline__ bool bad_values(const bf16* v, int lane, float (&x)[DH / 32]) {
    bool any = false;
#pragma unroll
    for (int u = 0; u < DH / 32; ++u) {
        const bf16 y = v[lane * (DH / 32) + u];
        const bool bad = not_finite2(__bfloat16_as_ushort(y)) != 0;
        x[u] = bad ? __bfloat162float(y) : 0.f;
        any |= bad;
    }
    return __any_sync(0xffffffffu, any) != 0;
}
// A wait of a whole warp, which agrees on how it ended
__device__ __forceinline__ bool all_wait(uint64_t* bar, uint32_t phase) { return __all_sync(0xffffffffu, mbar_wait(bar, phase)) != 0; }
// One thread of a warp issues its products, but all of it runs the code around them: descriptors and addresses
// are the same in every lane then, and stay in the uniform registers that the instruction reads them from.
__device__ __forceinline__ uint32_t elect_leader() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}
__device__ __forceinline__ void mma_ss(uint32_t leader, uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(accumulate), "r"(leader)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t leader, uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(id), "r"(accumulate), "r"(leader)
        : "memory");
}
__device__ __forceinline__ void commit(uint32_t leader, uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
        "r"(leader)
        : "memory");
}

// Issue of O += P V of tile `tile` of a lane over the first nv keys. accumulate: O holds earlier tiles.
template <int DH>
__device__ __forceinline__ void issue_pv(uint32_t leader, uint32_t lane, uint32_t tile, uint64_t vd, int nv, bool accumulate) {
    constexpr uint32_t id = idesc_bf16_f32_bmn(128, DH);
#pragma unroll
    for (int kk = 0; kk < tile_keys(DH) / 16; ++kk)
        if (kk * 16 < nv)
            mma_ts(leader, lane + o_col(DH), lane + p_col(DH, tile) + (uint32_t)(kk * 8), vd + (uint64_t)((kk * 16 * 128) >> 4), id,
                   (kk > 0 || accumulate) ? 1u : 0u);
}
// Issue of its S = Q K^T.
template <int DH>
__device__ __forceinline__ void issue_scores(uint32_t leader, uint32_t lane, uint32_t tile, uint64_t qd, uint64_t kd) {
    constexpr uint32_t id = idesc_bf16_f32(128, tile_keys(DH));
#pragma unroll
    for (int kk = 0; kk < DH / 16; ++kk)
        mma_ss(leader, lane + s_col(DH, tile), qd + (uint64_t)(((kk >> 2) * Q_ROWS * 128 + (kk & 3) * 32) >> 4),
               kd + (uint64_t)(((kk >> 2) * tile_keys(DH) * 128 + (kk & 3) * 32) >> 4), id, kk > 0 ? 1u : 0u);
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

// [seqs][heads][rows][dh] bf16, boxes of box_rows rows x 64 columns; rows outside read as zero.
inline bool make_rows_map(CUtensorMap* m, const void* base, int box_rows, int dh, int rows, int heads, int seqs, int64_t row,
                          int64_t head, int64_t seq) {
    const auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)dh, (cuuint64_t)rows, (cuuint64_t)heads, (cuuint64_t)seqs};
    const cuuint64_t r2 = rows > 1 ? (cuuint64_t)row * 2 : (cuuint64_t)dh * 2;
    const cuuint64_t h2 = heads > 1 ? (cuuint64_t)head * 2 : r2, s2 = seqs > 1 ? (cuuint64_t)seq * 2 : h2;
    const cuuint64_t strides[3] = {r2, h2, s2};
    const cuuint32_t box[4] = {64, (cuuint32_t)box_rows, 1, 1}, estr[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace attn
}  // namespace evs
