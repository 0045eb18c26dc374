// Attention for a batch whose sequences share a long prefix (evs_shared_attention): every query
// reads the shared rows, its sequence's own rows and the block rows of its candidate up to its
// own position. The shared rows are streamed once for all sequences: the queries of the whole
// batch that use a K/V head are the rows of one product.
//
//   o = sum_j exp(scale q.k_j - m) v_j / l over the three, lse = m + log l.
//
// Two launches: partial sums (o unnormalised, m, l) per run of keys, then a combine that merges
// a query's partials, adds its block rows and normalises.
//
// Measured, bf16, heads of 128: 4 sequences x 4 candidates x 13 positions x 32 heads behind 32768
// rows and 700 own 136 us (820 TFLOP/s, bound by the turns at the softmax); 64 sequences x 32 heads
// of 8 K/V heads behind 30001 rows and about 1024 own 79 us (its K/V at 6.4 TB/s between a start of
// 6 us and a combine of 5); 8 sequences x 8 heads behind 8192 rows and about 256 own 17.5 us, of
// which 12 do not depend on the rows.
#include <cudaTypedefs.h>

#include "evs_common.cuh"
#include "sm100_ptx.cuh"

namespace evs {
namespace {

using bf16 = __nv_bfloat16;

// What both launches know. A partial of a shared row r of K/V head g (r = m * group + head in the
// group, m = (b * C + c) * T + i) lies in segment g * sh_tiles + r / sh_rows, row r % sh_rows; of
// an own row r = (c * T + i) * group + head in segment (b * G + g) * own_tiles + r / own_rows.
// On CUDA cores a segment has `slots` partials, slot s of segment g is partial g * slots + s. On the
// tensor cores worker w's of segment g is partial w + g: the pieces of the axis in order step on to the
// next worker, the next segment or both, so no two share a number, and workers + segments are enough
// whatever the lengths. o is stored four columns at a time, [dh / 4][rows to a multiple of four][4], so that both the threads that write it (one a row) and those that read it (four
// columns each) touch consecutive addresses.
struct SharedArgs {
    const void *q, *kp, *vp, *ko, *vo, *kb, *vb;
    void* o;
    float* lse;
    const int32_t* own_len;
    uint32_t* flags;
    int64_t q_ld, o_ld, p_row, p_head, o_row, o_head, o_seq, b_row, b_head, b_cand;
    int B, C, T, H, G, dh, P, own_max, own_skip, q_bf16;
    float scale;
    float *sh_o, *own_o;       // [partial][dh / 4][rows4][4]
    float2 *sh_ml, *own_ml;    // [partial][rows] (m, l), natural units
    int sh_rows, sh_tiles, sh_slots, own_rows, own_tiles, own_slots;
    int partials;              // a partial kernel runs
    int tensor;                // the tensor-core kernel's partials (sh_slots: at most so many of a segment)
    int sh_pair, own_pair;     // 1: segments of up to 256 rows, a row tile a lane; 0: a lane of its own
    int* plan;                 // run lengths (shared, own), where own runs start, own costs before sequence b
    int q_vec, b_vec;          // q and block rows on 16 (8) bytes
};

__host__ __device__ inline int rows4(int rows) { return (rows + 3) & ~3; }

// fp32 problems keep the full precision of the exponential
template <typename T> __device__ __forceinline__ float exp_of(float x);
template <> __device__ __forceinline__ float exp_of<float>(float x) { return expf(x); }
template <> __device__ __forceinline__ float exp_of<bf16>(float x) { return __expf(x); }

// Own rows of sequence b, clamped to [0, own_max].
__device__ __forceinline__ int own_rows_of(const SharedArgs& a, int b, bool report) {
    if (!a.own_len) return 0;
    const int64_t n = (int64_t)__ldcg(a.own_len + b) - a.own_skip;   // any two 32-bit values
    if (n < 0 || n > a.own_max) {
        if (report && a.flags) atomicOr(a.flags, (uint32_t)EVS_FLAG_BAD_LEN);
        return n < 0 ? 0 : a.own_max;
    }
    return (int)n;
}

// A query enters its products in the type of K: fp32 queries of a bf16 cache are rounded to bf16 in
// every product, the block rows' and those on CUDA cores too, so that the result is that of the rounded
// queries whichever kernel the strides lead to. (The tensor cores multiply bf16 by bf16 only; the
// query's remainder as a second product would double the staged queries, 64 of the 227 KB.)
template <typename T> __device__ __forceinline__ float as_product(float q) { return to_f32(from_f32<T>(q)); }
template <typename T> __device__ __forceinline__ float load_q(const SharedArgs& a, int64_t at) {
    return a.q_bf16 ? __bfloat162float(((const bf16*)a.q)[at]) : as_product<T>(((const float*)a.q)[at]);
}

// Past L1, which may hold what an earlier kernel read: for loads ahead of the dependency wait.
__device__ __forceinline__ float load_l2(const float* p) { return __ldcg(p); }
__device__ __forceinline__ float load_l2(const bf16* p) {
    return __uint_as_float((uint32_t)__ldcg(reinterpret_cast<const unsigned short*>(p)) << 16);
}

// =========================================================================================
// Partials on CUDA cores: fp32, narrow heads, and strides that tensor maps cannot describe.
// A CTA takes 16 rows of one segment and one slot's share of its keys, 64 keys at a time: scores
// to shared memory, one running maximum and sum per row, o in registers.
// =========================================================================================
constexpr int SA_Q = 16, SA_K = 64;

template <typename T>
__global__ void __launch_bounds__(256) shared_simt_kernel(SharedArgs a, int sh_items) {
    pdl_wait();
    pdl_trigger();                // the combine may begin: all before this kernel is done
    __shared__ float qs[SA_Q][128];
    __shared__ float kvs[SA_K][129];
    __shared__ float ps[SA_Q][SA_K];
    __shared__ float row_m[SA_Q], row_l[SA_Q], row_scale[SA_Q];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int dh = a.dh, grp = a.H / a.G;
    int item = blockIdx.x;
    const bool sh = item < sh_items;
    if (!sh) item -= sh_items;
    const int slots = sh ? a.sh_slots : a.own_slots, rows = sh ? a.sh_rows : a.own_rows;
    const int groups = (rows + SA_Q - 1) / SA_Q;
    const int slot = item % slots, rg = (item / slots) % groups, seg = item / slots / groups;
    const int g = sh ? seg : seg % a.G, b = sh ? 0 : seg / a.G;
    const int r0 = rg * SA_Q;
    const int n = sh ? a.P : own_rows_of(a, b, rg == 0 && slot == 0 && tid == 0);
    const int k_lo = (int)((int64_t)n * slot / slots), k_hi = (int)((int64_t)n * (slot + 1) / slots);
    for (int e = tid; e < SA_Q * dh; e += 256) {
        const int r = r0 + e / dh, c = e % dh;
        float v = 0.f;
        if (r < rows) {
            const int64_t m = sh ? r / grp : (int64_t)b * a.C * a.T + r / grp;
            v = load_q<T>(a, m * a.q_ld + (int64_t)(g * grp + r % grp) * dh + c) * a.scale;
        }
        qs[e / dh][c] = v;
    }
    if (tid < SA_Q) { row_m[tid] = -INFINITY; row_l[tid] = 0.f; }
    const int orow = tid / 16, ocol = tid % 16;
    float o[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) o[u] = 0.f;
    const int64_t ld = sh ? a.p_row : a.o_row;
    const T* kbase = sh ? (const T*)a.kp + g * a.p_head : (const T*)a.ko + b * a.o_seq + g * a.o_head;
    const T* vbase = sh ? (const T*)a.vp + g * a.p_head : (const T*)a.vo + b * a.o_seq + g * a.o_head;
    __syncthreads();
    for (int t0 = k_lo; t0 < k_hi; t0 += SA_K) {
        const int nk = min(SA_K, k_hi - t0);
        for (int e = tid; e < SA_K * dh; e += 256) {
            const int r = e / dh, c = e % dh;
            kvs[r][c] = (r < nk) ? to_f32(kbase[(int64_t)(t0 + r) * ld + c]) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < SA_K / 16; ++u) {   // thread -> row tid / 16, keys tid % 16 + 16 u
            const int j = ocol + 16 * u;
            float acc = 0.f;
            for (int c = 0; c < dh; ++c) acc = fmaf(qs[orow][c], kvs[j][c], acc);
            ps[orow][j] = (j < nk) ? acc : -INFINITY;
        }
        __syncthreads();
#pragma unroll
        for (int rr = 0; rr < 2; ++rr) {        // warp w keeps rows 2w, 2w + 1
            const int r = warp * 2 + rr;
            const float x0 = ps[r][lane], x1 = ps[r][lane + 32];
            const float m_old = row_m[r];
            const float m_new = fmaxf(m_old, warp_max(fmaxf(x0, x1)));
            const float base = m_new == -INFINITY ? 0.f : m_new;   // a row of -inf scores keeps weight 0
            const float p0 = exp_of<T>(x0 - base), p1 = exp_of<T>(x1 - base);
            const float tsum = warp_sum(p0 + p1);
            ps[r][lane] = p0;
            ps[r][lane + 32] = p1;
            __syncwarp();
            if (lane == 0) {
                const float sc = exp_of<T>(m_old - base);
                row_scale[r] = sc;
                row_l[r] = row_l[r] * sc + tsum;
                row_m[r] = m_new;
            }
        }
        for (int e = tid; e < SA_K * dh; e += 256) {
            const int r = e / dh, c = e % dh;
            kvs[r][c] = (r < nk) ? to_f32(vbase[(int64_t)(t0 + r) * ld + c]) : 0.f;
        }
        __syncthreads();
        const float sc = row_scale[orow];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int c = ocol + 16 * u;
            if (c < dh) {
                float acc = o[u] * sc;
                for (int j = 0; j < nk; ++j) acc = fmaf(ps[orow][j], kvs[j][c], acc);
                o[u] = acc;
            }
        }
        __syncthreads();
    }
    const int r = r0 + orow;
    if (r < rows) {
        const int64_t at = (int64_t)seg * slots + slot;
        float* dst = (sh ? a.sh_o : a.own_o) + at * rows4(rows) * dh + r * 4;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int c = ocol + 16 * u;
            if (c < dh) dst[(int64_t)(c >> 2) * rows4(rows) * 4 + (c & 3)] = o[u];
        }
        if (ocol == 0) (sh ? a.sh_ml : a.own_ml)[at * rows + r] = make_float2(row_m[orow], row_l[orow]);
    }
}

// =========================================================================================
// Partials on the tensor cores (bf16, head width 64 or 128).
//
// Work: the 128-key tiles of every segment (a K/V head of the prefix with up to 256 query rows, or
// of one sequence's own rows) laid end to end, a segment's first tile behind ST_OVER tiles' worth of
// its own cost; workers take equal runs of that axis, so ragged lengths balance on the device. A
// run may cross segments; each piece of a segment leaves its own partials.
//
// A CTA has two lanes, each with its own score, weight and output columns in tensor memory, four
// softmax warps and a thread that issues its products. In segments of more than 128 rows the CTA is
// the worker: its lanes are two row tiles, and each K/V tile that TMA brings serves both. Otherwise
// each lane is a worker of its own, with half of the ring. Where the prefix is of the one kind and
// the own rows of the other, the CTAs are divided by cost.
//   S[q][key] = Q K^T (fp32, 128 columns) -> registers, one thread a row: running maximum, exp2,
//   sum -> bf16 weights back over the first half of S's columns -> O += P V with P read from
//   tensor memory, V MN-major from shared memory.
// Two row lanes take turns at the softmax: left alone they fall into step, both in it and then both
// waiting for the tensor core (155 us instead of 131 behind 32768 rows of 32 heads with 208 queries).
// The weights enter P V as bf16, the type that the products with V want: off by 2^-8 at most each,
// of both signs, while their sum l stays fp32. Against 64 bits outputs are 2.3e-3 off where the
// rounding of the output alone is 1.7e-3 (root mean square, relative); lse is not touched by it.
// The running maximum moves only when it grows by more than 2^8, as few rescales of O as that.
// A tile that the keys end in takes only the 16-key steps that hold keys, the rows behind them in
// the last step cleared in shared memory (they may hold anything, NaN included).
//
// Tensor memory, columns: S/P of lane 0 and 1 at 0 and 128, O at 256 and 384.
// Warps 0-3 and 4-7: the lanes' softmax and epilogue; 8 and 10: TMA; 9 and 11: products. Issuing
// eight products takes as long as they run (512 cycles), the waits and commits between two groups
// about 1600 more: one thread for both lanes left the tensor core idle half of the time.
// =========================================================================================
constexpr int ST_OVER = 1;
constexpr int ST_KEYS = 128;
constexpr int ST_THREADS = 384;
constexpr float ST_RESCALE_LOG2 = 8.f;

__device__ __forceinline__ uint32_t st_pack(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// 16 bytes, or as many zeros
__device__ __forceinline__ void st_cp_async16(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

__device__ __forceinline__ uint64_t st_pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void st_split(uint64_t v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t st_fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t st_add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ float st_max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// A worker's share of a segment: tiles t0 .. t0 + n - 1 of its nt, over `keys` keys; start: where
// the segment lies on the axis; seg numbers the prefix's segments or the own rows' ones.
struct Piece {
    int sh, b, g, rt, t0, n, nt, keys, seg, start;
};

template <int DH, int NST>
__global__ void __launch_bounds__(ST_THREADS, 1)
shared_tc_kernel(const __grid_constant__ CUtensorMap tmKP, const __grid_constant__ CUtensorMap tmVP,
                 const __grid_constant__ CUtensorMap tmKO, const __grid_constant__ CUtensorMap tmVO, SharedArgs a) {
    constexpr int HALVES = DH / 64;
    constexpr int HALF = ST_KEYS * 128;          // 64 columns of a tile
    constexpr int TILE = HALF * HALVES;
    constexpr uint32_t O_COL = 256;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint32_t tmem_slot[1];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    uint8_t* sQ = smem;                                        // [2 lanes][halves][128 rows][128 B]
    uint8_t* ring = sQ + 2 * TILE;                             // [NST]
    uint64_t* full = reinterpret_cast<uint64_t*>(ring + (size_t)NST * TILE);   // [NST]
    uint64_t* empty = full + NST;                              // [NST]
    uint64_t* s_full = empty + NST;                            // [2] scores of a tile in tensor memory
    uint64_t* p_full = s_full + 2;                             // [2] weights of a tile there
    uint64_t* pv_done = p_full + 2;                            // [2] P V of a tile complete
    uint64_t* q_ready = pv_done + 2;                           // [2] Q of a piece staged
    uint64_t* turn = q_ready + 2;                              // [2] the other lane's softmax is through
    uint64_t* drain = turn + 2;                                // [2]
    int* pre = reinterpret_cast<int*>(drain + 2);              // [B + 1] cost of one head's own rows before b
    int* len = pre + a.B + 1;                                  // [B]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    pdl_wait();
    pdl_trigger();                // the combine may begin: all before this kernel is done
    // not before the wait: a predecessor's CTA on this SM may have yet to allocate
    if (warp == 8) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    for (int b = tid; b < a.B; b += ST_THREADS) len[b] = own_rows_of(a, b, blockIdx.x == 0);
    __syncthreads();
    if (warp == 0) {
        int run = 0;
        for (int b0 = 0; b0 < a.B; b0 += 32) {
            const int b = b0 + lane;
            int x = b < a.B && len[b] > 0 ? (len[b] + ST_KEYS - 1) / ST_KEYS + ST_OVER : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            if (b < a.B) pre[b + 1] = run + x;
            run += __shfl_sync(0xffffffffu, x, 31);
        }
        if (lane == 0) pre[0] = 0;
    }
    __syncthreads();
    // ---- this CTA's axis: the prefix's tiles and then the own ones, or one of the two
    const int ntp = (a.P + ST_KEYS - 1) / ST_KEYS, per_b = a.G * a.own_tiles;
    const int sh_cost = ntp ? a.G * a.sh_tiles * (ntp + ST_OVER) : 0, own_cost = per_b * pre[a.B];
    const int grid = gridDim.x;
    const bool split = a.sh_pair != a.own_pair && sh_cost > 0 && own_cost > 0;
    // a tile takes a pair of lanes 1.76 us (measured with 208 rows), a lane of its own 2.3, its CTA half of that
    // (in fp32, the same for every CTA)
    const float sh_ctas = (float)(2 + a.sh_pair) * (float)sh_cost, own_ctas = (float)(2 + a.own_pair) * (float)own_cost;
    const int n_sh = split ? min(grid - 1, max(1, (int)((float)grid * __fdividef(sh_ctas, sh_ctas + own_ctas) + 0.5f))) : grid;
    const bool on_sh = split ? (int)blockIdx.x < n_sh : sh_cost > 0;      // axis starts with the prefix
    const bool rows2 = (on_sh ? a.sh_pair : a.own_pair) != 0;             // lanes are two row tiles
    auto run_of = [&](int cost, int ctas, int pair) { return max(1, (cost + ctas * (2 - pair) - 1) / (ctas * (2 - pair))); };
    const int sh_run = run_of(split ? sh_cost : sh_cost + own_cost, n_sh, sh_cost > 0 ? a.sh_pair : a.own_pair);
    const int own_run = split ? run_of(own_cost, grid - n_sh, a.own_pair) : sh_run;
    const int own_at = split ? 0 : sh_cost;                               // where the own tiles start
    const int total = split ? (on_sh ? sh_cost : own_cost) : sh_cost + own_cost;
    const int W = on_sh ? sh_run : own_run;
    if (blockIdx.x == 0) {
        for (int b = tid; b <= a.B; b += ST_THREADS) a.plan[3 + b] = pre[b];
        if (tid == 0) {
            a.plan[0] = sh_run;
            a.plan[1] = own_run;
            a.plan[2] = own_at;
        }
    }
    if (tid == 0) {
        for (int s = 0; s < NST; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], rows2 ? 2 : 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 4);
            mbar_init(&pv_done[i], 1);
            mbar_init(&q_ready[i], 4);
            mbar_init(&turn[i], 4);
            mbar_init(&drain[i], 1);
        }
        fence_barrier_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    // Lane L's run of the axis and slots of the ring
    const int L = warp < 8 ? warp >> 2 : (warp < 10 ? 0 : 1);
    const int cta = (int)blockIdx.x - (split && !on_sh ? n_sh : 0), worker = rows2 ? cta : 2 * cta + L;
    const int lo = min(total, W * worker), hi = min(lo + W, total);
    const int slot0 = rows2 || L == 0 ? 0 : NST / 2, nslots = rows2 ? NST : NST / 2;
    // the run's first piece, and the one behind p; n = 0: none
    auto first_piece = [&]() -> Piece {
        Piece p;
        p.n = 0;
        if (lo >= hi) return p;
        if (on_sh && lo < sh_cost) {
            p.sh = 1;
            p.b = 0;
            p.seg = lo / (ntp + ST_OVER);
            p.g = p.seg / a.sh_tiles;
            p.rt = p.seg - p.g * a.sh_tiles;
            p.start = p.seg * (ntp + ST_OVER);
            p.nt = ntp;
            p.keys = a.P;
        } else {
            const int q = lo - own_at;
            int b0 = 0, b1 = a.B - 1;             // the last b with per_b * pre[b] <= q
            while (b0 < b1) {
                const int mid = (b0 + b1 + 1) >> 1;
                if (per_b * pre[mid] <= q) b0 = mid; else b1 = mid - 1;
            }
            const int cost = pre[b0 + 1] - pre[b0], r = (q - per_b * pre[b0]) / cost;
            p.nt = cost - ST_OVER;
            p.sh = 0;
            p.b = b0;
            p.g = r / a.own_tiles;
            p.rt = r - p.g * a.own_tiles;
            p.seg = b0 * per_b + r;
            p.start = own_at + per_b * pre[b0] + r * cost;
            p.keys = len[b0];
        }
        p.t0 = max(0, lo - p.start - ST_OVER);
        p.n = max(0, min(p.nt, hi - p.start - ST_OVER) - p.t0);
        return p;
    };
    auto next_piece = [&](const Piece& c) -> Piece {
        Piece p = c;
        p.start = c.start + c.nt + ST_OVER;
        p.n = 0;
        if (p.start >= hi) return p;
        p.t0 = 0;
        ++p.seg;
        if (++p.rt == (c.sh ? a.sh_tiles : a.own_tiles)) {
            p.rt = 0;
            if (++p.g == a.G) {                   // on to the next sequence that has rows
                p.g = 0;
                p.b = c.sh ? 0 : c.b + 1;
                while (p.b < a.B - 1 && pre[p.b + 1] == pre[p.b]) ++p.b;
                p.sh = 0;
                p.seg = p.b * per_b;
                p.nt = pre[p.b + 1] - pre[p.b] - ST_OVER;
                p.keys = len[p.b];
            }
        }
        p.n = max(0, min(p.nt, hi - p.start - ST_OVER));
        return p;
    };

    // Ring steps of a worker: K0 V0 K1 V1 ... over all its pieces, in the order of use.
    // The softmax threads hold a row of scores each: they take registers that the other warps leave
    // (of the launch's 384 x 168: 256 x 208 + 128 x 80).
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        if ((warp & 1) == 0) {
            if (lane == 0 && (L == 0 || !rows2)) {
                // ---- TMA
                const uint64_t stream = policy_evict_first(), keep = policy_evict_last();
                int s = 0;
                uint32_t ph = 1, used = 0;        // parity that a free slot has; slots in use so far
                bool ok = true;
                for (Piece p = first_piece(); p.n > 0 && ok; p = next_piece(p)) {
                    const uint64_t pol = p.sh && a.sh_tiles > 1 ? keep : stream;
                    for (int j = 0; j < 2 * p.n; ++j) {
                        const int at = slot0 + s;
                        if ((used >> s & 1u) && !mbar_wait(&empty[at], ph)) { ok = false; break; }
                        used |= 1u << s;
                        const CUtensorMap* m = p.sh ? (j & 1 ? &tmVP : &tmKP) : (j & 1 ? &tmVO : &tmKO);
                        uint8_t* dst = ring + (size_t)at * TILE;
                        mbar_arrive_expect_tx(&full[at], (uint32_t)TILE);
#pragma unroll
                        for (int hf = 0; hf < HALVES; ++hf)
                            tma_load_4d(dst + hf * HALF, m, hf * 64, (p.t0 + (j >> 1)) * ST_KEYS, p.g, p.b, &full[at], pol);
                        if (++s == nslots) {
                            s = 0;
                            ph ^= 1u;
                        }
                    }
                }
                if (!ok) {
                    // loads in flight into this CTA's shared memory end before it does (bounded)
                    for (int i = 0; i < nslots; ++i)
                        if (used >> i & 1u) mbar_wait(&full[slot0 + i], i < s ? ph ^ 1u : ph);
                }
            }
            __syncwarp();
            tc_fence_before();
            __syncthreads();
            if (warp == 8) {
                tc_fence_after();
                tmem_dealloc(tmem, 512);
            }
            return;
        }
        if (lane == 0) {
            // ---- products of lane L
            constexpr uint32_t id_s = idesc_bf16_f32(128, ST_KEYS), id_o = idesc_bf16_f32_bmn(128, DH);
            const uint64_t qd = smem_desc_sw128(smem_u32(sQ + L * TILE)),
                           dk = smem_desc_sw128(smem_u32(ring + slot0 * TILE)),
                           dv = smem_desc_sw128_mn(smem_u32(ring + slot0 * TILE), HALF);
            const uint32_t s_at = tmem + (uint32_t)L * 128u, o_at = tmem + O_COL + (uint32_t)L * 128u;
            int s = 0;                            // next slot, its phase
            uint32_t ph = 0, cnt = 0, qn = 0;
            bool ok = true;
            auto take = [&]() -> int {            // wait for the next step's tile
                const int at = s;
                if (!mbar_wait(&full[slot0 + at], ph)) ok = false;
                if (++s == nslots) {
                    s = 0;
                    ph ^= 1u;
                }
                return at;
            };
            auto score = [&](int at) {            // S = Q K^T
                const uint64_t kd = dk + (uint64_t)((uint32_t)(at * TILE) >> 4);
#pragma unroll
                for (int kk = 0; kk < DH / 16; ++kk) {
                    const uint32_t off = (uint32_t)((kk >> 2) * HALF + (kk & 3) * 32) >> 4;
                    tc_mma_f16(s_at, qd + off, kd + off, id_s, kk > 0 ? 1u : 0u);
                }
            };
            for (Piece p = first_piece(); p.n > 0 && ok; p = next_piece(p)) {
                if (!mbar_wait(&q_ready[L], qn & 1u)) { ok = false; break; }
                ++qn;
                int k = take();
                if (!ok) break;
                tc_fence_after();
                score(k);
                tc_commit(&s_full[L]);
                tc_commit(&empty[slot0 + k]);
                for (int t = 0; t < p.n; ++t) {
                    // O += P V of this tile, then the next one's scores before any of the commits
                    const bool next = t + 1 < p.n;
                    const int v = take();
                    if (next) k = take();
                    if (!ok || !mbar_wait(&p_full[L], cnt & 1u)) { ok = false; break; }
                    ++cnt;
                    tc_fence_after();
                    const int nv = min(ST_KEYS, p.keys - (p.t0 + t) * ST_KEYS);
                    const uint64_t vd = dv + (uint64_t)((uint32_t)(v * TILE) >> 4);
                    if (nv > ST_KEYS - 16) {
#pragma unroll
                        for (int kk = 0; kk < ST_KEYS / 16; ++kk)
                            tc_mma_f16_ta(o_at, s_at + kk * 8u, vd + (uint64_t)((kk * 16 * 128) >> 4), id_o,
                                          (kk > 0 || t > 0) ? 1u : 0u);
                    } else {
                        for (int kk = 0; kk < (nv + 15) / 16; ++kk)
                            tc_mma_f16_ta(o_at, s_at + kk * 8u, vd + (uint64_t)((kk * 16 * 128) >> 4), id_o,
                                          (kk > 0 || t > 0) ? 1u : 0u);
                    }
                    if (next) {
                        score(k);
                        tc_commit(&s_full[L]);
                        tc_commit(&empty[slot0 + k]);
                    }
                    tc_commit(&empty[slot0 + v]);
                    tc_commit(&pv_done[L]);
                }
            }
            tc_commit(&drain[L]);                 // nothing of this thread's in tensor memory in flight
            mbar_wait(&drain[L], 0);
        }
        __syncwarp();
        tc_fence_before();
        __syncthreads();
        return;
    }
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // ---- softmax of lane L: thread = row r of the lane's tile
    const int q4 = warp & 3, r = q4 * 32 + lane;
    const uint32_t trow = tmem + ((uint32_t)(q4 * 32) << 16);
    const uint32_t s_col = (uint32_t)L * 128u, o_col = O_COL + (uint32_t)L * 128u;
    const int grp = a.H / a.G;
    const float sl = a.scale * 1.4426950408889634f;
    // where this thread's row of a piece lies: in its segment, and of the head
    auto rows_of = [&](const Piece& p, int& r_seg, int& r_all) -> bool {
        const int all_rows = p.sh ? a.B * a.C * a.T * grp : a.C * a.T * grp;
        const int seg_rows = p.sh ? a.sh_rows : a.own_rows;
        r_seg = rows2 ? L * 128 + r : r;
        r_all = p.rt * seg_rows + r_seg;
        return r_seg < seg_rows && r_all < all_rows;
    };
    // Q row -> bf16, K-major, 128-byte swizzle. bf16 rows on 16 bytes are copied asynchronously, so
    // that the next piece's come while this one's last tile is worked on; staged() ends a staging.
    auto stage = [&](const Piece& p) {
        int r_seg, r_all;
        const bool live = rows_of(p, r_seg, r_all);
        if (!__any_sync(0xffffffffu, live)) return;
        const int m_in = r_all / grp;
        const int64_t m = p.sh ? m_in : (int64_t)p.b * a.C * a.T + m_in;
        const int64_t at = m * a.q_ld + (int64_t)(p.g * grp + r_all - m_in * grp) * DH;
        uint8_t* dst = sQ + L * TILE + r * 128;
        if (a.q_bf16 && a.q_vec) {
            const bf16* src = (const bf16*)a.q + (live ? at : 0);
            const uint32_t to = smem_u32(dst);
#pragma unroll 1
            for (int hf = 0; hf < HALVES; ++hf)
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    st_cp_async16(to + hf * HALF + (uint32_t)((c ^ (r & 7)) << 4), src + hf * 64 + c * 8, live);
            return;
        }
#pragma unroll 1
        for (int e = 0; e < DH; e += 8) {
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = 0.f;
            if (live && a.q_vec) {
                const float4 x0 = *reinterpret_cast<const float4*>((const float*)a.q + at + e);
                const float4 x1 = *reinterpret_cast<const float4*>((const float*)a.q + at + e + 4);
                x[0] = x0.x; x[1] = x0.y; x[2] = x0.z; x[3] = x0.w;
                x[4] = x1.x; x[5] = x1.y; x[6] = x1.z; x[7] = x1.w;
            } else if (live) {
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = load_q<bf16>(a, at + e + j);
            }
            *reinterpret_cast<uint4*>(dst + (e >> 6) * HALF + (((e >> 3 & 7) ^ (r & 7)) << 4)) =
                make_uint4(st_pack(x[0], x[1]), st_pack(x[2], x[3]), st_pack(x[4], x[5]), st_pack(x[6], x[7]));
        }
    };
    auto staged = [&]() {
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_ready[L]);
    };
    auto wait_all = [&](uint64_t* bar, uint32_t phase) { return __all_sync(0xffffffffu, mbar_wait(bar, phase)) != 0; };
    uint32_t cnt = 0;                             // tiles so far
    bool ok = true;
    Piece p = first_piece();
    if (p.n > 0) {
        stage(p);
        staged();
    }
    while (p.n > 0) {
        const int seg_rows = p.sh ? a.sh_rows : a.own_rows;
        int r_seg, r_all;
        const bool live = rows_of(p, r_seg, r_all), work = __any_sync(0xffffffffu, live);
        const Piece nx = next_piece(p);
        float m_run = -INFINITY, l = 0.f;
        for (int t = 0; ok && t < p.n; ++t) {
            if (!wait_all(&s_full[L], cnt & 1u)) { ok = false; break; }
            if (t == p.n - 1 && nx.n > 0) stage(nx);   // the last scores are out: Q's place is free
            uint32_t x[8][16];
            if (work) {
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < 8; ++c) tmem_ld16_issue(trow + s_col + (uint32_t)(c * 16), x[c]);
                tmem_wait_ld();
            }
            const int nv = min(ST_KEYS, p.keys - (p.t0 + t) * ST_KEYS);
            // row lanes: lane 1's turn follows lane 0's of the same tile, lane 0's the one before of lane 1
            if (rows2 && (L == 1 || cnt > 0) && !wait_all(&turn[L], (cnt & 1u) ^ (uint32_t)(L ^ 1))) { ok = false; break; }
            if ((nv & 15) && (!rows2 || L == 0)) {
                // clear the V rows behind the last key, up to the end of its 16-key step (for both of
                // two row lanes: lane 1's weights come after this turn)
                const uint32_t st = 2 * cnt + 1;
                const int at = slot0 + (int)(st % (uint32_t)nslots);
                if (!wait_all(&full[at], st / (uint32_t)nslots & 1u)) { ok = false; break; }
                const int rows = 16 - (nv & 15);
                for (int e = r; e < rows * 8 * HALVES; e += 128) {
                    const int hf = e / (rows * 8), k = nv + (e - hf * rows * 8) / 8;
                    *reinterpret_cast<uint4*>(ring + (size_t)at * TILE + hf * HALF + k * 128 + e % 8 * 16) =
                        make_uint4(0u, 0u, 0u, 0u);
                }
                fence_proxy_async_smem();
            }
            if (work) {
                if (nv < ST_KEYS) {               // keys behind the last one: no weight
#pragma unroll
                    for (int c = 0; c < 8; ++c)
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (c * 16 + j >= nv) x[c][j] = 0xff800000u;
                }
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < 8; ++c)
#pragma unroll
                    for (int j = 0; j < 16; j += 2)
                        mx[(j >> 1) & 3] = st_max3(mx[(j >> 1) & 3], __uint_as_float(x[c][j]), __uint_as_float(x[c][j + 1]));
                const float m_new = fmaxf(m_run, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl);
                const bool move = m_new > m_run + ST_RESCALE_LOG2 || (m_run == -INFINITY && m_new > -INFINITY);
                if (t > 0 && __any_sync(0xffffffffu, move)) {
                    // rescale the rows of O once P V of the previous tile is in it
                    if (!wait_all(&pv_done[L], (cnt - 1) & 1u)) { ok = false; break; }
                    tc_fence_after();
                    const float f = move ? ex2_approx_ftz(m_run - m_new) : 1.f;
#pragma unroll
                    for (int c = 0; c < DH / 16; ++c) {
                        uint32_t o[16];
                        tmem_ld16_issue(trow + o_col + (uint32_t)(c * 16), o);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                        tmem_st16(trow + o_col + (uint32_t)(c * 16), o);
                    }
                    l *= f;
                }
                if (move) m_run = m_new;
                const float mb = m_run == -INFINITY ? 0.f : m_run;   // only -inf scores so far: weights 0
                const uint64_t sl2 = st_pair(sl, sl), mb2 = st_pair(-mb, -mb);
                uint64_t sum0 = 0, sum1 = 0;      // two fp32 each
#pragma unroll
                for (int c = 0; c < 4; ++c) {     // 32 keys: 16 columns of weights
                    uint32_t w[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const uint32_t* at = &x[2 * c + j / 8][(2 * j) & 15];
                        float e0, e1;
                        st_split(st_fma2(st_pair(__uint_as_float(at[0]), __uint_as_float(at[1])), sl2, mb2), e0, e1);
                        e0 = ex2_approx_ftz(e0);
                        e1 = ex2_approx_ftz(e1);
                        if (j & 1) sum1 = st_add2(sum1, st_pair(e0, e1));
                        else sum0 = st_add2(sum0, st_pair(e0, e1));
                        w[j] = st_pack(e0, e1);
                    }
                    tmem_st16(trow + s_col + (uint32_t)(c * 16), w);
                }
                float l0, l1;
                st_split(st_add2(sum0, sum1), l0, l1);
                l += l0 + l1;
            }
            __syncwarp();
            if (rows2 && lane == 0) mbar_arrive(&turn[L ^ 1]);
            if (work) {
                tmem_wait_st();
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[L]);
            ++cnt;
        }
        if (ok && nx.n > 0) staged();             // the next scores need not wait for the rest
        // ---- the piece's partials: o, then (m, l). Once a wait has run out, this piece's and those of the
        // worker's later ones are void: l = NaN makes the rows' outputs NaN, whether or not the caller
        // looks at the flag (a row of NaN scores leaves the same pair).
        if (ok && !wait_all(&pv_done[L], (cnt - 1) & 1u)) ok = false;
        tc_fence_after();
        if (!ok && lane == 0 && a.flags) atomicOr(a.flags, (uint32_t)EVS_FLAG_TIMEOUT);
        if (work) {
            const int64_t at = worker + p.seg;
            const int ld = rows4(seg_rows) * 4;
            float* dst = (p.sh ? a.sh_o : a.own_o) + at * rows4(seg_rows) * DH + r_seg * 4;
            if (ok) {
#pragma unroll
                for (int c = 0; c < DH / 32; ++c) {
                    uint32_t o[2][16];
                    tmem_ld16_issue(trow + o_col + (uint32_t)(c * 32), o[0]);
                    tmem_ld16_issue(trow + o_col + (uint32_t)(c * 32 + 16), o[1]);
                    tmem_wait_ld();
                    if (live) {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            *reinterpret_cast<uint4*>(dst + (c * 8 + j) * ld) =
                                make_uint4(o[j >> 2][4 * (j & 3)], o[j >> 2][4 * (j & 3) + 1], o[j >> 2][4 * (j & 3) + 2],
                                           o[j >> 2][4 * (j & 3) + 3]);
                    }
                }
            }
            if (live)
                (p.sh ? a.sh_ml : a.own_ml)[at * seg_rows + r_seg] =
                    ok ? make_float2(m_run * 0.6931471805599453f, l) : make_float2(-INFINITY, __int_as_float(0x7fc00000));
        }
        tc_fence_before();                        // these reads precede the next piece's products
        p = nx;
    }
    tc_fence_before();
    __syncthreads();
}

// =========================================================================================
// Combine. A CTA takes 512 / dh consecutive (candidate, position, head) rows of a sequence and K/V
// head, 128 threads for them, four columns of one row each, and up to four such groups, which deal
// the row's partials and the chunks of its block rows among them. First the block rows j <= i
// (scores by a dot product over the row's threads, 16 keys at a time), which need nothing of the
// partial kernel and are done while that runs out; then the partials; then the groups' sums.
// =========================================================================================
constexpr int SC_GROUPS = 4;
template <typename T, int DH>
__global__ void __launch_bounds__(128 * SC_GROUPS) shared_combine_kernel(SharedArgs a) {
    constexpr int RW = 512 / DH, KB = 16;
    __shared__ float part[SC_GROUPS][4][KB][RW];  // a warp's share of the dot products
    __shared__ float4 sum_o[SC_GROUPS - 1][128];
    __shared__ float2 sum_ml[SC_GROUPS - 1][128];
    // The partial kernel starts its dependents when all before it is done, so the inputs are there (in
    // L2); without one, wait for that.
    if (!a.partials) {
        pdl_wait();
        pdl_trigger();
    }
    const int tid = threadIdx.x & 127, part_of = threadIdx.x >> 7, parts = blockDim.x >> 7, warp = tid >> 5;
    const int grp = a.H / a.G, rows = a.C * a.T * grp;
    const int b = blockIdx.z, g = blockIdx.y, row = tid % RW, c4 = tid / RW;
    const int r_own = blockIdx.x * RW + row;
    const bool live = r_own < rows;
    const int ci = (live ? r_own : rows - 1) / grp, hg = (live ? r_own : rows - 1) - ci * grp;   // (c, i), head
    const int c = ci / a.T, i = ci - c * a.T;
    const int64_t m = (int64_t)b * a.C * a.T + ci;
    const int h = g * grp + hg;
    float M = -INFINITY, L = 0.f;
    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
    auto rebase = [&](float mb) {
        if (mb > M) {
            const float f = M == -INFINITY ? 0.f : exp_of<T>(M - mb);
            L *= f;
            O.x *= f; O.y *= f; O.z *= f; O.w *= f;
            M = mb;
        }
    };
    auto add = [&](float w, float4 v) {
        O.x = fmaf(w, v.x, O.x);
        O.y = fmaf(w, v.y, O.y);
        O.z = fmaf(w, v.z, O.z);
        O.w = fmaf(w, v.w, O.w);
    };
    const int own = own_rows_of(a, b, false);
    // block rows j <= i: of this candidate, or own rows own + j when the block is in the cache
    const T *kb, *vb;
    int64_t ld;
    int last = i;
    if (a.kb) {
        const int64_t at = ((int64_t)b * a.C + c) * a.b_cand + g * a.b_head + c4 * 4;
        kb = (const T*)a.kb + at;
        vb = (const T*)a.vb + at;
        ld = a.b_row;
    } else {
        const int64_t at = b * a.o_seq + g * a.o_head + own * a.o_row + c4 * 4;
        kb = (const T*)a.ko + at;
        vb = (const T*)a.vo + at;
        ld = a.o_row;
        if (own + i >= a.own_max) {                // rows past the capacity do not exist
            last = a.own_max - 1 - own;
            if (a.flags && live && c4 == 0 && part_of == 0) atomicOr(a.flags, (uint32_t)EVS_FLAG_KV_OVERFLOW);
        }
    }
    auto load4 = [&](const T* p) -> float4 {
        if (a.b_vec) {
            if constexpr (sizeof(T) == 4) {
                return __ldcg(reinterpret_cast<const float4*>(p));
            } else {
                const uint2 u = __ldcg(reinterpret_cast<const uint2*>(p));
                const float2 lo = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.x));
                const float2 hi = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.y));
                return make_float4(lo.x, lo.y, hi.x, hi.y);
            }
        }
        return make_float4(load_l2(p), load_l2(p + 1), load_l2(p + 2), load_l2(p + 3));
    };
    float q[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int64_t at = m * a.q_ld + (int64_t)h * DH + c4 * 4 + u;
        q[u] = (a.q_bf16 ? load_l2((const bf16*)a.q + at) : as_product<T>(load_l2((const float*)a.q + at))) * a.scale;
    }
    for (int j1 = 0; j1 < a.T; j1 += KB * parts) {  // the same count for every thread of the CTA
        const int j0 = j1 + part_of * KB, n = min(KB, a.T - j0);
        float4 v[KB];
        if (j1 > 0) __syncthreads();
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            if (j >= n) break;
            const bool on = live && j0 + j <= last;
            float4 k = make_float4(0.f, 0.f, 0.f, 0.f);
            v[j] = k;
            if (on) {
                k = load4(kb + (j0 + j) * ld);
                v[j] = load4(vb + (j0 + j) * ld);
            }
            float s = fmaf(q[0], k.x, fmaf(q[1], k.y, fmaf(q[2], k.z, q[3] * k.w)));
#pragma unroll
            for (int o = RW; o < 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            if ((tid & 31) < RW) part[part_of][warp][j][row] = s;
        }
        __syncthreads();
        float s[KB], mb = -INFINITY;
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            s[j] = -INFINITY;
            if (j < n && j0 + j <= last)
                s[j] = (part[part_of][0][j][row] + part[part_of][1][j][row]) + (part[part_of][2][j][row] + part[part_of][3][j][row]);
            mb = fmaxf(mb, s[j]);
        }
        rebase(mb);
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            if (j >= n || s[j] == -INFINITY) continue;
            const float w = exp_of<T>(s[j] - M);
            L += w;
            add(w, v[j]);
        }
    }
    if (a.partials) {
        pdl_wait();
        pdl_trigger();
        // The row's partials: those of the prefix, dealt among the groups but the last, and those of
        // the own rows, the last group's
        constexpr int PB = 8;                      // in flight
        const int dealt = max(1, parts - 1);
#pragma unroll 1
        for (int kind = part_of < dealt ? 0 : 1; kind < (part_of == parts - 1 ? 2 : 1); ++kind) {
            const float* o_at;
            const float2* ml_at;
            int rows_seg, s = 0, step = 1, used = 0;
            int64_t first;                         // partial
            // the runs that a segment's nt tiles from position at on meet
            auto runs = [&](int at, int nt, int W) {
                first = at / W;
                used = (at + nt - 1) / W - at / W + 1;
            };
            if (kind == 0) {
                if (!live || a.P == 0) continue;
                const int r = (int)(m * grp + hg), t = r / a.sh_rows, in = r - t * a.sh_rows;
                const int seg = g * a.sh_tiles + t, nt = (a.P + 127) / 128;
                rows_seg = a.sh_rows;
                s = part_of;
                step = dealt;
                if (a.tensor) {
                    runs(seg * (nt + ST_OVER) + ST_OVER, nt, a.plan[0]);
                    first += seg;
                } else {
                    first = (int64_t)seg * a.sh_slots;
                    used = a.sh_slots;
                }
                ml_at = a.sh_ml + first * rows_seg + in;
                o_at = a.sh_o + (first * DH + c4 * 4) * rows4(rows_seg) + in * 4;
            } else {
                if (!live || own == 0) continue;
                const int t = r_own / a.own_rows, in = r_own - t * a.own_rows, in_b = g * a.own_tiles + t;
                const int per_b = a.G * a.own_tiles;
                const int64_t seg = (int64_t)b * per_b + in_b;
                rows_seg = a.own_rows;
                if (a.tensor) {
                    const int before = a.plan[3 + b], cost = a.plan[4 + b] - before;
                    runs(a.plan[2] + per_b * before + in_b * cost + ST_OVER, cost - ST_OVER, a.plan[1]);
                    first += seg;
                } else {
                    first = seg * a.own_slots;
                    used = a.own_slots;
                }
                ml_at = a.own_ml + first * rows_seg + in;
                o_at = a.own_o + (first * DH + c4 * 4) * rows4(rows_seg) + in * 4;
            }
            const int64_t ml_step = (int64_t)step * rows_seg, o_step = (int64_t)step * DH * rows4(rows_seg);
            ml_at += (int64_t)s * rows_seg;
            o_at += (int64_t)s * DH * rows4(rows_seg);
#pragma unroll 1
            for (; s < used; s += PB * step) {
                float2 ml[PB];
                float4 os[PB];
#pragma unroll
                for (int j = 0; j < PB; ++j) {
                    ml[j] = make_float2(-INFINITY, 0.f);
                    os[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (s + j * step < used) {
                        ml[j] = *ml_at;
                        os[j] = *reinterpret_cast<const float4*>(o_at);
                    }
                    ml_at += ml_step;
                    o_at += o_step;
                }
                float mb = -INFINITY;
#pragma unroll
                for (int j = 0; j < PB; ++j) mb = fmaxf(mb, ml[j].x);
                rebase(mb);
#pragma unroll
                for (int j = 0; j < PB; ++j) {
                    // an empty partial leaves its o unwritten (one of NaN scores, or void, has l = NaN)
                    if (ml[j].x == -INFINITY && ml[j].y == 0.f) continue;
                    const float w = exp_of<T>(ml[j].x - M);
                    L = fmaf(ml[j].y, w, L);
                    add(w, os[j]);
                }
            }
        }
    }
    if (parts > 1) {
        if (part_of > 0) {
            sum_o[part_of - 1][tid] = O;
            sum_ml[part_of - 1][tid] = make_float2(M, L);
        }
        __syncthreads();
        if (part_of > 0) return;
        for (int p = 0; p < parts - 1; ++p) {
            const float2 ml = sum_ml[p][tid];
            if (ml.x == -INFINITY && ml.y == 0.f) continue;
            rebase(ml.x);
            const float w = exp_of<T>(ml.x - M);
            L = fmaf(ml.y, w, L);
            add(w, sum_o[p][tid]);
        }
    }
    if (!live) return;
    // no key with any weight: zero output, lse -inf
    const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
    T* dst = (T*)a.o + m * a.o_ld + (int64_t)h * DH + c4 * 4;
    dst[0] = from_f32<T>(O.x * inv);
    dst[1] = from_f32<T>(O.y * inv);
    dst[2] = from_f32<T>(O.z * inv);
    dst[3] = from_f32<T>(O.w * inv);
    if (a.lse && c4 == 0) a.lse[m * a.H + h] = L == 0.f ? -INFINITY : M + logf(L);
}

// ---- host side ----------------------------------------------------------------------------------
size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

bool valid_shape(const evs_shared_attn_args* c) {
    if (!c || c->batch < 0 || c->n_cand < 1 || c->block < 1 || c->heads < 1 || c->kv_heads < 1) return false;
    if (c->batch > 1024 || c->n_cand > 64 || c->block > 128 || c->heads > 1024 || c->heads % c->kv_heads) return false;
    if ((long long)c->batch * c->n_cand * c->block * c->heads > (1 << 24)) return false;
    if (!(c->head_dim == 16 || c->head_dim == 32 || c->head_dim == 64 || c->head_dim == 128)) return false;
    if (c->prefix < 0 || c->own_max < 0 || c->prefix > (1 << 30) || c->own_max > (1 << 30)) return false;
    if (c->dtype != EVS_DTYPE_F32 && c->dtype != EVS_DTYPE_BF16) return false;
    if (c->q_dtype != EVS_DTYPE_F32 && c->q_dtype != EVS_DTYPE_BF16) return false;
    return true;
}

// Slots and row tiles of the CUDA-core path: enough CTAs for about four waves of the SMs.
void plan_simt(const evs_shared_attn_args& c, SharedArgs& a) {
    const int grp = c.heads / c.kv_heads;
    a.sh_rows = c.batch * c.n_cand * c.block * grp;
    a.own_rows = c.n_cand * c.block * grp;
    a.sh_tiles = a.own_tiles = 1;
    const long long sh = (long long)c.kv_heads * ((a.sh_rows + SA_Q - 1) / SA_Q);
    const long long own = (long long)c.batch * c.kv_heads * ((a.own_rows + SA_Q - 1) / SA_Q);
    auto slots = [](long long items, int keys) {
        long long s = (4 * 152 + items - 1) / items;
        s = s < (keys + SA_K - 1) / SA_K ? s : (keys + SA_K - 1) / SA_K;
        return (int)(s < 1 ? 1 : s);
    };
    a.sh_slots = c.prefix > 0 ? slots(sh, c.prefix) : 0;
    a.own_slots = c.own_max > 0 ? slots(own, c.own_max) : 0;
}

// The tensor-core path: bf16 with heads of 64 or 128, rows that tensor maps describe.
bool map_ok(const void* p, long long row, long long head, long long seq, bool heads, bool seqs) {
    return (uintptr_t)p % 16 == 0 && row % 8 == 0 && row < (1LL << 38) &&
           (!heads || (head % 8 == 0 && head > 0 && head < (1LL << 38))) &&
           (!seqs || (seq % 8 == 0 && seq > 0 && seq < (1LL << 38)));
}
bool tensor_ok(const evs_shared_attn_args& c) {
    if (c.dtype != EVS_DTYPE_BF16 || (c.head_dim != 64 && c.head_dim != 128)) return false;
    if (c.prefix == 0 && c.own_max == 0) return false;
    if (c.prefix > 0 && !(map_ok(c.k_prefix, c.prefix_row, c.prefix_head, 0, c.kv_heads > 1, false) &&
                          map_ok(c.v_prefix, c.prefix_row, c.prefix_head, 0, c.kv_heads > 1, false)))
        return false;
    if (c.own_max > 0 && !(map_ok(c.k_own, c.own_row, c.own_head, c.own_seq, c.kv_heads > 1, c.batch > 1) &&
                           map_ok(c.v_own, c.own_row, c.own_head, c.own_seq, c.kv_heads > 1, c.batch > 1)))
        return false;
    return true;
}

// Tiles, slots and grid. A prefix segment of nt tiles meets at most (nt - 1) / W + 2 runs, and a run is
// at least the segments' cost over the workers. false: sizes past the kernel's 32-bit positions.
bool plan_tensor(const evs_shared_attn_args& c, SharedArgs& a, int& grid) {
    const int grp = c.heads / c.kv_heads;
    const long long sh = (long long)c.batch * c.n_cand * c.block * grp, own = (long long)c.n_cand * c.block * grp;
    const long long ntp = (c.prefix + ST_KEYS - 1) / ST_KEYS, nto = (c.own_max + ST_KEYS - 1) / ST_KEYS;
    a.sh_pair = sh > 128;
    a.own_pair = own > 128;
    a.sh_rows = (int)(sh < 256 ? sh : 256);
    a.own_rows = (int)(own < 256 ? own : 256);
    a.sh_tiles = (int)((sh + 255) / 256);
    a.own_tiles = (int)((own + 255) / 256);
    const long long shs = c.kv_heads * (long long)a.sh_tiles, owns = c.kv_heads * (long long)a.own_tiles;
    const long long tiles = shs * ntp + c.batch * owns * nto;
    if (tiles + shs * ST_OVER + c.batch * owns * ST_OVER >= (1LL << 30)) return false;
    grid = (int)(tiles < kAttnGrid ? tiles : kAttnGrid);
    const long long s = ntp ? ntp * grid * (2 - a.sh_pair) / (shs * (ntp + ST_OVER)) + 2 : 0;
    a.sh_slots = (int)(s < ntp ? s : ntp);
    a.tensor = 1;
    return true;
}

// Lays the partials out from base (or sizes them).
size_t carve_partials(const evs_shared_attn_args& c, SharedArgs& a, int grid_tc, char* base) {
    size_t off = 0;
    auto take = [&](size_t bytes) {
        char* p = base ? base + off : nullptr;
        off = round256(off + bytes);
        return p;
    };
    size_t sh = (size_t)c.kv_heads * a.sh_tiles, own = (size_t)c.batch * c.kv_heads * a.own_tiles;   // segments
    sh = c.prefix == 0 ? 0 : a.tensor ? sh + (size_t)grid_tc * (2 - a.sh_pair) : sh * a.sh_slots;
    own = c.own_max == 0 ? 0 : a.tensor ? own + (size_t)grid_tc * (2 - a.own_pair) : own * a.own_slots;
    a.sh_o = (float*)take(sh * rows4(a.sh_rows) * c.head_dim * 4);
    a.own_o = (float*)take(own * rows4(a.own_rows) * c.head_dim * 4);
    a.sh_ml = (float2*)take(sh * a.sh_rows * 8);
    a.own_ml = (float2*)take(own * a.own_rows * 8);
    a.plan = (int*)take(((size_t)c.batch + 4) * 4);
    return off;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
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

// [seqs][heads][rows][dh] bf16, boxes of 128 rows x 64 columns. The stride of a dimension of one
// is not used; it only has to be a legal one.
bool make_rows_map(CUtensorMap* m, const void* base, int dh, int rows, int heads, int seqs, int64_t row, int64_t head,
                   int64_t seq) {
    const auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)dh, (cuuint64_t)rows, (cuuint64_t)heads, (cuuint64_t)seqs};
    const cuuint64_t r2 = rows > 1 ? (cuuint64_t)row * 2 : (cuuint64_t)dh * 2;
    const cuuint64_t h2 = heads > 1 ? (cuuint64_t)head * 2 : r2, s2 = seqs > 1 ? (cuuint64_t)seq * 2 : h2;
    const cuuint64_t strides[3] = {r2, h2, s2};
    const cuuint32_t box[4] = {64, ST_KEYS, 1, 1}, estr[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// alignment, two Q tiles, the barriers, lengths and their running sums, the ring
constexpr int tc_smem(int dh, int stages, int batch) {
    return 1024 + (2 + stages) * ST_KEYS * dh * 2 + (2 * stages + 12) * 8 + (2 * batch + 1) * 4 + 16;
}

constexpr int TC_SMEM_MAX = 227 * 1024 - 256;   // the kernel's own variables beside it
template <int DH, int NST>
cudaError_t launch_tensor(const evs_shared_attn_args& c, const SharedArgs& a, int grid, cudaStream_t stream) {
    // First: the runtime makes the device's context this thread's own, which the driver's encoding of the
    // maps does not and wants to find. The limit is that of any batch: this call's own would be lowered by
    // another thread's smaller call before the launch.
    const int smem = tc_smem(DH, NST, c.batch);
    constexpr int most = tc_smem(DH, NST, 1024) < TC_SMEM_MAX ? tc_smem(DH, NST, 1024) : TC_SMEM_MAX;
    const cudaError_t e =
        cudaFuncSetAttribute(shared_tc_kernel<DH, NST>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return e;
    CUtensorMap kp, vp, ko, vo;
    bool ok = true;
    if (c.prefix > 0)
        ok = make_rows_map(&kp, c.k_prefix, DH, c.prefix, c.kv_heads, 1, c.prefix_row, c.prefix_head, 0) &&
             make_rows_map(&vp, c.v_prefix, DH, c.prefix, c.kv_heads, 1, c.prefix_row, c.prefix_head, 0);
    if (ok && c.own_max > 0)
        ok = make_rows_map(&ko, c.k_own, DH, c.own_max, c.kv_heads, c.batch, c.own_row, c.own_head, c.own_seq) &&
             make_rows_map(&vo, c.v_own, DH, c.own_max, c.kv_heads, c.batch, c.own_row, c.own_head, c.own_seq);
    if (!ok) return cudaErrorInvalidValue;
    if (c.prefix == 0) { kp = ko; vp = vo; }
    if (c.own_max == 0) { ko = kp; vo = vp; }
    return launch_s(stream, shared_tc_kernel<DH, NST>, dim3(grid), dim3(ST_THREADS), (size_t)smem, kp, vp, ko, vo, a);
}

}  // namespace

cudaError_t launch_shared_attention(const evs_shared_attn_args& c, cudaStream_t stream) {
    SharedArgs a{};
    a.q = c.q; a.kp = c.k_prefix; a.vp = c.v_prefix; a.ko = c.k_own; a.vo = c.v_own; a.kb = c.k_block; a.vb = c.v_block;
    a.o = c.o; a.lse = c.lse; a.own_len = c.own_len; a.flags = c.flags;
    a.q_ld = c.q_ld; a.o_ld = c.o_ld; a.p_row = c.prefix_row; a.p_head = c.prefix_head;
    a.o_row = c.own_row; a.o_head = c.own_head; a.o_seq = c.own_seq;
    a.b_row = c.block_row; a.b_head = c.block_head; a.b_cand = c.block_cand;
    a.B = c.batch; a.C = c.n_cand; a.T = c.block; a.H = c.heads; a.G = c.kv_heads; a.dh = c.head_dim;
    a.P = c.prefix; a.own_max = c.own_max; a.own_skip = c.own_skip; a.q_bf16 = c.q_dtype == EVS_DTYPE_BF16;
    a.scale = c.scale != 0.f ? c.scale : 1.f / sqrtf((float)c.head_dim);
    const bool half = c.dtype == EVS_DTYPE_BF16;
    int grid_tc = 0;
    const bool tensor = tensor_ok(c) && plan_tensor(c, a, grid_tc);
    if (!tensor) plan_simt(c, a);
    const int es = half ? 2 : 4;
    const bool in_cache = !c.k_block;
    const int64_t b0 = in_cache ? c.own_row : c.block_row, b1 = in_cache ? c.own_head : c.block_head,
                  b2 = in_cache ? c.own_seq : c.block_cand;
    a.b_vec = ((uintptr_t)(in_cache ? c.k_own : c.k_block) | (uintptr_t)(in_cache ? c.v_own : c.v_block)) % (4 * es) == 0 &&
              b0 % 4 == 0 && b1 % 4 == 0 && b2 % 4 == 0;
    a.q_vec = (uintptr_t)c.q % 16 == 0 && c.q_ld * (a.q_bf16 ? 2 : 4) % 16 == 0;
    carve_partials(c, a, grid_tc, (char*)c.workspace);
    const int sh_items = c.kv_heads * a.sh_slots * ((a.sh_rows + SA_Q - 1) / SA_Q);
    const int own_items = c.batch * c.kv_heads * a.own_slots * ((a.own_rows + SA_Q - 1) / SA_Q);
    a.partials = tensor || sh_items + own_items > 0;
    cudaError_t e = cudaSuccess;
    if (tensor)
        // the ring takes what 227 KB leave: five tiles of 32 KB, four where the lengths need their place
        e = c.head_dim == 64                                 ? launch_tensor<64, 8>(c, a, grid_tc, stream)
            : tc_smem(128, 5, c.batch) <= TC_SMEM_MAX ? launch_tensor<128, 5>(c, a, grid_tc, stream)
                                                             : launch_tensor<128, 4>(c, a, grid_tc, stream);
    else if (sh_items + own_items > 0)
        e = half ? launch_s(stream, shared_simt_kernel<bf16>, dim3(sh_items + own_items), dim3(256), 0, a, sh_items)
                 : launch_s(stream, shared_simt_kernel<float>, dim3(sh_items + own_items), dim3(256), 0, a, sh_items);
    if (e != cudaSuccess) return e;
    const int rw = 512 / c.head_dim;
    const dim3 grid((c.n_cand * c.block * (c.heads / c.kv_heads) + rw - 1) / rw, c.kv_heads, c.batch);   // y and z end at 65535
    // groups: one for eight partials of a row's prefix, which it loads at once, and one for its own, as
    // many as all run at once
    const long long most = 4 * 152 / ((long long)grid.x * grid.y * grid.z);
    int groups = ((a.P > 0 ? a.sh_slots : 0) + 7) / 8 + (a.own_max > 0);
    groups = groups < most ? groups : (int)most;
    groups = groups < 1 ? 1 : groups > SC_GROUPS ? SC_GROUPS : groups;
    auto combine = [&](auto kernel) { return launch_s(stream, kernel, grid, dim3(128 * groups), 0, a); };
    switch (c.head_dim) {
        case 128: return half ? combine(shared_combine_kernel<bf16, 128>) : combine(shared_combine_kernel<float, 128>);
        case 64: return half ? combine(shared_combine_kernel<bf16, 64>) : combine(shared_combine_kernel<float, 64>);
        case 32: return half ? combine(shared_combine_kernel<bf16, 32>) : combine(shared_combine_kernel<float, 32>);
        default: return half ? combine(shared_combine_kernel<bf16, 16>) : combine(shared_combine_kernel<float, 16>);
    }
}

}  // namespace evs

extern "C" size_t evs_shared_attention_workspace(const evs_shared_attn_args* c) {
    using namespace evs;
    if (!valid_shape(c)) return 0;
    // the larger of the two paths: which one runs depends on addresses too
    SharedArgs a{}, t{};
    int grid = 0;
    plan_simt(*c, a);
    size_t n = carve_partials(*c, a, 0, nullptr);
    if (c->dtype == EVS_DTYPE_BF16 && (c->head_dim == 64 || c->head_dim == 128) && plan_tensor(*c, t, grid)) {
        const size_t m = carve_partials(*c, t, grid, nullptr);
        n = m > n ? m : n;
    }
    return n ? n : 256;
}

extern "C" evs_status evs_shared_attention(const evs_shared_attn_args* c, void* stream) {
    using namespace evs;
    if (!valid_shape(c)) return EVS_ERR_INVALID_ARG;
    if (c->batch == 0) return EVS_OK;
    const long long row = (long long)c->heads * c->head_dim;
    if (!c->q || !c->o || c->q_ld < row || c->o_ld < row) return EVS_ERR_INVALID_ARG;
    if (c->prefix > 0 && (!c->k_prefix || !c->v_prefix || c->prefix_row < c->head_dim)) return EVS_ERR_INVALID_ARG;
    if (c->own_max > 0 && (!c->k_own || !c->v_own || !c->own_len || c->own_row < c->head_dim)) return EVS_ERR_INVALID_ARG;
    if ((c->k_block == nullptr) != (c->v_block == nullptr)) return EVS_ERR_INVALID_ARG;
    if (c->k_block && c->block_row < c->head_dim) return EVS_ERR_INVALID_ARG;
    if (!c->k_block && (c->n_cand != 1 || c->own_max == 0)) return EVS_ERR_INVALID_ARG;
    if (!(c->scale >= 0.f) || isinf(c->scale)) return EVS_ERR_INVALID_ARG;
    if (!c->workspace || (uintptr_t)c->workspace % 256) return EVS_ERR_INVALID_ARG;
    if (c->ws_bytes < evs_shared_attention_workspace(c)) return EVS_ERR_CAPACITY;
    return status_of(launch_shared_attention(*c, (cudaStream_t)stream));
}
