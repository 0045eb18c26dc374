// The filtered draw of the next token (evs_sample): temperature, top-k, top-p, min-p and the
// inverse CDF at a given uniform, one thread-block cluster per row.
//
//   w_i = exp((l_i - max l) / T). In the order (l descending, id ascending): the first top_k
//   tokens, of these the shortest prefix whose mass before the token is below top_p of theirs,
//   of these the ones with w_i >= min_p. The token is the smallest id whose cumulative kept
//   mass, over ascending ids, exceeds u times the total.
//
// The decisions are comparisons of sums over the whole vocabulary, so weights are computed to
// about 2^-37 relative and summed as 64-bit fixed point (2^-44): the sums do not depend on their
// order, every run gives the same token, and it is the one that exact arithmetic gives unless a
// border falls within about 1e-11 of the total mass. In fp32 the error of one such sum,
// about 1e-6 of the mass, would move the draw in several percent of rows of 131072 flat logits.
//
// The row is read once: the CTAs of the cluster keep their slices in shared memory and search
// there. The cut (top-k and top-p are both prefixes of the sorted row, so one pair (logit, id)
// describes what is kept) is found by a histogram over (max - l) / T in steps of 1/64, narrowed
// by digits of (ordered logit, id) while the bin that holds the cut has more than CAP tokens;
// those few are then sorted. (Ranking them pairwise took 15 us for the 461 tokens left of a
// 512-entry row, and one CTA's 17 us held the other seven of a large row's cluster.)
#include "evs_common.cuh"
#include "sm100_ptx.cuh"

namespace evs {
namespace {

using bf16 = __nv_bfloat16;
typedef unsigned long long u64;

constexpr int SMP_MAX_V = 1 << 18;      // ids take 18 bits of the order
constexpr int SMP_IDBITS = 18;
constexpr int SMP_ORDER_BITS = 32 + SMP_IDBITS;
constexpr int SMP_DIGIT = 11;
constexpr int SMP_BINS = 1 << SMP_DIGIT;
constexpr int SMP_CAP = 1024;           // tokens sorted
constexpr int SMP_FRAC = 44;            // fixed point of weights; 2^18 of them stay below 2^63
constexpr int SMP_MAX_CS = 8;           // portable cluster size

// 2^(j/32) for j = -16..16, each the sum of two floats
__constant__ float2 kPow2[33] = {
    {0.7071067690849304f, 1.2101617485882343e-08f}, {0.7225903868675232f, 1.662099968768871e-08f}, {0.7384130954742432f, -2.250449426810519e-08f},
    {0.7545822262763977f, -1.2479686617439256e-08f}, {0.7711054086685181f, 4.035452416673024e-09f}, {0.7879904508590698f, -2.830512713103417e-08f},
    {0.8052451610565186f, 4.918108587048664e-09f}, {0.8228777647018433f, -2.5624860455764065e-08f}, {0.8408964276313782f, -1.2377663338725142e-08f},
    {0.8593096733093262f, -2.4248087981959543e-08f}, {0.8781260848045349f, -4.617885185353998e-09f}, {0.8973545432090759f, -5.707522454656555e-09f},
    {0.9170040488243103f, -5.619638976384067e-09f}, {0.9370838403701782f, -2.331502813035513e-08f}, {0.9576032757759094f, 4.922664054163306e-09f},
    {0.9785720705986023f, -8.510902205216553e-09f}, {1.0f, 0.0f}, {1.0218971967697144f, -4.811559861650494e-08f},
    {1.0442737340927124f, 4.8334701574503924e-08f}, {1.0671404600143433f, -5.9337519786595294e-08f}, {1.0905077457427979f, -1.3077539939843064e-08f},
    {1.114386796951294f, -5.435540018083884e-08f}, {1.1387885808944702f, 5.386222312608879e-08f}, {1.1637248992919922f, -4.051441493402308e-08f},
    {1.1892070770263672f, 3.797635272917432e-08f}, {1.215247392654419f, -3.267394887984665e-08f}, {1.2418577671051025f, 4.496838101886169e-08f},
    {1.2690509557724f, 1.419333317542737e-09f}, {1.2968395948410034f, -4.018999533172973e-08f}, {1.3252366781234741f, -3.496373324196611e-08f},
    {1.3542555570602417f, -1.0123349269974824e-08f}, {1.3839099407196045f, -5.875577357983275e-08f}, {1.4142135381698608f, 2.4203234971764687e-08f}
};

struct SampleArgs {
    const void* logits;
    int64_t ld, ldp;
    int V;
    const float *temperature, *top_p, *min_p, *uniforms;
    const int32_t* top_k;
    int32_t* token;
    float* logprob;
    float* probs;
    uint32_t* flags;
    int slice;             // slots of shared memory for logits
};

// ---- cluster helpers --------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void st_peer_u64(uint32_t addr, u64 v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ void st_peer_u32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_peer_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t atom_peer_add(uint32_t addr, uint32_t v) {
    uint32_t o;
    asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(o) : "r"(addr), "r"(v) : "memory");
    return o;
}
template <bool CLUSTER> __device__ __forceinline__ void sync_all() {
    if constexpr (CLUSTER) cluster_sync(); else __syncthreads();
}

__device__ __forceinline__ float load_logit(float v) { return v != v ? -INFINITY : v; }   // NaN: ruled out
__device__ __forceinline__ float load_logit(bf16 v) { return load_logit(__bfloat162float(v)); }

// Position in the order: larger is earlier. The logit's bits mapped to an ascending integer,
// then the id descending.
__device__ __forceinline__ u64 order_of(float l, int id) {
    uint32_t k = __float_as_uint(l + 0.f);             // -0 and +0 are one value
    k = (k & 0x80000000u) ? ~k : (k | 0x80000000u);
    return ((u64)k << SMP_IDBITS) | (u64)((1 << SMP_IDBITS) - 1 - id);
}

__device__ __forceinline__ u64 warp_sum_u64(u64 v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Exclusive scan over the block, and the total; red holds one word per warp.
template <int THREADS>
__device__ __forceinline__ u64 block_scan_u64(u64 v, u64* red, u64& total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    u64 x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) red[w] = x;
    __syncthreads();
    u64 before = 0, all = 0;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) {
        const u64 r = red[i];
        before += i < w ? r : 0;
        all += r;
    }
    total = all;
    return before + x - v;
}

// p in [0, 1) as 2^-bits fixed point, rounded down or up (p >= 1: `one`; p <= 0 or NaN: 0). By its
// bits: fp64 runs at 1/64 of fp32's rate.
__device__ __forceinline__ u64 unit_fixed(float p, int bits, bool up, u64 one) {
    if (!(p > 0.f)) return 0;
    if (p >= 1.f) return one;
    const uint32_t u = __float_as_uint(p), e = u >> 23;
    const u64 m = e ? (u & 0x7fffffu) | 0x800000u : u & 0x7fffffu;
    const int sh = (int)(e ? e : 1) - 150 + bits;          // p = m 2^(sh - bits)
    if (sh >= 0) return m << sh;
    if (sh <= -24) return up ? 1 : 0;
    return (m >> -sh) + (up && (m & ((1ull << -sh) - 1)) ? 1 : 0);
}

// ---- weights ------------------------------------------------------------------------------------
// exp((l - M) / T) = 2^y, y = (l - M) * c with c = log2(e) / T held as the sum of two floats. The
// difference and the product are formed exactly (two-sum, fused multiply-add remainders);
// y = n + j/32 + g, |g| <= 1/64, and 2^g - 1 by its Taylor series, whose first term is kept as a
// sum of two floats too. Relative error about 2^-37; weights below 2^-45 are 0. Integers are taken
// from the low bits of sums with 1.5 * 2^23: conversions run at an eighth of the rate.
constexpr float kRound = 12582912.f;      // 1.5 * 2^23
struct WeightFn {
    float M, c_hi, c_lo;
    const float2* tab;    // shared copy of kPow2

    // the weight times 2^22, as the sum of two floats; false: 0 (or l is not below M)
    __device__ __forceinline__ bool scaled(float l, float& hi, float& lo) const {
        const float dh = l - M;
        const float bb = dh - l;
        const float dl = (l - (dh - bb)) + (-M - bb);
        const float p = dh * c_hi;
        if (!(p > -64.f)) return false;
        const float e = fmaf(dh, c_hi, -p) + fmaf(dh, c_lo, dl * c_hi);
        const float tn = p + kRound;
        const float r0 = p - (tn - kRound);
        const float r = r0 + e;
        const float e1 = (r0 - r) + e;                    // what the sum dropped, below 2^-25
        const float tj = fmaf(r, 32.f, kRound);
        const float g = fmaf(tj - kRound, -0.03125f, r);
        const float L_hi = 0.693147182464599609375f, L_lo = -1.904654299957768e-09f;   // ln 2
        const float q = g * L_hi;
        const float q_lo = fmaf(g, L_lo, fmaf(g, L_hi, -q));
        float h = fmaf(q, 1.f / 120.f, 1.f / 24.f);
        h = fmaf(h, q, 1.f / 6.f);
        h = fmaf(h, q, 0.5f);
        const float rest = fmaf(h * q, q, fmaf(e1 * L_hi, 1.f + q, q_lo));
        const float2 t = tab[16 + (__float_as_int(tj) - __float_as_int(kRound))];
        const float m = t.x * q;
        const float s = t.x + m;
        const float s_lo = ((t.x - s) + m) + (fmaf(t.x, q, -m) + fmaf(t.x, rest, t.y));
        const float w = s + s_lo, w_lo = (s - w) + s_lo;  // w_lo within half a step of w
        const float two_n = __int_as_float((__float_as_int(tn) - __float_as_int(kRound) + 127 + 22) << 23);
        hi = w * two_n;
        lo = w_lo * two_n;
        return true;
    }
    __device__ __forceinline__ u64 fixed(float l) const {
        float hi, lo;
        if (l == M) return 1ull << SMP_FRAC;
        if (!scaled(l, hi, lo)) return 0;
        const float t = hi + kRound;
        const float rest = (hi - (t - kRound)) + lo;      // exact, then rounded once
        const float t2 = fmaf(rest, 4194304.f, kRound);
        const int a = __float_as_int(t) - __float_as_int(kRound), b = __float_as_int(t2) - __float_as_int(kRound);
        return (u64)((long long)a * (1ll << (SMP_FRAC - 22)) + b);
    }
    __device__ __forceinline__ float real(float l) const {   // fp32, for probabilities
        float hi, lo;
        if (l == M) return 1.f;
        return scaled(l, hi, lo) ? (hi + lo) * 2.384185791015625e-7f : 0.f;   // 2^-22
    }
};

// 16 bytes of a row
template <typename T> union Raw16 {
    uint4 q;
    T v[16 / sizeof(T)];
    __device__ Raw16() {}
};

// The set of tokens that holds a cut, and what precedes it: level-0 bin bin0, of it the tokens
// whose order has `prefix` above bit `shift` (shift SMP_ORDER_BITS: all of the bin).
struct Found {
    int bin0, shift;
    uint32_t count, above_count;
    u64 above_mass, prefix;
};

// =========================================================================================
template <typename T, int THREADS, bool CLUSTER>
__global__ void __launch_bounds__(THREADS, THREADS == 512 ? 2 : 1) sample_kernel(SampleArgs a) {
    constexpr int VEC = 16 / sizeof(T);
    constexpr int BPT = SMP_BINS / THREADS;     // bins a thread sums when the CTA is alone
    extern __shared__ __align__(16) uint8_t smem[];
    float* l_s = reinterpret_cast<float*>(smem);
    uint32_t* hist = reinterpret_cast<uint32_t*>(smem + (size_t)a.slice * 4);   // [4][BINS]: count, mass planes
    u64* list_o = reinterpret_cast<u64*>(hist);                                 // [CAP], after a search
    u64* list_w = list_o + SMP_CAP;                                             // [CAP]
    __shared__ float2 tab[33];
    __shared__ u64 red[THREADS / 32];
    __shared__ u64 warp_mass[THREADS / 32];
    __shared__ float x_max[SMP_MAX_CS];
    __shared__ u64 x_cnt[SMP_MAX_CS], x_mass[SMP_MAX_CS], x_sum[SMP_MAX_CS], x_arg[SMP_MAX_CS];
    __shared__ u64 f_above_mass, f_cut, pick_before;
    __shared__ uint32_t f_bin, f_count, f_above_count, list_n[2];
    __shared__ int pick_warp, last_kept;
    __shared__ float inv_total;
    __shared__ struct {
        u64 p64, u64_, mp;
        float c_hi, c_lo, bin_scale, temp;
        int k, greedy, need_p;
    } par;

    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t cs = CLUSTER ? cluster_size() : 1u, rank = CLUSTER ? cluster_rank() : 0u;
    const int row = blockIdx.x / cs;
    if (tid < 33) tab[tid] = kPow2[tid];
    if (tid < 2) list_n[tid] = 0;
    // peers may write here once every CTA of the cluster runs: arrive now, wait before the first
    if constexpr (CLUSTER) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    pdl_wait();

    // ---- parameters of the row: one thread's few fp64 operations (their rate is 1/64 of fp32's)
    if (tid == 0) {
        const float temp = a.temperature ? a.temperature[row] : 1.f;
        const int k = a.top_k ? a.top_k[row] : 0;
        const float p = a.top_p ? a.top_p[row] : 1.f, mp = a.min_p ? a.min_p[row] : 0.f;
        const bool greedy = !(temp > 0.f);
        // log2(e) / T, the quotient's remainder by a fused multiply-add
        const float L2E = 1.44269502162933349609375f, L2E_lo = 1.9259629911266175e-8f, t = greedy ? 1.f : temp;
        par.c_hi = L2E / t;
        const float rest = fmaf(-par.c_hi, t, L2E) + L2E_lo;
        par.c_lo = isfinite(par.c_hi) && isfinite(rest) ? rest / t : 0.f;
        par.bin_scale = 64.f / (greedy ? 1.f : temp);
        par.temp = greedy ? 1.f : temp;
        par.greedy = greedy;
        par.k = !greedy && k > 0 && k < a.V ? k : 0;
        par.need_p = !greedy && p < 1.f;
        par.p64 = unit_fixed(p, 64, false, ~0ull);
        par.u64_ = unit_fixed(a.uniforms[row], 64, false, ~0ull);
        par.mp = greedy ? 0 : unit_fixed(mp, SMP_FRAC, true, 1ull << SMP_FRAC);
    }

    // ---- the slice: granules of 16 bytes of the row, the first and last ones partly filled
    const T* rp = (const T*)a.logits + (size_t)row * a.ld;
    const int mis = (int)(((uintptr_t)rp % 16) / sizeof(T));
    const int grans = (mis + a.V + VEC - 1) / VEC;
    const int g0 = (int)((long long)grans * rank / cs), g1 = (int)((long long)grans * (rank + 1) / cs);
    const int n = (g1 - g0) * VEC;              // slots; slot s holds id base + s
    const int base = g0 * VEC - mis;
    float mx = -INFINITY;
    for (int gb = 0; gb < g1 - g0; gb += 4 * THREADS) {
        Raw16<T> r[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int g = gb + u * THREADS + tid;
            if (g < g1 - g0) {
                const int id0 = base + g * VEC;
                if (id0 >= 0 && id0 + VEC <= a.V) {
                    r[u].q = *reinterpret_cast<const uint4*>(rp + id0);
                } else {
#pragma unroll
                    for (int j = 0; j < VEC; ++j)
                        r[u].v[j] = (id0 + j >= 0 && id0 + j < a.V) ? rp[id0 + j] : from_f32<T>(-INFINITY);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int g = gb + u * THREADS + tid;
            if (g < g1 - g0) {
#pragma unroll
                for (int j = 0; j < VEC; j += 4) {
                    const float4 f = make_float4(load_logit(r[u].v[j]), load_logit(r[u].v[j + 1]),
                                                 load_logit(r[u].v[j + 2]), load_logit(r[u].v[j + 3]));
                    mx = fmaxf(mx, fmaxf(fmaxf(f.x, f.y), fmaxf(f.z, f.w)));
                    *reinterpret_cast<float4*>(l_s + g * VEC + j) = f;
                }
            }
        }
    }
    mx = block_max(mx, reinterpret_cast<float*>(red));
    if constexpr (CLUSTER) {
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (tid < (int)cs) st_peer_f32(map_peer(smem_u32(&x_max[rank]), tid), mx);
        cluster_sync();
        mx = x_max[0];
        for (uint32_t i = 1; i < cs; ++i) mx = fmaxf(mx, x_max[i]);
    } else {
        __syncthreads();
    }
    WeightFn wf{mx, par.c_hi, par.c_lo, tab};      // written before the barriers of the maximum
    const float bin_scale = par.bin_scale;
    const bool greedy = par.greedy, need_p = par.need_p;
    const int k_in = par.k;
    const bool need_k = k_in > 0;
    if (mx == -INFINITY) {                       // every token ruled out: no draw
        if (rank == 0 && tid == 0) {
            a.token[row] = -1;
            if (a.logprob) a.logprob[row] = -INFINITY;
            if (a.flags) atomicOr(a.flags, (uint32_t)EVS_FLAG_EMPTY_ROW);
        }
        if (a.probs)
            for (int s = tid; s < n; s += THREADS)
                if (base + s >= 0 && base + s < a.V) a.probs[(size_t)row * a.ldp + base + s] = 0.f;
        if constexpr (CLUSTER) cluster_sync();
        return;
    }

    u64 cut = 0;           // tokens with order >= cut are kept (before min-p): logits above cut_l,
    float cut_l = -INFINITY;   // and of that value ids up to cut_id
    int cut_id = 0;
    auto set_cut = [&](u64 c) {
        cut = c;
        const uint32_t k = (uint32_t)(c >> SMP_IDBITS);
        cut_l = __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
        cut_id = (1 << SMP_IDBITS) - 1 - (int)(c & ((1ull << SMP_IDBITS) - 1));
    };
    auto above_cut = [&](float l, int id) -> bool { return l > cut_l || (l == cut_l && id <= cut_id && cut != 0); };
    auto bin0_of = [&](float l) -> int {
        const float d = (mx - l) * bin_scale;
        return l == mx ? 0 : (d < (float)(SMP_BINS - 1) ? (int)d : SMP_BINS - 1);
    };
    auto in_found = [&](const Found& f, float l, u64 o) -> bool {
        return bin0_of(l) == f.bin0 && (f.shift == SMP_ORDER_BITS || (o >> f.shift) == f.prefix);
    };
    // The set of at most CAP tokens (or the single one) where the cumulative count reaches k
    // (k > 0), or the cumulative mass of the tokens above the cut so far reaches
    // x = ceil(p64 * their mass). Level 0 bins by (max - l) / T, later levels by a digit of the
    // order. bin0 is BINS where fewer than k tokens are left. Uniform over the cluster.
    auto search = [&](uint32_t k, u64 p64, u64& x) -> Found {
        Found f{SMP_BINS, SMP_ORDER_BITS, 0, 0, 0, 0};
        for (int level = 0;; ++level) {
            const int to = max(0, f.shift - SMP_DIGIT), width = f.shift - to;   // this level's digit
            for (int i = tid; i < (k ? 1 : 4) * SMP_BINS; i += THREADS) hist[i] = 0;
            __syncthreads();
            if (tid == 0) f_bin = SMP_BINS;      // read by all before that barrier, written next after another
            for (int s = tid; s < n; s += THREADS) {
                const float l = l_s[s];
                if (!above_cut(l, base + s)) continue;
                int bin;
                if (level == 0) {
                    bin = bin0_of(l);
                } else {
                    const u64 o = order_of(l, base + s);
                    if (!in_found(f, l, o)) continue;
                    // digits descend, so that a lower bin is earlier in the order
                    bin = (1 << width) - 1 - (int)((o >> to) & ((1ull << width) - 1));
                }
                atomicAdd(&hist[bin], 1u);
                if (k == 0) {
                    const u64 w = wf.fixed(l);
                    const uint32_t w0 = (uint32_t)w & 0xffffu, w1 = (uint32_t)(w >> 16) & 0xffffu,
                                   w2 = (uint32_t)(w >> 32);
                    if (w0) atomicAdd(&hist[SMP_BINS + bin], w0);
                    if (w1) atomicAdd(&hist[2 * SMP_BINS + bin], w1);
                    if (w2) atomicAdd(&hist[3 * SMP_BINS + bin], w2);
                }
            }
            sync_all<CLUSTER>();
            // this CTA's share of the bins, summed over the cluster; a thread takes PT in a row
            const int nb = SMP_BINS / cs, b_lo = nb * rank, PT = (nb + THREADS - 1) / THREADS;
            uint32_t cnt[BPT];
            u64 mass[BPT], tc = 0, tm = 0;
#pragma unroll
            for (int i = 0; i < BPT; ++i) {
                cnt[i] = 0;
                mass[i] = 0;
                if (i < PT && tid * PT + i < nb) {
                    const int b = b_lo + tid * PT + i;
                    for (uint32_t r = 0; r < cs; ++r) {
                        auto at = [&](int plane) -> u64 {
                            if constexpr (CLUSTER) return ld_peer_u32(map_peer(smem_u32(&hist[plane * SMP_BINS + b]), r));
                            else return hist[plane * SMP_BINS + b];
                        };
                        cnt[i] += (uint32_t)at(0);
                        if (k == 0) mass[i] += at(1) + (at(2) << 16) + (at(3) << 32);
                    }
                }
                tc += cnt[i];
                tm += mass[i];
            }
            u64 all_c, all_m;
            u64 ec = block_scan_u64<THREADS>(tc, red, all_c);
            u64 em = 0;
            all_m = 0;
            if (k == 0) em = block_scan_u64<THREADS>(tm, red, all_m);
            if constexpr (CLUSTER) {
                if (tid < (int)cs) {
                    st_peer_u64(map_peer(smem_u32(&x_cnt[rank]), tid), all_c);
                    st_peer_u64(map_peer(smem_u32(&x_mass[rank]), tid), all_m);
                }
                cluster_sync();
                all_m = 0;
                for (uint32_t i = 0; i < cs; ++i) {
                    if (i < rank) {
                        ec += x_cnt[i];
                        em += x_mass[i];
                    }
                    all_m += x_mass[i];
                }
            }
            if (level == 0 && k == 0) {           // mass before a kept token < p * total
                x = __umul64hi(p64, all_m) + ((p64 * all_m) != 0 ? 1 : 0);
                if (x == 0) x = 1;                // the first token is always kept
            }
            ec += f.above_count;
            em += f.above_mass;
#pragma unroll
            for (int i = 0; i < BPT; ++i) {
                const bool hit = k ? (ec < k && ec + cnt[i] >= k) : (em < x && em + mass[i] >= x);
                if (hit) {
                    const uint32_t bin = b_lo + tid * PT + i;
                    for (uint32_t r = 0; r < cs; ++r) {
                        if constexpr (CLUSTER) {
                            st_peer_u32(map_peer(smem_u32(&f_bin), r), bin);
                            st_peer_u32(map_peer(smem_u32(&f_count), r), cnt[i]);
                            st_peer_u32(map_peer(smem_u32(&f_above_count), r), (uint32_t)ec);
                            st_peer_u64(map_peer(smem_u32(&f_above_mass), r), em);
                        } else {
                            f_bin = bin;
                            f_count = cnt[i];
                            f_above_count = (uint32_t)ec;
                            f_above_mass = em;
                        }
                    }
                }
                ec += cnt[i];
                em += mass[i];
            }
            sync_all<CLUSTER>();
            if (f_bin == SMP_BINS) return f;
            f.count = f_count;
            f.above_count = f_above_count;
            f.above_mass = f_above_mass;
            if (level == 0) {
                f.bin0 = (int)f_bin;
            } else {
                const u64 digit = (u64)((1 << width) - 1 - (int)f_bin);
                f.prefix = f.shift == SMP_ORDER_BITS ? digit : ((f.prefix << width) | digit);
                f.shift = to;
            }
            if (f.count <= SMP_CAP || f.shift == 0) return f;
        }
    };
    int list_at = 0;
    // Sorts the gathered tokens (first CTA) and returns the order of the last one kept: the first
    // k overall (k > 0), and with do_p of these the nucleus of mass x, or where x is 0 of
    // ceil(p64 * mass of the k). above_*: what precedes all of them.
    auto finish = [&](uint32_t above_count, u64 above_mass, uint32_t k, bool do_p, u64 p64, u64 x) -> u64 {
        sync_all<CLUSTER>();                      // every CTA's entries have arrived
        if (rank == 0) {
            const int m = min((int)list_n[list_at], SMP_CAP);
            // Bitonic, descending, an element a thread (and every THREADS further): neighbours closer
            // than a warp through shuffles, others through shared memory. The place in the list
            // rides in the low bits.
            constexpr int PER = SMP_CAP / THREADS, PLACE = 10;
            u64 v[PER];
            int n2 = 2;
            while (n2 < m) n2 *= 2;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int e = tid + i * THREADS;
                v[i] = e < m ? (list_o[e] << PLACE) | (u64)e : 0;
            }
            for (int k2 = 2; k2 <= n2; k2 *= 2)
                for (int j = k2 / 2; j > 0; j /= 2) {
                    u64 o[PER];
                    if (j < 32) {
#pragma unroll
                        for (int i = 0; i < PER; ++i) o[i] = __shfl_xor_sync(0xffffffffu, v[i], j);
                    } else if (j < THREADS) {
                        __syncthreads();
#pragma unroll
                        for (int i = 0; i < PER; ++i) list_o[tid + i * THREADS] = v[i];
                        __syncthreads();
#pragma unroll
                        for (int i = 0; i < PER; ++i) o[i] = list_o[(tid ^ j) + i * THREADS];
                    } else {
#pragma unroll
                        for (int i = 0; i < PER; ++i) {
                            o[i] = v[i];
#pragma unroll
                            for (int x = 0; x < PER; ++x)
                                if (x == (i ^ (j / THREADS))) o[i] = v[x];
                        }
                    }
#pragma unroll
                    for (int i = 0; i < PER; ++i) {
                        const int e = tid + i * THREADS;
                        const bool larger = ((e & k2) == 0) == ((e & j) == 0);
                        if ((o[i] > v[i]) == larger) v[i] = o[i];
                    }
                }
            // consecutive entries to a thread again
            __syncthreads();
#pragma unroll
            for (int i = 0; i < PER; ++i) list_o[tid + i * THREADS] = v[i];
            if (tid == 0) last_kept = 0;
            __syncthreads();
            u64 w[PER], mine = 0, total;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int e = tid * PER + i;
                w[i] = e < m && (k == 0 || above_count + e < k) ? list_w[list_o[e] & ((1 << PLACE) - 1)] : 0;
                mine += w[i];
            }
            u64 before = block_scan_u64<THREADS>(mine, red, total) + above_mass;
            total += above_mass;
            if (do_p && x == 0) {
                x = __umul64hi(p64, total) + ((p64 * total) != 0 ? 1 : 0);
                if (x == 0) x = 1;
            }
            int kept_to = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int e = tid * PER + i;
                if (e < m && (k == 0 || above_count + e < k) && (!do_p || before < x)) kept_to = e;
                before += w[i];
            }
            kept_to = __reduce_max_sync(0xffffffffu, kept_to);
            if (lane == 0 && kept_to > 0) atomicMax(&last_kept, kept_to);
            __syncthreads();
            if (tid < (int)cs) {
                const u64 lowest = list_o[last_kept] >> PLACE;
                if constexpr (CLUSTER) st_peer_u64(map_peer(smem_u32(&f_cut), tid), lowest);
                else f_cut = lowest;
            }
        }
        sync_all<CLUSTER>();
        ++list_at;                                // a second list counts anew
        return f_cut;
    };
    // Appends the tokens that `take` names to the first CTA's list; a warp's share by one counter update.
    auto gather = [&](auto take) {
        for (int s0 = 0; s0 < n; s0 += THREADS) {
            const int s = s0 + tid;
            const float l = s < n ? l_s[s] : -INFINITY;
            u64 o = 0;
            const bool yes = l > -INFINITY && take(l, s, o);
            const unsigned who = __ballot_sync(0xffffffffu, yes);
            if (who == 0) continue;
            uint32_t at = 0;
            if (lane == 0) {
                if constexpr (CLUSTER) at = atom_peer_add(map_peer(smem_u32(&list_n[list_at]), 0), __popc(who));
                else at = atomicAdd(&list_n[list_at], __popc(who));
            }
            at = __shfl_sync(0xffffffffu, at, 0) + __popc(who & ((1u << lane) - 1));
            if (yes && at < SMP_CAP) {
                const u64 w = wf.fixed(l);
                if constexpr (CLUSTER) {
                    st_peer_u64(map_peer(smem_u32(&list_o[at]), 0), o);
                    st_peer_u64(map_peer(smem_u32(&list_w[at]), 0), w);
                } else {
                    list_o[at] = o;
                    list_w[at] = w;
                }
            }
        }
    };

    if (greedy) {
        u64 best = 0;
        for (int s = tid; s < n; s += THREADS)
            if (l_s[s] == mx) {
                const u64 o = order_of(mx, base + s);
                if (o > best) best = o;
            }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const u64 t = __shfl_xor_sync(0xffffffffu, best, o);
            if (t > best) best = t;
        }
        __syncthreads();
        if (lane == 0) red[warp] = best;
        __syncthreads();
        for (int i = 0; i < THREADS / 32; ++i)
            if (red[i] > best) best = red[i];
        if constexpr (CLUSTER) {
            if (tid < (int)cs) st_peer_u64(map_peer(smem_u32(&x_arg[rank]), tid), best);
            cluster_sync();
            for (uint32_t i = 0; i < cs; ++i)
                if (x_arg[i] > best) best = x_arg[i];
        }
        set_cut(best);
    } else if (need_k || need_p) {
        const u64 p64 = par.p64;
        u64 x = 0;
        bool p_left = need_p;
        if (a.V <= SMP_CAP) {                     // all of them sorted, no search
            gather([&](float l, int s, u64& o) {
                o = order_of(l, base + s);
                return true;
            });
            set_cut(finish(0, 0, need_k ? (uint32_t)k_in : 0u, need_p, p64, 0));
            p_left = false;
        } else if (need_k) {
            // the whole top-k as one list where it fits, else only the set that holds its end
            const Found f = search((uint32_t)k_in, 0, x);
            if (f.bin0 < SMP_BINS) {
                const bool all = f.shift == SMP_ORDER_BITS && f.above_count + f.count <= SMP_CAP;
                gather([&](float l, int s, u64& o) {
                    if (all ? bin0_of(l) > f.bin0 : bin0_of(l) != f.bin0) return false;
                    o = order_of(l, base + s);
                    return all || in_found(f, l, o);
                });
                set_cut(finish(all ? 0 : f.above_count, 0, (uint32_t)k_in, need_p && all, p64, 0));
                if (all) p_left = false;
            }
        }
        if (p_left) {
            const Found f = search(0, p64, x);
            gather([&](float l, int s, u64& o) {
                if (bin0_of(l) != f.bin0 || !above_cut(l, base + s)) return false;
                o = order_of(l, base + s);
                return in_found(f, l, o);
            });
            set_cut(finish(f.above_count, f.above_mass, 0, true, p64, x));
        }
    }

    // ---- the kept mass by ids: a warp owns consecutive slots ------------------------------------
    const u64 mp = par.mp;
    auto kept = [&](int s) -> u64 {
        const float l = l_s[s];
        if (!above_cut(l, base + s)) return 0;
        const u64 w = wf.fixed(l);
        return w >= mp ? w : 0;
    };
    const int seg = (n + THREADS - 1) / THREADS * 32;
    {
        u64 m = 0;
        const int hi = min(n, (warp + 1) * seg);
        for (int s = warp * seg + lane; s < hi; s += 32) m += kept(s);
        m = warp_sum_u64(m);
        if (lane == 0) warp_mass[warp] = m;
    }
    __syncthreads();
    u64 mine = 0, total, before = 0;
    for (int i = 0; i < THREADS / 32; ++i) mine += warp_mass[i];
    total = mine;
    if constexpr (CLUSTER) {
        if (tid < (int)cs) st_peer_u64(map_peer(smem_u32(&x_sum[rank]), tid), mine);
        cluster_sync();
        total = 0;
        for (uint32_t i = 0; i < cs; ++i) {
            if (i < rank) before += x_sum[i];
            total += x_sum[i];
        }
    }
    // cumulative mass > u * total: integers, so > its floor
    const u64 thr = __umul64hi(par.u64_, total);
    if (before <= thr && thr < before + mine) {
        if (tid == 0) {
            u64 c = before;
            int w = 0;
            while (w < THREADS / 32 - 1 && c + warp_mass[w] <= thr) c += warp_mass[w++];
            pick_warp = w;
            pick_before = c;
        }
        __syncthreads();
        // the warp's slots, dealt out to the whole CTA in order
        const int lo = pick_warp * seg, hi = min(n, lo + seg), per = (seg + THREADS - 1) / THREADS;
        u64 m = 0;
        for (int i = 0; i < per; ++i)
            if (lo + tid * per + i < hi) m += kept(lo + tid * per + i);
        u64 all;
        u64 c = pick_before + block_scan_u64<THREADS>(m, red, all);
        if (c <= thr && thr < c + m) {
            int s = lo + tid * per;
            for (;; ++s) {
                const u64 w = kept(s);
                if (thr < c + w) break;
                c += w;
            }
            a.token[row] = base + s;
            if (a.logprob) {
                // log(w / total): the logit's distance less the log of the total over the largest weight,
                // which is at least 1 and relative to it where it is near
                const float lw = l_s[s] == mx ? 0.f : (l_s[s] - mx) / par.temp;
                const u64 one = 1ull << SMP_FRAC;
                const float lt = total < 2 * one ? log1pf((float)(total - one) * 5.684341886080802e-14f)   // 2^-44
                                                 : logf((float)total * 5.684341886080802e-14f);
                a.logprob[row] = lw - lt;
            }
        }
    }
    if (a.probs) {
        if (tid == 0) inv_total = (float)((double)(1ull << SMP_FRAC) / (double)total);
        __syncthreads();
        const float inv = inv_total;
        float* pr = a.probs + (size_t)row * a.ldp;
        for (int s = tid; s < n; s += THREADS) {
            const int id = base + s;
            if (id >= 0 && id < a.V) pr[id] = kept(s) ? wf.real(l_s[s]) * inv : 0.f;
        }
    }
    if constexpr (CLUSTER) cluster_sync();        // peers may still write into this CTA
}

// Cluster size: slices of at most 16384 slots (64 KiB, so that two CTAs share an SM), then more
// CTAs a row while the rows alone leave SMs idle and a slice still has 4096 slots.
int sample_cluster(int rows, int V) {
    int cs = 1;
    while (cs < SMP_MAX_CS && V > cs * 16384) cs *= 2;
    while (cs < SMP_MAX_CS && (long long)rows * cs < 2 * 152 && V > cs * 4096) cs *= 2;
    return cs;
}

template <typename T, int THREADS, bool CLUSTER>
cudaError_t sample_launch(const SampleArgs& a, int rows, int cs, size_t smem, cudaStream_t stream) {
    auto kernel = sample_kernel<T, THREADS, CLUSTER>;
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)rows * cs);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cs;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CLUSTER ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <typename T>
cudaError_t sample_dispatch(SampleArgs a, int rows, cudaStream_t stream) {
    constexpr int VEC = 16 / sizeof(T);
    const int cs = sample_cluster(rows, a.V);
    const int grans = (VEC - 1 + a.V + VEC - 1) / VEC;
    a.slice = (grans + cs - 1) / cs * VEC;
    const size_t smem = (size_t)a.slice * 4 + (a.V <= SMP_CAP ? (size_t)SMP_CAP * 16 : (size_t)SMP_BINS * 16);
    if (cs > 1) return sample_launch<T, 512, true>(a, rows, cs, smem, stream);
    if (a.V > 2048) return sample_launch<T, 512, false>(a, rows, 1, smem, stream);
    return sample_launch<T, 256, false>(a, rows, 1, smem, stream);
}

}  // namespace

cudaError_t launch_sample(const evs_sample_args& c, cudaStream_t stream) {
    SampleArgs a{c.logits, c.ld, c.probs_ld, c.vocab, c.temperature, c.top_p, c.min_p, c.uniforms, c.top_k,
                 c.token, c.logprob, c.probs, c.flags, 0};
    return c.dtype == EVS_DTYPE_BF16 ? sample_dispatch<bf16>(a, c.rows, stream)
                                     : sample_dispatch<float>(a, c.rows, stream);
}

}  // namespace evs

extern "C" evs_status evs_sample(const evs_sample_args* c, void* stream) {
    using namespace evs;
    if (!c || c->rows < 0 || c->vocab < 1 || c->vocab > SMP_MAX_V || c->ld < c->vocab) return EVS_ERR_INVALID_ARG;
    if (c->dtype != EVS_DTYPE_F32 && c->dtype != EVS_DTYPE_BF16) return EVS_ERR_INVALID_ARG;
    if (c->rows == 0) return EVS_OK;
    if (c->rows > (1 << 24) || !c->logits || !c->token || !c->uniforms) return EVS_ERR_INVALID_ARG;
    if ((uintptr_t)c->logits % (c->dtype == EVS_DTYPE_BF16 ? 2 : 4)) return EVS_ERR_INVALID_ARG;
    if (c->probs && c->probs_ld < c->vocab) return EVS_ERR_INVALID_ARG;
    return launch_sample(*c, (cudaStream_t)stream) == cudaSuccess ? EVS_OK : EVS_ERR_CUDA;
}
