// The filtered draw of the next token (evs_sample): temperature, top-k, top-p, min-p and the
// inverse CDF at a given uniform, one thread-block cluster per row.
//
//   w_i = exp((l_i - max l) / T). In the order (l descending, id ascending): the first top_k
//   tokens, of these the shortest prefix whose mass before the token is below top_p of theirs,
//   of these the ones with w_i >= min_p. The token is the smallest id whose cumulative kept
//   mass, over ascending ids, exceeds u times the total.
//
// The decisions are comparisons of sums over the whole vocabulary, so weights are computed to
// about 2^-32 relative and summed as 64-bit fixed point (2^-45): the sums do not depend on their
// order, every run gives the same token, and it is the one that exact arithmetic gives unless a
// border falls within about 2e-10 of the total mass. In fp32 the error of one such sum,
// about 1e-6 of the mass, would move the draw in several percent of rows of 131072 flat logits.
//
// The row is read once: the CTAs of the cluster keep their slices in shared memory and search
// there. The cut (top-k and top-p are both prefixes of the sorted row, so one pair (logit, id)
// describes what is kept) is found by a histogram over the weight's exponent in steps of 1/32,
// narrowed by digits of (ordered logit, id) while the bin that holds the cut has more than CAP
// tokens; those few are then ranked. A bin's mass is the sum of its tokens' mantissas, of 33 bits,
// in two 32-bit counters (three took 13.5 thousand cycles of a large row's histogram, two 12.9).
//
// A chain of dependent phases, each with a barrier, bounds small and large rows alike. 4 x 512 fp32
// with every filter 6.8 us, 208 x 4096 with probabilities 17, 64 x 50021 bf16 23, 256 x 131072 fp32
// with top-p and min-p 261: 2048 CTAs, two an SM, of 33 us each, in thousands of cycles launch and loads
// 7, maximum 4, histogram 13 and the wait for the cluster 3, its scan 8, gathering the bin 8, ranking it
// 11 (one CTA of the eight works), the kept mass 11, its total 3, the rest 1. Two of four issue slots are
// used; the row is read once (134 MB, 20 us).
#include "evs_common.cuh"
#include "sm100_ptx.cuh"

#include <cfloat>
#include <climits>

namespace evs {
namespace {

using bf16 = __nv_bfloat16;
typedef unsigned long long u64;

constexpr int SMP_MAX_V = 1 << 18;      // ids take 18 bits of the order
constexpr int SMP_IDBITS = 18;
constexpr int SMP_ORDER_BITS = 32 + SMP_IDBITS;
constexpr int SMP_DIGIT = 11;
constexpr int SMP_BINS = 1 << SMP_DIGIT;
constexpr int SMP_CAP = 1024;           // tokens ranked at once
constexpr int SMP_FEW = 128;            // of them by counting instead of sorting
constexpr int SMP_FRAC = 45;            // fixed point of weights; 2^18 of them reach 2^63
constexpr int SMP_ZERO = SMP_FRAC + 1;  // weights of 2^-46 and less are 0
constexpr int SMP_AREA = SMP_CAP * 20;   // bytes of shared memory behind the logits: two lists of 8 bytes, two of 2
constexpr int SMP_MAX_CS = 8;           // portable cluster size
constexpr int SMP_MAX_SMEM = (SMP_MAX_V / SMP_MAX_CS + 16) * 4 + SMP_AREA;   // of the largest slice, its ends off the grid

// 2^(j/32) for j = 0..31, each the sum of two floats
__constant__ float2 kPow2[32] = {
    {1.0f, 0.0f}, {1.0218971967697144f, -4.811559861650494e-08f}, {1.0442737340927124f, 4.8334701574503924e-08f},
    {1.0671404600143433f, -5.9337519786595294e-08f}, {1.0905077457427979f, -1.3077539939843064e-08f}, {1.1143867969512939f, -5.4355400180838842e-08f},
    {1.1387885808944702f, 5.3862223126088793e-08f}, {1.1637248992919922f, -4.051441493402308e-08f}, {1.1892070770263672f, 3.7976352729174323e-08f},
    {1.2152473926544189f, -3.2673948879846648e-08f}, {1.2418577671051025f, 4.4968381018861692e-08f}, {1.2690509557723999f, 1.4193333175427369e-09f},
    {1.2968395948410034f, -4.0189995331729733e-08f}, {1.3252366781234741f, -3.4963733241966111e-08f}, {1.3542555570602417f, -1.0123349269974824e-08f},
    {1.3839099407196045f, -5.8755773579832749e-08f}, {1.4142135381698608f, 2.4203234971764687e-08f}, {1.4451807737350464f, 3.3241999375377418e-08f},
    {1.4768261909484863f, -4.5008988536210381e-08f}, {1.5091644525527954f, -2.4959373234878512e-08f}, {1.5422108173370361f, 8.0709048333460487e-09f},
    {1.5759809017181396f, -5.6610254262068338e-08f}, {1.6104903221130371f, 9.8362171740973281e-09f}, {1.6457555294036865f, -5.1249720911528129e-08f},
    {1.6817928552627563f, -2.4755326677450284e-08f}, {1.7186193466186523f, -4.8496175963919086e-08f}, {1.7562521696090698f, -9.2357703707079963e-09f},
    {1.7947090864181519f, -1.141504490931311e-08f}, {1.8340080976486206f, -1.1239277952768134e-08f}, {1.8741676807403564f, -4.6630056260710262e-08f},
    {1.9152065515518188f, 9.845328108326612e-09f}, {1.9571441411972046f, -1.7021804410433106e-08f},
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

__device__ __forceinline__ float logit_of(u64 order) {
    const uint32_t k = (uint32_t)(order >> SMP_IDBITS);
    return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
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
// difference and the product are formed exactly (two-sum, fused multiply-add remainders), so that
// y = p + e; p = i/32 + r, |r| <= 1/64, i taken from the low bits of p + 1.5 * 2^18 (one fused operation); and
// 2^(r + e) - 1 = q + rest with q = r ln 2 rounded and rest its tail, q^2/2 + q^3/6 + q^4/24 and
// e ln 2 * exp(q). In fixed point of 2^-34 the sum of the two is off by 2^-34 at most; times
// 2^(i/32), a weight is within about 2^-33 of its value. Two logits at a time: 26 packed
// instructions for both, where one by one in the same arithmetic takes 51 for each.
constexpr float kRound = 393216.f;        // 1.5 * 2^18: its last bit is 1/32

__device__ __forceinline__ u64 pk(float a, float b) {
    u64 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ u64 pk(float a) { return pk(a, a); }
__device__ __forceinline__ float2 unpk(u64 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ u64 add2(u64 a, u64 b) {
    u64 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ u64 mul2(u64 a, u64 b) {
    u64 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ u64 fma2(u64 a, u64 b, u64 c) {
    u64 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ u64 sub2(u64 a, u64 b) { return fma2(b, pk(-1.f), a); }

struct Parts {
    int i0, i1;           // the weight is 2^(i/32) (1 + q + rest) where p > -SMP_ZERO; else 0
    float2 p, q, rest;
};
struct WeightFn {
    float M, c_hi, c_lo;
    const u64* tab;       // 2^(j/32) * 2^62

    __device__ __forceinline__ Parts parts(float l0, float l1) const {
        const u64 l = pk(l0, l1), nM = pk(-M), ch = pk(c_hi);
        const u64 dh = add2(l, nM);
        const u64 bb = sub2(dh, l);
        const u64 dl = add2(sub2(l, sub2(dh, bb)), sub2(nM, bb));
        const u64 p = mul2(dh, ch);
        const u64 e = fma2(dl, ch, fma2(dh, pk(c_lo), fma2(dh, ch, mul2(dh, pk(-c_hi)))));
        const u64 tn = fma2(dh, ch, pk(kRound));
        const u64 r = sub2(p, add2(tn, pk(-kRound)));
        const float L_hi = 0.693147182464599609375f, L_lo = -1.904654299957768e-09f;   // ln 2
        const u64 q = mul2(r, pk(L_hi));
        const u64 q_lo = fma2(r, pk(L_lo), fma2(r, pk(L_hi), mul2(r, pk(-L_hi))));
        const u64 d = fma2(e, pk(L_hi), q_lo);
        const u64 h = fma2(fma2(q, pk(1.f / 24.f), pk(1.f / 6.f)), q, pk(0.5f));
        const u64 ex = fma2(fma2(q, pk(0.5f), pk(1.f)), q, pk(1.f));
        const u64 rest = fma2(mul2(h, q), q, mul2(d, ex));
        const float2 t = unpk(tn);
        return {__float_as_int(t.x) - __float_as_int(kRound), __float_as_int(t.y) - __float_as_int(kRound), unpk(p),
                unpk(q), unpk(rest)};
    }
    // q + rest in steps of 2^-34, or of 2^-32
    static __device__ __forceinline__ int frac(float q, float rest, float steps = 17179869184.f) {
        return __float2int_rn(q * steps) + __float2int_rn(rest * steps);
    }
    __device__ __forceinline__ u64 scaled(int i, float p, float q, float rest) const {
        const u64 t = tab[i & 31];
        const u64 w = t + (u64)((long long)(int)(t >> 34) * frac(q, rest));
        return p > (float)-SMP_ZERO ? w >> ((62 - SMP_FRAC - (i >> 5)) & 63) : 0;
    }
    __device__ __forceinline__ void fixed2(float l0, float l1, u64& w0, u64& w1) const {
        const Parts a = parts(l0, l1);
        w0 = scaled(a.i0, a.p.x, a.q.x, a.rest.x);
        w1 = scaled(a.i1, a.p.y, a.q.y, a.rest.y);
    }
    __device__ __forceinline__ u64 fixed(float l) const {
        u64 w0, w1;
        fixed2(l, l, w0, w1);
        return w0;
    }
    // The step of 1/32 that parts() takes, of two. One fused operation wherever a bin is worked out, so
    // that a token counted in a bin is ranked in it: a rounded product and a sum are one operation or two
    // as the compiler finds in each place, and a token within 2^-23 of a border fell into two bins.
    __device__ __forceinline__ u64 step(float l0, float l1) const {
        return fma2(add2(pk(l0, l1), pk(-M)), pk(c_hi), pk(kRound));
    }
    // Which step of 1/32 of the exponent: bins that ascend as the logit falls
    // (far from M the integer is no multiple of anything, but larger all the same)
    static __device__ __forceinline__ int bin(int i) { return (int)min((unsigned)-i, (unsigned)SMP_BINS - 1u); }
    __device__ __forceinline__ int bin(float l) const {
        return bin(__float_as_int(__fmaf_rn(__fadd_rn(l, -M), c_hi, kRound)) - __float_as_int(kRound));
    }
    // The mass of a bin whose tokens' 1 + q + rest sum to s 2^-32
    __device__ __forceinline__ u64 mass(int b, u64 s) const {
        if (b > 32 * SMP_ZERO) return 0;
        const u64 t = tab[-b & 31], hi = __umul64hi(t, s << 13), lo = t * (s << 13);   // in 2^-43, 2^-107
        return (hi << (SMP_FRAC - 43) | lo >> (64 - (SMP_FRAC - 43))) >> ((b + 31) >> 5);
    }
};
// fp32 of it, for probabilities
__device__ __forceinline__ float real_weight(int i, float p, float q, float rest, const float2* pow2) {
    const float2 t = pow2[i & 31];
    const float w = t.x + fmaf(t.x, q + rest, t.y);
    return p > (float)-SMP_ZERO ? w * __int_as_float((127 + (i >> 5)) << 23) : 0.f;
}

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
    uint32_t count;        // at most so many
    u64 above, prefix;     // above: count or mass of what precedes
};

// =========================================================================================
template <typename T, int THREADS, bool CLUSTER>
__global__ void __launch_bounds__(THREADS, THREADS == 512 ? 2 : 1) sample_kernel(SampleArgs a) {
    constexpr int VEC = 16 / sizeof(T);
    constexpr int BPT = SMP_BINS / THREADS;     // bins a thread sums when the CTA is alone
    extern __shared__ __align__(16) uint8_t smem[];
    float* l_s = reinterpret_cast<float*>(smem);
    // [2][BINS]: count, or sum of mantissas (low 16 bits, high 17 bits: 32776 slots stay below 2^32)
    uint32_t* hist = reinterpret_cast<uint32_t*>(smem + (size_t)a.slice * 4);
    // after a search: what the row's first CTA ranks, with its weights; and before these are
    // worked out, what each CTA found of it, after that two lists of places
    u64* list_o = reinterpret_cast<u64*>(hist);                                 // [CAP]
    u64* list_w = list_o + SMP_CAP;                                             // [CAP]
    u64* own_o = CLUSTER ? list_w : list_o;                                     // [CAP]
    uint16_t* places = reinterpret_cast<uint16_t*>(list_w + SMP_CAP);           // [2][CAP]
    // after the cut: 192 kept logits a warp
    float* queue = reinterpret_cast<float*>(hist) + (threadIdx.x >> 5) * 192;
    static_assert(THREADS / 32 * 192 * 4 <= SMP_AREA && SMP_BINS * 8 <= SMP_AREA, "shared memory behind the logits");
    __shared__ float2 pow2[32];
    __shared__ u64 tab[32];
    __shared__ u64 red[THREADS / 32];
    __shared__ u64 warp_mass[THREADS / 32];
    __shared__ float x_max[SMP_MAX_CS];
    __shared__ u64 x_cnt[SMP_MAX_CS], x_sum[SMP_MAX_CS], x_arg[SMP_MAX_CS];
    __shared__ u64 f_above, f_cut, last_o;
    __shared__ u64 piv_o[THREADS / 32], piv_w[THREADS / 32];
    __shared__ int piv_c[THREADS / 32];
    __shared__ uint32_t piv_n;
    __shared__ uint32_t f_bin, f_count, list_n[2], own_n[2], own_at;
    __shared__ int last_kept;
    __shared__ struct {
        u64 p64, u64_, mp;
        float c_hi, c_lo, temp;
        int k, greedy, need_p;
    } par;

    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t cs = CLUSTER ? cluster_size() : 1u, rank = CLUSTER ? cluster_rank() : 0u;
    const int row = blockIdx.x / cs;
    if (tid < 32) {
        const float2 t = kPow2[tid];
        pow2[tid] = t;
        tab[tid] = (u64)(__float2ll_rn(t.x * 4611686018427387904.f) + __float2ll_rn(t.y * 4611686018427387904.f));
    }
    if (tid < 2) list_n[tid] = own_n[tid] = 0;
    // peers may write here once every CTA of the cluster runs: arrive now, wait before the first
    if constexpr (CLUSTER) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    pdl_wait();

    // ---- parameters of the row, by one thread: loaded here, worked out while the row arrives
    float temp = 1.f, p_in = 1.f, mp_in = 0.f, u_in = 0.f;
    int top_k = 0;
    if (tid == 0) {
        if (a.temperature) temp = a.temperature[row];
        if (a.top_k) top_k = a.top_k[row];
        if (a.top_p) p_in = a.top_p[row];
        if (a.min_p) mp_in = a.min_p[row];
        u_in = a.uniforms[row];
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
    if (tid == 0) {
        const bool greedy = !(temp > 0.f);
        // log2(e) / T, the quotient's remainder by a fused multiply-add
        const float L2E = 1.44269502162933349609375f, L2E_lo = 1.9259629911266175e-8f, t = greedy ? 1.f : temp;
        const float c = L2E / t, left = fmaf(-c, t, L2E) + L2E_lo;
        par.c_hi = fminf(fmaxf(c, 1.4e-45f), FLT_MAX);   // finite, and no 0 to meet an infinite difference
        par.c_lo = c <= FLT_MAX && isfinite(left) ? left / t : 0.f;
        par.temp = t;
        par.greedy = greedy;
        par.k = !greedy && top_k > 0 && top_k < a.V ? top_k : 0;
        par.need_p = !greedy && p_in < 1.f;
        par.p64 = unit_fixed(p_in, 64, false, ~0ull);
        par.u64_ = unit_fixed(u_in, 64, false, ~0ull);
        par.mp = greedy ? 0 : unit_fixed(mp_in, SMP_FRAC, true, 1ull << SMP_FRAC);
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
    if (mx == INFINITY) {                        // the infinite ones share the mass
        for (int s = tid; s < n; s += THREADS) l_s[s] = l_s[s] == INFINITY ? 0.f : -INFINITY;
        mx = 0.f;
        __syncthreads();
    }
    const WeightFn wf{mx, par.c_hi, par.c_lo, tab};      // written before the barriers of the maximum
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
        return;
    }

    // Kept (before min-p): logits above cut_l, and of that value ids up to cut_id
    float cut_l = -INFINITY;
    int cut_id = INT_MIN;
    auto set_cut = [&](u64 c) {
        cut_l = logit_of(c);
        cut_id = (1 << SMP_IDBITS) - 1 - (int)(c & ((1ull << SMP_IDBITS) - 1));
    };
    auto above_cut = [&](float l, int id) -> bool { return l > cut_l || (l == cut_l && id <= cut_id); };
    auto in_found = [&](const Found& f, int bin, u64 o) -> bool {
        return bin == f.bin0 && (f.shift == SMP_ORDER_BITS || (o >> f.shift) == f.prefix);
    };
    // The set of at most CAP tokens (or the single one) where the cumulative count reaches k
    // (k > 0), or the cumulative mass of the tokens above the cut so far reaches
    // x = ceil(p64 * their mass). Level 0 bins by the weight's exponent, later levels by a digit of the
    // order. bin0 is BINS where fewer than k tokens are left. Uniform over the cluster.
    // Masses are rounded down, so those of a bin's digits may fall short of the bin's own, and a cut
    // in between would have no digit. Digits are therefore summed as mantissas, which add exactly, and
    // a mass is formed of all of the bin up to a digit: the last digit reaches what the bin does.
    auto search = [&](uint32_t k, u64 p64, u64& x) -> Found {
        Found f{SMP_BINS, SMP_ORDER_BITS, 0, 0, 0};
        u64 bin_above = 0, part = 0;              // mass before bin0; mantissas of bin0 before the digit
        for (int level = 0;; ++level) {
            const int to = max(0, f.shift - SMP_DIGIT), width = f.shift - to;   // this level's digit
            for (int i = tid; i < (k ? 1 : 2) * SMP_BINS; i += THREADS) hist[i] = 0;
            __syncthreads();
            if (tid == 0) f_bin = SMP_BINS;      // read by all before that barrier, written next after another
            for (int s = 4 * tid; s < n; s += 4 * THREADS) {
                const float4 l4 = *reinterpret_cast<const float4*>(l_s + s);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float l0 = h ? l4.z : l4.x, l1 = h ? l4.w : l4.y;
                    const bool in0 = above_cut(l0, base + s + 2 * h), in1 = above_cut(l1, base + s + 2 * h + 1);
                    if (!in0 && !in1) continue;
                    auto place = [&](float l, int id, int bin) -> int {       // -1: not in the set
                        if (level == 0) return bin;
                        const u64 o = order_of(l, id);
                        if (!in_found(f, bin, o)) return -1;
                        // digits descend, so that a lower bin is earlier in the order
                        return (1 << width) - 1 - (int)((o >> to) & ((1ull << width) - 1));
                    };
                    if (k) {
                        const int b0 = in0 ? place(l0, base + s + 2 * h, wf.bin(l0)) : -1;
                        const int b1 = in1 ? place(l1, base + s + 2 * h + 1, wf.bin(l1)) : -1;
                        if (b0 >= 0) atomicAdd(&hist[b0], 1u);
                        if (b1 >= 0) atomicAdd(&hist[b1], 1u);
                    } else {
                        const Parts w = wf.parts(l0, l1);
                        auto add = [&](int b, float p, float q, float rest) {
                            if (!(p > (float)-SMP_ZERO)) return;
                            const int x = WeightFn::frac(q, rest, 4294967296.f);
                            atomicAdd(&hist[b], (uint32_t)x & 0xffffu);
                            atomicAdd(&hist[SMP_BINS + b], (uint32_t)((x >> 16) + 65536));
                        };
                        const int b0 = in0 ? place(l0, base + s + 2 * h, wf.bin(w.i0)) : -1;
                        const int b1 = in1 ? place(l1, base + s + 2 * h + 1, wf.bin(w.i1)) : -1;
                        if (b0 >= 0) add(b0, w.p.x, w.q.x, w.rest.x);
                        if (b1 >= 0) add(b1, w.p.y, w.q.y, w.rest.y);
                    }
                }
            }
            sync_all<CLUSTER>();
            // this CTA's share of the bins, summed over the cluster; a thread takes PT in a row
            const int nb = SMP_BINS / cs, b_lo = nb * rank, PT = (nb + THREADS - 1) / THREADS;
            u64 sum[BPT], cnt[BPT], tc = 0;       // of counts, masses or mantissas
#pragma unroll
            for (int i = 0; i < BPT; ++i) {
                cnt[i] = sum[i] = 0;
                if (i < PT && tid * PT + i < nb) {
                    const int b = b_lo + tid * PT + i;
                    for (uint32_t r = 0; r < cs; ++r) {
                        auto at = [&](int plane) -> uint32_t {
                            if constexpr (CLUSTER) return ld_peer_u32(map_peer(smem_u32(&hist[plane * SMP_BINS + b]), r));
                            else return hist[plane * SMP_BINS + b];
                        };
                        sum[i] += at(0);
                        if (k == 0) sum[i] += (u64)at(1) << 16;
                    }
                    cnt[i] = sum[i];
                    if (k == 0) {
                        // |q + rest| < 0.011: at most this many tokens
                        cnt[i] = (sum[i] >> 32) + (sum[i] >> 38) + 1;
                        if (level == 0) sum[i] = wf.mass(b, sum[i]);
                    }
                }
                tc += sum[i];
            }
            u64 all;
            u64 before = block_scan_u64<THREADS>(tc, red, all);
            if constexpr (CLUSTER) {
                if (tid < (int)cs) st_peer_u64(map_peer(smem_u32(&x_cnt[rank]), tid), all);
                cluster_sync();
                all = 0;
                for (uint32_t i = 0; i < cs; ++i) {
                    if (i < rank) before += x_cnt[i];
                    all += x_cnt[i];
                }
            }
            if (level == 0 && k == 0) {           // mass before a kept token < p * total
                x = __umul64hi(p64, all) + ((p64 * all) != 0 ? 1 : 0);
                if (x == 0) x = 1;                // the first token is always kept
            }
            const bool parts = k == 0 && level > 0;
            before += parts ? part : f.above;
            const u64 goal = k ? k : x;
            auto reach = [&](u64 v) -> u64 { return parts ? bin_above + wf.mass(f.bin0, v) : v; };
#pragma unroll
            for (int i = 0; i < BPT; ++i) {
                if (sum[i] && reach(before) < goal && reach(before + sum[i]) >= goal) {
                    const uint32_t bin = b_lo + tid * PT + i;
                    for (uint32_t r = 0; r < cs; ++r) {
                        if constexpr (CLUSTER) {
                            st_peer_u32(map_peer(smem_u32(&f_bin), r), bin);
                            st_peer_u32(map_peer(smem_u32(&f_count), r), (uint32_t)cnt[i]);
                            st_peer_u64(map_peer(smem_u32(&f_above), r), before);
                        } else {
                            f_bin = bin;
                            f_count = (uint32_t)cnt[i];
                            f_above = before;
                        }
                    }
                }
                before += sum[i];
            }
            sync_all<CLUSTER>();
            if (f_bin == SMP_BINS) return f;
            f.count = f_count;
            part = parts ? f_above : 0;
            f.above = reach(f_above);
            if (level == 0) {
                bin_above = f.above;
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
    // Ranks the gathered tokens (first CTA) and returns the order of the last one kept: the first
    // k overall (k > 0), and with do_p of these the nucleus of mass x, or where x is 0 of
    // ceil(p64 * mass of the k). above_*: what precedes all of them.
    auto finish = [&](u64 above_count, u64 above_mass, u64 k, bool do_p, u64 p64, u64 x) -> u64 {
        sync_all<CLUSTER>();                      // every CTA's entries have arrived
        if (rank == 0) {
            const int m = min((int)list_n[list_at], SMP_CAP);
            for (int e = tid; e < m; e += THREADS) list_w[e] = wf.fixed(logit_of(list_o[e]));
            auto nucleus = [&](u64 mine) {        // mass wanted of these and what precedes them
                u64 total;
                block_scan_u64<THREADS>(mine, red, total);
                total += above_mass;
                x = __umul64hi(p64, total) + ((p64 * total) != 0 ? 1 : 0);
                if (x == 0) x = 1;
            };
            // The last entry that has fewer than k - above_count before it (k > 0) and less mass than
            // x - above_mass (with_p). While more than FEW may be it, each warp weighs one of them
            // against the others, and what lies between two of those goes on.
            auto last = [&](u64 k, bool with_p) -> u64 {
                u64 before_c = above_count, before_m = above_mass;
                int left = m, at = 0;
                for (int e = tid; e < m; e += THREADS) places[e] = (uint16_t)e;
                __syncthreads();
                while (left > SMP_FEW) {
                    const uint16_t* from = places + at * SMP_CAP;
                    uint16_t* onto = places + (at ^ 1) * SMP_CAP;
                    const int pivot = from[(int)((long long)left * warp / (THREADS / 32))];
                    const u64 o = list_o[pivot];
                    int c = 0;
                    u64 w = 0;
#pragma unroll 4
                    for (int e = lane; e < left; e += 32) {
                        const int i = from[e];
                        const u64 y = list_w[i];
                        const bool earlier = list_o[i] > o;
                        c += earlier;
                        w += earlier ? y : 0;
                    }
                    c = __reduce_add_sync(0xffffffffu, c);
                    w = warp_sum_u64(w);
                    if (lane == 0) {
                        piv_o[warp] = o;
                        piv_c[warp] = c;
                        piv_w[warp] = w;
                    }
                    if (tid == 0) piv_n = 0;
                    __syncthreads();
                    // the last one known to stay, the first one known to go
                    const int y = lane % (THREADS / 32);
                    const u64 py = piv_o[y], wy = piv_w[y];
                    const int cy = piv_c[y];
                    const bool stays = (k == 0 || before_c + cy < k) && (!with_p || before_m + wy < x);
                    const int hi_c = __reduce_max_sync(0xffffffffu, stays ? cy : -1);
                    const int lo_c = __reduce_min_sync(0xffffffffu, stays ? INT_MAX : cy);
                    const unsigned is_hi = __ballot_sync(0xffffffffu, cy == hi_c), is_lo = __ballot_sync(0xffffffffu, cy == lo_c);
                    u64 hi = ~0ull, lo = 0;
                    if (is_lo) lo = __shfl_sync(0xffffffffu, py, __ffs(is_lo) - 1);
                    if (is_hi) {
                        hi = __shfl_sync(0xffffffffu, py, __ffs(is_hi) - 1);
                        before_c += hi_c;
                        before_m += __shfl_sync(0xffffffffu, wy, __ffs(is_hi) - 1);
                    }
                    for (int e0 = 0; e0 < left; e0 += THREADS) {
                        const int e = e0 + tid;
                        const int i = e < left ? from[e] : 0;
                        const bool goes_on = e < left && list_o[i] > lo && list_o[i] <= hi;
                        const unsigned who = __ballot_sync(0xffffffffu, goes_on);
                        uint32_t to = 0;
                        if (lane == 0 && who) to = atomicAdd(&piv_n, (uint32_t)__popc(who));
                        to = __shfl_sync(0xffffffffu, to, 0) + __popc(who & ((1u << lane) - 1));
                        if (goes_on) onto[to] = (uint16_t)i;
                    }
                    __syncthreads();
                    left = piv_n;
                    at ^= 1;
                    __syncthreads();
                }
                // 2^g lanes compare an entry with all others
                const int g = min(5, __clz(max(left - 1, 1)) - __clz(THREADS) - 1), G = 1 << g;
                const uint16_t* from = places + at * SMP_CAP;
                const int e = tid >> g, sub = tid & (G - 1);
                const int own = e < left ? from[e] : 0;
                const u64 own_w = list_w[own];
                const u64 o = e < left ? list_o[own] : ~0ull;
                int c = 0;
                u64 w = 0;
#pragma unroll 4
                for (int j = sub; j < left; j += G) {
                    const int i = from[j];
                    const u64 y = list_w[i];
                    const bool earlier = list_o[i] > o;
                    c += earlier;
                    w += earlier ? y : 0;
                }
                for (int d = 1; d < G; d *= 2) {
                    c += __shfl_xor_sync(0xffffffffu, c, d);
                    w += __shfl_xor_sync(0xffffffffu, w, d);
                }
                const bool in_k = e < left && (k == 0 || before_c + c < k);
                if (with_p && x == 0) nucleus(in_k && sub == 0 ? own_w : 0);
                if (tid == 0) last_kept = 0;
                __syncthreads();
                const bool stays = in_k && (!with_p || before_m + w < x);
                const int to = __reduce_max_sync(0xffffffffu, stays ? c : 0);
                if (lane == 0 && to > 0) atomicMax(&last_kept, to);
                __syncthreads();
                if (e < left && c == last_kept && sub == 0) last_o = o;
                __syncthreads();
                return last_o;
            };
            if (do_p && x == 0 && m > SMP_FEW) {
                const u64 c = last(k, false);
                u64 mine = 0;
                for (int e = tid; e < m; e += THREADS) mine += list_o[e] >= c ? list_w[e] : 0;
                nucleus(mine);
                k = 0;                            // what follows the k-th has x or more before it
            }
            const u64 c = last(k, do_p);
            if (tid < (int)cs) {
                if constexpr (CLUSTER) st_peer_u64(map_peer(smem_u32(&f_cut), tid), c);
                else f_cut = c;
            }
        }
        sync_all<CLUSTER>();
        ++list_at;                                // a second list counts anew
        return f_cut;
    };
    // Collects the orders of the tokens that `take` names, a warp's share by one counter update, and
    // in a cluster a CTA's share by one more.
    auto gather = [&](int first_bin, int last_bin, auto take) {
        const float highest = kRound - (float)first_bin * 0.03125f;
        const float lowest = last_bin < SMP_BINS - 1 ? kRound - (float)last_bin * 0.03125f : -INFINITY;
        uint32_t* count = CLUSTER ? &own_n[list_at] : &list_n[list_at];
        for (int s0 = 0; s0 < n; s0 += 4 * THREADS) {
            const int s = s0 + 4 * tid;
            const float4 l4 = s < n ? *reinterpret_cast<const float4*>(l_s + s)
                                    : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            const float l[4] = {l4.x, l4.y, l4.z, l4.w};
            // what WeightFn::bin rounds, two at a time
            const float2 a01 = unpk(wf.step(l4.x, l4.y)), a23 = unpk(wf.step(l4.z, l4.w));
            const float at_step[4] = {a01.x, a01.y, a23.x, a23.y};
            bool yes[4], mine = false;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                yes[j] = at_step[j] >= lowest && at_step[j] <= highest && l[j] > -INFINITY && take(l[j], base + s + j);
                mine |= yes[j];
            }
            if (!__any_sync(0xffffffffu, mine)) continue;
            uint32_t off[4], all = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const unsigned who = __ballot_sync(0xffffffffu, yes[j]);
                off[j] = all + __popc(who & ((1u << lane) - 1));
                all += __popc(who);
            }
            uint32_t at = 0;
            if (lane == 0) at = atomicAdd(count, all);
            at = __shfl_sync(0xffffffffu, at, 0);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (yes[j] && at + off[j] < SMP_CAP) own_o[at + off[j]] = order_of(l[j], base + s + j);
        }
        if constexpr (CLUSTER) {
            __syncthreads();
            const int m = min((int)*count, SMP_CAP);
            if (tid == 0) own_at = m ? atom_peer_add(map_peer(smem_u32(&list_n[list_at]), 0), m) : 0;
            __syncthreads();
            const uint32_t at = own_at;
            for (int e = tid; e < m; e += THREADS)
                if (at + e < SMP_CAP) st_peer_u64(map_peer(smem_u32(&list_o[at + e]), 0), own_o[e]);
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
        if (need_k) {
            // the whole top-k as one list where it fits, else only the set that holds its end
            const Found f = search((uint32_t)k_in, 0, x);
            if (f.bin0 < SMP_BINS) {
                const bool all = f.shift == SMP_ORDER_BITS && f.above + f.count <= SMP_CAP;
                gather(all ? 0 : f.bin0, f.bin0, [&](float l, int id) { return all || in_found(f, f.bin0, order_of(l, id)); });
                set_cut(finish(all ? 0 : f.above, 0, (uint32_t)k_in, need_p && all, p64, 0));
                if (all) p_left = false;
            }
        }
        if (p_left) {
            const Found f = search(0, p64, x);
            gather(f.bin0, f.bin0, [&](float l, int id) { return above_cut(l, id) && in_found(f, f.bin0, order_of(l, id)); });
            set_cut(finish(0, f.above, 0, true, p64, x));
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
    const int seg = (n + 4 * THREADS - 1) / (4 * THREADS) * 128;
    {
        // Few tokens stay of many and they lie apart: a warp queues them and weighs 64 at a time
        u64 m = 0;
        int held = 0;
        auto weigh = [&](int first) {
            __syncwarp();
            const int e = first + lane;
            u64 w0, w1;
            wf.fixed2(e < held ? queue[e] : -INFINITY, e + 32 < held ? queue[e + 32] : -INFINITY, w0, w1);
            m += (w0 >= mp ? w0 : 0) + (w1 >= mp ? w1 : 0);
            __syncwarp();
        };
        const int hi = min(n, (warp + 1) * seg);
        for (int s0 = warp * seg; s0 < hi; s0 += 128) {
            const int s = s0 + 4 * lane;
            const float4 l4 = s < hi ? *reinterpret_cast<const float4*>(l_s + s)
                                     : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            const float l[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool yes = above_cut(l[j], base + s + j);
                const unsigned who = __ballot_sync(0xffffffffu, yes);
                if (yes) queue[held + __popc(who & ((1u << lane) - 1))] = l[j];
                held += __popc(who);
            }
            for (; held >= 64; held -= 64) weigh(held - 64);
        }
        if (held > 0) weigh(0);
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
        // the first warp whose tokens reach past it
        const u64 in_warp = lane < THREADS / 32 ? warp_mass[lane] : 0;
        u64 upto = in_warp;
#pragma unroll
        for (int o = 1; o < THREADS / 32; o *= 2) {
            const u64 y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        const int pick_warp = __ffs(__ballot_sync(0xffffffffu, lane < THREADS / 32 && before + upto > thr)) - 1;
        const u64 pick_before = before + __shfl_sync(0xffffffffu, upto - in_warp, pick_warp);
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
                const float lt = total < 2 * one ? log1pf((float)(total - one) * 2.842170943040401e-14f)   // 2^-45
                                                 : logf((float)total * 2.842170943040401e-14f);
                a.logprob[row] = lw - lt;
            }
        }
    }
    if (a.probs) {
        const float inv = (float)(1ull << SMP_FRAC) / (float)total;
        float* pr = a.probs + (size_t)row * a.ldp;
        const bool wide = (uintptr_t)(pr + base) % 16 == 0;
        for (int s = 4 * tid; s < n; s += 4 * THREADS) {
            const float4 l4 = *reinterpret_cast<const float4*>(l_s + s);
            const float l[4] = {l4.x, l4.y, l4.z, l4.w};
            const int id = base + s;
            bool in[4];
            float p[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < 4; ++j) in[j] = above_cut(l[j], id + j);
            if (in[0] || in[1] || in[2] || in[3]) {
#pragma unroll
                for (int j = 0; j < 4; j += 2) {
                    const Parts w = wf.parts(l[j], l[j + 1]);
                    if (in[j] && (mp == 0 || wf.scaled(w.i0, w.p.x, w.q.x, w.rest.x) >= mp))
                        p[j] = real_weight(w.i0, w.p.x, w.q.x, w.rest.x, pow2) * inv;
                    if (in[j + 1] && (mp == 0 || wf.scaled(w.i1, w.p.y, w.q.y, w.rest.y) >= mp))
                        p[j + 1] = real_weight(w.i1, w.p.y, w.q.y, w.rest.y, pow2) * inv;
                }
            }
            if (wide && id >= 0 && id + 4 <= a.V) {
                *reinterpret_cast<float4*>(pr + id) = make_float4(p[0], p[1], p[2], p[3]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (id + j >= 0 && id + j < a.V) pr[id + j] = p[j];
            }
        }
    }
}

// Cluster size: slices of at most 16384 slots (64 KiB, so that two CTAs share an SM), then more
// CTAs a row while the rows alone leave SMs idle and the row is long enough to repay the cluster's
// barriers, about 3 us. Measured with top-k and top-p: 1 x 32000 23, 19, 15, 13.5 us with 1, 2, 4, 8
// CTAs; 1 x 8192 11.4, 13.2, 12.2, 12.3; 100 x 8192 13.2 with one, 17.1 with two. No further than 256
// CTAs: clusters of eight do not fill every SM twice (38 x 50021 takes 22 us with 152, 30 with 304).
int sample_cluster(int rows, int V) {
    int cs = 1;
    while (cs < SMP_MAX_CS && V > cs * 16384) cs *= 2;
    while (cs < SMP_MAX_CS && (long long)rows * cs * 2 <= 256 && V > cs * 4096 + 8192) cs *= 2;
    return cs;
}

template <typename T, int THREADS, bool CLUSTER>
cudaError_t sample_launch(const SampleArgs& a, int rows, int cs, size_t smem, cudaStream_t stream) {
    auto kernel = sample_kernel<T, THREADS, CLUSTER>;
    if (smem > SMP_MAX_SMEM) return cudaErrorInvalidValue;
    if (smem > 40 * 1024) {   // with the kernel's own 2 KB above the 48 KB that need no asking
        // the same limit in every call: one of this call's own would be lowered by another thread's smaller
        // call between here and the launch
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMP_MAX_SMEM);
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
    const size_t smem = (size_t)a.slice * 4 + SMP_AREA;
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
    return status_of(launch_sample(*c, (cudaStream_t)stream));
}
