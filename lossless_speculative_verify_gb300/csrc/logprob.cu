// Log probabilities of given tokens, with the row's entropy and its largest tokens
// (evs_token_logprobs).
//
//   y_i = (l_i - max l) / T,  Z = sum e^y_i:  log p(t) = y_t - log Z,
//   entropy = -sum p log p = log Z - sum (e^y_i y_i) / Z.
//
// One pass over the row: each thread keeps the running maximum m of what it has seen, s = sum e^y and
// w = sum e^y (l - m), rescaled when m grows; a row's threads (and the CTAs of a cluster, where there are
// too few rows for the GPU) join theirs at the end.
//
// The largest K tokens, in the order (logit descending, id ascending): K threads' own maxima reach a border
// that the K-th largest token reaches, too, and a token that does is one of a thread whose maximum does. So
// only those threads' tokens (K / 256 of the row, from L2) are read a second time, and the few that reach the
// border (its leading bits, found by counting) are ranked by one warp in registers. Where more than 256 do,
// as among equal logits, every warp keeps a sorted list and the lists are joined (512 x 131072 of zeros: 330 us). No order of execution shows.
//
// Measured (replayed graphs): 13 x 512 fp32 2.2 us, 208 x 4096 with eight alternatives 6.8, 64 x 50021 bf16 with
// 20 10.8, 512 x 131072 fp32 with five 56 (4.8 TB/s; the row's passage is 40 at the rate of a copy, the uneven last
// place on an SM a fifth of it, start and ranking about 10).
#include "evs_common.cuh"
#include "sm100_ptx.cuh"

#include <cfloat>

namespace evs {
namespace {

using bf16 = __nv_bfloat16;
typedef unsigned long long u64;

constexpr int LP_MAX_CS = 8;             // portable cluster size
constexpr int LP_MAX_TOP = 64;
constexpr uint32_t FULL = 0xffffffffu;
constexpr float LP_LOG2E = 1.44269502162933349609375f, LP_LOG2E_REST = 1.9259629911e-8f;
constexpr int LP_FOUND = 256;            // tokens that one warp ranks
constexpr int LP_BORDER_BIT = 14;        // the border's sign, exponent and nine bits of its mantissa

struct LogprobArgs {
    const void* logits;
    int64_t ld;
    int V, n, K;
    const float* temperature;
    const int32_t* tokens;
    float *logprob, *entropy, *top_logprob;
    int32_t* top_token;
    uint32_t* flags;
};

// A logit's bits as an ascending integer; NaN and -inf, which are ruled out, are the lowest.
constexpr uint32_t LP_RULED_OUT = 0x007fffffu;         // of -inf
__device__ __forceinline__ uint32_t lp_order(float l) {
    const uint32_t k = __float_as_uint(fmaxf(l, -INFINITY) + 0.f);   // NaN: -inf; -0 and +0 are one value
    return (k & 0x80000000u) ? ~k : (k | 0x80000000u);
}
__device__ __forceinline__ float lp_of_order(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
// Position in the order: larger is earlier, 0 is no token.
__device__ __forceinline__ u64 lp_key(float l, int id) {
    const uint32_t k = lp_order(l);
    return k <= LP_RULED_OUT ? 0 : ((u64)k << 32) | (u64)(0xffffffffu - (uint32_t)id);
}
__device__ __forceinline__ float lp_value(u64 key) { return lp_of_order((uint32_t)(key >> 32)); }
__device__ __forceinline__ int lp_id(u64 key) { return (int)(0xffffffffu - (uint32_t)key); }

__device__ __forceinline__ u64 lp_max(u64 a, u64 b) { return a > b ? a : b; }
__device__ __forceinline__ u64 lp_min(u64 a, u64 b) { return a > b ? b : a; }

// A bitonic sequence over the lanes, sorted descending
__device__ __forceinline__ u64 lp_merge32(u64 v, int lane) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const u64 o = __shfl_xor_sync(FULL, v, d);
        v = (lane & d) ? lp_min(v, o) : lp_max(v, o);
    }
    return v;
}
__device__ __forceinline__ u64 lp_sort32(u64 v, int lane) {
#pragma unroll
    for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
        for (int d = k >> 1; d > 0; d >>= 1) {
            const u64 o = __shfl_xor_sync(FULL, v, d);
            v = (((lane & d) == 0) == ((lane & k) == 0)) ? lp_max(v, o) : lp_min(v, o);
        }
    return v;
}

// A warp's largest 32 L keys, descending: place 32 j + lane.
template <int L> struct WarpTop {
    u64 a[L];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int j = 0; j < L; ++j) a[j] = 0;
    }
    // 32 keys in descending order
    __device__ __forceinline__ void push_sorted(u64 b, int lane) {
#pragma unroll
        for (int j = L - 1; j >= 0; --j) {
            // the larger half of (a[j], b) stays, and goes on against the places before
            const u64 r = __shfl_xor_sync(FULL, b, 31);
            const u64 hi = lp_merge32(lp_max(a[j], r), lane);
            if (j + 1 < L) a[j + 1] = lp_merge32(lp_min(a[j], r), lane);
            b = hi;
        }
        a[0] = b;
    }
    // The smallest of them
    __device__ __forceinline__ u64 last() const { return __shfl_sync(FULL, a[L - 1], 31); }
    __device__ __forceinline__ void push(u64 b, int lane) { push_sorted(lp_sort32(b, lane), lane); }
};

// All warps' lists into warp 0's, by halves; lists: [WARPS / 2][32 L]. Ends with a barrier only
// between its steps: callers synchronise before lists is used again.
template <int L, int WARPS> __device__ __forceinline__ void join_warps(WarpTop<L>& top, u64* lists, int warp, int lane) {
#pragma unroll 1
    for (int half = WARPS / 2; half > 0; half >>= 1) {
        __syncthreads();
        if (warp >= half && warp < 2 * half) {
#pragma unroll
            for (int j = 0; j < L; ++j) lists[(warp - half) * 32 * L + j * 32 + lane] = top.a[j];
        }
        __syncthreads();
        if (warp < half) {
#pragma unroll
            for (int j = 0; j < L; ++j) top.push_sorted(lists[warp * 32 * L + j * 32 + lane], lane);
        }
    }
}

// Vectors of 16 bytes on their own grid: vector v holds the ids v E - off .. v E - off + E - 1, of which
// those outside the row are read as -inf.
template <typename T> struct Row {
    static constexpr int E = 16 / (int)sizeof(T);
    const T* base;                       // id 0
    int off, V;
    // vector v as it lies in memory
    __device__ __forceinline__ uint4 raw(int v) const {
        const int id0 = v * E - off;
        if (id0 >= 0 && id0 + E <= V) return __ldg(reinterpret_cast<const uint4*>(base + id0));
        alignas(16) T x[E];
#pragma unroll
        for (int j = 0; j < E; ++j) x[j] = (id0 + j >= 0 && id0 + j < V) ? base[id0 + j] : from_f32<T>(-INFINITY);
        return *reinterpret_cast<const uint4*>(x);
    }
    static __device__ __forceinline__ uint4 nothing() {
        const uint32_t w = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;
        return make_uint4(w, w, w, w);
    }
    static __device__ __forceinline__ void values(const uint4& u, float (&x)[E]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (sizeof(T) == 4) {
                x[j] = __uint_as_float(w[j]);
            } else {
                x[2 * j] = __uint_as_float(w[j] << 16);
                x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
            }
        }
    }
    __device__ __forceinline__ void load(int v, float (&x)[E]) const { values(raw(v), x); }
};

// (m, s, w) of two disjoint parts of a row; c: log2(e) / T in two parts
struct Stat {
    float m, s, w;
};
__device__ __forceinline__ float lp_exp(float x, float2 c) { return ex2_approx_ftz(fmaf(x, c.y, x * c.x)); }
__device__ __forceinline__ Stat join(Stat a, Stat b, float2 c) {
    Stat r;
    r.m = fmaxf(a.m, b.m);
    // -FLT_MAX: a part of ruled-out tokens, or one beside +inf, has no weight
    const float da = a.m == r.m ? 0.f : fmaxf(a.m - r.m, -FLT_MAX), db = b.m == r.m ? 0.f : fmaxf(b.m - r.m, -FLT_MAX);
    const float fa = lp_exp(da, c), fb = lp_exp(db, c);
    r.s = a.s * fa + b.s * fb;
    // a part's w moves by its shift; a part without weight has no shift worth the name
    r.w = (fa > 0.f ? fmaf(a.s, da, a.w) * fa : 0.f) + (fb > 0.f ? fmaf(b.s, db, b.w) * fb : 0.f);
    return r;
}

template <typename T, int L, int LP_THREADS>
__global__ void __launch_bounds__(LP_THREADS) logprob_kernel(LogprobArgs a) {
    constexpr int E = Row<T>::E, U = 4, LL = L ? L : 1, LP_WARPS = LP_THREADS / 32;
    __shared__ u64 lists[LP_WARPS / 2 * 32 * LL];
    __shared__ u64 parts[LP_MAX_CS * 32 * LL];           // of the cluster's CTAs, in its first
    __shared__ Stat part_stat[LP_MAX_CS];
    __shared__ uint32_t warp_keys[LP_WARPS], thread_keys[LP_THREADS], border_key;
    __shared__ float2 warp_sums[LP_WARPS];
    __shared__ u64 found[LP_FOUND];
    __shared__ int n_found;
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint32_t cs, rank;
    asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(cs));
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    // the first CTA's shared memory is written to below: not before it runs
    if (cs > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    const int64_t r = blockIdx.x / cs;
    Row<T> row;
    row.base = (const T*)a.logits + r * a.ld;
    row.V = a.V;
    row.off = (int)(((uintptr_t)row.base & 15) / sizeof(T));
    const int vectors = (a.V + row.off + E - 1) / E, per = (vectors + (int)cs - 1) / (int)cs;
    const int lo = min(vectors, per * (int)rank), hi = min(vectors, lo + per);

    const float t_in = a.temperature ? a.temperature[r] : 1.f;
    const bool greedy = !(t_in > 0.f);
    const float t = greedy ? 1.f : fminf(t_in, 1e30f);   // above: as 1e30, so that ruled-out tokens stay so
    // log2(e) / T rounded would move every exponent the same way: its remainder is kept (and that of log2(e) itself)
    float2 c;
    c.x = fminf(LP_LOG2E / t, FLT_MAX);
    c.y = c.x < FLT_MAX ? (fmaf(-c.x, t, LP_LOG2E) + LP_LOG2E_REST) / t : 0.f;

    // ---- the pass. A thread has up to 65536 tokens, and terms that are alike make every addition to a sum round the same
    // way (off by 8e-4 of the sum with 2^24 tokens a row, where a step of the result is 1e-6): so the U E tokens that it
    // works on at a time are added up by themselves, and their sum goes to s (w) with what the additions before lost
    // (sums of 32 bits compensated as Kahan described): 55.7 us for 54.7 (512 x 131072); the sums alone cost nothing, and
    // leave 2e-5.
    float m = -INFINITY, s = 0.f, w = 0.f, s_lost = 0.f, w_lost = 0.f;
    auto add_to = [](float& sum, float& lost, float x) {
        const float y = x - lost, t = sum + y;
        lost = (t - sum) - y;
        sum = t;
    };
    // U vectors at a time, the next ones on their way while these are worked on
    uint4 ahead[U];
    auto fetch = [&](int v0) {
#pragma unroll
        for (int u = 0; u < U; ++u) ahead[u] = v0 + u * LP_THREADS < hi ? row.raw(v0 + u * LP_THREADS) : Row<T>::nothing();
    };
    fetch(lo + tid);
    for (int v0 = lo + tid; v0 < hi; v0 += U * LP_THREADS) {
        uint4 now[U];
#pragma unroll
        for (int u = 0; u < U; ++u) now[u] = ahead[u];
        if (v0 + U * LP_THREADS < hi) fetch(v0 + U * LP_THREADS);
        float cm = -INFINITY;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float x[E];
            Row<T>::values(now[u], x);
#pragma unroll
            for (int j = 0; j < E; ++j) cm = fmaxf(cm, x[j]);
        }
        if (cm > m) {
            if (m > -INFINITY) {
                const float d = fmaxf(m - cm, -FLT_MAX), f = lp_exp(d, c);
                w = f > 0.f ? fmaf(s, d, w) * f : 0.f;
                w_lost = f > 0.f ? fmaf(s_lost, d, w_lost) * f : 0.f;
                s *= f;
                s_lost *= f;
            }
            m = cm;
        }
        float part_s = 0.f, part_w = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float x[E];
            Row<T>::values(now[u], x);
#pragma unroll
            for (int j = 0; j < E; ++j) {
                // -inf, NaN and what +inf leaves behind: no weight, and no NaN in w
                const float d = fmaxf(x[j] - m, -FLT_MAX), e = lp_exp(d, c);
                part_s += e;
                part_w = fmaf(e, d, part_w);
            }
        }
        add_to(s, s_lost, part_s);
        add_to(w, w_lost, part_w);
    }
    // ---- the row's statistics: the maximum of all, then every thread's sums moved to it once
    uint32_t key = lp_order(m);
    const uint32_t warp_key = __reduce_max_sync(FULL, key);
    if (lane == 0) warp_keys[warp] = warp_key;
    __syncthreads();
    uint32_t top_key = warp_keys[0];
#pragma unroll
    for (int i = 1; i < LP_WARPS; ++i) top_key = max(top_key, warp_keys[i]);
    Stat st;
    st.m = lp_of_order(top_key);
    {
        const Stat mine = join(Stat{m, s, w}, Stat{st.m, 0.f, 0.f}, c);
        const float ws = warp_sum(mine.s), ww = warp_sum(mine.w);
        if (lane == 0) warp_sums[warp] = make_float2(ws, ww);
    }
    __syncthreads();
    st.s = st.w = 0.f;
#pragma unroll
    for (int i = 0; i < LP_WARPS; ++i) {
        st.s += warp_sums[i].x;
        st.w += warp_sums[i].y;
    }
    if (st.m == INFINITY) {                              // the +inf tokens share the mass: count them
        float mine = 0.f;
        for (int v = lo + tid; v < hi; v += LP_THREADS) {
            float x[E];
            row.load(v, x);
#pragma unroll
            for (int j = 0; j < E; ++j) mine += x[j] == INFINITY ? 1.f : 0.f;
        }
        mine = warp_sum(mine);
        __syncthreads();
        if (lane == 0) warp_sums[warp].x = mine;
        __syncthreads();
        st.s = st.w = 0.f;
        for (int i = 0; i < LP_WARPS; ++i) st.s += warp_sums[i].x;
    }

    // ---- the largest tokens
    WarpTop<LL> top;
    top.clear();
    const bool keys = L > 0 || greedy;
    const int K = L > 0 ? a.K : 1;                       // greedy: the argmax
    if (keys) {
        thread_keys[tid] = key;
        if (tid == 0) n_found = 0;
        __syncthreads();
        if (warp == 0) {
            // a border that at least K threads' largest reach (if as many have any): its first bits, which is enough
            uint32_t mine[LP_WARPS], border = 0;
#pragma unroll
            for (int i = 0; i < LP_WARPS; ++i) mine[i] = thread_keys[i * 32 + lane];
#pragma unroll 1
            for (uint32_t bit = 1u << 31; bit >= 1u << LP_BORDER_BIT; bit >>= 1) {
                int n = 0;
#pragma unroll
                for (int i = 0; i < LP_WARPS; ++i) n += mine[i] >= (border | bit) ? 1 : 0;
                if (__reduce_add_sync(FULL, n) >= K) border |= bit;
            }
            if (lane == 0) border_key = max(border, LP_RULED_OUT + 1);
        }
        __syncthreads();
        const uint32_t border = border_key;
        // the tokens of the threads that reach it: a warp reads each such thread's vectors again
        auto each = [&](auto use) {
            for (uint32_t who = __ballot_sync(FULL, key >= border); who; who &= who - 1) {
                const int first = lo + warp * 32 + __ffs(who) - 1, count = (hi - first + LP_THREADS - 1) / LP_THREADS;
#pragma unroll 1
                for (int i0 = 0; i0 < count; i0 += 32) {
                    const int i = i0 + lane, v = first + i * LP_THREADS;
                    float x[E];
                    if (i < count) {
                        row.load(v, x);
                    } else {
#pragma unroll
                        for (int j = 0; j < E; ++j) x[j] = -INFINITY;
                    }
#pragma unroll
                    for (int j = 0; j < E; ++j) use(x[j], v * E - row.off + j);
                }
            }
        };
        each([&](float x, int id) {
            if (lp_order(x) < border) return;
            const int at = atomicAdd(&n_found, 1);
            if (at < LP_FOUND) found[at] = lp_key(x, id);
        });
        __syncthreads();
        if (n_found <= LP_FOUND) {
            if (warp == 0)
                for (int i = 0; i < n_found; i += 32) top.push(i + lane < n_found ? found[i + lane] : 0, lane);
        } else {
            // many equal or nearly equal tokens: every warp keeps a list, and they are joined
            each([&](float x, int id) {
                const u64 k = lp_order(x) < border ? 0 : lp_key(x, id);
                if (__any_sync(FULL, k > top.last())) top.push(k, lane);
            });
            join_warps<LL, LP_WARPS>(top, lists, warp, lane);
        }
    }

    // ---- the cluster's parts to its first CTA
    if (cs > 1) {
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (warp == 0) {
            if (keys) {
#pragma unroll
                for (int j = 0; j < LL; ++j) {
                    const uint32_t to = map_peer(smem_u32(&parts[rank * 32 * LL + j * 32 + lane]), 0);
                    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(to), "l"(top.a[j]) : "memory");
                }
            }
            if (lane == 0) {
                const uint32_t to = map_peer(smem_u32(&part_stat[rank]), 0);
                st_peer_f32(to, st.m);
                st_peer_f32(to + 4, st.s);
                st_peer_f32(to + 8, st.w);
            }
        }
        cluster_sync();
        if (rank != 0) return;
        st = part_stat[0];
        for (int i = 1; i < (int)cs; ++i) st = join(st, part_stat[i], c);
        if (keys && warp == 0) {
            for (int i = 1; i < (int)cs; ++i)
#pragma unroll
                for (int j = 0; j < LL; ++j) top.push_sorted(parts[i * 32 * LL + j * 32 + lane], lane);
        }
    }

    // ---- out
    const bool empty = st.m == -INFINITY;
    const float log_z = empty ? 0.f : logf(st.s);
    auto logprob = [&](float l) -> float {
        if (empty || !(l > -INFINITY)) return -INFINITY;
        if (l == st.m) return -log_z;                    // also +inf
        return st.m == INFINITY ? -INFINITY : (l - st.m) / t - log_z;
    };
    if (greedy && tid == 0) found[0] = top.a[0];
    __syncthreads();
    const int best = greedy ? lp_id(found[0]) : 0;       // -1 of an empty row is no token's id
    if (tid == 0) {
        if (a.entropy) a.entropy[r] = greedy || empty ? 0.f : st.m == INFINITY ? log_z : fmaxf(log_z - st.w / st.s / t, 0.f);
        if (empty && a.flags) atomicOr(a.flags, (uint32_t)EVS_FLAG_EMPTY_ROW);
    }
    for (int i = tid; i < a.n; i += LP_THREADS) {
        const int id = a.tokens[r * a.n + i];
        float lp = -INFINITY;
        if ((uint32_t)id >= (uint32_t)a.V) {
            if (a.flags) atomicOr(a.flags, (uint32_t)EVS_FLAG_BAD_TOKEN);
        } else if (greedy) {
            lp = id == best && !empty ? 0.f : -INFINITY;
        } else {
            lp = logprob(to_f32(row.base[id]));
        }
        a.logprob[r * a.n + i] = lp;
    }
    if (L > 0 && warp == 0) {
#pragma unroll
        for (int j = 0; j < LL; ++j) {
            const int at = j * 32 + lane;
            if (at >= a.K) continue;
            const u64 key = top.a[j];
            const float lp = key == 0 ? -INFINITY : greedy ? (at == 0 ? 0.f : -INFINITY) : logprob(lp_value(key));
            a.top_logprob[r * a.K + at] = lp;
            a.top_token[r * a.K + at] = key == 0 ? -1 : lp_id(key);
        }
    }
}

template <typename T, int L, int NT> cudaError_t launch_as(const evs_logprob_args& c, const LogprobArgs& a, int cs, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)c.rows * cs);
    cfg.blockDim = dim3(NT);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cs;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cs > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, logprob_kernel<T, L, NT>, a);
}
template <typename T, int L>
cudaError_t launch(const evs_logprob_args& c, const LogprobArgs& a, int nt, int cs, cudaStream_t stream) {
    return nt == 128 ? launch_as<T, L, 128>(c, a, cs, stream) : launch_as<T, L, 256>(c, a, cs, stream);
}

}  // namespace
}  // namespace evs

extern "C" evs_status evs_token_logprobs(const evs_logprob_args* c, void* stream) {
    using namespace evs;
    if (!c || c->rows < 0 || c->vocab < 1 || c->n_tokens < 0 || c->top < 0) return EVS_ERR_INVALID_ARG;
    if (c->rows > (1 << 24) || c->vocab > (1 << 24) || c->n_tokens > (1 << 20) || c->top > LP_MAX_TOP || c->top > c->vocab)
        return EVS_ERR_INVALID_ARG;
    if (c->dtype != EVS_DTYPE_F32 && c->dtype != EVS_DTYPE_BF16) return EVS_ERR_INVALID_ARG;
    if (c->rows == 0) return EVS_OK;
    const int es = c->dtype == EVS_DTYPE_F32 ? 4 : 2;
    if (!c->logits || (uintptr_t)c->logits % es || (c->rows > 1 && c->ld < c->vocab)) return EVS_ERR_INVALID_ARG;
    if (c->n_tokens > 0 && (!c->tokens || !c->logprob)) return EVS_ERR_INVALID_ARG;
    if (c->top > 0 && (!c->top_logprob || !c->top_token)) return EVS_ERR_INVALID_ARG;
    if (c->n_tokens == 0 && c->top == 0 && !c->entropy) return EVS_ERR_INVALID_ARG;
    LogprobArgs a{c->logits, c->ld, c->vocab, c->n_tokens, c->top, c->temperature, c->tokens, c->logprob, c->entropy,
                  c->top_logprob, c->top_token, c->flags};
    // CTAs of a row: two, four or eight where the rows leave SMs without any and a CTA's share stays some passes long,
    // or where rows of the largest vocabularies would make an uneven wave (64 x 50021 bf16: 10.7 us with two, 11.5
    // with one, 13.0 with four; 256 x 131072: 31 with two, 39 with one, 34 with four). A CTA has 128 threads for a short
    // share, whose time is the ranking's steps (4096 x 4096: 24 us, 256 threads 40), and 256 for a long one (512 x
    // 131072: 55, 128 threads 83).
    const long long rows = c->rows;
    int cs = 1;
    while (cs < LP_MAX_CS && ((2 * rows * cs <= 152 && c->vocab / (2 * cs) >= 8192) || (rows * cs < 304 && c->vocab / (2 * cs) >= 65536)))
        cs *= 2;
    const int nt = c->vocab / cs <= 8192 ? 128 : 256;
    const int lists = c->top == 0 ? 0 : c->top <= 32 ? 1 : 2;
    const cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
    if (c->dtype == EVS_DTYPE_F32)
        e = lists == 0 ? launch<float, 0>(*c, a, nt, cs, s) : lists == 1 ? launch<float, 1>(*c, a, nt, cs, s) : launch<float, 2>(*c, a, nt, cs, s);
    else
        e = lists == 0 ? launch<bf16, 0>(*c, a, nt, cs, s) : lists == 1 ? launch<bf16, 1>(*c, a, nt, cs, s) : launch<bf16, 2>(*c, a, nt, cs, s);
    return status_of(e);
}
