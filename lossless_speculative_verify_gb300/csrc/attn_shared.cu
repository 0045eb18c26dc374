// Attention for a batch whose sequences share a long prefix (evs_shared_attention): every query
// reads the shared rows, its sequence's own rows and the block rows of its candidate up to its
// own position. The shared rows are streamed once for all sequences: the queries of the whole
// batch that use a K/V head are the rows of one product.
//
//   o = sum_j exp(scale q.k_j - m) v_j / l over the three, lse = m + log l.
//
// Two launches: partial sums (o unnormalised, m, l) per run of keys, then a combine that merges
// a query's partials, adds its block rows and normalises.
#include "evs_common.cuh"
#include "sm100_ptx.cuh"

namespace evs {
namespace {

using bf16 = __nv_bfloat16;

// What both launches know. A partial of a shared row r of K/V head g (r = m * group + head in the
// group, m = (b * C + c) * T + i) lies in segment g * sh_tiles + r / sh_rows, row r % sh_rows; of
// an own row r = (c * T + i) * group + head in segment (b * G + g) * own_tiles + r / own_rows.
// Segments have `slots` partials of `rows` rows each.
struct SharedArgs {
    const void *q, *kp, *vp, *ko, *vo, *kb, *vb;
    void* o;
    float* lse;
    const int32_t* own_len;
    uint32_t* flags;
    int64_t q_ld, o_ld, p_row, p_head, o_row, o_head, o_seq, b_row, b_head, b_cand;
    int B, C, T, H, G, dh, P, own_max, own_skip, q_bf16;
    float scale;
    float *sh_o, *own_o;       // [segment][slot][rows][dh]
    float2 *sh_ml, *own_ml;    // [segment][slot][rows] (m, l), natural units
    int sh_rows, sh_tiles, sh_slots, own_rows, own_tiles, own_slots;
};

// fp32 problems keep the full precision of the exponential
template <typename T> __device__ __forceinline__ float exp_of(float x);
template <> __device__ __forceinline__ float exp_of<float>(float x) { return expf(x); }
template <> __device__ __forceinline__ float exp_of<bf16>(float x) { return __expf(x); }

// Own rows of sequence b, clamped to [0, own_max].
__device__ __forceinline__ int own_rows_of(const SharedArgs& a, int b, bool report) {
    if (!a.own_len) return 0;
    const int n = a.own_len[b] - a.own_skip;
    if (n < 0 || n > a.own_max) {
        if (report && a.flags) atomicOr(a.flags, (uint32_t)EVS_FLAG_BAD_LEN);
        return n < 0 ? 0 : a.own_max;
    }
    return n;
}

__device__ __forceinline__ float load_q(const SharedArgs& a, int64_t at) {
    return a.q_bf16 ? __bfloat162float(((const bf16*)a.q)[at]) : ((const float*)a.q)[at];
}

// =========================================================================================
// Partials on CUDA cores: fp32, narrow heads, and strides that tensor maps cannot describe.
// A CTA takes 16 rows of one segment and one slot's share of its keys, 64 keys at a time: scores
// to shared memory, one running maximum and sum per row, o in registers.
// =========================================================================================
constexpr int SA_Q = 16, SA_K = 64;

template <typename T>
__global__ void __launch_bounds__(256) shared_simt_kernel(SharedArgs a, int sh_items) {
    pdl_trigger();
    pdl_wait();
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
            v = load_q(a, m * a.q_ld + (int64_t)(g * grp + r % grp) * dh + c) * a.scale;
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
        const int64_t at = ((int64_t)seg * slots + slot) * rows + r;
        float* dst = (sh ? a.sh_o : a.own_o) + at * dh;
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (ocol + 16 * u < dh) dst[ocol + 16 * u] = o[u];
        if (ocol == 0) (sh ? a.sh_ml : a.own_ml)[at] = make_float2(row_m[orow], row_l[orow]);
    }
}

// =========================================================================================
// Combine: a warp per (query, head); lanes own dh / 32 consecutive columns (dh 16: 16 lanes one).
// =========================================================================================
template <typename T, int EPL>
__global__ void __launch_bounds__(128) shared_combine_kernel(SharedArgs a) {
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t id = (int64_t)blockIdx.x * 4 + warp;
    const int dh = a.dh, grp = a.H / a.G;
    if (id >= (int64_t)a.B * a.C * a.T * a.H) return;
    // id -> (b, c, g, i, head in group), so that the four warps of a CTA share block rows
    const int hg = (int)(id % grp), i = (int)(id / grp % a.T), g = (int)(id / grp / a.T % a.G);
    const int bc = (int)(id / grp / a.T / a.G), b = bc / a.C, c = bc % a.C;
    const int64_t m = (int64_t)bc * a.T + i;
    const int h = g * grp + hg;
    const int e0 = lane * EPL;
    const bool act = e0 < dh;
    float M = -INFINITY, L = 0.f, O[EPL];
#pragma unroll
    for (int u = 0; u < EPL; ++u) O[u] = 0.f;
    auto rebase = [&](float mb) {
        if (mb > M) {
            const float f = M == -INFINITY ? 0.f : exp_of<T>(M - mb);
            L *= f;
#pragma unroll
            for (int u = 0; u < EPL; ++u) O[u] *= f;
            M = mb;
        }
    };
    auto fold = [&](const float* po, const float2* pml, int64_t row, int64_t stride, int used) {
        constexpr int PB = 8;                      // partials in flight
        for (int s0 = 0; s0 < used; s0 += PB) {
            float2 ml[PB];
            float os[PB][EPL];
#pragma unroll
            for (int j = 0; j < PB; ++j) {
                const bool on = s0 + j < used;
                ml[j] = on ? pml[row + (s0 + j) * stride] : make_float2(-INFINITY, 0.f);
#pragma unroll
                for (int u = 0; u < EPL; ++u) os[j][u] = 0.f;
                if (on && act) {
                    const float* src = po + (row + (s0 + j) * stride) * dh + e0;
#pragma unroll
                    for (int u = 0; u < EPL; ++u) os[j][u] = src[u];
                }
            }
            float mb = -INFINITY;
#pragma unroll
            for (int j = 0; j < PB; ++j) mb = fmaxf(mb, ml[j].x);
            rebase(mb);
#pragma unroll
            for (int j = 0; j < PB; ++j) {
                // an empty partial leaves its o unwritten (one of NaN scores has l = NaN)
                if (ml[j].x == -INFINITY && ml[j].y == 0.f) continue;
                const float w = exp_of<T>(ml[j].x - M);
                L = fmaf(ml[j].y, w, L);
#pragma unroll
                for (int u = 0; u < EPL; ++u) O[u] = fmaf(os[j][u], w, O[u]);
            }
        }
    };
    const int r_sh = (int)(m * grp + hg), r_own = (c * a.T + i) * grp + hg;
    const int own = own_rows_of(a, b, false);
    if (a.P > 0) {
        const int64_t seg = (int64_t)g * a.sh_tiles + r_sh / a.sh_rows;
        fold(a.sh_o, a.sh_ml, seg * a.sh_slots * a.sh_rows + r_sh % a.sh_rows, a.sh_rows, a.sh_slots);
    }
    if (own > 0) {
        const int64_t seg = ((int64_t)b * a.G + g) * a.own_tiles + r_own / a.own_rows;
        fold(a.own_o, a.own_ml, seg * a.own_slots * a.own_rows + r_own % a.own_rows, a.own_rows, a.own_slots);
    }
    // block rows j <= i: of this candidate, or own rows own + j when the block is in the cache
    const T *kb, *vb;
    int64_t ld;
    int last = i;
    if (a.kb) {
        kb = (const T*)a.kb + bc * a.b_cand + g * a.b_head;
        vb = (const T*)a.vb + bc * a.b_cand + g * a.b_head;
        ld = a.b_row;
    } else {
        kb = (const T*)a.ko + b * a.o_seq + g * a.o_head + own * a.o_row;
        vb = (const T*)a.vo + b * a.o_seq + g * a.o_head + own * a.o_row;
        ld = a.o_row;
        if (own + i >= a.own_max) {                // rows past the capacity do not exist
            last = a.own_max - 1 - own;
            if (a.flags && lane == 0) atomicOr(a.flags, (uint32_t)EVS_FLAG_KV_OVERFLOW);
        }
    }
    float qv[EPL];
#pragma unroll
    for (int u = 0; u < EPL; ++u)
        qv[u] = act ? load_q(a, m * a.q_ld + (int64_t)h * dh + e0 + u) * a.scale : 0.f;
    for (int j0 = 0; j0 <= last; j0 += 4) {
        float kv[4][EPL], vv[4][EPL], s[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int u = 0; u < EPL; ++u) {
                const bool on = j0 + j <= last && act;
                kv[j][u] = on ? to_f32(kb[(int64_t)(j0 + j) * ld + e0 + u]) : 0.f;
                vv[j][u] = on ? to_f32(vb[(int64_t)(j0 + j) * ld + e0 + u]) : 0.f;
            }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            s[j] = 0.f;
#pragma unroll
            for (int u = 0; u < EPL; ++u) s[j] = fmaf(qv[u], kv[j][u], s[j]);
        }
#pragma unroll
        for (int x = 16; x > 0; x >>= 1)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[j] += __shfl_xor_sync(0xffffffffu, s[j], x);
        float mb = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j0 + j > last) s[j] = -INFINITY;
            mb = fmaxf(mb, s[j]);
        }
        rebase(mb);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (s[j] == -INFINITY) continue;
            const float w = exp_of<T>(s[j] - M);
            L += w;
#pragma unroll
            for (int u = 0; u < EPL; ++u) O[u] = fmaf(w, vv[j][u], O[u]);
        }
    }
    // a query without any key: zero output, lse -inf
    if (act) {
        const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
        T* dst = (T*)a.o + m * a.o_ld + (int64_t)h * dh + e0;
#pragma unroll
        for (int u = 0; u < EPL; ++u) dst[u] = from_f32<T>(O[u] * inv);
    }
    if (a.lse && lane == 0) a.lse[m * a.H + h] = L == 0.f ? -INFINITY : M + logf(L);
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

// Lays the partials out from base (or sizes them).
size_t carve_partials(const evs_shared_attn_args& c, SharedArgs& a, char* base) {
    size_t off = 0;
    auto take = [&](size_t bytes) {
        char* p = base ? base + off : nullptr;
        off = round256(off + bytes);
        return p;
    };
    const size_t sh = (size_t)c.kv_heads * a.sh_tiles * a.sh_slots * a.sh_rows;
    const size_t own = (size_t)c.batch * c.kv_heads * a.own_tiles * a.own_slots * a.own_rows;
    a.sh_o = (float*)take(sh * c.head_dim * 4);
    a.own_o = (float*)take(own * c.head_dim * 4);
    a.sh_ml = (float2*)take(sh * 8);
    a.own_ml = (float2*)take(own * 8);
    return off;
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
    plan_simt(c, a);
    carve_partials(c, a, (char*)c.workspace);
    const bool half = c.dtype == EVS_DTYPE_BF16;
    const int sh_items = c.kv_heads * a.sh_slots * ((a.sh_rows + SA_Q - 1) / SA_Q);
    const int own_items = c.batch * c.kv_heads * a.own_slots * ((a.own_rows + SA_Q - 1) / SA_Q);
    cudaError_t e = cudaSuccess;
    if (sh_items + own_items > 0)
        e = half ? launch_s(stream, shared_simt_kernel<bf16>, dim3(sh_items + own_items), dim3(256), 0, a, sh_items)
                 : launch_s(stream, shared_simt_kernel<float>, dim3(sh_items + own_items), dim3(256), 0, a, sh_items);
    if (e != cudaSuccess) return e;
    const long long queries = (long long)c.batch * c.n_cand * c.block * c.heads;
    const dim3 grid((unsigned)((queries + 3) / 4));
    if (half)
        e = c.head_dim == 128  ? launch_s(stream, shared_combine_kernel<bf16, 4>, grid, dim3(128), 0, a)
            : c.head_dim == 64 ? launch_s(stream, shared_combine_kernel<bf16, 2>, grid, dim3(128), 0, a)
                               : launch_s(stream, shared_combine_kernel<bf16, 1>, grid, dim3(128), 0, a);
    else
        e = c.head_dim == 128  ? launch_s(stream, shared_combine_kernel<float, 4>, grid, dim3(128), 0, a)
            : c.head_dim == 64 ? launch_s(stream, shared_combine_kernel<float, 2>, grid, dim3(128), 0, a)
                               : launch_s(stream, shared_combine_kernel<float, 1>, grid, dim3(128), 0, a);
    return e;
}

}  // namespace evs

extern "C" size_t evs_shared_attention_workspace(const evs_shared_attn_args* c) {
    using namespace evs;
    if (!valid_shape(c)) return 0;
    SharedArgs a{};
    plan_simt(*c, a);
    const size_t n = carve_partials(*c, a, nullptr);
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
    return launch_shared_attention(*c, (cudaStream_t)stream) == cudaSuccess ? EVS_OK : EVS_ERR_CUDA;
}
