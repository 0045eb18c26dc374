// Stand-alone recurrent mixers: the short causal convolution and the selective scan, for
// prompts, verify blocks and single tokens (evs_causal_conv, evs_selective_scan).
//
// Both take ragged lengths from the device and keep the state they read apart from the state
// they write, so a verify pass leaves the carried state alone and slicing at k is the same call
// with lengths k + 1 (and no output rows wanted). Every reduction has a fixed order.
#include "evs_common.cuh"

namespace evs {
namespace {

using bf16 = __nv_bfloat16;

// ---- vectors of consecutive channels --------------------------------------------------------
// Raw words, so that a vector is one load, and loads are never conditional: out of range they take
// a valid neighbour. (Loads under a condition each wait for the one before: 14 of them, at 700
// cycles apiece, made a chunk of the scan take 10400 cycles.)
template <int BYTES> struct Word;
template <> struct Word<2> { using type = unsigned short; };
template <> struct Word<4> { using type = uint32_t; };
template <> struct Word<8> { using type = uint2; };
template <> struct Word<16> { using type = uint4; };
struct TwoWords { uint4 a, b; };
template <> struct Word<32> { using type = TwoWords; };
template <typename T, int VEC> union Chunk {
    typename Word<sizeof(T) * VEC>::type raw;
    T v[VEC];
    __device__ Chunk() {}
};
template <typename T, int VEC>
__device__ __forceinline__ Chunk<T, VEC> load_chunk(const T* p) {
    Chunk<T, VEC> c;
    c.raw = *reinterpret_cast<const typename Word<sizeof(T) * VEC>::type*>(p);
    return c;
}
template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T* p, float (&f)[VEC]) {
    const Chunk<T, VEC> c = load_chunk<T, VEC>(p);
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = to_f32(c.v[i]);
}
template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const float (&f)[VEC]) {
    Chunk<T, VEC> c;
#pragma unroll
    for (int i = 0; i < VEC; ++i) c.v[i] = from_f32<T>(f[i]);
    *reinterpret_cast<typename Word<sizeof(T) * VEC>::type*>(p) = c.raw;
}

__device__ __forceinline__ float silu(float v) { return __fdividef(v, 1.f + __expf(-v)); }

// A sequence's length: lens[b] clamped to [0, T], flagged if it lay outside.
__device__ __forceinline__ int seq_len(const int32_t* lens, int b, int T, uint32_t* flags, bool report) {
    if (!lens) return T;
    const int n = lens[b];
    if (n < 0 || n > T) {
        if (report && flags) atomicOr(flags, (uint32_t)EVS_FLAG_BAD_LEN);
        return n < 0 ? 0 : T;
    }
    return n;
}

// =========================================================================================
// Short causal convolution, y_t[c] = act(bias[c] + sum_{j<L} w[c][j] x_{t-j}[c]).
//
// A thread owns VEC consecutive channels and a run of consecutive positions: the window slides
// through registers, so x is read once but for the L - 1 rows before a run, and the weights once a
// run. The next four rows are requested before the last four are used. The thread of the first
// run also writes the tail (after it has read the old one), so the two may be the same buffer.
// HBM-bound: x read + y written.
// =========================================================================================
constexpr int CONV_THREADS = 128;

struct ConvArgs {
    const void* x;
    void* y;
    const float *w, *bias, *tail_in;
    float* tail_out;
    const int32_t* lens;
    uint32_t* flags;
    int64_t x_ld, x_seq, y_ld, y_seq;
    int T, D, L, act, run;
};

template <typename T, int LMAX, int VEC>
__global__ void __launch_bounds__(CONV_THREADS) conv_kernel(ConvArgs a) {
    pdl_wait();
    const int L = a.L;
    const int ch = (blockIdx.x * CONV_THREADS + threadIdx.x) * VEC;
    const int b = blockIdx.z, t0 = blockIdx.y * a.run;
    if (ch >= a.D) return;
    const int len = seq_len(a.lens, b, a.T, a.flags, ch == 0 && t0 == 0);
    if (t0 >= len && t0 > 0) return;
    const T* x = (const T*)a.x + (size_t)b * a.x_seq + ch;
    T* y = a.y ? (T*)a.y + (size_t)b * a.y_seq + ch : nullptr;
    const float* tin = a.tail_in ? a.tail_in + (size_t)b * (L - 1) * a.D + ch : nullptr;
    // hist[j] = x_{t0-1-j}; w[j] multiplies x_{t-j}
    float w[LMAX][VEC], hist[LMAX - 1][VEC], bias[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) bias[i] = a.bias ? a.bias[ch + i] : 0.f;
    if constexpr (VEC * LMAX % 4 == 0 && LMAX <= 4) {   // instances of one length, rows on 16 bytes
        float4 v[VEC * LMAX / 4];
#pragma unroll
        for (int i = 0; i < VEC * LMAX / 4; ++i) v[i] = reinterpret_cast<const float4*>(a.w + (size_t)ch * LMAX)[i];
        const float* f = reinterpret_cast<const float*>(v);
#pragma unroll
        for (int j = 0; j < LMAX; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) w[j][i] = f[i * LMAX + j];
    } else {
#pragma unroll
        for (int j = 0; j < LMAX; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) w[j][i] = j < L ? a.w[(size_t)(ch + i) * L + j] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < LMAX - 1; ++j) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) hist[j][i] = 0.f;
        const int t = t0 - 1 - j;
        if (j < L - 1) {
            if (t >= 0) load_vec<T, VEC>(x + (size_t)t * a.x_ld, hist[j]);
            else if (tin) load_vec<float, VEC>(tin + (size_t)(L - 1 + t) * a.D, hist[j]);
        }
    }
    if (t0 == 0 && a.tail_out) {
        // tail row r is the input at position len - (L - 1) + r, from x or, before its start,
        // from the old tail, which is in hist: position -1-j is hist[j]
        float* tout = a.tail_out + (size_t)b * (L - 1) * a.D + ch;
        for (int r = 0; r < L - 1; ++r) {
            const int t = len - (L - 1) + r;
            float v[VEC];
            if (t >= 0) {
                load_vec<T, VEC>(x + (size_t)t * a.x_ld, v);
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i) v[i] = 0.f;
#pragma unroll
                for (int j = 0; j < LMAX - 1; ++j)
                    if (j == -1 - t)
#pragma unroll
                        for (int i = 0; i < VEC; ++i) v[i] = hist[j][i];
            }
            store_vec<float, VEC>(tout + (size_t)r * a.D, v);
        }
    }
    if (!y) return;
    const int t1 = min(t0 + a.run, len);
    if (t0 >= t1) return;
    constexpr int AHEAD = 4;                       // rows requested while as many are worked on
    Chunk<T, VEC> buf[2][AHEAD];
    auto fetch = [&](int s, Chunk<T, VEC> (&c)[AHEAD]) {
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) c[u] = load_chunk<T, VEC>(x + (int64_t)min(s + u, t1 - 1) * a.x_ld);
    };
    auto work = [&](int s, const Chunk<T, VEC> (&in)[AHEAD]) {
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            if (s + u >= t1) return;
            float out[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float v = to_f32(in[u].v[i]);
                float acc = fmaf(w[0][i], v, bias[i]);
#pragma unroll
                for (int j = 1; j < LMAX; ++j)
                    if (j < L) acc = fmaf(w[j][i], hist[j - 1][i], acc);
#pragma unroll
                for (int j = LMAX - 2; j > 0; --j) hist[j][i] = hist[j - 1][i];
                hist[0][i] = v;
                out[i] = a.act ? silu(acc) : acc;
            }
            store_vec<T, VEC>(y + (int64_t)(s + u) * a.y_ld, out);
        }
    };
    fetch(t0, buf[0]);
    for (int s = t0; s < t1; s += 2 * AHEAD) {
        fetch(s + AHEAD, buf[1]);
        work(s, buf[0]);
        fetch(s + 2 * AHEAD, buf[0]);
        work(s + AHEAD, buf[1]);
    }
    pdl_trigger();
}

// Runs: about three CTAs an SM over all sequences, at least 16 positions each.
template <typename T, int LMAX, int VEC>
void conv_launch(ConvArgs a, int B, cudaStream_t s) {
    const int cols = (a.D + VEC * CONV_THREADS - 1) / (VEC * CONV_THREADS);
    int runs = 1;
    if (a.y) {
        const long long want = (3 * 152 + (long long)cols * B - 1) / ((long long)cols * B);
        const long long most = (a.T + 15) / 16;
        runs = (int)(want < most ? want : most);
        a.run = ((a.T + runs - 1) / runs + 7) / 8 * 8;
        runs = (a.T + a.run - 1) / a.run;
    } else {
        a.run = a.T > 0 ? a.T : 1;
    }
    launch_s(s, conv_kernel<T, LMAX, VEC>, dim3(cols, runs, B), dim3(CONV_THREADS), 0, a);
}

template <typename T>
void conv_dispatch(const ConvArgs& a, int B, bool wide, cudaStream_t s) {
    constexpr int V = 16 / sizeof(T);   // 16-byte accesses
    if (!wide) {
        conv_launch<T, 16, 1>(a, B, s);
    } else if (a.L == 2) {
        conv_launch<T, 2, V>(a, B, s);
    } else if (a.L == 3) {
        conv_launch<T, 3, V>(a, B, s);
    } else if (a.L == 4) {
        conv_launch<T, 4, V>(a, B, s);
    } else if (a.L <= 8) {
        conv_launch<T, 8, V / 2>(a, B, s);
    } else {
        conv_launch<T, 16, 2>(a, B, s);
    }
}

// =========================================================================================
// Selective scan, per channel c and state n of a sequence:
//   dl_t = softplus(dt_t + dt_bias), s_t = exp(dl_t A) s_{t-1} + dl_t x_t B_t,
//   y_t  = (sum_n C_t[n] s_t[n] + D x_t) silu(z_t).
// One exponential and three multiply-adds per (t, c, n); everything in fp32.
// =========================================================================================
struct ScanArgs {
    const void *x, *dt, *z, *Bm, *Cm;
    void* y;
    const float *A, *Dskip, *dt_bias, *state_in;
    float* state_out;
    const int32_t* lens;
    uint32_t* flags;
    int64_t x_ld, x_seq, dt_ld, dt_seq, z_ld, z_seq, b_ld, b_seq, c_ld, c_seq, y_ld, y_seq;
    int T, D, softplus;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr float kLog2e = 1.4426950408889634f, kLog2eLo = 1.9259629911266175e-8f;   // log2 e and its rest

// softplus(v) = max(v, 0) + log(1 + e), e = exp(-|v|): the exponential's argument with its rounding
// carried along, and log(1 + e) = 2 atanh(z), z = e / (2 + e) <= 1/3, by its series (the terms left
// out are below 2e-8 of it), so that it stays relatively exact where e is small.
__device__ __forceinline__ float step_size(float v, int softplus) {
    if (!softplus) return v;
    const float t = fmaxf(-fabsf(v), -100.f);
    const float hi = t * kLog2e;
    const float lo = fmaf(t, kLog2eLo, fmaf(t, kLog2e, -hi));
    float e = ex2(hi);
    e = fmaf(e, lo * 0.69314718f, e);
    const float z = __fdividef(e, 2.f + e), w = z * z;
    float p = fmaf(w, 1.f / 13.f, 1.f / 11.f);
    p = fmaf(p, w, 1.f / 9.f);
    p = fmaf(p, w, 1.f / 7.f);
    p = fmaf(p, w, 1.f / 5.f);
    p = fmaf(p, w, 1.f / 3.f);
    p = fmaf(p, w, 1.f);
    const float r = fmaf(2.f * z, p, fmaxf(v, 0.f));
    return v != v ? v : r;
}

// ---- pairs of fp32 ---------------------------------------------------------------------------
__device__ __forceinline__ uint64_t pair_of(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// A few tokens (single tokens, verify blocks): lanes of a channel hold NPL states each, straight
// from global memory; HBM-bound on the state read and written.
template <typename T, int N, int LPC>
__global__ void __launch_bounds__(256) scan_step_kernel(ScanArgs a) {
    constexpr int NPL = N / LPC;
    pdl_trigger();
    pdl_wait();
    const int b = blockIdx.y;
    const int g = blockIdx.x * 256 + threadIdx.x;
    const int ch_raw = g / LPC, k0 = (g % LPC) * NPL;
    const bool on = ch_raw < a.D;              // whole warps stay for the shuffles
    const int ch = on ? ch_raw : a.D - 1;
    const int len = seq_len(a.lens, b, a.T, a.flags, g == 0);
    float A2[NPL], s[NPL];
    load_vec<float, NPL>(a.A + (size_t)ch * N + k0, A2);
    const size_t so = ((size_t)b * a.D + ch) * N + k0;
    if (a.state_in) {
        load_vec<float, NPL>(a.state_in + so, s);
    } else {
#pragma unroll
        for (int k = 0; k < NPL; ++k) s[k] = 0.f;
    }
#pragma unroll
    for (int k = 0; k < NPL; ++k) A2[k] *= kLog2e;
    const float bias = a.dt_bias ? a.dt_bias[ch] : 0.f, Ds = a.Dskip ? a.Dskip[ch] : 0.f;
    const T* x = (const T*)a.x + (size_t)b * a.x_seq + ch;
    const T* dt = (const T*)a.dt + (size_t)b * a.dt_seq + ch;
    const T* z = a.z ? (const T*)a.z + (size_t)b * a.z_seq + ch : nullptr;
    const T* Bm = (const T*)a.Bm + (size_t)b * a.b_seq + k0;
    const T* Cm = (const T*)a.Cm + (size_t)b * a.c_seq + k0;
    for (int t = 0; t < len; ++t) {
        const float xv = to_f32(x[(size_t)t * a.x_ld]);
        const float dl = step_size(to_f32(dt[(size_t)t * a.dt_ld]) + bias, a.softplus);
        const float u = dl * xv;
        float q = 0.f;
#pragma unroll
        for (int k = 0; k < NPL; ++k) {
            s[k] = fmaf(ex2(dl * A2[k]), s[k], u * to_f32(Bm[(size_t)t * a.b_ld + k]));
            q = fmaf(s[k], to_f32(Cm[(size_t)t * a.c_ld + k]), q);
        }
        if (a.y) {
#pragma unroll
            for (int o = LPC / 2; o > 0; o >>= 1) q += __shfl_xor_sync(0xffffffffu, q, o);
            if (k0 == 0 && on) {
                float v = fmaf(Ds, xv, q);
                if (z) v *= silu(to_f32(z[(size_t)t * a.z_ld]));
                ((T*)a.y)[(size_t)b * a.y_seq + (size_t)t * a.y_ld + ch] = from_f32<T>(v);
            }
        }
    }
    if (a.state_out && on) store_vec<float, NPL>(a.state_out + so, s);
}

// Prompts. A CTA owns CH channels of one sequence and walks its tokens SCAN_TC at a time: the
// chunk's dl and dl x are formed once per (t, channel) into shared memory together with B_t and
// C_t, then LPC lanes of each channel run the recurrence over it, two states to an instruction, then
// the outputs leave with coalesced stores. The next chunk's raw values are requested before the
// recurrence of this one starts. The recurrence's own chain is one multiply-add a step: the
// exponentials of later steps do not depend on it, so they fill the pipe. Bound by issue: one
// exponential, half of four packed operations and its share of the staging per (t, c, n).
constexpr int SCAN_TC = 32;

template <typename T, int N, int LPC, bool V2>
__global__ void __launch_bounds__(256) scan_kernel(ScanArgs a) {
    constexpr int NPL = N / LPC;
    constexpr int CH = 256 / LPC;
    constexpr int RP = 512 / CH;                     // rows that one pass of the threads stages
    constexpr int PER = SCAN_TC / RP;
    constexpr int PBC = (SCAN_TC * N / 2 + 255) / 256;
    constexpr int YS = CH + 4;                       // eight steps of a channel's lanes in different banks
    __shared__ __align__(16) float2 du_s[SCAN_TC][CH];   // dl, dl * x
    __shared__ __align__(16) float y_s[SCAN_TC][YS];
    __shared__ __align__(16) float b_s[SCAN_TC][N], c_s[SCAN_TC][N];
    pdl_wait();
    const int b = blockIdx.y, tid = threadIdx.x;
    const int ch0 = blockIdx.x * CH;
    const int len = seq_len(a.lens, b, a.T, a.flags, blockIdx.x == 0 && tid == 0);
    const int lch = tid / LPC, sub = tid % LPC, k0 = sub * NPL;
    const int ch = min(ch0 + lch, a.D - 1);
    const bool on = ch0 + lch < a.D;
    float A2[NPL], s[NPL];
    load_vec<float, NPL>(a.A + (size_t)ch * N + k0, A2);
    const size_t so = ((size_t)b * a.D + ch) * N + k0;
    if (a.state_in) {
        load_vec<float, NPL>(a.state_in + so, s);
    } else {
#pragma unroll
        for (int k = 0; k < NPL; ++k) s[k] = 0.f;
    }
#pragma unroll
    for (int k = 0; k < NPL; ++k) A2[k] *= kLog2e;
    // staging: thread -> channels 2 (tid % (CH / 2)) and the next, positions tid / (CH / 2) + i RP
    const int sc = tid % (CH / 2) * 2, sr = tid / (CH / 2);
    const bool s1 = ch0 + sc < a.D, s2 = ch0 + sc + 1 < a.D;
    const int gch = min(ch0 + sc, a.D - (V2 ? 2 : 1)), gch2 = min(gch + 1, a.D - 1);
    const float2 bias = a.dt_bias ? make_float2(a.dt_bias[gch], a.dt_bias[gch2]) : make_float2(0.f, 0.f);
    const float2 Ds = a.Dskip ? make_float2(a.Dskip[gch], a.Dskip[gch2]) : make_float2(0.f, 0.f);
    const T* x = (const T*)a.x + (size_t)b * a.x_seq + gch;
    const T* dt = (const T*)a.dt + (size_t)b * a.dt_seq + gch;
    const T* z = a.z ? (const T*)a.z + (size_t)b * a.z_seq + gch : nullptr;
    const T* Bm = (const T*)a.Bm + (size_t)b * a.b_seq;
    const T* Cm = (const T*)a.Cm + (size_t)b * a.c_seq;
    T* y = a.y ? (T*)a.y + (size_t)b * a.y_seq + gch : nullptr;
    Chunk<T, 2> xr[PER], dr[PER], zr[PER], br[PBC], cr[PBC];
    const int other = gch2 - gch;                 // the second channel's place; 0: there is none
    auto two = [&](const T* p, int second) -> Chunk<T, 2> {
        if (V2) return load_chunk<T, 2>(p);
        Chunk<T, 2> r;
        r.v[0] = p[0];
        r.v[1] = p[second];
        return r;
    };
    auto fetch = [&](int t0) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int t = min(t0 + sr + i * RP, len - 1);
            xr[i] = two(x + (int64_t)t * a.x_ld, other);
            dr[i] = two(dt + (int64_t)t * a.dt_ld, other);
            if (z) zr[i] = two(z + (int64_t)t * a.z_ld, other);
        }
#pragma unroll
        for (int i = 0; i < PBC; ++i) {
            const int e = (tid + i * 256) * 2 % (SCAN_TC * N), t = min(t0 + e / N, len - 1);
            br[i] = two(Bm + (int64_t)t * a.b_ld + e % N, 1);
            cr[i] = two(Cm + (int64_t)t * a.c_ld + e % N, 1);
        }
    };
    if (len > 0) fetch(0);
    for (int t0 = 0; t0 < len; t0 += SCAN_TC) {
        Chunk<T, 2> xc[PER], zc[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            // positions past the end keep the state: dl = 0 gives a decay of one and no input
            const bool in = t0 + sr + i * RP < len;
            const float d0 = in ? step_size(to_f32(dr[i].v[0]) + bias.x, a.softplus) : 0.f;
            const float d1 = in ? step_size(to_f32(dr[i].v[1]) + bias.y, a.softplus) : 0.f;
            *reinterpret_cast<float4*>(&du_s[sr + i * RP][sc]) =
                make_float4(d0, d0 * to_f32(xr[i].v[0]), d1, d1 * to_f32(xr[i].v[1]));
            xc[i] = xr[i];
            zc[i] = zr[i];
        }
#pragma unroll
        for (int i = 0; i < PBC; ++i) {
            const int e = (tid + i * 256) * 2;
            if (e < SCAN_TC * N) {
                *reinterpret_cast<float2*>(&b_s[e / N][e % N]) = make_float2(to_f32(br[i].v[0]), to_f32(br[i].v[1]));
                *reinterpret_cast<float2*>(&c_s[e / N][e % N]) = make_float2(to_f32(cr[i].v[0]), to_f32(cr[i].v[1]));
            }
        }
        __syncthreads();
        if (t0 + SCAN_TC < len) fetch(t0 + SCAN_TC);
#pragma unroll 1
        for (int i0 = 0; i0 < SCAN_TC; i0 += 8) {
            float q[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const float2 du = du_s[i0 + u][lch];
                float bv[NPL], cv[NPL];
                load_vec<float, NPL>(&b_s[i0 + u][k0], bv);
                load_vec<float, NPL>(&c_s[i0 + u][k0], cv);
                if constexpr (NPL % 2 == 0) {
                    const uint64_t dl2 = pair_of(du.x, du.x), u2 = pair_of(du.y, du.y);
                    uint64_t acc = 0;
#pragma unroll
                    for (int k = 0; k < NPL; k += 2) {
                        const float2 r = unpair(mul2(dl2, pair_of(A2[k], A2[k + 1])));
                        const uint64_t ns = fma2(pair_of(ex2(r.x), ex2(r.y)), pair_of(s[k], s[k + 1]),
                                                 mul2(u2, pair_of(bv[k], bv[k + 1])));
                        acc = fma2(ns, pair_of(cv[k], cv[k + 1]), acc);
                        const float2 sv = unpair(ns);
                        s[k] = sv.x;
                        s[k + 1] = sv.y;
                    }
                    const float2 v = unpair(acc);
                    q[u] = v.x + v.y;
                } else {
                    float acc = 0.f;
#pragma unroll
                    for (int k = 0; k < NPL; ++k) {
                        s[k] = fmaf(ex2(du.x * A2[k]), s[k], du.y * bv[k]);
                        acc = fmaf(s[k], cv[k], acc);
                    }
                    q[u] = acc;
                }
            }
            // sum the eight steps over the channel's lanes; each lane is left with 8 / LPC of them
            int first = 0;
#pragma unroll
            for (int o = LPC / 2, n = 4; o > 0; o >>= 1, n >>= 1) {
                const bool up = (sub & o) != 0;
#pragma unroll
                for (int u = 0; u < n; ++u) {
                    const float give = up ? q[u] : q[u + n], keep = up ? q[u + n] : q[u];
                    q[u] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                }
                first += up ? n : 0;
            }
#pragma unroll
            for (int u = 0; u < 8 / LPC; ++u) y_s[i0 + first + u][lch] = q[u];
        }
        __syncthreads();
        if (y) {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int r = sr + i * RP, t = t0 + r;
                if (t >= len) break;
                const float2 v = *reinterpret_cast<const float2*>(&y_s[r][sc]);
                float o[2] = {fmaf(Ds.x, to_f32(xc[i].v[0]), v.x), fmaf(Ds.y, to_f32(xc[i].v[1]), v.y)};
                if (z) {
                    o[0] *= silu(to_f32(zc[i].v[0]));
                    o[1] *= silu(to_f32(zc[i].v[1]));
                }
                T* to = y + (int64_t)t * a.y_ld;
                if (V2) {
                    if (s1) store_vec<T, 2>(to, o);
                } else {
                    if (s1) to[0] = from_f32<T>(o[0]);
                    if (s2) to[1] = from_f32<T>(o[1]);
                }
            }
        }
        // the next chunk's y_s writes come after its own barrier, which follows these reads
    }
    if (a.state_out && on) store_vec<float, NPL>(a.state_out + so, s);
    // not before: CTAs of a successor placed early would share SMs that this grid keeps busy
    pdl_trigger();
}

constexpr int SCAN_STEP_MAX = 16;   // up to this many tokens the staging is not worth its barriers

// Pairs of channels load and store as one where every row starts on a pair.
bool pairs_ok(const ScanArgs& a, size_t es) {
    auto ok = [&](const void* p, int64_t ld, int64_t seq) {
        return !p || ((uintptr_t)p % (2 * es) == 0 && ld % 2 == 0 && seq % 2 == 0);
    };
    return a.D % 2 == 0 && ok(a.x, a.x_ld, a.x_seq) && ok(a.dt, a.dt_ld, a.dt_seq) && ok(a.z, a.z_ld, a.z_seq) &&
           ok(a.Bm, a.b_ld, a.b_seq) && ok(a.Cm, a.c_ld, a.c_seq) && ok(a.y, a.y_ld, a.y_seq);
}

template <typename T, int N, int LPC>
void scan_launch(const ScanArgs& a, int B, cudaStream_t s) {
    const dim3 grid((a.D * LPC + 255) / 256, B);
    if (a.T <= SCAN_STEP_MAX)
        launch_s(s, scan_step_kernel<T, N, LPC>, grid, dim3(256), 0, a);
    else if (pairs_ok(a, sizeof(T)))
        launch_s(s, scan_kernel<T, N, LPC, true>, grid, dim3(256), 0, a);
    else
        launch_s(s, scan_kernel<T, N, LPC, false>, grid, dim3(256), 0, a);
}

template <typename T>
bool scan_dispatch(const ScanArgs& a, int B, int N, cudaStream_t s) {
    switch (N) {
        case 4: scan_launch<T, 4, 4>(a, B, s); return true;
        case 8: scan_launch<T, 8, 4>(a, B, s); return true;
        case 16: scan_launch<T, 16, 4>(a, B, s); return true;
        case 32: scan_launch<T, 32, 8>(a, B, s); return true;
        default: return false;
    }
}

bool aligned(const void* p, size_t n) { return ((uintptr_t)p % n) == 0; }

}  // namespace
}  // namespace evs

extern "C" evs_status evs_causal_conv(const evs_conv_args* c, void* stream) {
    using namespace evs;
    if (!c || c->batch < 0 || c->tokens < 0 || c->width < 1 || c->taps < 2 || c->taps > 16) return EVS_ERR_INVALID_ARG;
    if (c->dtype != EVS_DTYPE_F32 && c->dtype != EVS_DTYPE_BF16) return EVS_ERR_INVALID_ARG;
    if (c->batch > 65535 || c->tokens > (1 << 30) || c->width > (1 << 24)) return EVS_ERR_INVALID_ARG;
    if (c->batch == 0) return EVS_OK;
    if (!c->weight || (c->tokens > 0 && !c->x) || (!c->y && !c->tail_out)) return EVS_ERR_INVALID_ARG;
    if (c->x_ld < c->width || (c->y && c->y_ld < c->width)) return EVS_ERR_INVALID_ARG;
    if (c->tokens == 0 && !c->tail_out) return EVS_OK;
    ConvArgs a{c->x, c->tokens > 0 ? c->y : nullptr, c->weight, c->bias, c->tail_in, c->tail_out, c->lens, c->flags,
               c->x_ld, c->x_seq, c->y_ld, c->y_seq, c->tokens, c->width, c->taps, c->silu ? 1 : 0, 0};
    const int es = c->dtype == EVS_DTYPE_BF16 ? 2 : 4, v = 16 / es;
    // 16-byte accesses when every row starts on 16 bytes and the width is a whole number of them
    const bool wide = c->width % v == 0 && c->x_ld % v == 0 && c->x_seq % v == 0 && aligned(c->x, 16) &&
                      (!c->y || (c->y_ld % v == 0 && c->y_seq % v == 0 && aligned(c->y, 16))) &&
                      aligned(c->weight, 16) && (!c->tail_in || aligned(c->tail_in, 16)) && (!c->tail_out || aligned(c->tail_out, 16));
    if (es == 2) conv_dispatch<bf16>(a, c->batch, wide, (cudaStream_t)stream);
    else conv_dispatch<float>(a, c->batch, wide, (cudaStream_t)stream);
    return cudaGetLastError() == cudaSuccess ? EVS_OK : EVS_ERR_CUDA;
}

extern "C" evs_status evs_selective_scan(const evs_scan_args* c, void* stream) {
    using namespace evs;
    if (!c || c->batch < 0 || c->tokens < 0 || c->width < 1) return EVS_ERR_INVALID_ARG;
    if (c->states != 4 && c->states != 8 && c->states != 16 && c->states != 32) return EVS_ERR_INVALID_ARG;
    if (c->dtype != EVS_DTYPE_F32 && c->dtype != EVS_DTYPE_BF16) return EVS_ERR_INVALID_ARG;
    if (c->batch > 65535 || c->width > (1 << 24) || c->tokens > (1 << 30)) return EVS_ERR_INVALID_ARG;
    if (c->batch == 0) return EVS_OK;
    if (!c->A || (!c->y && !c->state_out)) return EVS_ERR_INVALID_ARG;
    if (c->tokens > 0 && (!c->x || !c->dt || !c->B || !c->C)) return EVS_ERR_INVALID_ARG;
    if (c->x_ld < c->width || c->dt_ld < c->width || (c->z && c->z_ld < c->width) || (c->y && c->y_ld < c->width) ||
        c->b_ld < c->states || c->c_ld < c->states)
        return EVS_ERR_INVALID_ARG;
    // a lane's states are read and written as one vector
    if (!aligned(c->A, 16) || (c->state_in && !aligned(c->state_in, 16)) || (c->state_out && !aligned(c->state_out, 16)))
        return EVS_ERR_INVALID_ARG;
    if (c->tokens == 0 && !c->state_out) return EVS_OK;
    ScanArgs a{c->x, c->dt, c->z, c->B, c->C, c->y, c->A, c->D, c->dt_bias, c->state_in, c->state_out, c->lens,
               c->flags, c->x_ld, c->x_seq, c->dt_ld, c->dt_seq, c->z_ld, c->z_seq, c->b_ld, c->b_seq, c->c_ld,
               c->c_seq, c->y_ld, c->y_seq, c->tokens, c->width, c->softplus ? 1 : 0};
    const bool ok = c->dtype == EVS_DTYPE_BF16 ? scan_dispatch<bf16>(a, c->batch, c->states, (cudaStream_t)stream)
                                               : scan_dispatch<float>(a, c->batch, c->states, (cudaStream_t)stream);
    if (!ok) return EVS_ERR_INVALID_ARG;
    return cudaGetLastError() == cudaSuccess ? EVS_OK : EVS_ERR_CUDA;
}
