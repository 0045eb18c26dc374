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
template <int N> struct Words { uint4 w[N]; };
template <> struct Word<32> { using type = Words<2>; };
template <> struct Word<64> { using type = Words<4>; };
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

__device__ __forceinline__ uint64_t both(float v) { return pair_of(v, v); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr float kLog2e = 1.4426950408889634f, kLog2eLo = 1.9259629911266175e-8f;   // log2 e and its rest

// ex2.approx is low by 0.1 to 0.45 u (u = 2^-24) in the mean over arguments of -2^-14 to -1, and a
// decay's error of one sign adds up over all the steps that a state remembers. 0.2 u in the exponent
// halves it (0.1 to -0.25 u) at no cost, in the product's own operation; 2^kDecay is 1 exactly, so that
// a step of size 0 keeps the state. Eight sequences of 64 tokens, 16 states: 8.1e-7 off in the state
// without it, 3.8e-7 with it (fp32 composed pairwise with exact exponentials, 3.4e-7).
constexpr float kDecay = 0.2f * 5.9604645e-8f * 1.4426950f;

// v / (1 + exp(-v)) for two: 8 instructions, where the scalar one takes about 11 for each
__device__ __forceinline__ uint64_t silu2(uint64_t v) {
    const float2 t = unpair(mul2(v, both(-kLog2e)));
    const float2 d = unpair(fma2(pair_of(ex2(t.x), ex2(t.y)), both(1.f), both(1.f)));
    return mul2(v, pair_of(rcp(d.x), rcp(d.y)));
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
// HBM-bound: x read + y written; 8192 x 8192 positions x channels of bf16 in 50 us, 5.3 TB/s. Four
// channels of bf16 a thread instead of eight halve its registers: seven CTAs an SM instead of three
// stream as fast, and a step of 64 single tokens x 4096 takes 3.0 us, not 3.9.
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
            if constexpr (VEC % 2 == 0 && LMAX <= 4) {
                // pairs of channels: the taps and the activation in packed fp32
#pragma unroll
                for (int i = 0; i < VEC; i += 2) {
                    const float v0 = to_f32(in[u].v[i]), v1 = to_f32(in[u].v[i + 1]);
                    uint64_t acc = fma2(pair_of(w[0][i], w[0][i + 1]), pair_of(v0, v1), pair_of(bias[i], bias[i + 1]));
#pragma unroll
                    for (int j = 1; j < LMAX; ++j)
                        acc = fma2(pair_of(w[j][i], w[j][i + 1]), pair_of(hist[j - 1][i], hist[j - 1][i + 1]), acc);
#pragma unroll
                    for (int j = LMAX - 2; j > 0; --j) {
                        hist[j][i] = hist[j - 1][i];
                        hist[j][i + 1] = hist[j - 1][i + 1];
                    }
                    hist[0][i] = v0;
                    hist[0][i + 1] = v1;
                    if (a.act) acc = silu2(acc);
                    const float2 r = unpair(acc);
                    out[i] = r.x;
                    out[i + 1] = r.y;
                }
            } else {
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

// Runs: as many as run at once, seven CTAs an SM over all sequences, at least 16
// positions each: only the first run then reads the old tail, which its thread may overwrite.
template <typename T, int LMAX, int VEC>
cudaError_t conv_launch(ConvArgs a, int B, cudaStream_t s) {
    const int cols = (a.D + VEC * CONV_THREADS - 1) / (VEC * CONV_THREADS);
    int runs = 1;
    if (a.y) {
        const long long want = 7 * 152 / ((long long)cols * B);
        const long long most = a.T / 16;
        runs = want < 1 || most < 1 ? 1 : (int)(want < most ? want : most);
        a.run = (a.T + runs - 1) / runs;
        runs = (a.T + a.run - 1) / a.run;
    } else {
        a.run = a.T > 0 ? a.T : 1;
    }
    return launch_s(s, conv_kernel<T, LMAX, VEC>, dim3(cols, runs, B), dim3(CONV_THREADS), 0, a);
}

template <typename T>
cudaError_t conv_dispatch(const ConvArgs& a, int B, bool wide, cudaStream_t s) {
    constexpr int V = 4;
    if (!wide) return conv_launch<T, 16, 1>(a, B, s);
    if (a.L == 2) return conv_launch<T, 2, V>(a, B, s);
    if (a.L == 3) return conv_launch<T, 3, V>(a, B, s);
    if (a.L == 4) return conv_launch<T, 4, V>(a, B, s);
    if (a.L <= 8) return conv_launch<T, 8, V / 2>(a, B, s);
    return conv_launch<T, 16, 2>(a, B, s);
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

__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
// The same for two at a time: 25 instructions where the scalar one takes 28 for each
__device__ __forceinline__ float2 step_sizes(float v0, float v1) {
    const uint64_t t = pair_of(fmaxf(-fabsf(v0), -100.f), fmaxf(-fabsf(v1), -100.f));
    const uint64_t hi = mul2(t, both(kLog2e));
    const uint64_t lo = fma2(t, both(kLog2eLo), fma2(t, both(kLog2e), mul2(t, both(-kLog2e))));
    const float2 h = unpair(hi);
    uint64_t e = pair_of(ex2(h.x), ex2(h.y));
    e = fma2(e, mul2(lo, both(0.69314718f)), e);
    const float2 d = unpair(fma2(e, both(1.f), both(2.f)));
    const uint64_t z = mul2(e, pair_of(rcp(d.x), rcp(d.y))), w = mul2(z, z);
    uint64_t p = fma2(w, both(1.f / 13.f), both(1.f / 11.f));
    p = fma2(p, w, both(1.f / 9.f));
    p = fma2(p, w, both(1.f / 7.f));
    p = fma2(p, w, both(1.f / 5.f));
    p = fma2(p, w, both(1.f / 3.f));
    p = fma2(p, w, both(1.f));
    return unpair(fma2(fma2(z, both(1.f), z), p, pair_of(max_nan(v0, 0.f), max_nan(v1, 0.f))));
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
            s[k] = fmaf(ex2(fmaf(dl, A2[k], kDecay)), s[k], u * to_f32(Bm[(size_t)t * a.b_ld + k]));
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

// Prompts. A lane owns a channel (LPC lanes do, with N / LPC states each, where that would leave few
// warps) with its states in registers, a warp 32 / LPC neighbouring channels. x, dt and z come
// asynchronously into the warp's own ring of SCAN_RING groups of eight positions, B_t and C_t into
// shared memory for the CTA, 32 positions at a time, which all lanes read as one address. What is
// per position and channel (softplus, gate) one of its lanes works out for the others, two
// positions at a time in packed arithmetic. Bound by instructions, 107 for a warp's step: 16
// sequences of 2048 x 4096 take 669 us, 97 ns a step on a quarter of an SM. The compiler is left all
// the registers (156): three CTAs an SM with more of the eight positions under way beat four (720
// us, 110 registers), five (737) and six (785).
//
// That leaves few warps for few sequences, so the tokens are cut into segments: a first pass runs
// each segment from a zero state (the first from state_in) and leaves its last state and the sum of
// its step sizes; the second starts every segment from
//   s(j) = exp(A sum dl(j-1)) s(j-1) + last(j-1),
// folded over the segments before it, and writes the outputs. The first pass costs the
// exponentials once more: segments are taken only where warps are short.
constexpr int SCAN_TC = 32, SCAN_WARPS = 4, SCAN_RING = 6;

template <int BYTES> __device__ __forceinline__ void cp_async(void* dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
                 "n"(BYTES)
                 : "memory");
}

struct ScanSeg {
    float* ws;          // [b][segment][N + 1][D]: last states and the sum of dl; then [b][N][D] state_in of
                        // the sequences of more than one segment
    int segs, len;      // segments of a sequence, positions of one
    int lanes;          // of a channel
};

// COPY: bytes of an asynchronous copy, 16 where rows start on 16 bytes, else 4 (bf16: where they
// start on two channels), else 0: element by element.
template <typename T, int N, int LPC, bool FIRST, int COPY>
__global__ void __launch_bounds__(32 * SCAN_WARPS, 1) scan_kernel(ScanArgs a, ScanSeg sg) {
    constexpr int NPL = N / LPC, THREADS = 32 * SCAN_WARPS, CPW = 32 / LPC;
    constexpr int EL = COPY ? COPY / (int)sizeof(T) : 1, PER_ROW = CPW / EL;   // channels of a copy, copies of a row
    constexpr int GROUP = 8 * CPW;                   // values of one array in a ring slot
    extern __shared__ __align__(16) uint8_t ring_raw[];
    constexpr int PBC = (SCAN_TC * N / 2 + THREADS - 1) / THREADS;
    __shared__ __align__(16) float b_s[2][SCAN_TC][N], c_s[2][SCAN_TC][N];
    pdl_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int b = blockIdx.y, j = blockIdx.z, t0 = j * sg.len;
    const int len = seq_len(a.lens, b, a.T, a.flags, FIRST == (sg.segs > 1) && blockIdx.x == 0 && j == 0 && tid == 0);
    const int t1 = min(t0 + sg.len, len);
    const bool last = t1 == len && (t0 < len || j == 0);   // the sequence ends here
    const int raw = (blockIdx.x * SCAN_WARPS + warp) * CPW + lane / LPC, k0 = lane % LPC * NPL;
    const bool on = raw < a.D;
    const int ch = on ? raw : a.D - 1;
    // a first pass serves segments that another one follows; a second one without outputs the last
    if (FIRST ? t0 + sg.len >= len : (t0 >= len && j > 0) || (!a.y && !last)) {
        pdl_trigger();
        return;
    }
    uint64_t A2[NPL / 2], s[NPL / 2];                // pairs of states
    auto of_state = [&](const float* p, int64_t step, int k) { return on ? p[(k0 + k) * step] : 0.f; };
    {
        float v[NPL];
        load_vec<float, NPL>(a.A + (size_t)ch * N + k0, v);
#pragma unroll
        for (int k = 0; k < NPL; k += 2) A2[k / 2] = pair_of(v[k] * kLog2e, v[k + 1] * kLog2e);
#pragma unroll
        for (int k = 0; k < NPL; ++k) v[k] = 0.f;
        float* keep = sg.ws + (size_t)gridDim.y * sg.segs * (N + 1) * a.D + (size_t)b * N * a.D + ch;
        if (j == 0 && a.state_in) {
            // Where a later segment writes state_out, which may be state_in, the first pass kept a copy. A
            // sequence that ends in this segment has none, and no other writer than this lane.
            if (!FIRST && !last) {
#pragma unroll
                for (int k = 0; k < NPL; ++k) v[k] = of_state(keep, a.D, k);
            } else {
                load_vec<float, NPL>(a.state_in + ((size_t)b * a.D + ch) * N + k0, v);
            }
        }
        if (FIRST && j == 0 && a.state_in && on) {
#pragma unroll
            for (int k = 0; k < NPL; ++k) keep[(int64_t)(k0 + k) * a.D] = v[k];
        }
        if (!FIRST) {
            const float* w = sg.ws + (size_t)b * sg.segs * (N + 1) * a.D + ch;
            for (int i = 0; i < j; ++i, w += (size_t)(N + 1) * a.D) {
                const float sum = w[(int64_t)N * a.D];
#pragma unroll
                for (int k = 0; k < NPL; k += 2) {
                    const float2 r = unpair(mul2(pair_of(sum, sum), A2[k / 2]));
                    v[k] = fmaf(ex2(r.x), v[k], w[(int64_t)(k0 + k) * a.D]);
                    v[k + 1] = fmaf(ex2(r.y), v[k + 1], w[(int64_t)(k0 + k + 1) * a.D]);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < NPL; k += 2) s[k / 2] = pair_of(v[k], v[k + 1]);
    }
    const float bias = a.dt_bias ? a.dt_bias[ch] : 0.f, Ds = a.Dskip ? a.Dskip[ch] : 0.f;
    const T* xb = (const T*)a.x + (size_t)b * a.x_seq;
    const T* db = (const T*)a.dt + (size_t)b * a.dt_seq;
    const bool out = !FIRST && a.y != nullptr, gated = out && a.z != nullptr;
    const T* zb = gated ? (const T*)a.z + (size_t)b * a.z_seq : xb;
    const int64_t z_ld = gated ? a.z_ld : a.x_ld;
    const T* Bm = (const T*)a.Bm + (size_t)b * a.b_seq;
    const T* Cm = (const T*)a.Cm + (size_t)b * a.c_seq;
    T* y = out ? (T*)a.y + (size_t)b * a.y_seq + ch : nullptr;
    float sum = 0.f;
    T* ring = reinterpret_cast<T*>(ring_raw) + (size_t)warp * SCAN_RING * 3 * GROUP;
    const int c0 = (blockIdx.x * SCAN_WARPS + warp) * CPW;    // the warp's first channel
    const int groups = (max(t1 - t0, 0) + 7) / 8;
    // Positions t0 + 8 g .. + 7 into the ring; past the end the last row again, past the width the
    // last channels.
    auto request = [&](int g) {
        if (g < groups) {
            T* to = ring + g % SCAN_RING * (3 * GROUP);
#pragma unroll
            for (int i = 0; i < (8 * PER_ROW + 31) / 32; ++i) {
                const int e = lane + 32 * i, c = min(c0 + e % PER_ROW * EL, a.D - EL);
                if (8 * PER_ROW % 32 && e >= 8 * PER_ROW) break;
                const int64_t t = min(t0 + 8 * g + e / PER_ROW, t1 - 1);
                const T *px = xb + t * a.x_ld + c, *pd = db + t * a.dt_ld + c, *pz = zb + t * z_ld + c;
                if constexpr (COPY > 0) {
                    cp_async<COPY>(to + EL * e, px);
                    cp_async<COPY>(to + GROUP + EL * e, pd);
                    if (gated) cp_async<COPY>(to + 2 * GROUP + EL * e, pz);
                } else {
                    const T vx = *px, vd = *pd, vz = *pz;
                    to[e] = vx;
                    to[GROUP + e] = vd;
                    to[2 * GROUP + e] = vz;
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    T br[PBC][2], cr[PBC][2];
    auto fetch_bc = [&](int t) {
#pragma unroll
        for (int i = 0; i < PBC; ++i) {
            const int e = (tid + i * THREADS) * 2 % (SCAN_TC * N);
            const int64_t at = min(t + e / N, t1 - 1);
            br[i][0] = Bm[at * a.b_ld + e % N];
            br[i][1] = Bm[at * a.b_ld + e % N + 1];
            if (!FIRST) {
                cr[i][0] = Cm[at * a.c_ld + e % N];
                cr[i][1] = Cm[at * a.c_ld + e % N + 1];
            }
        }
    };
    auto place_bc = [&](int buf) {
#pragma unroll
        for (int i = 0; i < PBC; ++i) {
            const int e = (tid + i * THREADS) * 2;
            if (e < SCAN_TC * N) {
                *reinterpret_cast<float2*>(&b_s[buf][0][0] + e) = make_float2(to_f32(br[i][0]), to_f32(br[i][1]));
                if (!FIRST)
                    *reinterpret_cast<float2*>(&c_s[buf][0][0] + e) = make_float2(to_f32(cr[i][0]), to_f32(cr[i][1]));
            }
        }
    };
    constexpr int PER = 8 / LPC;
    const int part = lane % LPC;
    const int my = max(0, min(ch - c0, CPW - 1));    // this lane's channel in a ring row
    auto steps = [&](int g, int row, int buf) {
        // the three parts apart, each eight positions wide, so that their chains fill one another;
        // what belongs to a position alone is worked out by one of a channel's lanes for all
        const T* from = ring + g % SCAN_RING * (3 * GROUP) + my;
        const int t = t0 + 8 * g, u0 = part * PER;
        float xv[PER], dl[PER], ux[PER], q[8];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            xv[i] = to_f32(from[(u0 + i) * CPW]);
            dl[i] = to_f32(from[GROUP + (u0 + i) * CPW]) + bias;
        }
        if (a.softplus) {
#pragma unroll
            for (int i = 0; i < PER; i += 2) {
                const float2 d = step_sizes(dl[i], dl[i + 1]);
                dl[i] = d.x;
                dl[i + 1] = d.y;
            }
        }
        const bool whole = t + 8 <= t1;
        if (!whole) {
            // positions past the end keep the state: dl = 0 gives a decay of one, and no input
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (t + u0 + i >= t1) dl[i] = xv[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (FIRST) sum += dl[i];
            ux[i] = dl[i] * xv[i];
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const float dlu = LPC == 1 ? dl[u % PER] : __shfl_sync(0xffffffffu, dl[u % PER], u / PER, LPC);
            const float uxu = LPC == 1 ? ux[u % PER] : __shfl_sync(0xffffffffu, ux[u % PER], u / PER, LPC);
            const uint64_t dl2 = pair_of(dlu, dlu), u2 = pair_of(uxu, uxu);
            uint64_t acc0 = 0, acc1 = 0;
#pragma unroll
            for (int k = 0; k < NPL / 2; k += 2) {
                // four states' B and C, one address for all lanes of a part
                const ulonglong2 bv = *reinterpret_cast<const ulonglong2*>(&b_s[buf][row + u][k0 + 2 * k]);
                const float2 r0 = unpair(fma2(dl2, A2[k], both(kDecay))), r1 = unpair(fma2(dl2, A2[k + 1], both(kDecay)));
                s[k] = fma2(pair_of(ex2(r0.x), ex2(r0.y)), s[k], mul2(u2, bv.x));
                s[k + 1] = fma2(pair_of(ex2(r1.x), ex2(r1.y)), s[k + 1], mul2(u2, bv.y));
                if (!FIRST) {
                    const ulonglong2 cv = *reinterpret_cast<const ulonglong2*>(&c_s[buf][row + u][k0 + 2 * k]);
                    acc0 = k == 0 ? mul2(s[k], cv.x) : fma2(s[k], cv.x, acc0);
                    acc1 = k == 0 ? mul2(s[k + 1], cv.y) : fma2(s[k + 1], cv.y, acc1);
                }
            }
            const float2 v0 = unpair(acc0), v1 = unpair(acc1);
            q[u] = (v0.x + v0.y) + (v1.x + v1.y);
        }
        if (out) {
            // the lanes' sums, each keeping half of the positions
#pragma unroll
            for (int o = LPC / 2, n = 4; o > 0; o >>= 1, n >>= 1)
#pragma unroll
                for (int i = 0; i < n; ++i) {
                    const bool up = part & o;
                    const float other = __shfl_xor_sync(0xffffffffu, up ? q[i] : q[i + n], o);
                    q[i] = (up ? q[i + n] : q[i]) + other;
                }
            T* yt = y + (int64_t)(t + u0) * a.y_ld;
#pragma unroll
            for (int i = 0; i < PER; i += 2) {
                uint64_t v = fma2(both(Ds), pair_of(xv[i], xv[i + 1]), pair_of(q[i], q[i + 1]));
                if (gated)
                    v = mul2(v, silu2(pair_of(to_f32(from[2 * GROUP + (u0 + i) * CPW]), to_f32(from[2 * GROUP + (u0 + i + 1) * CPW]))));
                const float2 w = unpair(v);
                q[i] = w.x;
                q[i + 1] = w.y;
            }
            if (on && whole) {
#pragma unroll
                for (int i = 0; i < PER; ++i, yt += a.y_ld) *yt = from_f32<T>(q[i]);
            } else if (on) {
#pragma unroll
                for (int i = 0; i < PER; ++i, yt += a.y_ld)
                    if (t + u0 + i < t1) *yt = from_f32<T>(q[i]);
            }
        }
    };
    if (t0 < t1) {
        fetch_bc(t0);
        for (int g = 0; g < SCAN_RING - 1; ++g) request(g);
        int buf = 0, g = 0;
        for (int tc = t0; tc < t1; tc += SCAN_TC, buf ^= 1) {
            place_bc(buf);
            __syncthreads();                       // the other buffer's readers passed the one before
            fetch_bc(tc + SCAN_TC);
#pragma unroll 1
            for (int row = 0; row < SCAN_TC; row += 8, ++g) {
                asm volatile("cp.async.wait_group %0;" ::"n"(SCAN_RING - 2) : "memory");
                __syncwarp();
                steps(g, row, buf);                // a group past the end changes nothing
                __syncwarp();
                request(g + SCAN_RING - 1);        // into the slot of group g - 1
            }
        }
    }
    if (FIRST) {
#pragma unroll
        for (int o = LPC / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    if (on && (FIRST || (last && a.state_out))) {
        float v[NPL];
#pragma unroll
        for (int k = 0; k < NPL; k += 2) {
            const float2 p = unpair(s[k / 2]);
            v[k] = p.x;
            v[k + 1] = p.y;
        }
        if (FIRST) {
            float* w = sg.ws + ((size_t)b * sg.segs + j) * (N + 1) * a.D + ch;
#pragma unroll
            for (int k = 0; k < NPL; ++k) w[(int64_t)(k0 + k) * a.D] = v[k];
            if (k0 == 0) w[(int64_t)N * a.D] = sum;
        } else {
            store_vec<float, NPL>(a.state_out + ((size_t)b * a.D + ch) * N + k0, v);
        }
    }
    // not before: CTAs of a successor placed early would share SMs that this grid keeps busy
    pdl_trigger();
}

constexpr int SCAN_STEP_MAX = 16;   // up to this many tokens the staging is not worth its barriers

// Lanes and segments of a prompt. One lane a channel, unless that leaves schedulers without a warp
// even with segments (512 x 2048 positions x channels of 16 states: 27 us with four lanes, 44 with
// one). Segments where fewer than a warp for each scheduler would run, of at least 128 positions
// (a multiple of the staged 32), enough for about three times the 12 warps that an SM holds:
// 2 x 4096 x 4096 takes 224 us so, 257 with a third of that and 731 in one piece.
constexpr int SCAN_FEW = 152 * 4, SCAN_FILL = 152 * 36, SCAN_MAX_SEGS = 64;
ScanSeg scan_segments(int B, int T, int D, int N) {
    ScanSeg sg{nullptr, 1, T, 1};
    if (T <= SCAN_STEP_MAX) return sg;
    for (int lanes = N == 32 ? 2 : 1;; lanes = N == 32 ? 4 : N / 4) {
        const long long warps = (long long)B * ((D * (long long)lanes + 31) / 32);
        long long segs = 1;
        if (warps < SCAN_FEW) {
            segs = SCAN_FILL / warps;
            if (segs > T / 128) segs = T / 128;
            if (segs > SCAN_MAX_SEGS) segs = SCAN_MAX_SEGS;
            if (segs < 3) segs = 1;                // two segments pay twice and gain at most that
        }
        const bool most = lanes >= (N == 32 ? 4 : N / 4);
        if (warps * segs >= SCAN_FEW || most) {
            sg.lanes = lanes;
            if (segs > 1) {
                sg.len = (int)(((T + segs - 1) / segs + SCAN_TC - 1) / SCAN_TC * SCAN_TC);
                sg.segs = (T + sg.len - 1) / sg.len;
            }
            return sg;
        }
    }
}
size_t scan_ws_bytes(const ScanSeg& sg, int B, int D, int N) {
    return sg.segs > 1 ? ((size_t)B * sg.segs * (N + 1) + (size_t)B * N) * D * 4 : 0;
}

template <typename T, int N, int LPC, int COPY>
cudaError_t scan_prompt(const ScanArgs& a, const ScanSeg& sg, int B, cudaStream_t s) {
    const int cols = (a.D * LPC + 32 * SCAN_WARPS - 1) / (32 * SCAN_WARPS);
    constexpr size_t smem = SCAN_WARPS * SCAN_RING * 3 * 8 * (32 / LPC) * sizeof(T);
    const dim3 block(32 * SCAN_WARPS);
    auto first = scan_kernel<T, N, LPC, true, COPY>;
    auto second = scan_kernel<T, N, LPC, false, COPY>;
    cudaError_t e = cudaSuccess;
    if (smem > 24 * 1024) {   // with the static part above 48 KB
        if (sg.segs > 1) e = cudaFuncSetAttribute(first, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(second, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    }
    if (sg.segs > 1 && e == cudaSuccess) e = launch_s(s, first, dim3(cols, B, sg.segs - 1), block, smem, a, sg);
    return e != cudaSuccess ? e : launch_s(s, second, dim3(cols, B, sg.segs), block, smem, a, sg);
}

// Every row of x, dt and z starts on n channels.
bool rows_on(const ScanArgs& a, size_t es, int n) {
    auto ok = [&](const void* p, int64_t ld, int64_t seq) {
        return !p || ((uintptr_t)p % (n * es) == 0 && ld % n == 0 && seq % n == 0);
    };
    return a.D % n == 0 && ok(a.x, a.x_ld, a.x_seq) && ok(a.dt, a.dt_ld, a.dt_seq) && ok(a.z, a.z_ld, a.z_seq);
}

template <typename T, int N, int LPC>
cudaError_t scan_copies(const ScanArgs& a, const ScanSeg& sg, int B, cudaStream_t s) {
    constexpr int es = sizeof(T);
    if (rows_on(a, es, 16 / es)) return scan_prompt<T, N, LPC, 16>(a, sg, B, s);
    if (es == 4 || rows_on(a, es, 4 / es)) return scan_prompt<T, N, LPC, 4>(a, sg, B, s);
    if constexpr (es < 4) return scan_prompt<T, N, LPC, 0>(a, sg, B, s);
    return cudaSuccess;
}
template <typename T, int N, int SLPC, int FEW, int MANY>
cudaError_t scan_launch(const ScanArgs& a, const ScanSeg& sg, int B, cudaStream_t s) {
    if (a.T <= SCAN_STEP_MAX)
        return launch_s(s, scan_step_kernel<T, N, SLPC>, dim3((a.D * SLPC + 255) / 256, B), dim3(256), 0, a);
    return sg.lanes == MANY ? scan_copies<T, N, MANY>(a, sg, B, s) : scan_copies<T, N, FEW>(a, sg, B, s);
}

template <typename T>
cudaError_t scan_dispatch(const ScanArgs& a, const ScanSeg& sg, int B, int N, cudaStream_t s) {
    switch (N) {
        case 4: return scan_launch<T, 4, 4, 1, 1>(a, sg, B, s);
        case 8: return scan_launch<T, 8, 4, 1, 2>(a, sg, B, s);
        case 16: return scan_launch<T, 16, 4, 1, 4>(a, sg, B, s);
        default: return scan_launch<T, 32, 8, 2, 4>(a, sg, B, s);
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
    const int es = c->dtype == EVS_DTYPE_BF16 ? 2 : 4, v = 4;
    // four channels at a time where every row starts on them and the width is a whole number of fours
    const bool wide = c->width % v == 0 && c->x_ld % v == 0 && c->x_seq % v == 0 && aligned(c->x, v * es) &&
                      (!c->y || (c->y_ld % v == 0 && c->y_seq % v == 0 && aligned(c->y, v * es))) &&
                      aligned(c->weight, 16) && (!c->tail_in || aligned(c->tail_in, 16)) && (!c->tail_out || aligned(c->tail_out, 16));
    const cudaError_t e = es == 2 ? conv_dispatch<bf16>(a, c->batch, wide, (cudaStream_t)stream)
                                  : conv_dispatch<float>(a, c->batch, wide, (cudaStream_t)stream);
    return status_of(e);
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
    ScanSeg sg = scan_segments(c->batch, c->tokens, c->width, c->states);
    if (sg.segs > 1) {
        if (!c->workspace || !aligned(c->workspace, 16)) return EVS_ERR_INVALID_ARG;
        if (c->ws_bytes < scan_ws_bytes(sg, c->batch, c->width, c->states)) return EVS_ERR_CAPACITY;
        sg.ws = (float*)c->workspace;
    }
    const cudaError_t e = c->dtype == EVS_DTYPE_BF16 ? scan_dispatch<bf16>(a, sg, c->batch, c->states, (cudaStream_t)stream)
                                                     : scan_dispatch<float>(a, sg, c->batch, c->states, (cudaStream_t)stream);
    return status_of(e);
}

extern "C" size_t evs_selective_scan_workspace(int32_t batch, int32_t tokens, int32_t width, int32_t states) {
    using namespace evs;
    if (batch < 1 || tokens < 1 || width < 1 || batch > 65535 || width > (1 << 24) || tokens > (1 << 30)) return 0;
    if (states != 4 && states != 8 && states != 16 && states != 32) return 0;
    return scan_ws_bytes(scan_segments(batch, tokens, width, states), batch, width, states);
}
