// Attention of a few query rows on CUDA cores, in fp32 whatever the type: for fp32 problems, narrow heads
// and strides that tensor maps cannot describe. 256 threads, 16 R rows by tiles of 64 keys: thread (ty, tx)
// has rows ty R .. and keys tx + 16 j of the scores, then the same rows and DH / 16 columns of the output,
// both in registers, multiplied two at a time. The 16 threads of a row are neighbours in a warp, so its
// maximum and sum take four shuffles.
#pragma once

#include "evs_common.cuh"

namespace evs {
namespace attn {

template <typename T> __device__ __forceinline__ float simt_exp(float x);
// fp32 problems keep the full precision of the exponential; in bf16 ones its fast form is off by 2^-19 at most where a
// weight counts (x > -10), far inside the 2^-9 of the output's own rounding
template <> __device__ __forceinline__ float simt_exp<float>(float x) { return expf(x); }
template <> __device__ __forceinline__ float simt_exp<__nv_bfloat16>(float x) { return __expf(x); }

template <typename T, int DH, int R> struct Simt {
    static constexpr int ROWS = 16 * R, KEYS = 64, LD = DH + 4, LDP = KEYS + 4;
    static constexpr int CW = DH / 16, VEC = CW < 4 ? CW : 4, NU = CW / VEC;   // columns of a thread, in a piece, pieces
    static constexpr int PIECES = KEYS * DH / 4 / 256;   // of four columns, of a tile of K or V, a thread brings
    // V of a tile on its way while its scores are worked out, where registers allow
    static constexpr bool AHEAD = R * DH <= 256;
    struct Smem {
        float q[ROWS][LD];
        float kv[KEYS][LD];
        float p[ROWS][LDP];
    };
    Smem& sm;
    const int tid, ty, tx;
    float m[R], l[R], o[R][CW];

    __device__ __forceinline__ Simt(Smem& s) : sm(s), tid(threadIdx.x), ty(threadIdx.x / 16), tx(threadIdx.x % 16) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int c = 0; c < CW; ++c) o[i][c] = 0.f;
        }
    }
    // rows(r): row r of q, or null
    template <typename F> __device__ __forceinline__ void stage_q(F rows, float scale) {
        for (int e = tid; e < ROWS * DH; e += 256) {
            const int r = e / DH, c = e % DH;
            const T* p = rows(r);
            sm.q[r][c] = p ? to_f32(p[c]) * scale : 0.f;
        }
    }
    template <typename F> __device__ __forceinline__ float4 fetch(F rows, int nk, int piece) {
        const int e = tid + piece * 256, r = e / (DH / 4), c = e % (DH / 4) * 4;
        if (r >= nk) return make_float4(0.f, 0.f, 0.f, 0.f);
        const T* p = rows(r) + c;
        if (sizeof(T) == 4 && (uintptr_t)p % 16 == 0) return *reinterpret_cast<const float4*>(p);
        return make_float4(to_f32(p[0]), to_f32(p[1]), to_f32(p[2]), to_f32(p[3]));
    }
    __device__ __forceinline__ void put(int piece, float4 x) {
        const int e = tid + piece * 256;
        *reinterpret_cast<float4*>(&sm.kv[e / (DH / 4)][e % (DH / 4) * 4]) = x;
    }
    template <typename F> __device__ __forceinline__ void stage_kv(F rows, int nk) {
#pragma unroll 4
        for (int i = 0; i < PIECES; ++i) put(i, fetch(rows, nk, i));
    }
    static __device__ __forceinline__ uint64_t as_pair(float a, float b) {
        uint64_t r;
        asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
        return r;
    }
    static __device__ __forceinline__ void fma_pair(uint64_t a, uint64_t b, uint64_t& c) {
        asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(c) : "l"(a), "l"(b));
    }
    static __device__ __forceinline__ void of_pair(uint64_t v, float& a, float& b) {
        asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
    }
    // nk keys (1 .. 64) whose rows k(j) and v(j) are; sees(r, j): row r reads key j. MASKED: some may not, and V that
    // is not finite is kept from those (a weight of 0 does not)
    template <bool MASKED, typename FK, typename FV, typename FM>
    __device__ __forceinline__ void tile(FK k, FV v, int nk, FM sees) {
        float4 ahead[AHEAD ? PIECES : 1];
        if constexpr (AHEAD) {
            float4 x[PIECES];
#pragma unroll
            for (int i = 0; i < PIECES; ++i) x[i] = fetch(k, nk, i);
#pragma unroll
            for (int i = 0; i < PIECES; ++i) ahead[i] = fetch(v, nk, i);
#pragma unroll
            for (int i = 0; i < PIECES; ++i) put(i, x[i]);
        } else {
            stage_kv(k, nk);
        }
        __syncthreads();
        uint64_t acc[R][4];
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = 0;
#pragma unroll 4
        for (int d = 0; d < DH; d += 4) {
            uint64_t q2[R][2], k2[4][2];
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const float4 x = *reinterpret_cast<const float4*>(&sm.q[ty * R + i][d]);
                q2[i][0] = as_pair(x.x, x.y);
                q2[i][1] = as_pair(x.z, x.w);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float4 x = *reinterpret_cast<const float4*>(&sm.kv[tx + 16 * j][d]);
                k2[j][0] = as_pair(x.x, x.y);
                k2[j][1] = as_pair(x.z, x.w);
            }
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    fma_pair(q2[i][0], k2[j][0], acc[i][j]);
                    fma_pair(q2[i][1], k2[j][1], acc[i][j]);
                }
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            float s[4], mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float a, b;
                of_pair(acc[i][j], a, b);
                s[j] = tx + 16 * j < nk && sees(ty * R + i, tx + 16 * j) ? a + b : -INFINITY;
                mx = fmaxf(mx, s[j]);
            }
#pragma unroll
            for (int x = 8; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
            const float m_new = fmaxf(m[i], mx), base = m_new == -INFINITY ? 0.f : m_new;   // only -inf scores: weights 0
            const float f = simt_exp<T>(m[i] - base);
            m[i] = m_new;
            l[i] *= f;
#pragma unroll
            for (int c = 0; c < CW; ++c) o[i][c] *= f;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[j] = simt_exp<T>(s[j] - base);
                sum += s[j];
                sm.p[ty * R + i][tx + 16 * j] = s[j];
            }
#pragma unroll
            for (int x = 8; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
            l[i] += sum;
        }
        __syncthreads();
        if constexpr (AHEAD) {
#pragma unroll
            for (int i = 0; i < PIECES; ++i) put(i, ahead[i]);
        } else {
            stage_kv(v, nk);
        }
        __syncthreads();
        const int end = (nk + 3) & ~3;                   // rows behind nk are zero, and so are their weights
#pragma unroll 1
        for (int j0 = 0; j0 < end; j0 += 4) {
            float4 p[R];
#pragma unroll
            for (int i = 0; i < R; ++i) p[i] = *reinterpret_cast<const float4*>(&sm.p[ty * R + i][j0]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
                for (int u = 0; u < NU; ++u) {
                    const float* row = &sm.kv[j0 + j][u * 16 * VEC + tx * VEC];
                    if constexpr (VEC == 4) {
                        const float4 x = *reinterpret_cast<const float4*>(row);
                        const uint64_t v01 = as_pair(x.x, x.y), v23 = as_pair(x.z, x.w);
#pragma unroll
                        for (int i = 0; i < R; ++i) {
                            const float w = (&p[i].x)[j];
                            if (MASKED && w == 0.f) continue;
                            const uint64_t w2 = as_pair(w, w);
                            uint64_t o01 = as_pair(o[i][u * 4], o[i][u * 4 + 1]), o23 = as_pair(o[i][u * 4 + 2], o[i][u * 4 + 3]);
                            fma_pair(w2, v01, o01);
                            fma_pair(w2, v23, o23);
                            of_pair(o01, o[i][u * 4], o[i][u * 4 + 1]);
                            of_pair(o23, o[i][u * 4 + 2], o[i][u * 4 + 3]);
                        }
                    } else {
#pragma unroll
                        for (int c = 0; c < VEC; ++c) {
                            const float x = row[c];
#pragma unroll
                            for (int i = 0; i < R; ++i)
                                if (!MASKED || (&p[i].x)[j] != 0.f) o[i][u * VEC + c] = fmaf((&p[i].x)[j], x, o[i][u * VEC + c]);
                        }
                    }
                }
            }
        }
        __syncthreads();
    }
    // out(r, c, o, m, l) for every column c of every row r: the sum of weighted values, the maximum and the
    // sum of weights (natural units)
    template <typename F> __device__ __forceinline__ void finish(F out) {
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int u = 0; u < NU; ++u)
#pragma unroll
                for (int c = 0; c < VEC; ++c) out(ty * R + i, u * 16 * VEC + tx * VEC + c, o[i][u * VEC + c], m[i], l[i]);
    }
};

}  // namespace attn
}  // namespace evs
