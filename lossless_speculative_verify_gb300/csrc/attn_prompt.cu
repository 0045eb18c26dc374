// Causal attention over whole prompts packed behind each other (evs_prompt_attention).
//
//   o_i = sum_{j <= i} exp(scale q_i.k_j - m) v_j / l,  lse_i = m + log l, within each sequence.
//
// On the tensor cores an item is 256 query rows of one head of one sequence, 128 for each lane (see
// attn_tiles.cuh), and the K/V tiles up to its diagonal, which TMA brings once for both. A persistent grid
// takes the items in the order of their length, longest first, forwards and backwards in turn, so that the
// CTAs end together: lengths are on the device, and each role of a CTA walks the same order by itself.
#include "attn_simt.cuh"
#include "attn_tiles.cuh"

namespace evs {
namespace {

using namespace attn;

struct PromptArgs {
    const void *q, *k, *v;
    void* o;
    float* lse;
    const int32_t* starts;
    uint32_t* flags;
    int64_t q_row, q_head, kv_row, kv_head, o_row;
    int N, B, H, G, zero_rest, o_vec;
    float scale;
};

// Row where sequence b starts, in ascending order within [0, N] whatever starts holds; st: [B + 1] in
// shared memory. All threads of the CTA; a warp scans.
__device__ __forceinline__ void load_starts(const PromptArgs& a, int* st) {
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int run = 0;
        bool bad = false;
        for (int b0 = 0; b0 <= a.B; b0 += 32) {
            const int b = b0 + lane;
            const int raw = b <= a.B ? __ldcg(a.starts + b) : 0;
            int x = min(max(raw, 0), a.N);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x = max(x, y);
            }
            x = max(x, run);
            if (b <= a.B) {
                st[b] = x;
                bad |= x != raw;
            }
            run = __shfl_sync(0xffffffffu, x, 31);
        }
        if (bad && a.flags && blockIdx.x == 0) atomicOr(a.flags, (uint32_t)EVS_FLAG_BAD_LEN);
    }
    __syncthreads();
}

// Rows of no sequence, dealt among `parts` CTAs of `threads`
template <typename T>
__device__ __forceinline__ void rest_rows(const PromptArgs& a, int s0, int s1, int dh, int part, int parts, int t, int threads) {
    const int rest = s0 + (a.N - s1);
    for (int i = part; i < rest; i += parts) {
        const int64_t row = i < s0 ? i : s1 + (i - s0);
        if (a.zero_rest)
            for (int c = t; c < a.H * dh; c += threads) ((T*)a.o)[row * a.o_row + c] = from_f32<T>(0.f);
        if (a.lse)
            for (int h = t; h < a.H; h += threads) a.lse[row * a.H + h] = -INFINITY;
    }
}

// Shared memory of the tensor-core kernel: exchange [2][128] floats, barriers, then st [B + 1], order [B] and of [B]
// (sequences by length, longest first: which, and their items of 256 rows), then Q and the ring on 1024 bytes.
constexpr int BARRIERS = 320;
constexpr int small_smem(int B) { return 1024 + BARRIERS + (3 * B + 1) * 4; }

// The CTA's items. Level v holds the items of v x 256 rows and their keys: one for each head of each
// sequence that is as long.
struct Items {
    const PromptArgs& a;
    int round, base, level, count;
    int first, len, head, tile;          // the item: its sequence's first row and length, its head and 256 rows

    static __device__ __forceinline__ int* starts() {
        extern __shared__ uint8_t smem_raw[];
        return reinterpret_cast<int*>(smem_raw + 1024 + BARRIERS);
    }
    static __device__ __forceinline__ int* order(const PromptArgs& a) { return starts() + a.B + 1; }
    static __device__ __forceinline__ int* of(const PromptArgs& a) { return starts() + 2 * a.B + 1; }

    __device__ __forceinline__ Items(const PromptArgs& args) : a(args), round(0), base(0), count(0) {
        level = of(a)[0];
        widen();
    }
    __device__ __forceinline__ void widen() {
        while (count < a.B && of(a)[count] >= level) ++count;
    }
    __device__ __forceinline__ bool next() {
        const int grid = gridDim.x, at = round * grid + ((round & 1) ? grid - 1 - (int)blockIdx.x : (int)blockIdx.x);
        ++round;
        while (level > 0 && at >= base + count * a.H) {
            base += count * a.H;
            --level;
            widen();
        }
        if (level <= 0) return false;
        const int in = at - base, i = in / a.H, s = order(a)[i];
        first = starts()[s];
        len = starts()[s + 1] - first;
        head = in - i * a.H;
        tile = level - 1;
        return true;
    }
    // of lane L: its first row, rows, keys, tiles of K keys; of the item: tiles
    __device__ __forceinline__ int row0(int L) const { return tile * 256 + L * 128; }
    __device__ __forceinline__ int rows(int L) const { return min(128, len - row0(L)); }
    __device__ __forceinline__ int keys(int L) const { return min(len, row0(L) + 128); }
    template <int K> __device__ __forceinline__ int key_tiles(int L) const { return rows(L) > 0 ? (keys(L) + K - 1) / K : 0; }
    template <int K> __device__ __forceinline__ int key_tiles() const { return (keys(1) + K - 1) / K; }
};

constexpr int prompt_smem(int dh, int B) { return small_smem(B) + 1024 + 2 * Q_ROWS * dh * 2 + ring_slots(dh) * tile_bytes(dh); }
static_assert(prompt_smem(64, 1024) <= 227 * 1024 && prompt_smem(128, 1024) <= 227 * 1024, "shared memory of an SM");

template <int DH>
__global__ void __launch_bounds__(THREADS, 1)
prompt_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                 const __grid_constant__ CUtensorMap tmV, PromptArgs a) {
    constexpr int KEYS = tile_keys(DH), HALVES = DH / 64, HALF = KEYS * 128, TILE = HALF * HALVES;
    constexpr int NST = ring_slots(DH), Q_HALF = Q_ROWS * 128, Q_TILE = Q_HALF * HALVES;
    extern __shared__ uint8_t smem_raw[];
    float* exchange = reinterpret_cast<float*>(smem_raw);                  // [2][128]
    uint64_t* full = reinterpret_cast<uint64_t*>(smem_raw + 1024);         // [NST]
    uint64_t* empty = full + NST;                                          // [NST]
    uint64_t* s_full = empty + NST;                                        // [2] scores of a tile in tensor memory
    uint64_t* s_free = s_full + 2;                                         // [2] and in registers
    uint64_t* p_full = s_free + 2;                                         // [2][2] weights of an even, an odd tile there
    uint64_t* pv_done = p_full + 4;                                        // [2][2] P V of an even, an odd tile complete
    uint64_t* q_full = pv_done + 4;                                        // [2] Q of an item there
    uint64_t* q_free = q_full + 2;                                         // [2] and read for the last time
    uint64_t* drain = q_free + 2;                                          // [4]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 4);
    int* st = Items::starts();
    uint8_t* sQ = smem_raw + ((smem_u32(smem_raw) + small_smem(a.B) + 1023u & ~1023u) - smem_u32(smem_raw));
    uint8_t* ring = sQ + 2 * Q_TILE;
    static_assert((2 * NST + 20) * 8 + 4 <= BARRIERS, "barriers");
    // an even number: a slot is K's or V's, and each thread that waits for one has seen its phase before
    static_assert(NST % 2 == 0 && NST >= 4, "ring");
    static_assert(TILE == tile_bytes(DH) && HALF % 1024 == 0, "tiles on 1024 bytes");
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

    pdl_wait();
    pdl_trigger();
    // not before the wait: a predecessor's CTA on this SM may have yet to allocate
    if (warp == SOFT_WARPS) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    if (tid == 0) {
        for (int s = 0; s < NST; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_free[i], 8);
            mbar_init(&p_full[2 * i], 8);
            mbar_init(&p_full[2 * i + 1], 8);
            mbar_init(&pv_done[2 * i], 1);
            mbar_init(&pv_done[2 * i + 1], 1);
            mbar_init(&q_full[i], 1);
            mbar_init(&q_free[i], 1);
            mbar_init(&drain[i], 1);
            mbar_init(&drain[2 + i], 1);
        }
        fence_barrier_init();
    }
    load_starts(a, st);
    for (int s = tid; s < a.B; s += THREADS) {           // sequences by tiles, longest first
        const int n = (st[s + 1] - st[s] + 255) >> 8;
        int before = 0;
        for (int o = 0; o < a.B; ++o) {
            const int m = (st[o + 1] - st[o] + 255) >> 8;
            before += m > n || (m == n && o < s);
        }
        Items::order(a)[before] = s;
        Items::of(a)[before] = n;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    Items it(a);

    if (warp >= SOFT_WARPS) {
        asm volatile(EVS_ATTN_AUX_REGS);
        const int role = warp - SOFT_WARPS;
        if (role == 0 && lane == 0) {
            // ---- K and V tiles: K0 V0 K1 V1 ... of all items
            const uint64_t keep = policy_evict_last();
            int s = 0;
            uint32_t ph = 1, used = 0;                   // parity that a free slot has; slots in use so far
            bool ok = true;
            while (ok && it.next()) {
                const int n = 2 * it.key_tiles<KEYS>(), g = it.head / (a.H / a.G);
                for (int j = 0; j < n; ++j) {
                    if ((used >> s & 1u) && !mbar_wait(&empty[s], ph)) { ok = false; break; }
                    used |= 1u << s;
                    uint8_t* dst = ring + (size_t)s * TILE;
                    mbar_arrive_expect_tx(&full[s], (uint32_t)TILE);
#pragma unroll
                    for (int hf = 0; hf < HALVES; ++hf)
                        tma_load_4d(dst + hf * HALF, j & 1 ? &tmV : &tmK, hf * 64, it.first + (j >> 1) * KEYS, g, 0, &full[s], keep);
                    if (++s == NST) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            if (!ok)                                     // loads in flight end before this CTA does (bounded)
                for (int i = 0; i < NST; ++i)
                    if (used >> i & 1u) mbar_wait(&full[i], i < s ? ph ^ 1u : ph);
        } else if (role == 1 || role == 2) {
            // ---- Q and the scores of lane L: those of the next tile as soon as this one's are in registers
            const int L = role - 1;
            const uint64_t qd = smem_desc_sw128(smem_u32(sQ + L * Q_TILE)), dk = smem_desc_sw128(smem_u32(ring));
            const uint64_t once = policy_evict_first();
            const uint32_t at = tmem + (uint32_t)L * LANE_COLS, leader = elect_leader();
            Cursor k(0, NST);
            uint32_t cnt = 0, qn = 0;                    // tiles, items
            bool ok = true;
            while (ok && it.next()) {
                const int n = it.key_tiles<KEYS>(L), all = it.key_tiles<KEYS>();
                if (n > 0) {
                    if (qn > 0 && !all_wait(&q_free[L], (qn - 1) & 1u)) { ok = false; break; }
                    if (leader) {
                        mbar_arrive_expect_tx(&q_full[L], (uint32_t)Q_TILE);
#pragma unroll
                        for (int hf = 0; hf < HALVES; ++hf)
                            tma_load_4d(sQ + L * Q_TILE + hf * Q_HALF, &tmQ, hf * 64, it.first + it.row0(L), it.head, 0, &q_full[L],
                                        once);
                    }
                    __syncwarp();
                    if (!all_wait(&q_full[L], qn & 1u)) { ok = false; break; }
                    ++qn;
                }
                for (int t = 0; t < all; ++t, k.next()) {
                    if (t >= n) {                        // only the other lane reads it
                        if (!all_wait(&full[k.slot], k.phase)) { ok = false; break; }
                        if (leader) mbar_arrive(&empty[k.slot]);
                        continue;
                    }
                    // S goes over the scores of the tile before and the weights of the one before that
                    if ((cnt > 0 && !all_wait(&s_free[L], (cnt - 1) & 1u)) ||
                        (cnt > 1 && !all_wait(&pv_done[2 * L + (cnt & 1u)], (cnt - 2) >> 1 & 1u)) || !all_wait(&full[k.slot], k.phase)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    issue_scores<DH>(leader, at, cnt, qd, dk + (uint64_t)((uint32_t)(k.slot * TILE) >> 4));
                    commit(leader, &s_full[L]);
                    commit(leader, &empty[k.slot]);
                    if (t == n - 1) commit(leader, &q_free[L]);
                    ++cnt;
                }
            }
            commit(leader, &drain[L]);                   // nothing of this thread's in tensor memory in flight
            mbar_wait(&drain[L], 0);
        } else if (role == 3 || role == 4) {
            // ---- P V of lane L
            const int L = role - 3;
            const uint64_t dv = smem_desc_sw128_mn(smem_u32(ring), HALF);
            const uint32_t at = tmem + (uint32_t)L * LANE_COLS, leader = elect_leader();
            Cursor v(1, NST);
            uint32_t cnt = 0;
            bool ok = true;
            while (ok && it.next()) {
                const int n = it.key_tiles<KEYS>(L), all = it.key_tiles<KEYS>(), keys = it.keys(L);
                for (int t = 0; t < all; ++t, v.next()) {
                    if (!all_wait(&full[v.slot], v.phase)) { ok = false; break; }
                    if (t >= n) {
                        if (leader) mbar_arrive(&empty[v.slot]);
                        continue;
                    }
                    const int nv = keys - t * KEYS;      // keys from this tile on
                    if (nv < KEYS && (nv & 15)) clear_rows<DH>(ring + (size_t)v.slot * TILE, nv, lane);
                    if (!all_wait(&p_full[2 * L + (cnt & 1u)], cnt >> 1 & 1u)) { ok = false; break; }
                    tc_fence_after();
                    issue_pv<DH>(leader, at, cnt, dv + (uint64_t)((uint32_t)(v.slot * TILE) >> 4), nv, t > 0);
                    commit(leader, &pv_done[2 * L + (cnt & 1u)]);
                    commit(leader, &empty[v.slot]);
                    ++cnt;
                }
            }
            commit(leader, &drain[2 + L]);
            mbar_wait(&drain[2 + L], 0);
        }
        __syncwarp();
        tc_fence_before();
        __syncthreads();
        if (warp == SOFT_WARPS) {
            tc_fence_after();
            tmem_dealloc(tmem, 512);
        }
        return;
    }

    // ---- softmax and epilogue
    asm volatile(EVS_ATTN_SOFT_REGS);
    SoftThread<DH> th;
    th.init(warp, lane, tmem, exchange);
    const int L = th.lane;
    const float sl = a.scale * LOG2E;
    uint32_t cnt = 0;                                    // tiles of this lane
    bool ok = true;                                      // a wait that ran out ends all later ones; barriers go on
    auto wait = [&](uint64_t* bar, uint32_t phase) {
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar, phase)) != 0;
    };
    auto arrive = [&](uint64_t* bar) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };
    // P V of tile cnt - 1. That of two tiles before a tile whose scores are there is done, since S went over its
    // weights: so a barrier for even and one for odd tiles are never a phase ahead of a wait.
    auto before = [&]() {
        if (cnt > 0) wait(&pv_done[2 * L + ((cnt - 1) & 1u)], (cnt - 1) >> 1 & 1u);
    };
    bool more = it.next();
    while (more) {
        const int rows = it.rows(L), n = it.key_tiles<KEYS>(L), row0 = it.row0(L), head = it.head;
        const int row_at = it.first + row0;
        const bool work = (th.row & ~31) < rows;         // of this warp
        th.begin();
        for (int t = 0; t < n; ++t) {
            wait(&s_full[L], cnt & 1u);
            uint32_t x[SoftThread<DH>::N];
            if (work) {
                tc_fence_after();
                th.load(x, cnt);
            }
            arrive(&s_free[L]);
            if (work) {
                if ((t + 1) * KEYS > row0 + 1) th.mask_from(x, row0 + th.row + 1 - t * KEYS - th.half * (KEYS / 2));
                th.tile(x, sl, cnt, t == 0, before);
                tmem_wait_st();
            }
            arrive(&p_full[2 * L + (cnt & 1u)]);
            ++cnt;
        }
        // what needs nothing of the last product, while that runs
        float l = 0.f;
        if (rows > 0 && work) l = th.exchange(th.l, [](float x, float y) { return x + y; });
        more = it.next();
        if (rows <= 0) continue;
        before();
        if (work) {
            tc_fence_after();
            const bool live = th.row < rows;
            const int64_t row = row_at + th.row;
            // no key with any weight: zero output, lse -inf; a void row: NaN
            const float inv = ok ? (l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l)) : __int_as_float(0x7fc00000);
            bf16* dst = (bf16*)a.o + row * a.o_row + (int64_t)head * DH + th.half * (DH / 2);
#pragma unroll
            for (int c = 0; c < DH / 32; ++c) {
                uint32_t o[16], w[8];
                tmem_ld16_issue(th.o_at + (uint32_t)(c * 16), o);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = pack2(__uint_as_float(o[2 * j]) * inv, __uint_as_float(o[2 * j + 1]) * inv);
                if (live && a.o_vec) {
                    *reinterpret_cast<uint4*>(dst + c * 16) = make_uint4(w[0], w[1], w[2], w[3]);
                    *reinterpret_cast<uint4*>(dst + c * 16 + 8) = make_uint4(w[4], w[5], w[6], w[7]);
                } else if (live) {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        reinterpret_cast<uint16_t*>(dst)[c * 16 + j] = (uint16_t)(w[j >> 1] >> (j & 1) * 16);
                }
            }
            if (live && th.half == 0 && a.lse)
                a.lse[row * a.H + head] = !ok ? inv : l == 0.f ? -INFINITY : th.m * LN2 + logf(l);
            tc_fence_before();                           // these reads precede the next item's products
        }
        __syncwarp();
    }
    if (!ok && lane == 0 && a.flags) atomicOr(a.flags, (uint32_t)EVS_FLAG_TIMEOUT);
    rest_rows<bf16>(a, st[0], st[a.B], DH, blockIdx.x, gridDim.x, tid, 32 * SOFT_WARPS);
    tc_fence_before();
    __syncthreads();
}

// =========================================================================================
// On CUDA cores (fp32, narrow heads, strides that tensor maps cannot describe): a CTA takes 64 rows of one
// head. Tiles are numbered over the sequences as if each began a new 64 rows; a CTA behind the last one
// takes rows of no sequence.
// =========================================================================================
template <typename T, int DH> __global__ void __launch_bounds__(256) prompt_simt_kernel(PromptArgs a) {
    using S = Simt<T, DH, 4>;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    int* st = reinterpret_cast<int*>(smem_raw);
    typename S::Smem& sm = *reinterpret_cast<typename S::Smem*>(smem_raw + ((a.B + 1) * 4 + 15) / 16 * 16);
    pdl_wait();
    pdl_trigger();
    load_starts(a, st);
    const int h = blockIdx.y;
    int item = blockIdx.x, s = 0;
    for (; s < a.B; ++s) {
        const int n = (st[s + 1] - st[s] + S::ROWS - 1) / S::ROWS;
        if (item < n) {
            item = n - 1 - item;                         // the longest rows first
            break;
        }
        item -= n;
    }
    if (s == a.B) {
        if (h == 0) rest_rows<T>(a, st[0], st[a.B], DH, item, gridDim.x - (blockIdx.x - item), threadIdx.x, 256);
        return;
    }
    const int first = st[s], len = st[s + 1] - first, r0 = item * S::ROWS;
    const int g = h / (a.H / a.G);
    const T* q = (const T*)a.q + h * a.q_head;
    const T* k = (const T*)a.k + first * a.kv_row + g * a.kv_head;
    const T* v = (const T*)a.v + first * a.kv_row + g * a.kv_head;
    S w(sm);
    w.stage_q([&](int r) -> const T* { return r0 + r < len ? q + (int64_t)(first + r0 + r) * a.q_row : nullptr; }, a.scale);
    const int end = min(len, r0 + S::ROWS);
    for (int j0 = 0; j0 < end; j0 += S::KEYS) {
        const int nk = min(S::KEYS, end - j0);
        w.tile([&](int j) { return k + (int64_t)(j0 + j) * a.kv_row; }, [&](int j) { return v + (int64_t)(j0 + j) * a.kv_row; }, nk,
               [&](int r, int j) { return j0 + j <= r0 + r; });
    }
    w.finish([&](int r, int c, float o, float m, float l) {
        if (r0 + r >= len) return;
        const int64_t row = first + r0 + r;
        ((T*)a.o)[row * a.o_row + (int64_t)h * DH + c] = from_f32<T>(l > 0.f ? o / l : (l == 0.f ? 0.f : l));
        if (c == 0 && a.lse) a.lse[row * a.H + h] = l == 0.f ? -INFINITY : m + logf(l);
    });
}

// ---- host side ----------------------------------------------------------------------------------
bool valid_shape(const evs_prompt_attn_args* c) {
    if (!c || c->tokens < 0 || c->batch < 0 || c->heads < 1 || c->kv_heads < 1) return false;
    if (c->tokens > (1 << 24) || c->batch > 1024 || c->heads > 1024 || c->heads % c->kv_heads) return false;
    if (!(c->head_dim == 16 || c->head_dim == 32 || c->head_dim == 64 || c->head_dim == 128)) return false;
    if (c->batch == 0 && c->tokens > 0) return false;
    return c->dtype == EVS_DTYPE_F32 || c->dtype == EVS_DTYPE_BF16;
}

bool tensor_ok(const evs_prompt_attn_args& c) {
    return c.dtype == EVS_DTYPE_BF16 && (c.head_dim == 64 || c.head_dim == 128) &&
           map_ok(c.q, c.q_row, c.q_head, 0, c.heads > 1, false) && map_ok(c.k, c.kv_row, c.kv_head, 0, c.kv_heads > 1, false) &&
           map_ok(c.v, c.kv_row, c.kv_head, 0, c.kv_heads > 1, false);
}

template <int DH>
cudaError_t launch_tensor(const evs_prompt_attn_args& c, const PromptArgs& a, cudaStream_t stream) {
    // First: the runtime makes the device's context this thread's own, which the driver's encoding of the
    // maps does not and wants to find. The limit is that of any batch: this call's own would be lowered by
    // another thread's smaller call before the launch.
    const cudaError_t e =
        cudaFuncSetAttribute(prompt_tc_kernel<DH>, cudaFuncAttributeMaxDynamicSharedMemorySize, prompt_smem(DH, 1024));
    if (e != cudaSuccess) return e;
    CUtensorMap q, k, v;
    if (!make_rows_map(&q, c.q, Q_ROWS, DH, c.tokens, c.heads, 1, c.q_row, c.q_head, 0) ||
        !make_rows_map(&k, c.k, tile_keys(DH), DH, c.tokens, c.kv_heads, 1, c.kv_row, c.kv_head, 0) ||
        !make_rows_map(&v, c.v, tile_keys(DH), DH, c.tokens, c.kv_heads, 1, c.kv_row, c.kv_head, 0))
        return cudaErrorInvalidValue;
    const long long items = ((long long)c.tokens / 256 + c.batch) * c.heads;     // at most
    const int grid = (int)(items < kAttnGrid ? items : kAttnGrid);
    return launch_s(stream, prompt_tc_kernel<DH>, dim3(grid), dim3(THREADS), (size_t)prompt_smem(DH, c.batch), q, k, v, a);
}

template <typename T, int DH>
cudaError_t launch_simt(const evs_prompt_attn_args& c, const PromptArgs& a, cudaStream_t stream) {
    using S = Simt<T, DH, 4>;
    constexpr size_t most = sizeof(typename S::Smem) + (1024 + 1) * 4 + 16;
    const cudaError_t e = cudaFuncSetAttribute(prompt_simt_kernel<T, DH>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
    if (e != cudaSuccess) return e;
    const size_t smem = sizeof(typename S::Smem) + ((c.batch + 1) * 4 + 15) / 16 * 16;
    // one more than the sequences can fill, for the rest
    const dim3 grid(c.tokens / S::ROWS + c.batch + 1, c.heads);
    return launch_s(stream, prompt_simt_kernel<T, DH>, grid, dim3(256), smem, a);
}

cudaError_t launch(const evs_prompt_attn_args& c, cudaStream_t stream) {
    PromptArgs a{};
    a.q = c.q; a.k = c.k; a.v = c.v; a.o = c.o; a.lse = c.lse; a.starts = c.starts; a.flags = c.flags;
    a.q_row = c.q_row; a.q_head = c.q_head; a.kv_row = c.kv_row; a.kv_head = c.kv_head; a.o_row = c.o_row;
    a.N = c.tokens; a.B = c.batch; a.H = c.heads; a.G = c.kv_heads; a.zero_rest = c.zero_rest != 0;
    a.scale = c.scale != 0.f ? c.scale : 1.f / sqrtf((float)c.head_dim);
    a.o_vec = (uintptr_t)c.o % 16 == 0 && c.o_row % 8 == 0;
    if (tensor_ok(c)) {
        return c.head_dim == 64 ? launch_tensor<64>(c, a, stream) : launch_tensor<128>(c, a, stream);
    }
    const bool half = c.dtype == EVS_DTYPE_BF16;
    switch (c.head_dim) {
        case 128: return half ? launch_simt<bf16, 128>(c, a, stream) : launch_simt<float, 128>(c, a, stream);
        case 64: return half ? launch_simt<bf16, 64>(c, a, stream) : launch_simt<float, 64>(c, a, stream);
        case 32: return half ? launch_simt<bf16, 32>(c, a, stream) : launch_simt<float, 32>(c, a, stream);
        default: return half ? launch_simt<bf16, 16>(c, a, stream) : launch_simt<float, 16>(c, a, stream);
    }
}

}  // namespace
}  // namespace evs

extern "C" size_t evs_prompt_attention_workspace(const evs_prompt_attn_args* c) {
    return 0;
}

extern "C" evs_status evs_prompt_attention(const evs_prompt_attn_args* c, void* stream) {
    using namespace evs;
    if (!valid_shape(c)) return EVS_ERR_INVALID_ARG;
    if (c->tokens == 0) return EVS_OK;
    const int es = c->dtype == EVS_DTYPE_F32 ? 4 : 2;
    if (!c->q || !c->k || !c->v || !c->o || !c->starts) return EVS_ERR_INVALID_ARG;
    if (((uintptr_t)c->q | (uintptr_t)c->k | (uintptr_t)c->v | (uintptr_t)c->o) % es) return EVS_ERR_INVALID_ARG;
    if (c->q_row < c->head_dim || c->kv_row < c->head_dim || c->o_row < (long long)c->heads * c->head_dim) return EVS_ERR_INVALID_ARG;
    if ((c->heads > 1 && c->q_head < c->head_dim) || (c->kv_heads > 1 && c->kv_head < c->head_dim)) return EVS_ERR_INVALID_ARG;
    if (!(c->scale >= 0.f) || isinf(c->scale) || (c->scale > 0.f && c->scale < 1e-30f)) return EVS_ERR_INVALID_ARG;
    return status_of(launch(*c, (cudaStream_t)stream));
}
