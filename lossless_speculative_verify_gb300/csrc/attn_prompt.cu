// Causal attention over whole prompts packed behind each other (evs_prompt_attention).
//
//   o_i = sum_{j <= i} exp(scale q_i.k_j - m) v_j / l,  lse_i = m + log l, within each sequence.
//
// On the tensor cores an item is 256 query rows of one head of one sequence, 128 for each lane (see
// attn_tiles.cuh), and the K/V tiles up to its diagonal, which TMA brings once for both. A persistent grid
// takes the items in the order of their length, longest first, forwards and backwards in turn, so that the
// CTAs end together: lengths are on the device, and each role of a CTA walks the same order by itself. Few
// items are dealt in runs of tiles instead.
// Warps 0-15: softmax and output; 16: TMA of K and V; 17 and 18: Q and the scores of the lanes; 19 and 20: P V;
// 21-23 look through V.
//
// Measured, bf16, heads of 128: 32768 tokens x 8 heads 1.30 ms alone (1.7 PFLOP/s; 0.92 us for a tile of 80 keys x 256
// rows, 0.82 with the products alone) and up to 1.44 back to back, at the power limit; 8192 x 8 100 us (256 items on
// 152 SMs), 13 prompts of 16381 tokens x 32 heads 205 us (an item's start and end about 2.5 us, and a third of its
// tiles' work is on the diagonal). Heads of 64: 16384 x 16 600 us (0.92 PFLOP/s: a score's softmax costs the same
// beside half of the products).
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
    // Items in runs (below): of worker w slot 2 w + 1 is for an item that begins in its run, 2 w for one that began
    // before. o four columns at a time, [slot][dh / 4][256][4]; (m, l) in natural units. jobs[w]: the item that w's
    // run begins within.
    float* po;
    float2* pml;
    struct Job* jobs;
};
struct Job {
    int valid, first, len, head, tile, start, run, pad;
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
// (sequences by length, longest first: which, and their items of 256 rows; or with runs where each begins on the
// axis), then Q and the ring on 1024 bytes.
constexpr int SCANNERS = 3;              // warps that look through V
constexpr int BARRIERS = 384;           // and whether V had values that are not finite
constexpr int small_smem(int B) { return 1024 + BARRIERS + (3 * B + 3) * 4; }

// The item a CTA is at: its sequence's first row and length, its head and 256 rows.
struct Item {
    int first, len, head, tile;

    static __device__ __forceinline__ int* starts() {
        extern __shared__ uint8_t smem_raw[];
        return reinterpret_cast<int*>(smem_raw + 1024 + BARRIERS);
    }
    // of lane L: its first row, rows, keys, tiles of K keys; of the item: tiles
    __device__ __forceinline__ int row0(int L) const { return tile * 256 + L * 128; }
    __device__ __forceinline__ int rows(int L) const { return min(128, len - row0(L)); }
    __device__ __forceinline__ int keys(int L) const { return min(len, row0(L) + 128); }
    template <int K> __device__ __forceinline__ int lane_tiles(int L) const { return rows(L) > 0 ? (keys(L) + K - 1) / K : 0; }
    template <int K> __device__ __forceinline__ int item_tiles() const { return (keys(1) + K - 1) / K; }
};

// Whole items. Level v holds the items of v x 256 rows and their keys: one for each head of each
// sequence that is as long.
struct Items : Item {
    static constexpr bool RUNS = false;
    const PromptArgs& a;
    int round, base, level, count;

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
    template <int K> __device__ __forceinline__ int t_lo() const { return 0; }
    template <int K> __device__ __forceinline__ int tiles() const { return item_tiles<K>(); }
    template <int K> __device__ __forceinline__ int tiles(int L) const { return lane_tiles<K>(L); }
    // fills what the kernel's start gives: sequences by length
    static __device__ __forceinline__ void prepare(const PromptArgs& a) {
        const int* st = starts();
        for (int s = threadIdx.x; s < a.B; s += THREADS) {
            const int n = (st[s + 1] - st[s] + 255) >> 8;
            int before = 0;
            for (int o = 0; o < a.B; ++o) {
                const int m = (st[o + 1] - st[o] + 255) >> 8;
                before += m > n || (m == n && o < s);
            }
            order(a)[before] = s;
            of(a)[before] = n;
        }
    }
};

// Where there are too few items for that to end evenly, or for every SM to have one: the items of all heads of all
// sequences lie end to end on an axis in units of 16 keys, each behind RUN_OVER units of its own cost, and worker w
// takes the tiles that begin in [W w, W (w + 1)). Items that a run ends in leave partials, which a second launch
// joins.
constexpr int RUN_OVER = 20;             // Q, first scores, output or partials: about 4 us, a tile of 5 units takes 0.92
__host__ __device__ inline int item_cost(int tile) { return 16 * (tile + 1) + RUN_OVER; }
__host__ __device__ inline int items_cost(int n) { return 8 * n * (n + 1) + RUN_OVER * n; }   // of the first n of a head
// the item's first tile of K keys that begins at unit u of it or behind
template <int K> __device__ __forceinline__ int run_tile(int u) { return (max(u - RUN_OVER, 0) + K / 16 - 1) / (K / 16); }

struct Runs : Item {
    static constexpr bool RUNS = true;
    const PromptArgs& a;
    int seq, start;                      // the item's sequence, where it begins on the axis (-1: before the first item)

    static __device__ __forceinline__ int* pre(const PromptArgs& a) { return starts() + a.B + 1; }   // [B + 1], then W
    // (registers are short in the softmax threads: what is needed once an item stays in shared memory)
    __device__ __forceinline__ int run() const { return pre(a)[a.B + 1]; }
    __device__ __forceinline__ int lo() const { return min(pre(a)[a.B], run() * (int)blockIdx.x); }
    __device__ __forceinline__ int hi() const { return min(pre(a)[a.B], run() * ((int)blockIdx.x + 1)); }
    __device__ __forceinline__ int n_tiles() const { return (len + 255) >> 8; }
    __device__ __forceinline__ void at_sequence(int s) {
        seq = s;
        first = starts()[s];
        len = starts()[s + 1] - first;
    }
    __device__ __forceinline__ Runs(const PromptArgs& args) : a(args), start(-1) {}
    __device__ __forceinline__ void find(int lo) {
        int s0 = 0, s1 = a.B - 1;                        // the last sequence that begins at lo or before
        while (s0 < s1) {
            const int mid = (s0 + s1 + 1) >> 1;
            if (pre(a)[mid] <= lo) s0 = mid; else s1 = mid - 1;
        }
        at_sequence(s0);
        const int per_head = items_cost(n_tiles());
        int in = lo - pre(a)[s0];
        head = in / per_head;
        in -= head * per_head;
        tile = 0;
        for (int step = 1 << 15; step > 0; step >>= 1)   // the last item that begins at in or before
            if (tile + step < n_tiles() && items_cost(tile + step) <= in) tile += step;
        start = lo - in + items_cost(tile);
    }
    __device__ __forceinline__ bool next() {
        if (start < 0) {
            if (lo() >= hi()) return false;
            find(lo());
            return true;
        }
        start += item_cost(tile);
        if (start >= hi()) return false;
        if (++tile == n_tiles()) {
            tile = 0;
            if (++head == a.H) {
                head = 0;
                int s = seq + 1;
                while (pre(a)[s + 1] == pre(a)[s]) ++s;  // (one is behind: the axis goes on)
                at_sequence(s);
            }
        }
        return true;
    }
    template <int K> __device__ __forceinline__ int t_lo() const { return min(run_tile<K>(lo() - start), item_tiles<K>()); }
    template <int K> __device__ __forceinline__ int t_hi() const { return min(run_tile<K>(hi() - start), item_tiles<K>()); }
    template <int K> __device__ __forceinline__ int tiles() const { return max(t_hi<K>() - t_lo<K>(), 0); }
    template <int K> __device__ __forceinline__ int tiles(int L) const { return max(min(t_hi<K>(), lane_tiles<K>(L)) - t_lo<K>(), 0); }
    static __device__ __forceinline__ void prepare(const PromptArgs& a) {
        if (threadIdx.x >= 32) return;
        const int* st = starts();
        const int lane = threadIdx.x;
        int run = 0;
        for (int b0 = 0; b0 < a.B; b0 += 32) {
            const int b = b0 + lane;
            int x = b < a.B ? a.H * items_cost((st[b + 1] - st[b] + 255) >> 8) : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            if (b < a.B) pre(a)[b + 1] = run + x;
            run += __shfl_sync(0xffffffffu, x, 31);
        }
        if (lane == 0) {
            pre(a)[0] = 0;
            pre(a)[a.B + 1] = max(2 * RUN_OVER, (run + (int)gridDim.x - 1) / (int)gridDim.x);
        }
    }
};

constexpr int prompt_smem(int dh, int B) { return small_smem(B) + 1024 + 2 * Q_ROWS * dh * 2 + ring_slots(dh) * tile_bytes(dh); }
static_assert(prompt_smem(64, 1024) <= 227 * 1024 && prompt_smem(128, 1024) <= 227 * 1024, "shared memory of an SM");

// Adds the values of V that are not finite, which were cleared in the item's tiles of its own rows, to the rows that
// read them: in the output, or in partials. A row reads what the row before it reads, and one key more: so their sums
// are carried from row to row, and each row is written once, however many there are (13 prompts of 1260 rows x 32 heads
// of nothing else: 1.15 ms, with a pass over the rows for each key 41). part: 0 and 1 are the lanes, the rest has
// nothing to do.
template <int DH, class It> __device__ __forceinline__ void mend(const PromptArgs& a, const It& it, int part, int lane) {
    constexpr int KEYS = tile_keys(DH);
    if (part > 1) return;
    const int L = part, n = it.template tiles<KEYS>(L), k0 = it.template t_lo<KEYS>() * KEYS, row0 = it.row0(L), rows = it.rows(L);
    int slot = -1;
    if constexpr (It::RUNS) {
        if (n < it.template lane_tiles<KEYS>(L)) slot = 2 * blockIdx.x + (it.lo() > it.start ? 0 : 1);
    }
    const bf16* v = (const bf16*)a.v + (int64_t)it.first * a.kv_row + it.head / (a.H / a.G) * a.kv_head;
    const int begin = max(it.tile * 256, k0), end = min(k0 + n * KEYS, row0 + rows);   // keys that were looked through
    float sum[DH / 32] = {};
    bool any = false;
    auto take = [&](int j) {
        float x[DH / 32];
        if (!bad_values<DH>(v + j * a.kv_row, lane, x)) return;
        any = true;
#pragma unroll
        for (int u = 0; u < DH / 32; ++u) sum[u] += x[u];
    };
#pragma unroll 1
    for (int j = begin; j < min(end, row0); ++j) take(j);
#pragma unroll 1
    for (int r = 0; r < rows; ++r) {
        if (row0 + r >= begin && row0 + r < end) take(row0 + r);
        if (!any) continue;
#pragma unroll
        for (int u = 0; u < DH / 32; ++u) {
            const int c = lane * (DH / 32) + u;
            if (sum[u] == 0.f) continue;
            if (slot >= 0) {
                a.po[((int64_t)slot * DH + (c & ~3)) * 256 + (L * 128 + r) * 4 + (c & 3)] += sum[u];
            } else {
                bf16* o = (bf16*)a.o + (int64_t)(it.first + row0 + r) * a.o_row + (int64_t)it.head * DH + c;
                *o = __float2bfloat16_rn(__bfloat162float(*o) + sum[u]);
            }
        }
    }
}

template <int DH, class It>
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
    uint64_t* scanned = drain + 4;                                         // [NST] V there and looked through
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(scanned + NST);
    volatile uint32_t* cleared = tmem_slot + 1;
    int* st = Items::starts();
    uint8_t* sQ = smem_raw + ((smem_u32(smem_raw) + small_smem(a.B) + 1023u & ~1023u) - smem_u32(smem_raw));
    uint8_t* ring = sQ + 2 * Q_TILE;
    static_assert((3 * NST + 20) * 8 + 2 * 4 <= BARRIERS, "barriers");
    // an even number: a slot is K's or V's, and each thread that waits for one has seen its phase before
    static_assert(NST % 2 == 0 && NST >= 4, "ring");
    static_assert(TILE == tile_bytes(DH) && HALF % 1024 == 0, "tiles on 1024 bytes");
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

    pdl_wait();
    // not before the wait: a predecessor's CTA on this SM may have yet to allocate
    if (warp == SOFT_WARPS) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    if (tid == 0) {
        for (int s = 0; s < NST; ++s) {
            mbar_init(&scanned[s], SCANNERS);
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
    if (tid == 0) *cleared = 0;
    load_starts(a, st);
    It::prepare(a);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // not before the allocation: a dependent's CTA that holds columns and waits for this grid could share the SM
    pdl_trigger();
    const uint32_t tmem = *tmem_slot;
    It it(a);
    if constexpr (It::RUNS) {
        if (tid == 0) {
            Runs r(a);
            const bool any = r.next();
            a.jobs[blockIdx.x] = Job{any && r.lo() > r.start, r.first, r.len, r.head, r.tile, r.start, r.run(), 0};
        }
    }

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
                const int n = 2 * it.template tiles<KEYS>(), g = it.head / (a.H / a.G), row = it.first + it.template t_lo<KEYS>() * KEYS;
                for (int j = 0; j < n; ++j) {
                    if ((used >> s & 1u) && !mbar_wait(&empty[s], ph)) { ok = false; break; }
                    used |= 1u << s;
                    uint8_t* dst = ring + (size_t)s * TILE;
                    mbar_arrive_expect_tx(&full[s], (uint32_t)TILE);
#pragma unroll
                    for (int hf = 0; hf < HALVES; ++hf)
                        tma_load_4d(dst + hf * HALF, j & 1 ? &tmV : &tmK, hf * 64, row + (j >> 1) * KEYS, g, 0, &full[s], keep);
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
                const int n = it.template tiles<KEYS>(L), all = it.template tiles<KEYS>();
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
                const int n = it.template tiles<KEYS>(L), all = it.template tiles<KEYS>(), k0 = it.template t_lo<KEYS>() * KEYS;
                const int keys = it.keys(L) - k0;        // from the piece's first on
                for (int t = 0; t < all; ++t, v.next()) {
                    if (!all_wait(&scanned[v.slot], v.phase)) { ok = false; break; }
                    if (t >= n) {
                        if (leader) mbar_arrive(&empty[v.slot]);
                        continue;
                    }
                    const int nv = keys - t * KEYS;      // keys from this tile on
                    uint8_t* tile = ring + (size_t)v.slot * TILE;
                    if (nv < KEYS && (nv & 15)) clear_rows<DH>(tile, nv, lane);
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
        } else if (role >= 5) {
            // ---- V of the item's own rows looked through
            const uint32_t leader = elect_leader();
            Cursor v(1, NST);
            bool ok = true;
            while (ok && it.next()) {
                const int all = it.template tiles<KEYS>(), k0 = it.template t_lo<KEYS>() * KEYS, end = it.keys(1) - k0, own = it.tile * 256 - k0;
                for (int t = 0; t < all; ++t, v.next()) {
                    if (!all_wait(&full[v.slot], v.phase)) { ok = false; break; }
                    const int from = max(own - t * KEYS, 0), to = min(end - t * KEYS, KEYS);
                    uint8_t* tile = ring + (size_t)v.slot * TILE;
                    if (from < to && scan_rows<DH>(tile, from, to, role - 5, SCANNERS, lane)) {
                        *cleared = 1;
                        clear_values<DH>(tile, from, to, role - 5, SCANNERS, lane);
                    }
                    if (leader) mbar_arrive(&scanned[v.slot]);
                }
            }
        }
        __syncwarp();
        tc_fence_before();
        __syncthreads();
        if (warp == SOFT_WARPS) {
            tc_fence_after();
            tmem_dealloc(tmem, 512);
        }
        if (*cleared) {
            // all is written: the lanes of this CTA's items, dealt among the warps here
            It again(a);
            for (int i = 0; again.next(); ++i) mend<DH>(a, again, (i + role) & 7, lane);
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
        const int rows = it.rows(L), n = it.template tiles<KEYS>(L), row0 = it.row0(L), head = it.head, row_at = it.first + row0;
        const int diagonal = row0 - it.template t_lo<KEYS>() * KEYS;   // the first row's own key, from the first tile on
        int slot = -1;                                   // for partials, where this is not all of the lane's tiles
        if constexpr (It::RUNS) {
            if (n < it.template lane_tiles<KEYS>(L)) slot = 2 * blockIdx.x + (it.lo() > it.start ? 0 : 1);
        }
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
                if ((t + 1) * KEYS > diagonal + 1) th.mask_from(x, diagonal + th.row + 1 - t * KEYS - th.half * (KEYS / 2));
                th.tile(x, sl, cnt, t == 0, before);
                tmem_wait_st();
            }
            arrive(&p_full[2 * L + (cnt & 1u)]);
            ++cnt;
        }
        // what needs nothing of the last product, while that runs
        float l = 0.f;
        if (n > 0 && work) l = th.exchange(th.l, [](float x, float y) { return x + y; });
        more = it.next();
        if (n == 0) continue;
        before();
        if (work && slot >= 0) {
            tc_fence_after();
            const int r = L * 128 + th.row;
            float* dst = a.po + ((int64_t)slot * DH + th.half * (DH / 2)) * 256 + r * 4;
#pragma unroll 1
            for (int c = 0; c < DH / 32; ++c) {
                uint32_t o[16];
                tmem_ld16_issue(th.o_at + (uint32_t)(c * 16), o);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    *reinterpret_cast<uint4*>(dst + (c * 4 + j) * 1024) = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
            }
            // once a wait has run out the rest is void: l = NaN makes the rows' outputs NaN
            if (th.half == 0)
                a.pml[slot * 256 + r] = ok ? make_float2(th.m * LN2, l) : make_float2(-INFINITY, __int_as_float(0x7fc00000));
            tc_fence_before();
        } else if (work) {
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
// Joins the partials of items that a run ended in: a CTA takes 1024 / dh rows of the item that worker
// blockIdx.y's run begins within, if that is the first run to do so; four columns of two rows a thread.
// A partial is scaled by __expf, of x <= 0: where it weighs (x > -10) off by 2^-19 at most, far inside the 2^-9 of the
// output's own rounding.
// Bounded by the latency of its loads: with those of one row behind the work on the other 2048 rows x 8 heads took
// 26.2 us in all for 24.6; two or four partials of both rows on their way at once take 24.6 and 26.1 (8192 rows: 100.6
// and 100.9 for 99.9).
// =========================================================================================
template <int DH> __global__ void __launch_bounds__(128) prompt_join_kernel(PromptArgs a) {
    constexpr int KEYS = tile_keys(DH), RW = 512 / DH, R = 2;
    pdl_wait();
    pdl_trigger();
    const int w = blockIdx.y + 1;
    const Job job = a.jobs[w];
    if (!job.valid || job.run * (w - 1) > job.start) return;
    Item it;
    it.first = job.first;
    it.len = job.len;
    it.head = job.head;
    it.tile = job.tile;
    const int c4 = threadIdx.x / RW, r0 = blockIdx.x * RW * R, L = r0 >> 7, all = it.lane_tiles<KEYS>(L);
    // the workers that have some of the lane's tiles (Runs::t_lo and t_hi): consecutive ones
    int v0 = w - 1, v1 = (job.start + item_cost(job.tile) - 1) / job.run;
    while (v0 <= v1 && run_tile<KEYS>(job.run * (v0 + 1) - job.start) == 0) ++v0;
    while (v1 >= v0 && run_tile<KEYS>(job.run * v1 - job.start) >= all) --v1;
    if (v0 >= v1) return;                                // one has written all of it
    float M[R] = {-INFINITY, -INFINITY}, l[R] = {};
    float4 O[R] = {};
    for (int v = v0; v <= v1; ++v) {
        const int64_t slot = 2 * v + (job.run * v > job.start ? 0 : 1);
        float2 mls[R];
        float4 os[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {                    // of both rows before either is worked on
            const int r = r0 + i * RW + threadIdx.x % RW;
            mls[i] = a.pml[slot * 256 + r];
            os[i] = *reinterpret_cast<const float4*>(a.po + (slot * DH + c4 * 4) * 256 + r * 4);
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float2 ml = mls[i];
            const float4 o = os[i];
            if (ml.x == -INFINITY && ml.y == 0.f) continue;   // only -inf scores
            if (ml.x > M[i]) {
                const float f = __expf(M[i] - ml.x);
                l[i] *= f;
                O[i].x *= f; O[i].y *= f; O[i].z *= f; O[i].w *= f;
                M[i] = ml.x;
            }
            const float p = ml.x == M[i] ? 1.f : __expf(ml.x - M[i]);
            l[i] = fmaf(ml.y, p, l[i]);
            O[i].x = fmaf(p, o.x, O[i].x);
            O[i].y = fmaf(p, o.y, O[i].y);
            O[i].z = fmaf(p, o.z, O[i].z);
            O[i].w = fmaf(p, o.w, O[i].w);
        }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int r = r0 + i * RW + threadIdx.x % RW;
        if (it.tile * 256 + r >= it.len) continue;
        const int64_t row = it.first + it.tile * 256 + r;
        const float inv = l[i] > 0.f ? 1.f / l[i] : (l[i] == 0.f ? 0.f : l[i]);
        bf16* dst = (bf16*)a.o + row * a.o_row + (int64_t)it.head * DH + c4 * 4;
        const uint32_t x = pack2(O[i].x * inv, O[i].y * inv), y = pack2(O[i].z * inv, O[i].w * inv);
        if (a.o_vec) {
            *reinterpret_cast<uint2*>(dst) = make_uint2(x, y);
        } else {
            uint16_t* to = reinterpret_cast<uint16_t*>(dst);
            to[0] = (uint16_t)x; to[1] = (uint16_t)(x >> 16); to[2] = (uint16_t)y; to[3] = (uint16_t)(y >> 16);
        }
        if (c4 == 0 && a.lse) a.lse[row * a.H + it.head] = l[i] == 0.f ? -INFINITY : M[i] + logf(l[i]);
    }
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
        auto k_at = [&](int j) { return k + (int64_t)(j0 + j) * a.kv_row; };
        auto v_at = [&](int j) { return v + (int64_t)(j0 + j) * a.kv_row; };
        if (j0 < r0) w.template tile<false>(k_at, v_at, nk, [](int, int) { return true; });
        else w.template tile<true>(k_at, v_at, nk, [&](int r, int j) { return j0 + j <= r0 + r; });
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

// Whether items are dealt in runs: where the longest of them would end far behind the mean of the SMs, if the
// sequences were of one length (the lengths are on the device). Runs cost their own starts, partials and a launch:
// 256 items of 8192 tokens, 54 units apart, 104 us in runs and 98 whole; 700 tokens x 8 heads (56) 19 and 14; 2048
// tokens x 8 heads (109) 24.6 and 29.6; 4096 (145) 43 and 52; 16384 x 2 heads 104 and 180. Batches of one long prompt
// and many short ones look shorter than they are: 16384 rows x 2 heads beside three requests of 24 rows take 97 to 105
// us, in runs, and 188 beside seven, in whole items; 8192 x 4 heads 60 to 64 alone, 99 beside four of 512.
constexpr int RUNS_WORTH = 80;
bool use_runs(const evs_prompt_attn_args& c) {
    if (c.dtype != EVS_DTYPE_BF16 || (c.head_dim != 64 && c.head_dim != 128)) return false;
    const long long n = ((long long)c.tokens + c.batch * 256LL - 1) / (c.batch * 256LL);   // items of a head
    if (n * c.batch * c.heads > 4096) return false;
    const double longest = item_cost((int)n - 1), mean = (double)items_cost((int)n) * c.batch * c.heads / kAttnGrid;
    return longest > mean + RUNS_WORTH;
}
size_t runs_workspace(const evs_prompt_attn_args& c, PromptArgs* a) {
    size_t off = 0;
    auto take = [&](size_t bytes) {
        char* p = a ? (char*)c.workspace + off : nullptr;
        off = round256(off + bytes);
        return p;
    };
    char* po = take((size_t)2 * kAttnGrid * 256 * c.head_dim * 4);
    char* ml = take((size_t)2 * kAttnGrid * 256 * 8);
    char* jobs = take((size_t)kAttnGrid * sizeof(Job));
    if (a) {
        a->po = (float*)po;
        a->pml = (float2*)ml;
        a->jobs = (Job*)jobs;
    }
    return off;
}

template <int DH, class It>
cudaError_t launch_items(const evs_prompt_attn_args& c, const PromptArgs& a, int grid, cudaStream_t stream) {
    // First: the runtime makes the device's context this thread's own, which the driver's encoding of the
    // maps does not and wants to find. The limit is that of any batch: this call's own would be lowered by
    // another thread's smaller call before the launch.
    const cudaError_t e =
        cudaFuncSetAttribute(prompt_tc_kernel<DH, It>, cudaFuncAttributeMaxDynamicSharedMemorySize, prompt_smem(DH, 1024));
    if (e != cudaSuccess) return e;
    CUtensorMap q, k, v;
    if (!make_rows_map(&q, c.q, Q_ROWS, DH, c.tokens, c.heads, 1, c.q_row, c.q_head, 0) ||
        !make_rows_map(&k, c.k, tile_keys(DH), DH, c.tokens, c.kv_heads, 1, c.kv_row, c.kv_head, 0) ||
        !make_rows_map(&v, c.v, tile_keys(DH), DH, c.tokens, c.kv_heads, 1, c.kv_row, c.kv_head, 0))
        return cudaErrorInvalidValue;
    return launch_s(stream, prompt_tc_kernel<DH, It>, dim3(grid), dim3(THREADS), (size_t)prompt_smem(DH, c.batch), q, k, v, a);
}

template <int DH> cudaError_t launch_tensor(const evs_prompt_attn_args& c, PromptArgs& a, cudaStream_t stream) {
    const long long items = ((long long)c.tokens / 256 + c.batch) * c.heads;     // at most
    if (!use_runs(c)) return launch_items<DH, Items>(c, a, (int)(items < kAttnGrid ? items : kAttnGrid), stream);
    runs_workspace(c, &a);
    const cudaError_t e = launch_items<DH, Runs>(c, a, kAttnGrid, stream);
    if (e != cudaSuccess) return e;
    return launch_s(stream, prompt_join_kernel<DH>, dim3(256 * DH / 1024, kAttnGrid - 1), dim3(128), 0, a);
}

template <typename T, int DH>
cudaError_t launch_simt(const evs_prompt_attn_args& c, const PromptArgs& a, cudaStream_t stream) {
    using S = Simt<T, DH, 4>;
    constexpr size_t most = sizeof(typename S::Smem) + (1024 + 1) * 4 + 16;
    if (most > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(prompt_simt_kernel<T, DH>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
        if (e != cudaSuccess) return e;
    }
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
    using namespace evs;
    return valid_shape(c) && c->tokens > 0 && use_runs(*c) ? runs_workspace(*c, nullptr) : 0;
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
    if (!(c->scale == 0.f || (c->scale >= 1e-30f && c->scale <= 1e30f))) return EVS_ERR_INVALID_ARG;
    const size_t need = evs_prompt_attention_workspace(c);
    if (need > 0 && (!c->workspace || (uintptr_t)c->workspace % 256)) return EVS_ERR_INVALID_ARG;
    if (c->ws_bytes < need) return EVS_ERR_CAPACITY;
    return status_of(launch(*c, (cudaStream_t)stream));
}
