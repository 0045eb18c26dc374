// Attention of a tree of drafted tokens over each sequence's cache (evs_tree_attention): a node reads the
// cached rows and the nodes on its path to the root.
//
//   o_i = sum_j exp(scale q_i.k_j - m) v_j / l over them, lse_i = m + log l.
//
// Two launches: partial sums (o unnormalised, m, l) per run of key tiles, then a combine that merges a
// row's partials and normalises. A segment is a K/V head of a sequence: its rows are the nodes' queries of
// the heads that share it (row r = node * group + head in the group), its keys the cached rows in tiles
// and then the nodes in one or two more, masked by ancestry. The segments' tiles laid end to end make an
// axis that workers take in equal runs, so ragged lengths balance on the device; a run may cross segments.
//
// Measured, bf16, heads of 128: 64 single tokens x 32 heads of 8 K/V heads over up to 4096 rows 104 us (its K/V at
// 6.5 TB/s), 4 x 41 nodes x 32 heads over up to 32768 rows 200 us (6.7 TB/s), 16 x 60 nodes x 32 heads of 8 over up
// to 8192 rows 82 us, of which the join is 10.
#include "attn_simt.cuh"
#include "attn_tiles.cuh"

namespace evs {
namespace {

using namespace attn;

constexpr int MAX_NODES = 128;
// What a segment costs beside its tiles, in tiles: Q, the partials. About 2.5 us, and 6 us where it has but a tile or
// two; a tile takes a pair of lanes 0.95 and a lane of its own 1.8 (heads of 64: half as much). With 1 everywhere the
// CTA with the segments of a sequence that has just begun ended 20 us behind the others of 60 (60 nodes x 32 heads x
// 16 sequences: 99 us, with 4 88, with 6 82), and 64 single tokens with heads of 64 took 65 us for 60.
constexpr int over_tiles(bool pair, int dh) { return pair ? 6 : dh == 64 ? 3 : 1; }

struct TreeArgs {
    const void *q, *kc, *vc, *kn, *vn;
    void* o;
    float* lse;
    const int32_t *cache_len, *parents, *lens;
    uint32_t* flags;
    int64_t q_ld, o_ld, c_row, c_head, c_seq, n_row, n_head, n_seq, parents_seq;
    int B, T, H, G, dh, cap, zero_rest;
    float scale;
    // Partials of up to seg_rows rows of a segment's row tile: o four columns at a time, [partial][dh / 4]
    // [rows to a multiple of four][4], so that those who write it (one a row) and those who read it (four
    // columns each) touch consecutive addresses; (m, l) in natural units. On the tensor cores worker w's of
    // segment s is number w + s: the pieces of the axis in order step on to the next worker, the next segment
    // or both, so no two share a number. On CUDA cores slot i of segment s is s * slots + i.
    float* po;
    float2* pml;
    int seg_rows, tiles, slots, tensor, pair, over;
    int* plan;                           // run length, then the axis' cost before each sequence, for one K/V head's row tile
    int q_vec, o_vec;                    // q on 16 bytes, o on four elements
};

__host__ __device__ inline int rows4(int rows) { return (rows + 3) & ~3; }

// Cached rows and nodes of sequence b. In the cache: nodes past the capacity do not exist as keys.
__device__ __forceinline__ int cached_of(const TreeArgs& a, int b, bool report) {
    const int n = __ldcg(a.cache_len + b);
    if (report && a.flags && (n < 0 || n > a.cap)) atomicOr(a.flags, (uint32_t)EVS_FLAG_BAD_LEN);
    return min(max(n, 0), a.cap);
}
__device__ __forceinline__ int nodes_of(const TreeArgs& a, int b, bool report) {
    if (!a.lens) return a.T;
    const int n = __ldcg(a.lens + b);
    if (report && a.flags && (n < 0 || n > a.T)) atomicOr(a.flags, (uint32_t)EVS_FLAG_BAD_LEN);
    return min(max(n, 0), a.T);
}
__device__ __forceinline__ int node_keys(const TreeArgs& a, int cached, int nodes, bool report) {
    if (a.kn || cached + nodes <= a.cap) return nodes;
    if (report && a.flags) atomicOr(a.flags, (uint32_t)EVS_FLAG_KV_OVERFLOW);
    return a.cap - cached;
}
// Parent of node i as stored: that plus one, 0 for a node below the cache
__device__ __forceinline__ uint8_t parent_of(const TreeArgs& a, int b, int i, bool report) {
    const int p = __ldcg(a.parents + b * a.parents_seq + i);
    if (p >= -1 && p < i) return (uint8_t)(p + 1);
    if (report && a.flags) atomicOr(a.flags, (uint32_t)EVS_FLAG_BAD_PARENT);
    return 0;
}

// =========================================================================================
// Partials on CUDA cores: a CTA takes 16 R rows of one segment and one slot's share of its keys.
// =========================================================================================
template <typename T, int DH, int R> __global__ void __launch_bounds__(256) tree_simt_kernel(TreeArgs a) {
    using S = Simt<T, DH, R>;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    typename S::Smem& sm = *reinterpret_cast<typename S::Smem*>(smem_raw);
    __shared__ uint8_t up[MAX_NODES];
    __shared__ uint32_t path[S::ROWS][MAX_NODES / 32];
    pdl_wait();
    pdl_trigger();
    const int grp = a.H / a.G, slot = blockIdx.x % a.slots, rt = blockIdx.x / a.slots, g = blockIdx.y, b = blockIdx.z;
    const bool report = rt == 0 && slot == 0 && g == 0 && threadIdx.x == 0;
    const int nodes = nodes_of(a, b, report), cached = cached_of(a, b, report), keys = node_keys(a, cached, nodes, report);
    const int r0 = rt * S::ROWS, rows = nodes * grp;
    if (a.slots == 1) {                                  // no second launch: nodes behind the tree's, too
        for (int r = max(r0, rows) + (int)threadIdx.x / 16; r < min(r0 + S::ROWS, a.T * grp); r += 16) {
            const int node = r / grp, h = g * grp + r - node * grp;
            const int64_t row = (int64_t)b * a.T + node;
            if (a.zero_rest)
                for (int c = threadIdx.x % 16; c < DH; c += 16) ((T*)a.o)[row * a.o_ld + (int64_t)h * DH + c] = from_f32<T>(0.f);
            if (a.lse && threadIdx.x % 16 == 0) a.lse[row * a.H + h] = -INFINITY;
        }
    }
    if (r0 >= rows) return;
    for (int i = threadIdx.x; i < nodes; i += 256) up[i] = parent_of(a, b, i, rt == 0 && slot == 0 && g == 0);
    S w(sm);
    const T* q = (const T*)a.q + (int64_t)b * a.T * a.q_ld + (int64_t)g * grp * DH;
    w.stage_q([&](int r) -> const T* {
        r += r0;
        return r < rows ? q + (int64_t)(r / grp) * a.q_ld + (int64_t)(r % grp) * DH : nullptr;
    }, a.scale);
    __syncthreads();
    if (threadIdx.x < S::ROWS) {
        uint32_t bits[MAX_NODES / 32] = {};
        for (int i = min(r0 + (int)threadIdx.x, rows - 1) / grp + 1; i > 0; i = up[i - 1])
#pragma unroll
            for (int u = 0; u < MAX_NODES / 32; ++u)
                if ((i - 1) / 32 == u) bits[u] |= 1u << ((i - 1) & 31);
#pragma unroll
        for (int u = 0; u < MAX_NODES / 32; ++u) path[threadIdx.x][u] = bits[u];
    }
    __syncthreads();
    // the cached rows of this slot, and in the last slot the nodes
    const T *kc = (const T*)a.kc + b * a.c_seq + g * a.c_head, *vc = (const T*)a.vc + b * a.c_seq + g * a.c_head;
    const int lo = (int)((int64_t)cached * slot / a.slots), hi = (int)((int64_t)cached * (slot + 1) / a.slots);
    for (int j0 = lo; j0 < hi; j0 += S::KEYS)
        w.template tile<false>([&](int j) { return kc + (int64_t)(j0 + j) * a.c_row; }, [&](int j) { return vc + (int64_t)(j0 + j) * a.c_row; },
               min(S::KEYS, hi - j0), [](int, int) { return true; });
    if (slot == a.slots - 1) {
        const T *kn = a.kn ? (const T*)a.kn + b * a.n_seq + g * a.n_head : kc + cached * a.c_row;
        const T *vn = a.kn ? (const T*)a.vn + b * a.n_seq + g * a.n_head : vc + cached * a.c_row;
        const int64_t ld = a.kn ? a.n_row : a.c_row;
        for (int j0 = 0; j0 < keys; j0 += S::KEYS)
            w.template tile<true>([&](int j) { return kn + (int64_t)(j0 + j) * ld; }, [&](int j) { return vn + (int64_t)(j0 + j) * ld; },
                   min(S::KEYS, keys - j0), [&](int r, int j) { return path[r][(j0 + j) >> 5] >> ((j0 + j) & 31) & 1u; });
    }
    if (a.slots == 1) {                                  // all of the keys: no partials
        w.finish([&](int r, int c, float o, float m, float l) {
            r += r0;
            const int node = r / grp, h = g * grp + r - node * grp;
            if (r >= rows) return;
            const int64_t row = (int64_t)b * a.T + node;
            ((T*)a.o)[row * a.o_ld + (int64_t)h * DH + c] = from_f32<T>(l > 0.f ? o / l : (l == 0.f ? 0.f : l));
            if (c == 0 && a.lse) a.lse[row * a.H + h] = l == 0.f ? -INFINITY : m + logf(l);
        });
        return;
    }
    const int64_t at = ((int64_t)b * a.G + g) * a.slots + slot;
    float* po = a.po + at * rows4(a.seg_rows) * DH;
    w.finish([&](int r, int c, float o, float m, float l) {
        r += r0;
        if (r >= rows) return;
        po[((c >> 2) * rows4(a.seg_rows) + r) * 4 + (c & 3)] = o;
        if (c == 0) a.pml[at * a.seg_rows + r] = make_float2(m, l);
    });
}

// =========================================================================================
// Partials on the tensor cores (bf16, head width 64 or 128; see attn_tiles.cuh). In segments of more than
// 128 rows a CTA is a worker: its lanes are two row tiles, and each K/V tile that TMA brings serves both.
// Otherwise each lane is a worker of its own, with half of the ring.
// Warps 16 and 17: TMA of the lanes; 18 and 19: their scores; 20 and 21: P V.
// =========================================================================================
// A worker's share of a segment: tiles t0 .. t0 + n - 1 of its nt, the first ntc of which are of the cache.
struct Piece {
    int b, g, rt, t0, n, nt, ntc, cached, nodes, keys, seg, start;
};
// Tiles of a segment
template <int DH> __device__ __forceinline__ int cache_tiles(int cached) { return (cached + tile_keys(DH) - 1) / tile_keys(DH); }
template <int DH> __device__ __forceinline__ int node_tiles(int nodes) { return (nodes + tile_keys(DH) - 1) / tile_keys(DH); }

constexpr int BARRIERS = 304;           // and whether nodes' V had values that are not finite
constexpr int small_smem(int B) { return 1024 + BARRIERS + 2 * MAX_NODES + (3 * B + 1) * 4; }
constexpr int tree_smem(int dh, int B) { return small_smem(B) + 1024 + 2 * Q_ROWS * dh * 2 + ring_slots(dh) * tile_bytes(dh); }
static_assert(tree_smem(64, 1024) <= 227 * 1024 && tree_smem(128, 1024) <= 227 * 1024, "shared memory of an SM");

// Adds the values of V that are not finite, which were cleared in the piece's tiles of nodes, to the partials of the
// rows below those nodes: the 128 of a lane from r_lane on. Each row is written once, with the sums over its node's path:
// those of the node before it where that is the same node or its parent, else gone through anew (a chain of 128 nodes of
// nothing else x 8 heads x 4 sequences: 0.16 ms, with a walk up for every node and row 75). The tree's parents and which nodes
// have such values are kept in the warp's registers.
template <int DH> __device__ __forceinline__ void mend(const TreeArgs& a, const Piece& p, int worker, int r_lane, int lane) {
    constexpr int KEYS = tile_keys(DH);
    const int grp = a.H / a.G, r_end = min(a.seg_rows, min(r_lane + 128, p.nodes * grp - p.rt * a.seg_rows));
    const int64_t ld = a.kn ? a.n_row : a.c_row;
    const bf16* v = a.kn ? (const bf16*)a.vn + p.b * a.n_seq + p.g * a.n_head
                         : (const bf16*)a.vc + p.b * a.c_seq + p.g * a.c_head + p.cached * a.c_row;
    float* po = a.po + (int64_t)(worker + p.seg) * rows4(a.seg_rows) * DH;
    uint32_t ups = 0, bad = 0;       // byte w: of node 32 w + lane; bits of nodes 32 lane ..
#pragma unroll
    for (int w = 0; w < MAX_NODES / 32; ++w)
        if (32 * w + lane < p.nodes) ups |= (uint32_t)parent_of(a, p.b, 32 * w + lane, false) << 8 * w;
    float x[DH / 32], sum[DH / 32] = {};
#pragma unroll 1
    for (int j = max(p.t0 - p.ntc, 0) * KEYS; j < min(p.keys, (p.t0 + p.n - p.ntc) * KEYS); ++j)
        if (bad_values<DH>(v + j * ld, lane, x) && lane == j >> 5) bad |= 1u << (j & 31);
    if (!__any_sync(0xffffffffu, bad != 0)) return;
    auto take = [&](int i) {
        if (!(__shfl_sync(0xffffffffu, bad, i >> 5) >> (i & 31) & 1u)) return;
        bad_values<DH>(v + i * ld, lane, x);
#pragma unroll
        for (int u = 0; u < DH / 32; ++u) sum[u] += x[u];
    };
    auto above = [&](int i) { return (int)(__shfl_sync(0xffffffffu, ups, i & 31) >> (i >> 5) * 8 & 0xffu) - 1; };
    int at = -1;                         // the node that sum is of
#pragma unroll 1
    for (int r = r_lane; r < r_end; ++r) {
        const int node = (p.rt * a.seg_rows + r) / grp;
        if (node != at) {
            const int parent = above(node);
            if (parent != at) {
#pragma unroll
                for (int u = 0; u < DH / 32; ++u) sum[u] = 0.f;
#pragma unroll 1
                for (int i = parent; i >= 0; i = above(i)) take(i);
            }
            take(node);
            at = node;
        }
#pragma unroll
        for (int u = 0; u < DH / 32; ++u) {
            const int c = lane * (DH / 32) + u;
            if (sum[u] != 0.f) po[((c >> 2) * rows4(a.seg_rows) + r) * 4 + (c & 3)] += sum[u];
        }
    }
}

template <int DH>
__global__ void __launch_bounds__(THREADS, 1)
tree_tc_kernel(const __grid_constant__ CUtensorMap tmKC, const __grid_constant__ CUtensorMap tmVC,
               const __grid_constant__ CUtensorMap tmKN, const __grid_constant__ CUtensorMap tmVN, TreeArgs a) {
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
    uint64_t* q_ready = pv_done + 4;                                       // [2] Q of a piece staged
    uint64_t* drain = q_ready + 2;                                         // [4]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 4);
    volatile uint32_t* cleared = tmem_slot + 1;                            // [2] of the lanes
    uint8_t* up = smem_raw + 1024 + BARRIERS;                               // [2][MAX_NODES] a lane's tree
    int* pre = reinterpret_cast<int*>(up + 2 * MAX_NODES);                 // [B + 1] cost of one row tile's axis before b
    int* len = pre + a.B + 1;                                              // [B] cached rows
    int* size = len + a.B;                                                 // [B] nodes
    uint8_t* sQ = smem_raw + ((smem_u32(smem_raw) + small_smem(a.B) + 1023u & ~1023u) - smem_u32(smem_raw));
    uint8_t* ring = sQ + 2 * Q_TILE;                                       // sQ: [2 lanes][halves][128 rows][128 B]
    static_assert((2 * NST + 18) * 8 + 3 * 4 <= BARRIERS, "barriers");
    static_assert(NST >= 6, "three slots a worker");
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const bool pairs = a.pair != 0;

    pdl_wait();
    // not before the wait: a predecessor's CTA on this SM may have yet to allocate
    if (warp == SOFT_WARPS) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    if (tid == 0) {
        for (int s = 0; s < NST; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], pairs ? 2 : 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&s_free[i], 8);
            mbar_init(&p_full[2 * i], 8);
            mbar_init(&p_full[2 * i + 1], 8);
            mbar_init(&pv_done[2 * i], 1);
            mbar_init(&pv_done[2 * i + 1], 1);
            mbar_init(&q_ready[i], 8);
            mbar_init(&drain[i], 1);
            mbar_init(&drain[2 + i], 1);
        }
        fence_barrier_init();
    }
    if (tid < 2) cleared[tid] = 0;
    for (int b = tid; b < a.B; b += THREADS) {
        len[b] = cached_of(a, b, blockIdx.x == 0);
        size[b] = nodes_of(a, b, blockIdx.x == 0);
        node_keys(a, len[b], size[b], blockIdx.x == 0);
    }
    __syncthreads();
    if (warp == 0) {
        int run = 0;
        for (int b0 = 0; b0 < a.B; b0 += 32) {
            const int b = b0 + lane;
            int x = b < a.B && size[b] > 0 ? cache_tiles<DH>(len[b]) + node_tiles<DH>(size[b]) + a.over : 0;
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
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // not before the allocation: a dependent's CTA that holds columns and waits for this grid could share the SM
    pdl_trigger();
    const uint32_t tmem = *tmem_slot;
    const int per_b = a.G * a.tiles, total = per_b * pre[a.B], workers = (int)gridDim.x * (pairs ? 1 : 2);
    const int W = max(1, (total + workers - 1) / workers);
    if (blockIdx.x == 0) {
        for (int b = tid; b <= a.B; b += THREADS) a.plan[1 + b] = pre[b];
        if (tid == 0) a.plan[0] = W;
    }
    // Lane L's run of the axis and slots of the ring
    const int L = warp < SOFT_WARPS ? warp >> 3 : warp & 1, role = (warp - SOFT_WARPS) >> 1;
    const int worker = pairs ? (int)blockIdx.x : 2 * (int)blockIdx.x + L;
    const int lo = min(total, W * worker), hi = min(lo + W, total);
    const int slot0 = pairs || L == 0 ? 0 : NST / 2, nslots = pairs ? NST : NST / 2;
    auto of_sequence = [&](Piece& p) {
        p.cached = len[p.b];
        p.nodes = size[p.b];
        p.ntc = cache_tiles<DH>(p.cached);
        p.nt = p.ntc + node_tiles<DH>(p.nodes);
        p.keys = node_keys(a, p.cached, p.nodes, false);
    };
    // keys of tile t, at least those
    auto keys_of = [&](const Piece& p, int t) { return t < p.ntc ? p.cached - t * KEYS : p.keys - (t - p.ntc) * KEYS; };
    // the run's first piece that has tiles, and the one behind p; n = 0: none
    auto fit = [&](Piece& p) {
        p.t0 = max(0, lo - p.start - a.over);
        p.n = max(0, min(p.nt, hi - p.start - a.over) - p.t0);
    };
    auto next_piece = [&](const Piece& c) -> Piece {
        Piece p = c;
        p.start = c.start + c.nt + a.over;
        p.n = 0;
        if (p.start >= hi) return p;
        ++p.seg;
        if (++p.rt == a.tiles) {
            p.rt = 0;
            if (++p.g == a.G) {                          // on to the next sequence that has nodes
                p.g = 0;
                do ++p.b; while (p.b < a.B - 1 && pre[p.b + 1] == pre[p.b]);
                p.seg = p.b * per_b;
                of_sequence(p);
            }
        }
        fit(p);
        return p;
    };
    auto first_piece = [&]() -> Piece {
        Piece p;
        p.n = 0;
        if (lo >= hi) return p;
        int b0 = 0, b1 = a.B - 1;                        // the last b with per_b * pre[b] <= lo
        while (b0 < b1) {
            const int mid = (b0 + b1 + 1) >> 1;
            if (per_b * pre[mid] <= lo) b0 = mid; else b1 = mid - 1;
        }
        const int cost = pre[b0 + 1] - pre[b0], r = (lo - per_b * pre[b0]) / cost;
        p.b = b0;
        p.g = r / a.tiles;
        p.rt = r - p.g * a.tiles;
        p.seg = b0 * per_b + r;
        p.start = per_b * pre[b0] + r * cost;
        of_sequence(p);
        fit(p);
        return p;
    };

    // Ring steps of a worker: K0 V0 K1 V1 ... over all its pieces, in the order of use.
    if (warp >= SOFT_WARPS) {
        asm volatile(EVS_ATTN_AUX_REGS);
        if (role == 0 && lane == 0 && (L == 0 || !pairs)) {
            // ---- TMA
            const uint64_t stream = policy_evict_first(), keep = policy_evict_last();
            int s = 0;
            uint32_t ph = 1, used = 0;                   // parity that a free slot has; slots in use so far
            bool ok = true;
            for (Piece p = first_piece(); p.n > 0 && ok; p = next_piece(p)) {
                const uint64_t pol = a.tiles > 1 ? keep : stream;
                for (int j = 0; j < 2 * p.n; ++j) {
                    const int at = slot0 + s, t = p.t0 + (j >> 1);
                    if ((used >> s & 1u) && !mbar_wait(&empty[at], ph)) { ok = false; break; }
                    used |= 1u << s;
                    const bool node = t >= p.ntc;
                    const CUtensorMap* m = node && a.kn ? (j & 1 ? &tmVN : &tmKN) : (j & 1 ? &tmVC : &tmKC);
                    const int row = !node ? t * KEYS : (t - p.ntc) * KEYS + (a.kn ? 0 : p.cached);
                    uint8_t* dst = ring + (size_t)at * TILE;
                    mbar_arrive_expect_tx(&full[at], (uint32_t)TILE);
#pragma unroll
                    for (int hf = 0; hf < HALVES; ++hf) tma_load_4d(dst + hf * HALF, m, hf * 64, row, p.g, p.b, &full[at], pol);
                    if (++s == nslots) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            if (!ok)                                     // loads in flight end before this CTA does (bounded)
                for (int i = 0; i < nslots; ++i)
                    if (used >> i & 1u) mbar_wait(&full[slot0 + i], i < s ? ph ^ 1u : ph);
        } else if (role == 1) {
            // ---- scores of lane L: those of the next tile as soon as this one's are in registers
            const uint64_t qd = smem_desc_sw128(smem_u32(sQ + L * Q_TILE)), dk = smem_desc_sw128(smem_u32(ring + slot0 * TILE));
            const uint32_t at = tmem + (uint32_t)L * LANE_COLS, leader = elect_leader();
            Cursor k(0, nslots);
            uint32_t cnt = 0, qn = 0;                    // tiles, pieces
            bool ok = true;
            for (Piece p = first_piece(); p.n > 0 && ok; p = next_piece(p)) {
                if (!all_wait(&q_ready[L], qn & 1u)) { ok = false; break; }
                ++qn;
                for (int t = 0; t < p.n; ++t, k.next()) {
                    // S goes over the scores of the tile before and the weights of the one before that. The ring's
                    // slot last: in a ring of three, V of the latter was in it, and a wait for a slot's next phase
                    // is one for that phase only if the one before is over
                    if ((cnt > 0 && !all_wait(&s_free[L], (cnt - 1) & 1u)) ||
                        (cnt > 1 && !all_wait(&pv_done[2 * L + (cnt & 1u)], (cnt - 2) >> 1 & 1u)) ||
                        !all_wait(&full[slot0 + k.slot], k.phase)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    issue_scores<DH>(leader, at, cnt, qd, dk + (uint64_t)((uint32_t)(k.slot * TILE) >> 4));
                    commit(leader, &s_full[L]);
                    commit(leader, &empty[slot0 + k.slot]);
                    ++cnt;
                }
            }
            commit(leader, &drain[L]);                   // nothing of this thread's in tensor memory in flight
            mbar_wait(&drain[L], 0);
        } else if (role == 2) {
            // ---- P V of lane L
            const uint64_t dv = smem_desc_sw128_mn(smem_u32(ring + slot0 * TILE), HALF);
            const uint32_t at = tmem + (uint32_t)L * LANE_COLS, leader = elect_leader();
            Cursor v(1, nslots);
            uint32_t cnt = 0;
            bool ok = true;
            for (Piece p = first_piece(); p.n > 0 && ok; p = next_piece(p)) {
                for (int t = 0; t < p.n; ++t, v.next()) {
                    if (!all_wait(&full[slot0 + v.slot], v.phase)) { ok = false; break; }
                    // a tile without keys (nodes past the capacity) still clears O where it is the first: one step of
                    // cleared rows
                    const int nv = max(keys_of(p, p.t0 + t), 0);
                    uint8_t* tile = ring + (size_t)(slot0 + v.slot) * TILE;
                    if (nv < KEYS && ((nv & 15) || nv == 0)) clear_rows<DH>(tile, nv, lane);
                    if (p.t0 + t >= p.ntc && scan_rows<DH>(tile, 0, min(nv, KEYS), 0, 1, lane)) {
                        cleared[L] = 1;
                        clear_values<DH>(tile, 0, min(nv, KEYS), 0, 1, lane);
                    } else if (pairs && p.t0 + t >= p.ntc) {
                        // zeros that the other lane's warp wrote and this one read are for this lane's products, too
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    if (!all_wait(&p_full[2 * L + (cnt & 1u)], cnt >> 1 & 1u)) { ok = false; break; }
                    tc_fence_after();
                    issue_pv<DH>(leader, at, cnt, dv + (uint64_t)((uint32_t)(v.slot * TILE) >> 4), max(nv, 1), t > 0);
                    commit(leader, &pv_done[2 * L + (cnt & 1u)]);
                    commit(leader, &empty[slot0 + v.slot]);
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
        // (where lanes share pieces, one may have cleared what the other would have found)
        if (role == 2 && (cleared[L] || (pairs && cleared[L ^ 1])))
            for (Piece p = first_piece(); p.n > 0; p = next_piece(p)) mend<DH>(a, p, worker, pairs ? L * 128 : 0, lane);
        return;
    }

    // ---- softmax
    asm volatile(EVS_ATTN_SOFT_REGS);
    SoftThread<DH> th;
    th.init(warp, lane, tmem, exchange);
    const int grp = a.H / a.G, in_lane = th.half * 128 + th.row;
    const float sl = a.scale * LOG2E;
    auto lane_sync = [&]() { named_bar_sync(9 + L, 256); };
    auto row_of = [&](const Piece& p) { return p.rt * a.seg_rows + (pairs ? L * 128 : 0) + th.row; };
    auto is_live = [&](const Piece& p, int r) {
        return (pairs ? L * 128 : 0) + th.row < a.seg_rows && r < p.nodes * grp;
    };
    // This thread's half of a Q row to shared memory, K-major, 128-byte swizzle. Rows on 16 bytes are copied
    // asynchronously, so that the next piece's come while this one's last tile is worked on; staged() ends it.
    auto stage = [&](const Piece& p) {
        const int r = row_of(p);
        const bool live = is_live(p, r);
        if (!__any_sync(0xffffffffu, live)) return;
        const int node = r / grp;
        const int64_t at = live ? ((int64_t)p.b * a.T + node) * a.q_ld + (int64_t)(p.g * grp + r - node * grp) * DH : 0;
        const bf16* src = (const bf16*)a.q + at;
        uint8_t* dst = sQ + L * Q_TILE + th.row * 128;
#pragma unroll
        for (int c = 0; c < DH / 16; ++c) {              // pieces of 8 columns
            const int col = th.half * (DH / 2) + c * 8;
            uint8_t* to = dst + (col >> 6) * Q_HALF + (((col >> 3 & 7) ^ (th.row & 7)) << 4);
            if (a.q_vec) {
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(to)), "l"(src + col), "r"(live ? 16 : 0)
                             : "memory");
            } else {
                uint32_t w[4] = {0, 0, 0, 0};
                if (live)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        w[j >> 1] |= (uint32_t) reinterpret_cast<const uint16_t*>(src)[col + j] << (j & 1) * 16;
                *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    };
    auto staged = [&]() {
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_ready[L]);
    };
    uint32_t cnt = 0;                                    // tiles so far
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
    Piece p = first_piece();
    if (p.n > 0) {
        stage(p);
        staged();
    }
    while (p.n > 0) {
        const int r = row_of(p);
        const bool live = is_live(p, r), work = __any_sync(0xffffffffu, live);
        const Piece nx = next_piece(p);
        // nodes that this row reads: bit j is the thread's j-th key of the first and of the second node tile
        uint64_t path0 = 0, path1 = 0;
        if (p.t0 + p.n > p.ntc) {
            if (in_lane < p.nodes) up[L * MAX_NODES + in_lane] = parent_of(a, p.b, in_lane, p.g == 0 && p.rt == 0);
            lane_sync();
            if (live)
                for (int i = r / grp + 1; i > 0; i = up[L * MAX_NODES + i - 1]) {
                    const int j = (i - 1) % KEYS - th.half * (KEYS / 2);
                    const uint64_t bit = j >= 0 && j < KEYS / 2 ? 1ull << j : 0;
                    path0 |= i > KEYS ? 0 : bit;
                    path1 |= i > KEYS ? bit : 0;
                }
            lane_sync();                                 // read before the next piece's
        }
        th.begin();
        for (int t = 0; t < p.n; ++t) {
            wait(&s_full[L], cnt & 1u);
            const int nv = keys_of(p, p.t0 + t), node = p.t0 + t - p.ntc;
            uint32_t x[SoftThread<DH>::N];
            if (work) {
                tc_fence_after();
                th.load(x, cnt);
            }
            arrive(&s_free[L]);
            if (t == p.n - 1 && nx.n > 0) stage(nx);     // the last scores are out: Q's place is free
            if (work) {
                if (nv < KEYS) th.mask_from(x, nv - th.half * (KEYS / 2));
                if (node >= 0) {
                    const uint64_t bits = node == 0 ? path0 : path1;
                    const uint32_t lo32 = (uint32_t)bits, hi32 = (uint32_t)(bits >> 32);
#pragma unroll
                    for (int j = 0; j < SoftThread<DH>::N; ++j)
                        if (!((j < 32 ? lo32 : hi32) >> (j & 31) & 1u)) x[j] = 0xff800000u;
                }
                th.tile(x, sl, cnt, t == 0, before);
                tmem_wait_st();
            }
            arrive(&p_full[2 * L + (cnt & 1u)]);
            ++cnt;
        }
        if (nx.n > 0) staged();                          // the next scores need not wait for the rest
        // ---- the piece's partials: o, then (m, l). Once a wait has run out, this piece's and those of the
        // worker's later ones are void: l = NaN makes the rows' outputs NaN, whether or not the caller
        // looks at the flag.
        before();
        if (work) {
            const float l = th.exchange(th.l, [](float x, float y) { return x + y; });
            tc_fence_after();
            const int64_t at = worker + p.seg;
            const int r_seg = (pairs ? L * 128 : 0) + th.row, ld = rows4(a.seg_rows) * 4;
            float* dst = a.po + at * rows4(a.seg_rows) * DH + (int64_t)th.half * (DH / 8) * ld + r_seg * 4;
#pragma unroll
            for (int c = 0; c < DH / 32; ++c) {
                uint32_t o[16];
                tmem_ld16_issue(th.o_at + (uint32_t)(c * 16), o);
                tmem_wait_ld();
                if (live) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        *reinterpret_cast<uint4*>(dst + (c * 4 + j) * ld) = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
                }
            }
            if (live && th.half == 0)
                a.pml[at * a.seg_rows + r_seg] = ok ? make_float2(th.m * LN2, l) : make_float2(-INFINITY, __int_as_float(0x7fc00000));
        }
        tc_fence_before();                               // these reads precede the next piece's products
        __syncwarp();
        p = nx;
    }
    if (!ok && lane == 0 && a.flags) atomicOr(a.flags, (uint32_t)EVS_FLAG_TIMEOUT);
    tc_fence_before();
    __syncthreads();
}

// =========================================================================================
// Combine. 128 threads take 512 / dh (node, head) rows of a sequence and K/V head at a time, four columns of
// one row each, and R such sets of rows at once, so that the loads of many small rows overlap (240 rows x 128
// segments of two or three partials: 18 us with one set, 10 with two; four were tried, and took 12). Where rows have many partials
// (and a CTA one set), up to four such groups of threads deal them among themselves.
// =========================================================================================
constexpr int GROUPS = 4;
template <typename T, int DH, int R> __global__ void __launch_bounds__(R == 1 ? 128 * GROUPS : 128) tree_combine_kernel(TreeArgs a) {
    constexpr int RW = 512 / DH, PB = R == 1 ? 8 : 2;    // rows of a set; partials of a row in flight
    const int tid = threadIdx.x & 127, part = R == 1 ? threadIdx.x >> 7 : 0, parts = R == 1 ? blockDim.x >> 7 : 1;
    const int grp = a.H / a.G, b = blockIdx.z, g = blockIdx.y, c4 = tid / RW, r0 = blockIdx.x * RW * R + tid % RW;
    // The partial kernel starts its dependents when all before it is done, so the lengths are there
    const int nodes = nodes_of(a, b, false);
    pdl_wait();
    pdl_trigger();
    float M[R] = {}, L[R] = {};
    float4 O[R] = {};
    auto add = [&](int i, float2 ml, float4 o) {
        // an empty partial may leave its o unwritten (one of NaN scores, or void, has l = NaN)
        if (ml.x == -INFINITY && ml.y == 0.f) return;
        if (ml.x > M[i]) {
            const float f = simt_exp<T>(M[i] - ml.x);
            L[i] *= f;
            O[i].x *= f; O[i].y *= f; O[i].z *= f; O[i].w *= f;
            M[i] = ml.x;
        }
        const float w = ml.x == M[i] ? 1.f : simt_exp<T>(ml.x - M[i]);
        L[i] = fmaf(ml.y, w, L[i]);
        O[i].x = fmaf(w, o.x, O[i].x);
        O[i].y = fmaf(w, o.y, O[i].y);
        O[i].z = fmaf(w, o.z, O[i].z);
        O[i].w = fmaf(w, o.w, O[i].w);
    };
    // The CTA's rows are of one row tile (where there are several, they have 256 rows, of which a CTA's are a part):
    // its partials, from the runs that the segment's tiles meet
    const int tile = a.tiles > 1 ? blockIdx.x * RW * R / a.seg_rows : 0;
    int64_t first = ((int64_t)b * a.G + g) * a.slots;
    int used = a.slots;
    if (a.tensor) {
        const int per_b = a.G * a.tiles, W = a.plan[0], before = a.plan[1 + b], cost = a.plan[2 + b] - before;
        const int in_b = g * a.tiles + tile, at = per_b * before + in_b * cost + a.over, run = at / W;
        first = run + (int64_t)b * per_b + in_b;
        used = (at + cost - a.over - 1) / W - run + 1;
    }
    const int in = r0 - tile * a.seg_rows, ml_step = a.seg_rows, o_step = DH * rows4(a.seg_rows);
    const float2* ml_at = a.pml + first * ml_step + in;
    const float* o_at = a.po + first * o_step + c4 * 4 * rows4(a.seg_rows) + in * 4;
    const int rows = nodes * grp;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        M[i] = -INFINITY;
        L[i] = 0.f;
        O[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll 1
    for (int s = part; s < used; s += PB * parts) {
        float2 ml[R][PB];
        float4 o[R][PB];
#pragma unroll
        for (int j = 0; j < PB; ++j) {
            const int at = s + j * parts;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                ml[i][j] = make_float2(-INFINITY, 0.f);
                o[i][j] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (at < used && r0 + i * RW < rows) {
                    ml[i][j] = ml_at[(int64_t)at * ml_step + i * RW];
                    o[i][j] = *reinterpret_cast<const float4*>(o_at + (int64_t)at * o_step + i * RW * 4);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < PB; ++j) add(i, ml[i][j], o[i][j]);
    }
    if constexpr (R == 1) {
        __shared__ float4 sum_o[GROUPS - 1][128];
        __shared__ float2 sum_ml[GROUPS - 1][128];
        if (parts > 1) {
            if (part > 0) {
                sum_o[part - 1][tid] = O[0];
                sum_ml[part - 1][tid] = make_float2(M[0], L[0]);
            }
            __syncthreads();
            if (part > 0) return;
            for (int p = 0; p < parts - 1; ++p) add(0, sum_ml[p][tid], sum_o[p][tid]);
        }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int r = r0 + i * RW, node = r / grp, h = g * grp + r - node * grp;
        if (r >= a.T * grp) break;
        const int64_t m = (int64_t)b * a.T + node;
        const bool live = node < nodes;
        if (a.lse && c4 == 0) a.lse[m * a.H + h] = !live || L[i] == 0.f ? -INFINITY : M[i] + logf(L[i]);
        if (!live && !a.zero_rest) continue;
        // no key with any weight: zero output, lse -inf
        const float inv = L[i] > 0.f ? 1.f / L[i] : (L[i] == 0.f ? 0.f : L[i]);
        T* dst = (T*)a.o + m * a.o_ld + (int64_t)h * DH + c4 * 4;
        const T w[4] = {from_f32<T>(O[i].x * inv), from_f32<T>(O[i].y * inv), from_f32<T>(O[i].z * inv), from_f32<T>(O[i].w * inv)};
        if (a.o_vec) {
            struct alignas(4 * sizeof(T)) Four { T x[4]; };
            *reinterpret_cast<Four*>(dst) = {{w[0], w[1], w[2], w[3]}};
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) dst[j] = w[j];
        }
    }
}

// ---- host side ----------------------------------------------------------------------------------
bool valid_shape(const evs_tree_attn_args* c) {
    if (!c || c->batch < 0 || c->nodes < 1 || c->heads < 1 || c->kv_heads < 1) return false;
    if (c->batch > 1024 || c->nodes > MAX_NODES || c->heads > 1024 || c->heads % c->kv_heads) return false;
    if ((long long)c->batch * c->nodes * c->heads > (1 << 24)) return false;
    if (!(c->head_dim == 16 || c->head_dim == 32 || c->head_dim == 64 || c->head_dim == 128)) return false;
    if (c->capacity < 0 || c->capacity > (1 << 30)) return false;
    return c->dtype == EVS_DTYPE_F32 || c->dtype == EVS_DTYPE_BF16;
}

// Row sizes and slots of the CUDA-core path: about four waves of the SMs at two CTAs each, or one slot, which needs
// no second launch, where the keys are few tiles of little work: that saves a call its host time and costs a replayed
// graph (4 sequences x 7 nodes x 4 heads of 16 over 128, 256, 448, 512 rows: a call 24 us with one slot and 28 with
// several; in a graph 6.7, 9.5, 13.6, 14.9 and 7.1, 7.4, 8.0, 8.4. The border lies between the last two).
constexpr long long ONE_SLOT = 2048;     // key tiles x rows x columns
int simt_rows(const evs_tree_attn_args& c) { return c.nodes * (c.heads / c.kv_heads) > 16 ? 64 : 16; }
void plan_simt(const evs_tree_attn_args& c, TreeArgs& a) {
    const int rows = c.nodes * (c.heads / c.kv_heads), per = simt_rows(c);
    const long long items = (long long)c.batch * c.kv_heads * ((rows + per - 1) / per);
    a.seg_rows = rows;
    a.tiles = 1;
    long long s = items > 0 ? (4 * 152 + items - 1) / items : 1;
    const long long most = c.capacity / 64 + 1;
    s = s < most ? s : most;
    if ((c.capacity / 64 + 1) * (long long)per * c.head_dim <= ONE_SLOT) s = 1;
    a.slots = (int)(s < 1 ? 1 : s);
}

bool tensor_ok(const evs_tree_attn_args& c) {
    if (c.dtype != EVS_DTYPE_BF16 || (c.head_dim != 64 && c.head_dim != 128)) return false;
    if (c.capacity > 0 && !(map_ok(c.k_cache, c.cache_row, c.cache_head, c.cache_seq, c.kv_heads > 1, c.batch > 1) &&
                            map_ok(c.v_cache, c.cache_row, c.cache_head, c.cache_seq, c.kv_heads > 1, c.batch > 1)))
        return false;
    return !c.k_nodes || (map_ok(c.k_nodes, c.node_row, c.node_head, c.node_seq, c.kv_heads > 1, c.batch > 1) &&
                          map_ok(c.v_nodes, c.node_row, c.node_head, c.node_seq, c.kv_heads > 1, c.batch > 1));
}

// false: sizes past the kernel's 32-bit positions
bool plan_tensor(const evs_tree_attn_args& c, TreeArgs& a, int& grid) {
    const long long rows = (long long)c.nodes * (c.heads / c.kv_heads);
    a.pair = rows > 128;
    a.over = over_tiles(a.pair, c.head_dim);
    a.seg_rows = (int)(rows < 256 ? rows : 256);
    a.tiles = (int)((rows + 255) / 256);
    const long long segs = (long long)c.batch * c.kv_heads * a.tiles, tiles =
        segs * (((long long)c.capacity + tile_keys(c.head_dim) - 1) / tile_keys(c.head_dim) + (c.nodes > tile_keys(c.head_dim) ? 2 : 1));
    if (tiles + segs * a.over >= (1LL << 30)) return false;
    grid = (int)(tiles < kAttnGrid ? tiles : kAttnGrid);
    a.tensor = 1;
    return true;
}

// Lays the partials out from base (or sizes them).
size_t carve(const evs_tree_attn_args& c, TreeArgs& a, int grid, char* base) {
    size_t off = 0;
    auto take = [&](size_t bytes) {
        char* p = base ? base + off : nullptr;
        off = round256(off + bytes);
        return p;
    };
    size_t n = (size_t)c.batch * c.kv_heads * a.tiles;   // segments
    n = a.tensor ? n + (size_t)grid * (a.pair ? 1 : 2) : n * a.slots;
    a.po = (float*)take(n * rows4(a.seg_rows) * c.head_dim * 4);
    a.pml = (float2*)take(n * a.seg_rows * 8);
    a.plan = (int*)take(((size_t)c.batch + 2) * 4);
    return off;
}

template <int DH>
cudaError_t launch_tensor(const evs_tree_attn_args& c, const TreeArgs& a, int grid, cudaStream_t stream) {
    // First: the runtime makes the device's context this thread's own, which the driver's encoding of the
    // maps does not and wants to find. The limit is that of any batch: this call's own would be lowered by
    // another thread's smaller call before the launch.
    const cudaError_t e = cudaFuncSetAttribute(tree_tc_kernel<DH>, cudaFuncAttributeMaxDynamicSharedMemorySize, tree_smem(DH, 1024));
    if (e != cudaSuccess) return e;
    CUtensorMap kc, vc, kn, vn;
    bool ok = true;
    if (c.capacity > 0)
        ok = make_rows_map(&kc, c.k_cache, tile_keys(DH), DH, c.capacity, c.kv_heads, c.batch, c.cache_row, c.cache_head, c.cache_seq) &&
             make_rows_map(&vc, c.v_cache, tile_keys(DH), DH, c.capacity, c.kv_heads, c.batch, c.cache_row, c.cache_head, c.cache_seq);
    if (ok && c.k_nodes)
        ok = make_rows_map(&kn, c.k_nodes, tile_keys(DH), DH, c.nodes, c.kv_heads, c.batch, c.node_row, c.node_head, c.node_seq) &&
             make_rows_map(&vn, c.v_nodes, tile_keys(DH), DH, c.nodes, c.kv_heads, c.batch, c.node_row, c.node_head, c.node_seq);
    if (!ok) return cudaErrorInvalidValue;
    if (c.capacity == 0) { kc = kn; vc = vn; }
    if (!c.k_nodes) { kn = kc; vn = vc; }
    return launch_s(stream, tree_tc_kernel<DH>, dim3(grid), dim3(THREADS), (size_t)tree_smem(DH, c.batch), kc, vc, kn, vn, a);
}

template <typename T, int DH, int R> cudaError_t launch_rows(const evs_tree_attn_args& c, const TreeArgs& a, cudaStream_t stream) {
    using S = Simt<T, DH, R>;
    if (sizeof(typename S::Smem) > 40 * 1024) {          // (beside the kernel's own)
        const cudaError_t e =
            cudaFuncSetAttribute(tree_simt_kernel<T, DH, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(typename S::Smem));
        if (e != cudaSuccess) return e;
    }
    const dim3 grid((a.seg_rows + S::ROWS - 1) / S::ROWS * a.slots, c.kv_heads, c.batch);
    return launch_s(stream, tree_simt_kernel<T, DH, R>, grid, dim3(256), sizeof(typename S::Smem), a);
}
template <typename T, int DH> cudaError_t launch_simt(const evs_tree_attn_args& c, const TreeArgs& a, cudaStream_t stream) {
    return simt_rows(c) == 64 ? launch_rows<T, DH, 4>(c, a, stream) : launch_rows<T, DH, 1>(c, a, stream);
}

template <typename T, int DH> cudaError_t combine(const TreeArgs& a, int sets, dim3 grid, dim3 block, cudaStream_t stream) {
    return sets == 2 ? launch_s(stream, tree_combine_kernel<T, DH, 2>, grid, block, 0, a)
                     : launch_s(stream, tree_combine_kernel<T, DH, 1>, grid, block, 0, a);
}

cudaError_t launch(const evs_tree_attn_args& c, cudaStream_t stream) {
    TreeArgs a{};
    a.q = c.q; a.kc = c.k_cache; a.vc = c.v_cache; a.kn = c.k_nodes; a.vn = c.v_nodes; a.o = c.o; a.lse = c.lse;
    a.cache_len = c.cache_len; a.parents = c.parents; a.lens = c.lens; a.flags = c.flags;
    a.q_ld = c.q_ld; a.o_ld = c.o_ld; a.c_row = c.cache_row; a.c_head = c.cache_head; a.c_seq = c.cache_seq;
    a.n_row = c.node_row; a.n_head = c.node_head; a.n_seq = c.node_seq; a.parents_seq = c.parents_seq;
    a.B = c.batch; a.T = c.nodes; a.H = c.heads; a.G = c.kv_heads; a.dh = c.head_dim; a.cap = c.capacity;
    a.zero_rest = c.zero_rest != 0;
    a.scale = c.scale != 0.f ? c.scale : 1.f / sqrtf((float)c.head_dim);
    a.q_vec = (uintptr_t)c.q % 16 == 0 && c.q_ld % 8 == 0;
    a.o_vec = (uintptr_t)c.o % (c.dtype == EVS_DTYPE_BF16 ? 8 : 16) == 0 && c.o_ld % 4 == 0;
    const bool half = c.dtype == EVS_DTYPE_BF16;
    int grid = 0;
    const bool tensor = tensor_ok(c) && plan_tensor(c, a, grid);
    if (!tensor) plan_simt(c, a);
    carve(c, a, grid, (char*)c.workspace);
    cudaError_t e;
    if (tensor)
        e = c.head_dim == 64 ? launch_tensor<64>(c, a, grid, stream) : launch_tensor<128>(c, a, grid, stream);
    else
        switch (c.head_dim) {
            case 128: e = half ? launch_simt<bf16, 128>(c, a, stream) : launch_simt<float, 128>(c, a, stream); break;
            case 64: e = half ? launch_simt<bf16, 64>(c, a, stream) : launch_simt<float, 64>(c, a, stream); break;
            case 32: e = half ? launch_simt<bf16, 32>(c, a, stream) : launch_simt<float, 32>(c, a, stream); break;
            default: e = half ? launch_simt<bf16, 16>(c, a, stream) : launch_simt<float, 16>(c, a, stream);
        }
    if (e != cudaSuccess || (!tensor && a.slots == 1)) return e;
    // sets of rows: two where one each would not run at once; groups: one for eight partials of a row, as many as do
    const int rw = 512 / c.head_dim, rows = c.nodes * (c.heads / c.kv_heads);
    const long long sets = (long long)((rows + rw - 1) / rw) * c.kv_heads * c.batch, room = 152 * 4;
    const int sets_each = sets > 4 * room ? 2 : 1;
    long long per_row = a.slots;
    if (tensor) per_row = grid * (a.pair ? 1 : 2) / ((long long)c.batch * c.kv_heads * a.tiles) + 2;
    long long groups = (per_row + 7) / 8;
    groups = groups < room / sets ? groups : room / sets;
    groups = groups < 1 ? 1 : groups > GROUPS ? GROUPS : groups;
    const dim3 cgrid((rows + rw * sets_each - 1) / (rw * sets_each), c.kv_heads, c.batch), cblock(128 * (unsigned)groups);
    switch (c.head_dim) {
        case 128: return half ? combine<bf16, 128>(a, sets_each, cgrid, cblock, stream) : combine<float, 128>(a, sets_each, cgrid, cblock, stream);
        case 64: return half ? combine<bf16, 64>(a, sets_each, cgrid, cblock, stream) : combine<float, 64>(a, sets_each, cgrid, cblock, stream);
        case 32: return half ? combine<bf16, 32>(a, sets_each, cgrid, cblock, stream) : combine<float, 32>(a, sets_each, cgrid, cblock, stream);
        default: return half ? combine<bf16, 16>(a, sets_each, cgrid, cblock, stream) : combine<float, 16>(a, sets_each, cgrid, cblock, stream);
    }
}

}  // namespace
}  // namespace evs

extern "C" size_t evs_tree_attention_workspace(const evs_tree_attn_args* c) {
    using namespace evs;
    if (!valid_shape(c)) return 0;
    // the larger of the two paths: which one runs depends on addresses too
    TreeArgs a{}, t{};
    int grid = 0;
    plan_simt(*c, a);
    size_t n = carve(*c, a, 0, nullptr);
    if (c->dtype == EVS_DTYPE_BF16 && (c->head_dim == 64 || c->head_dim == 128) && plan_tensor(*c, t, grid)) {
        const size_t m = carve(*c, t, grid, nullptr);
        n = m > n ? m : n;
    }
    return n ? n : 256;
}

extern "C" evs_status evs_tree_attention(const evs_tree_attn_args* c, void* stream) {
    using namespace evs;
    if (!valid_shape(c)) return EVS_ERR_INVALID_ARG;
    if (c->batch == 0) return EVS_OK;
    const int es = c->dtype == EVS_DTYPE_F32 ? 4 : 2;
    const long long row = (long long)c->heads * c->head_dim;
    if (!c->q || !c->o || c->q_ld < row || c->o_ld < row || !c->cache_len || !c->parents) return EVS_ERR_INVALID_ARG;
    if (c->parents_seq != 0 && c->parents_seq < c->nodes) return EVS_ERR_INVALID_ARG;
    if (c->capacity > 0 && (!c->k_cache || !c->v_cache || c->cache_row < c->head_dim)) return EVS_ERR_INVALID_ARG;
    if ((c->k_nodes == nullptr) != (c->v_nodes == nullptr)) return EVS_ERR_INVALID_ARG;
    if (c->k_nodes && c->node_row < c->head_dim) return EVS_ERR_INVALID_ARG;
    if (!c->k_nodes && c->capacity == 0) return EVS_ERR_INVALID_ARG;
    if (((uintptr_t)c->q | (uintptr_t)c->k_cache | (uintptr_t)c->v_cache | (uintptr_t)c->k_nodes | (uintptr_t)c->v_nodes |
         (uintptr_t)c->o) % es)
        return EVS_ERR_INVALID_ARG;
    if (!(c->scale == 0.f || (c->scale >= 1e-30f && c->scale <= 1e30f))) return EVS_ERR_INVALID_ARG;
    if (!c->workspace || (uintptr_t)c->workspace % 256) return EVS_ERR_INVALID_ARG;
    if (c->ws_bytes < evs_tree_attention_workspace(c)) return EVS_ERR_CAPACITY;
    return status_of(launch(*c, (cudaStream_t)stream));
}
