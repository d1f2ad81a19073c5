// Attention over a paged KV cache (sm_100a): the tile kernel, for many query
// rows a key (prompts, chunks of prompts, a prefix under many candidates), bf16
// heads of up to 128 values, pages of a multiple of 8 slots.
//
// The formula is the row kernel's.  A tile is 256 rows ((token, head of one
// key/value head's group) pairs), two sub-tiles of 128, the M of tcgen05.mma; a
// unit is 128 keys.  4 x 256 x 128 x 128 operations a unit are 2,048 clocks of
// the SM's tensor cores, its 32,768 exponentials 2,048 clocks of its 16
// exponential units a clock, its keys and values 64 KB: products and
// exponentials bound it together, and all must run at once:
//   warp 9  copies: keys and values of a unit by tensor maps, page by page, into
//           a ring of slots in the 128-byte swizzle;
//   warp 8  products: S_w = Q_w K^T into tensor memory, O_w += P_w V with P_w
//           read from tensor memory, for the sub-tiles w in turn: P_0 V, the
//           next S_0, P_1 V, the next S_1, so that one sub-tile's products run
//           under the other's softmax;
//   warps 0-3 and 4-7  softmax of sub-tiles 0 and 1, a row a thread: S out of
//           tensor memory, maximum, exponentials, sum, P (bf16) back over S.
// O stays in tensor memory; it is scaled only when a row's maximum has grown by
// more than 2^8 since the last time (P and l carry the factor until then; both
// are floating point, so nothing is lost).  Tensor memory: S_0, S_1, O_0, O_1,
// all 512 columns, one CTA an SM.
//
// The line of units is cut into equal shares, as in the row kernel; partial
// results go through the workspace and the last sub-tile to arrive joins them.
// Every wait is bounded in time.
#include "attention_common.cuh"
#include "tcgen05.cuh"

namespace arops {
namespace {

constexpr int kSubRows = 128;
constexpr int kTileRows = 2 * kSubRows;
constexpr int kTileUnit = 128;  // keys
constexpr int kTileThreads = 384;
constexpr int kTileWarps = kTileThreads / 32;
constexpr int kMmaWarp = 8;
constexpr int kLoadWarp = 9;

// Largest grid: the workspace holds four partial results a CTA.
constexpr int kMaxTileCtas = 160;

__host__ __device__ constexpr int tile_part_floats(int dp)
{
    return kSubRows * dp + 2 * kSubRows;
}

template <int DP>
struct TileTraits {
    static constexpr int kHalves = DP / 64;              // 128-byte column blocks
    static constexpr int kSlot = kTileUnit * DP * 2;     // keys or values of a unit
    static constexpr int kQ = kSubRows * DP * 2;         // of a sub-tile
    static constexpr int kSlots = DP == 128 ? 5 : 8;     // 160 / 128 KB
    static constexpr int kSmem = 2 * kQ + kSlots * kSlot + 1024;  // + alignment
    static constexpr uint32_t kS = 0, kO = 2 * kTileUnit;  // columns: S_w at kS + 128 w
};

struct TilePlan {
    ScoreMap score;
    int32_t* counters;
    float* parts;
    float* prefix_o;    // shared prefixes: results go here, not to out
    float* prefix_ml;
    int32_t g;
    int32_t box;        // keys of one tensor-map copy
};

struct TileCursor {
    int32_t seq, sub, kvh, unit;
};

// Keys of one (tile, key head) pair and of its sub-tiles: units [jlo, jhi).
struct TileSpan {
    int32_t tok0, ntok, len, bidir;
    int32_t lo, units;
    int32_t jlo[2], jhi[2];
    const int32_t* table;
};

// A group of sequences with a shared prefix, as an entity like a sequence: its
// members' query tokens on the prefix's keys.
__device__ __forceinline__ Ragged load_group(const AttentionParams& p, int32_t g, bool& bad)
{
    Ragged r;
    const int32_t a = __ldg(p.group_start + g), b = __ldg(p.group_start + g + 1);
    const bool ok = a >= 0 && b >= a && b <= p.n_seqs;
    bad = bad || !ok;
    r.t0 = ok ? a : 0;
    r.ntok = ok ? b - a : 0;
    r.len = clamp_length(__ldg(p.prefix_lens + g), p.max_prefix_pages * p.map.page_size, bad);
    r.bidir = 0;
    return r;
}

template <bool SHARED>
__device__ __forceinline__ Ragged load_entity(const AttentionParams& p, int32_t s, bool& bad)
{
    if constexpr (SHARED)
        return load_group(p, s, bad);
    else
        return load_ragged(p, s, bad);
}

__device__ __forceinline__ int32_t entity_tiles(const Ragged& r, int32_t g)
{
    return (int32_t)(((uint32_t)r.ntok * g + kTileRows - 1) / kTileRows);
}

template <bool SHARED>
__device__ __forceinline__ int32_t tile_units(const AttentionParams& p, const Ragged& r, int32_t g,
                                              int32_t sub)
{
    if constexpr (SHARED) {
        return max(1, units_between<kTileUnit>(0, r.len));
    } else {
        int32_t lo, hi;
        ragged_range<kTileUnit>(p, r, g, (uint32_t)sub * kTileRows, kTileRows, lo, hi);
        return max(1, units_between<kTileUnit>(lo, hi));
    }
}

// False: no tile `c.sub` in the entity at the cursor.
template <bool SHARED>
__device__ __forceinline__ bool load_span(const AttentionParams& p, int32_t g, const TileCursor& c,
                                          TileSpan& t)
{
    bool bad = false;
    const Ragged r = load_entity<SHARED>(p, c.seq, bad);
    if (c.sub >= entity_tiles(r, g))
        return false;
    t.tok0 = r.t0;
    t.ntok = r.ntok;
    t.len = r.len;
    t.bidir = r.bidir;
    t.table = SHARED ? p.prefix_table + (int64_t)c.seq * p.max_prefix_pages
                     : p.block_table + (int64_t)c.seq * p.max_pages;
    const uint32_t rows = (uint32_t)r.ntok * g;
    int32_t lo[2], hi[2];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const uint32_t row0 = (uint32_t)c.sub * kTileRows + w * kSubRows;
        lo[w] = hi[w] = 0;
        if (row0 < rows) {
            if constexpr (SHARED)
                hi[w] = r.len;
            else
                ragged_range<kTileUnit>(p, r, g, row0, kSubRows, lo[w], hi[w]);
        } else if (w == 1) {
            lo[1] = lo[0];
            hi[1] = lo[0];
        }
    }
    t.lo = lo[0];
    t.units = max(1, units_between<kTileUnit>(lo[0], max(hi[0], hi[1])));
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        t.jlo[w] = (lo[w] - t.lo) / kTileUnit;
        t.jhi[w] = units_between<kTileUnit>(t.lo, hi[w]);
    }
    return true;
}

// The first pair at or behind the cursor; false behind the last entity.
template <bool SHARED>
__device__ __forceinline__ bool seek(const AttentionParams& p, int32_t g, TileCursor& c,
                                     TileSpan& t)
{
    const int32_t entities = SHARED ? p.n_groups : p.n_seqs;
    while (c.seq < entities) {
        if (load_span<SHARED>(p, g, c, t))
            return true;
        ++c.seq;
        c.sub = 0;
    }
    return false;
}

// On along the line, past the pair at the cursor.
__device__ __forceinline__ void next_pair(TileCursor& c, int32_t hk)
{
    c.unit = 0;
    if (++c.kvh == hk) {
        c.kvh = 0;
        ++c.sub;
    }
}

// The CTA's barriers and flags in shared memory.
template <int DP>
struct TileShared {
    uint64_t full[TileTraits<DP>::kSlots];
    uint64_t empty[TileTraits<DP>::kSlots];
    uint64_t tail;      // a copy of values that reaches past the sequence's end
    uint64_t q_ready[2];
    uint64_t s_full[2];
    uint64_t p_ready[2];
    uint64_t o_done[2];
    uint64_t drain;
    uint32_t tmem;
    int stop;           // a wait ran out: everybody leaves
    int last[2];
    int64_t sums[kTileWarps];
    TileCursor found;
};

// Waits for `parity` of `bar`; false once anybody's wait has run out.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, int* stop, unsigned* err)
{
    const uint32_t b = smem_addr(bar);
    if (mbar_try_wait(b, parity))
        return true;
    const uint64_t t0 = global_timer_ns();
    for (;;) {
        for (int i = 0; i < 16; ++i)
            if (mbar_try_wait(b, parity))
                return true;
        if (*reinterpret_cast<volatile int*>(stop))
            return false;
        if (global_timer_ns() - t0 > kWaitTimeoutNs) {
            *reinterpret_cast<volatile int*>(stop) = 1;
            record_device_error(err, kDeviceErrTimeout);
            return false;
        }
    }
}

// ---------------------------------------------------------------------------
// Copies (one warp).
// ---------------------------------------------------------------------------
template <int DP, bool SHARED>
__device__ void tile_load_role(const AttentionParams& p, const TilePlan& plan,
                               const CUtensorMap* kmap, const CUtensorMap* vmap,
                               unsigned char* slots, TileShared<DP>& sh, TileCursor c, int64_t left,
                               int lane)
{
    using R = TileTraits<DP>;
    const int boxes = kTileUnit / plan.box;
    uint32_t n = 0;      // slots filled
    uint32_t tails = 0;  // copies waited for here
    bool ok = true;
    while (ok && left > 0) {
        TileSpan t;
        if (!seek<SHARED>(p, plan.g, c, t))
            break;
        const int32_t u1 = (int32_t)min((int64_t)t.units, c.unit + left);
        left -= u1 - c.unit;
        for (int32_t u = c.unit; ok && u < u1; ++u) {
            const int32_t key0 = t.lo + u * kTileUnit;
            const int32_t key = key0 + lane * plan.box;
            // a copy of a page that does not exist brings zeros
            int32_t page = (int32_t)p.map.num_pages, slot = 0;
            if (lane < boxes && key < t.len) {
                int32_t pi;
                split_position(p.map, key, pi, slot);
                page = __ldg(t.table + pi);
                if (page < 0 || page >= p.map.num_pages) {
                    page = (int32_t)p.map.num_pages;
                    record_device_error(p.err, kDeviceErrBadIndexBit);
                }
            }
            const bool tail = t.len - key0 < kTileUnit;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                const uint32_t s = n % R::kSlots;
                ok = wait_for(&sh.empty[s], ((n / R::kSlots) & 1) ^ 1, &sh.stop, p.err);
                if (!__all_sync(0xFFFFFFFFu, ok)) {
                    ok = false;
                    break;
                }
                unsigned char* dst = slots + s * R::kSlot;
                const bool clean = kv == 1 && tail;
                const uint32_t bar = smem_addr(clean ? &sh.tail : &sh.full[s]);
                if (lane == 0)
                    mbar_arrive_expect_tx(bar, R::kSlot);
                __syncwarp();
                if (lane < boxes) {
#pragma unroll
                    for (int h = 0; h < R::kHalves; ++h)
                        tensor_load4(smem_addr(dst) + h * (kTileUnit * 128) + lane * plan.box * 128,
                                     kv ? vmap : kmap, bar, h * 64, slot, c.kvh, page);
                }
                if (clean) {
                    // slots behind the sequence's end may hold anything, and 0
                    // times a NaN is one: their values become zeros
                    ok = wait_for(&sh.tail, tails & 1, &sh.stop, p.err);
                    ++tails;
                    if (!__all_sync(0xFFFFFFFFu, ok)) {
                        ok = false;
                        break;
                    }
                    const int first = max(t.len - key0, 0);
                    for (int i = first * 8 + lane; i < kTileUnit * 8; i += 32)
#pragma unroll
                        for (int h = 0; h < R::kHalves; ++h)
                            reinterpret_cast<uint4*>(dst + h * (kTileUnit * 128))[i] =
                                make_uint4(0, 0, 0, 0);
                    fence_async_proxy();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(smem_addr(&sh.full[s]));
                }
                ++n;
            }
        }
        next_pair(c, p.hk);
    }
    if (!ok) {
        // nothing is left in flight: the copies issued last (bounded)
        for (uint32_t i = n > R::kSlots ? n - R::kSlots : 0; i < n; ++i)
            mbar_wait(smem_addr(&sh.full[i % R::kSlots]), (i / R::kSlots) & 1);
    }
}

// ---------------------------------------------------------------------------
// Products (one thread).
// ---------------------------------------------------------------------------
template <int DP, bool SHARED>
__device__ void tile_mma_role(const AttentionParams& p, const TilePlan& plan,
                              const unsigned char* q, const unsigned char* slots,
                              TileShared<DP>& sh, TileCursor c, int64_t left)
{
    using R = TileTraits<DP>;
    constexpr uint32_t kWordS = mma_word(kSubRows, kTileUnit, false);
    constexpr uint32_t kWordO = mma_word(kSubRows, DP, true);
    const uint32_t tmem = sh.tmem;
    uint32_t used = 0;                   // slots consumed
    uint32_t qn[2] = {0, 0}, pn[2] = {0, 0};
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        return wait_for(bar, parity, &sh.stop, p.err);
    };
    while (left > 0) {
        TileSpan t;
        if (!seek<SHARED>(p, plan.g, c, t))
            break;
        const int32_t u0 = c.unit;
        const int32_t u1 = (int32_t)min((int64_t)t.units, u0 + left);
        left -= u1 - u0;
        int32_t a[2], b[2];  // the sub-tiles' units of this share
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            a[w] = max(t.jlo[w], u0);
            b[w] = min(t.jhi[w], u1);
        }
        // slots in order: keys u0, values u0, keys u0 + 1, ...
        for (int32_t u = u0 - 1; u < u1; ++u) {
            uint32_t vs = 0, ks = 0;
            if (u >= u0) {
                vs = used % R::kSlots;
                if (!wait(&sh.full[vs], (used / R::kSlots) & 1))
                    return;
                ++used;
            }
            if (u + 1 < u1) {
                ks = used % R::kSlots;
                if (!wait(&sh.full[ks], (used / R::kSlots) & 1))
                    return;
                ++used;
            }
            const uint32_t vaddr = smem_addr(slots + vs * R::kSlot);
            const uint32_t kaddr = smem_addr(slots + ks * R::kSlot);
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                if (u >= a[w] && u < b[w]) {  // O_w (+)= P_w V
                    if (!wait(&sh.p_ready[w], pn[w] & 1))
                        return;
                    ++pn[w];
                    tc_fence_after();
                    const uint32_t o = tmem + R::kO + w * DP;
                    const uint32_t s = tmem + R::kS + w * kTileUnit;
#pragma unroll
                    for (int k = 0; k < kTileUnit / 16; ++k)
                        tc_mma_ts(o, s + k * 8,
                                  operand_desc(vaddr + k * 2048, kTileUnit * 128, 1024), kWordO,
                                  u > a[w] || k > 0);
                    tc_commit(smem_addr(&sh.o_done[w]));
                }
                if (u + 1 >= a[w] && u + 1 < b[w]) {  // the next S_w = Q_w K^T
                    if (u + 1 == a[w]) {
                        if (!wait(&sh.q_ready[w], qn[w] & 1))
                            return;
                        ++qn[w];
                        tc_fence_after();
                    }
                    const uint32_t s = tmem + R::kS + w * kTileUnit;
                    const uint32_t qaddr = smem_addr(q + w * R::kQ);
#pragma unroll
                    for (int k = 0; k < DP / 16; ++k) {
                        const uint32_t off = (k / 4) * (kTileUnit * 128) + (k % 4) * 32;
                        tc_mma_ss(s, operand_desc(qaddr + off, 16, 1024),
                                  operand_desc(kaddr + off, 16, 1024), kWordS, k > 0);
                    }
                    tc_commit(smem_addr(&sh.s_full[w]));
                }
            }
            if (u >= u0)
                tc_commit(smem_addr(&sh.empty[vs]));
            if (u + 1 < u1)
                tc_commit(smem_addr(&sh.empty[ks]));
        }
        next_pair(c, p.hk);
    }
}

// ---------------------------------------------------------------------------
// Softmax (four warps a sub-tile, a row a thread).
// ---------------------------------------------------------------------------
__device__ __forceinline__ void sub_tile_barrier(int w)
{
    asm volatile("bar.sync %0, 128;" ::"r"(1 + w) : "memory");
}

// The sub-tile's query rows into shared memory (asynchronous copies).
template <int DP>
__device__ __forceinline__ void load_q_rows(const AttentionParams& p, int32_t g,
                                            const TileSpan& t, const TileCursor& c, int w,
                                            unsigned char* q, int tid)
{
    constexpr int kChunks = DP / 8;
    const int used = p.head_dim / 8;
    const uint32_t dst = smem_addr(q);
#pragma unroll 4
    for (int i = 0; i < kSubRows * kChunks / 128; ++i) {
        const int idx = i * 128 + tid;
        const int row = idx / kChunks, chunk = idx % kChunks;
        const uint32_t at = (uint32_t)c.sub * kTileRows + w * kSubRows + row;
        const uint32_t tok = at / (uint32_t)g;
        const uint32_t head = c.kvh * g + (at - tok * g);
        const bool ok = tok < (uint32_t)t.ntok && chunk < used;
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.q);
        if (ok)
            src += (int64_t)(t.tok0 + tok) * p.q_stride + (int64_t)head * p.head_dim + chunk * 8;
        const uint32_t d =
            dst + (chunk / 8) * (kSubRows * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src),
                     "r"(ok ? 16u : 0u)
                     : "memory");
    }
}

template <int DP, bool FULL, bool SHARED>
__device__ void tile_softmax_role(const AttentionParams& p, const TilePlan& plan, unsigned char* q,
                                  TileShared<DP>& sh, TileCursor c, int64_t left, int64_t begin,
                                  int64_t share, int w, int tid)
{
    using R = TileTraits<DP>;
    const int lane = tid & 31;
    const uint32_t lanes = (uint32_t)(tid & ~31) << 16;  // the warp's lanes of tensor memory
    const uint32_t s_addr = sh.tmem + lanes + R::kS + w * kTileUnit;
    const uint32_t o_addr = sh.tmem + lanes + R::kO + w * DP;
    uint32_t sn = 0, on = 0;  // S tiles seen, P V products asked for
    int64_t at = begin;

    // the first tile's queries; later ones are asked for under the last unit of
    // the tile before
    TileSpan t;
    auto next_queries = [&]() {
        if (!seek<SHARED>(p, plan.g, c, t)) {
            left = 0;
            return;
        }
        load_q_rows<DP>(p, plan.g, t, c, w, q, tid);
    };
    next_queries();
    // once a wait has run out a warp does nothing but keep the barriers
    bool dead = false;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        dead = !__all_sync(0xFFFFFFFFu, !dead && wait_for(bar, parity, &sh.stop, p.err));
        return !dead;
    };

    while (left > 0) {
        const int32_t u0 = c.unit;
        const int32_t u1 = (int32_t)min((int64_t)t.units, u0 + left);
        left -= u1 - u0;
        const int32_t a = max(t.jlo[w], u0), b = min(t.jhi[w], u1);

        // this thread's row
        const uint32_t row = (uint32_t)c.sub * kTileRows + w * kSubRows + tid;
        const int32_t index = (int32_t)(row / (uint32_t)plan.g);
        const int32_t head = c.kvh * plan.g + (int32_t)(row - (uint32_t)index * plan.g);
        const bool valid = index < t.ntok;
        int32_t pos, lo = 0, hi = t.len;
        if constexpr (SHARED) {
            bool ignore = false;
            pos = t.len - 1;
            if (FULL && valid)
                pos += clamp_length(__ldg(p.kv_lens + t.tok0 + index),
                                    p.max_pages * p.map.page_size, ignore);
        } else {
            pos = t.len - t.ntok + index;
            if (valid)
                visible_keys(pos, t.len, t.bidir, p.window, lo, hi);
            else
                hi = INT_MAX;  // nobody reads such a row
        }
        const float slope = FULL && p.slopes && valid ? __ldg(p.slopes + head) : 0.0f;
        const float scale = FULL ? 1.0f : plan.score.scale;

        const TileSpan span = t;
        bool asked = false;  // for the next tile's queries
        if (a < b) {
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_async_proxy();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_addr(&sh.q_ready[w]));
        }
        float m = -INFINITY, l = 0.0f;
        for (int32_t u = a; u < b; ++u) {
            if (!wait(&sh.s_full[w], sn & 1))
                break;
            ++sn;
            tc_fence_after();
            uint32_t s[kTileUnit];
#pragma unroll
            for (int i = 0; i < kTileUnit; i += 32)
                tc_load32(s + i, s_addr + i);
            if (u + 1 == b && left > 0) {
                // Q_w has been read for the last time: the next tile's queries
                next_pair(c, p.hk);
                next_queries();
                asked = true;
            }
            tc_wait_ld();
            tc_loaded<kTileUnit>(s);

            const int32_t key0 = span.lo + u * kTileUnit;
            if constexpr (FULL) {
#pragma unroll
                for (int i = 0; i < kTileUnit; ++i)
                    s[i] = __float_as_uint(map_score<true>(__uint_as_float(s[i]), plan.score,
                                                           slope, pos, key0 + i));
            }
            if (__any_sync(0xFFFFFFFFu, key0 < lo || hi - key0 < kTileUnit)) {
                const int32_t from = lo - key0, to = hi - key0;
#pragma unroll
                for (int i = 0; i < kTileUnit; ++i)
                    s[i] = i >= from && i < to ? s[i] : __float_as_uint(-INFINITY);
            }
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < kTileUnit; i += 8)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    mx[e] = fmaxf(fmaxf(mx[e], __uint_as_float(s[i + e])),
                                  __uint_as_float(s[i + 4 + e]));
            const float mu = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale;

            // scale what there is only when a maximum has grown by 2^8
            const bool grown = mu > m + 8.0f || (m == -INFINITY && mu > -INFINITY);
            if (__any_sync(0xFFFFFFFFu, grown)) {
                const float mn = fmaxf(m, mu);
                const float f = m == -INFINITY ? 0.0f : exp2_fast(m - mn);
                m = mn;
                l *= f;
                if (u > a) {
                    if (!wait(&sh.o_done[w], (on - 1) & 1))
                        break;
                    tc_fence_after();
#pragma unroll
                    for (int i = 0; i < DP; i += 32) {
                        uint32_t o[32];
                        tc_load32(o, o_addr + i);
                        tc_wait_ld();
                        tc_loaded<32>(o);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tc_store32(o_addr + i, o);
                    }
                }
            }
            const float base = m == -INFINITY ? 0.0f : -m;
            const float2 sc = make_float2(scale, scale), bs = make_float2(base, base);
            float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
            // the weights are rounded to bf16 (2^-8 of each at most), the type
            // of the values that they multiply; l keeps them in fp32
#pragma unroll
            for (int i = 0; i < kTileUnit; i += 64) {
                uint32_t pk[32];
#pragma unroll
                for (int e = 0; e < 64; e += 2) {
                    float2 x = make_float2(__uint_as_float(s[i + e]), __uint_as_float(s[i + e + 1]));
                    x = fma2(x, sc, bs);
                    x.x = exp2_fast(x.x);
                    x.y = exp2_fast(x.y);
                    sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], x);
                    pk[e >> 1] = pack_bf16x2(x.x, x.y);
                }
                tc_store32(s_addr + i / 2, pk);
            }
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(smem_addr(&sh.p_ready[w]));
            ++on;
            const float2 all = add2(sum[0], sum[1]);
            l += all.x + all.y;
        }
        if (!asked && left > 0) {  // no unit of this sub-tile here
            asm volatile("cp.async.wait_all;" ::: "memory");
            next_pair(c, p.hk);
            next_queries();
        }
        const bool has = a < b && wait(&sh.o_done[w], (on - 1) & 1);
        tc_fence_after();

        // -- results -----------------------------------------------------------
        const bool whole = u0 == 0 && u1 == span.units;
        const int64_t pair0 = at - u0;
        at += u1 - u0;
        const int32_t cta0 = (int32_t)(pair0 / share);
        const int32_t cta1 = (int32_t)((pair0 + span.units - 1) / share);
        auto part_of = [&](int32_t x) {
            return plan.parts + ((int64_t)x * 4 + (x == cta0 ? 2 : 0) + w) * tile_part_floats(DP);
        };
        const int64_t out_row = (int64_t)(span.tok0 + index) * p.hq + head;
        auto store_columns = [&](const float* f, int i, float mm, float ll) {
            if (!valid)
                return;
            if constexpr (SHARED) {
                float4* dst = reinterpret_cast<float4*>(plan.prefix_o + out_row * DP + i);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    dst[e] = make_float4(f[4 * e], f[4 * e + 1], f[4 * e + 2], f[4 * e + 3]);
                if (i == 0)
                    *reinterpret_cast<float2*>(plan.prefix_ml + out_row * 2) = make_float2(mm, ll);
            } else {
                const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
                __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + out_row * p.head_dim + i;
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    if (i + e >= p.head_dim)
                        break;
                    float y[8];
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        y[x] = ll == 0.0f ? 0.0f : f[e + x] * inv;
                    *reinterpret_cast<uint4*>(dst + e) = Vec<__nv_bfloat16>::pack(y);
                }
            }
        };
        float* part = part_of(blockIdx.x);
        if (u0 != 0)
            part = plan.parts + ((int64_t)blockIdx.x * 4 + w) * tile_part_floats(DP);
#pragma unroll
        for (int i = 0; i < DP; i += 32) {
            uint32_t o[32];
            if (has) {
                tc_load32(o, o_addr + i);
                tc_wait_ld();
                tc_loaded<32>(o);
            } else {
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    o[e] = 0;
            }
            if (whole) {
                store_columns(reinterpret_cast<const float*>(o), i, m, l);
            } else {
#pragma unroll
                for (int e = 0; e < 32; e += 4)
                    *reinterpret_cast<uint4*>(part + ((i + e) / 4 * kSubRows + tid) * 4) =
                        make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            }
        }
        if (!whole) {
            part[kSubRows * DP + tid] = m;
            part[kSubRows * DP + kSubRows + tid] = l;
            __threadfence();
            sub_tile_barrier(w);
            if (tid == 0) {
                int32_t* counter = plan.counters + kMaxAttentionCtas + cta0 * 2 + w;
                const int32_t n = cta1 - cta0 + 1;
                const int32_t old = atomicAdd(counter, 1);
                if (old < 0 || old >= n)
                    record_device_error(p.err, AROPS_DEVICE_ERR_WORKSPACE);
                sh.last[w] = old == n - 1;
                if (old == n - 1) {
                    *counter = 0;
                    __threadfence();
                }
            }
            sub_tile_barrier(w);
            if (sh.last[w]) {
                float mm = -INFINITY, ll = 0.0f;
                for (int32_t x = cta0; x <= cta1; ++x)
                    mm = fmaxf(mm, __ldcg(part_of(x) + kSubRows * DP + tid));
                for (int32_t x = cta0; x <= cta1; ++x) {
                    const float mx = __ldcg(part_of(x) + kSubRows * DP + tid);
                    if (mx != -INFINITY)
                        ll += __ldcg(part_of(x) + kSubRows * DP + kSubRows + tid) *
                              exp2_fast(mx - mm);
                }
#pragma unroll 1
                for (int i = 0; i < DP; i += 32) {
                    float f[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        f[e] = 0.0f;
                    for (int32_t x = cta0; x <= cta1; ++x) {
                        const float* src = part_of(x);
                        const float mx = __ldcg(src + kSubRows * DP + tid);
                        const float fx = mx == -INFINITY ? 0.0f : exp2_fast(mx - mm);
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            const float4 v = __ldcg(reinterpret_cast<const float4*>(
                                src + ((i + e) / 4 * kSubRows + tid) * 4));
                            f[e] += v.x * fx;
                            f[e + 1] += v.y * fx;
                            f[e + 2] += v.z * fx;
                            f[e + 3] += v.w * fx;
                        }
                    }
                    store_columns(f, i, mm, ll);
                }
            }
            sub_tile_barrier(w);  // the flag has been read
        }
    }
}

template <int DP, bool FULL, bool SHARED>
__global__ void __launch_bounds__(kTileThreads, 1)
attention_tiles_kernel(const __grid_constant__ AttentionParams p,
                       const __grid_constant__ TilePlan plan,
                       const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap)
{
    using R = TileTraits<DP>;
    extern __shared__ unsigned char raw[];
    __shared__ TileShared<DP> sh;
    unsigned char* smem = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
    unsigned char* q = smem;
    unsigned char* slots = smem + 2 * R::kQ;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

    if (threadIdx.x == 0) {
        for (int i = 0; i < R::kSlots; ++i) {
            mbar_init(smem_addr(&sh.full[i]), 1);
            mbar_init(smem_addr(&sh.empty[i]), 1);
        }
        mbar_init(smem_addr(&sh.tail), 1);
        mbar_init(smem_addr(&sh.drain), 1);
        for (int w = 0; w < 2; ++w) {
            mbar_init(smem_addr(&sh.q_ready[w]), 4);
            mbar_init(smem_addr(&sh.s_full[w]), 1);
            mbar_init(smem_addr(&sh.p_ready[w]), 4);
            mbar_init(smem_addr(&sh.o_done[w]), 1);
        }
        sh.stop = 0;
        mbar_init_fence();
    }
    pdl_wait();
    pdl_allow_dependents();

    // -- this CTA's share of the line of units --------------------------------
    const int32_t entities = SHARED ? p.n_groups : p.n_seqs;
    bool bad = false;
    const int32_t per = (entities + kTileThreads - 1) / kTileThreads;
    const int32_t e0 = (int32_t)min((int64_t)threadIdx.x * per, (int64_t)entities);
    const int32_t e1 = min(e0 + per, entities);
    auto count = [&](const Ragged& r) {
        const int32_t tiles = entity_tiles(r, plan.g);
        int64_t n = 0;
        for (int32_t i = 0; i < tiles; ++i)
            n += tile_units<SHARED>(p, r, plan.g, i);
        return n;
    };
    int64_t mine = 0;
    for (int32_t e = e0; e < e1; ++e)
        mine += count(load_entity<SHARED>(p, e, bad));
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if (lane >= o)
            upto += x;
    }
    if (lane == 31)
        sh.sums[warp] = upto;
    if (__syncthreads_or(SHARED && bad)) {  // malformed groups: nothing is written
        if (bad && blockIdx.x == 0)
            record_device_error(p.err, kDeviceErrBadIndexBit);
        return;
    }
    if (bad && blockIdx.x == 0)
        record_device_error(p.err, kDeviceErrBadIndexBit);
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < kTileWarps; ++w) {
        if (w < warp)
            upto += sh.sums[w];
        total += sh.sums[w];
    }
    const int64_t line = total * p.hk;
    const int64_t share = max((int64_t)1, (line + gridDim.x - 1) / gridDim.x);
    const int64_t begin = (int64_t)blockIdx.x * share;
    if (begin >= line)
        return;
    const int64_t left = min(share, line - begin);
    int64_t before = upto - mine;
    if (begin >= before * p.hk && begin < upto * p.hk) {
        TileCursor c;
        c.seq = e0;
        bool ignore = false;
        Ragged r;
        for (;; ++c.seq) {
            r = load_entity<SHARED>(p, c.seq, ignore);
            const int64_t n = count(r);
            if (begin < (before + n) * p.hk)
                break;
            before += n;
        }
        int64_t n = 1;
        for (c.sub = 0;; ++c.sub) {
            n = tile_units<SHARED>(p, r, plan.g, c.sub);
            if (begin < (before + n) * p.hk)
                break;
            before += n;
        }
        const int64_t rest = begin - before * p.hk;
        c.kvh = (int32_t)(rest / n);
        c.unit = (int32_t)(rest % n);
        sh.found = c;
    }
    if (warp == kMmaWarp)
        tc_alloc(smem_addr(&sh.tmem));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const TileCursor c = sh.found;

    // Registers: the softmax warps keep a row of 128 scores, the others little.
    // 256 x 216 + 128 x 72 = 384 x 168, what the launch gave out.
    if (warp < kMmaWarp) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int w = warp >> 2;
        tile_softmax_role<DP, FULL, SHARED>(p, plan, q + w * R::kQ, sh, c, left, begin, share, w,
                                            threadIdx.x & 127);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == kMmaWarp) {
            if (lane == 0) {
                tile_mma_role<DP, SHARED>(p, plan, q, slots, sh, c, left);
                // every product and every arrival asked for has happened
                tc_commit(smem_addr(&sh.drain));
                mbar_wait(smem_addr(&sh.drain), 0);
            }
            __syncwarp();
        } else if (warp == kLoadWarp) {
            tile_load_role<DP, SHARED>(p, plan, &kmap, &vmap, slots, sh, c, left, lane);
            __syncwarp();
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp)
        tc_dealloc(sh.tmem);
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled()
{
    static std::atomic<void*> cached{nullptr};
    void* f = cached.load(std::memory_order_acquire);
    if (f == nullptr) {
        cudaDriverEntryPointQueryResult res;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000,
                                             cudaEnableDefault, &res) != cudaSuccess ||
            res != cudaDriverEntryPointSuccess)
            return nullptr;
        cached.store(f, std::memory_order_release);
    }
    return reinterpret_cast<EncodeTiled>(f);
}

// The pool as [page][head][slot][value]; a copy takes 64 values of `box` slots
// of one page and head.
cudaError_t pool_map(CUtensorMap* map, const void* pool, const AttentionParams& p, int box)
{
    EncodeTiled encode = encode_tiled();
    if (encode == nullptr)
        return cudaErrorNotSupported;
    const cuuint64_t row = (cuuint64_t)p.head_dim * 2;
    const cuuint64_t head = row * p.map.page_size;
    const cuuint64_t dims[4] = {(cuuint64_t)p.head_dim, (cuuint64_t)p.map.page_size,
                                (cuuint64_t)p.hk, (cuuint64_t)p.map.num_pages};
    const cuuint64_t strides[3] = {row, head, head * p.hk};
    const cuuint32_t sizes[4] = {64, (cuuint32_t)box, 1, 1};
    const cuuint32_t steps[4] = {1, 1, 1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(pool),
                              dims, strides, sizes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

int box_slots(int page_size)
{
    int box = 8;
    while (box < kTileUnit && page_size % (2 * box) == 0)
        box *= 2;
    return box;
}

template <int DP, bool FULL, bool SHARED>
cudaError_t launch_tiles_f(const AttentionParams& p, const TilePlan& plan, const CUtensorMap& kmap,
                           const CUtensorMap& vmap, int sm_count, cudaStream_t st)
{
    auto kernel = attention_tiles_kernel<DP, FULL, SHARED>;
    int ctas = 0;
    const cudaError_t err = resident_ctas(kernel, kTileThreads, TileTraits<DP>::kSmem, &ctas);
    if (err != cudaSuccess)
        return err;
    if (ctas < 1)
        return cudaErrorNotSupported;
    // one CTA an SM: each takes all of its SM's tensor memory
    const int grid = std::min(sm_count, kMaxTileCtas);
    return launch(kernel, dim3(grid), dim3(kTileThreads), TileTraits<DP>::kSmem, st, p, plan, kmap,
                  vmap);
}

template <int DP>
cudaError_t launch_tiles_d(const AttentionParams& p, const TilePlan& plan, const CUtensorMap& kmap,
                           const CUtensorMap& vmap, bool full, int sm_count, cudaStream_t st)
{
    if (p.group_start)
        return full ? launch_tiles_f<DP, true, true>(p, plan, kmap, vmap, sm_count, st)
                    : launch_tiles_f<DP, false, true>(p, plan, kmap, vmap, sm_count, st);
    return full ? launch_tiles_f<DP, true, false>(p, plan, kmap, vmap, sm_count, st)
                : launch_tiles_f<DP, false, false>(p, plan, kmap, vmap, sm_count, st);
}

}  // namespace

bool tiles_can_run(const AttentionParams& p, arops_dtype dtype)
{
    return dtype == AROPS_BF16 && p.head_dim <= 128 && p.head_dim % 8 == 0 &&
           p.map.page_size % 8 == 0 && aligned16(p.k_pages) && aligned16(p.v_pages) &&
           aligned16(p.q) && p.q_stride % 8 == 0 && aligned16(p.out) &&
           // the tensor map's largest stride
           (int64_t)p.hk * p.map.page_size * p.head_dim * 2 < (1ll << 40);
}

size_t tile_part_bytes(int dp)
{
    return (size_t)kMaxTileCtas * 4 * tile_part_floats(dp) * sizeof(float);
}

cudaError_t launch_attention_tiles(const AttentionParams& p, int32_t* counters, float* parts,
                                   float* prefix_o, float* prefix_ml, int sm_count,
                                   cudaStream_t stream)
{
    TilePlan plan = {};
    // the plain form needs a positive factor: the largest product is then the
    // largest score
    const bool full = p.softcap > 0.0f || p.slopes != nullptr || !(p.scale > 0.0f);
    plan.score = make_score_map(p);
    if (full)
        plan.score.scale = p.scale;
    plan.counters = counters;
    plan.parts = parts;
    plan.prefix_o = prefix_o;
    plan.prefix_ml = prefix_ml;
    plan.g = p.hq / p.hk;
    plan.box = box_slots(p.map.page_size);
    CUtensorMap kmap, vmap;
    cudaError_t err = pool_map(&kmap, p.k_pages, p, plan.box);
    if (err == cudaSuccess)
        err = pool_map(&vmap, p.v_pages, p, plan.box);
    if (err != cudaSuccess)
        return err;
    return p.head_dim <= 64
               ? launch_tiles_d<64>(p, plan, kmap, vmap, full, sm_count, stream)
               : launch_tiles_d<128>(p, plan, kmap, vmap, full, sm_count, stream);
}

}  // namespace arops
