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
// Keys whose weights are handed to the products first, the rest follow: the
// products of the first run under the exponentials of the rest.
constexpr int kFirstKeys = 96;
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
    static constexpr int kSlots = DP == 128 ? 4 : 8;     // 128 KB
    static constexpr int kStage = kSubRows * 128;        // results of a sub-tile, 64 columns
    static constexpr int kSmem = 2 * kQ + kSlots * kSlot + 2 * kStage + 1024;  // + alignment
    static constexpr uint32_t kS = 0, kO = 2 * kTileUnit;  // columns: S_w at kS + 128 w
};

struct TilePlan {
    ScoreMap score;
    int32_t* counters;
    float* parts;
    float* prefix_o;    // shared prefixes: results go here, not to out
    float* prefix_ml;
    RowDivide g;        // query heads a key head
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

__device__ __forceinline__ int32_t entity_tiles(const Ragged& r, const RowDivide& g)
{
    return (int32_t)(((uint32_t)r.ntok * g.n + kTileRows - 1) / kTileRows);
}

template <bool SHARED>
__device__ __forceinline__ int32_t tile_units(const AttentionParams& p, const Ragged& r,
                                              const RowDivide& g, int32_t sub)
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
__device__ __forceinline__ bool load_span(const AttentionParams& p, const TilePlan& plan,
                                          const TileCursor& c, TileSpan& t)
{
    bool bad = false;
    const Ragged r = load_entity<SHARED>(p, c.seq, bad);
    const RowDivide g = plan.g;
    if (c.sub >= entity_tiles(r, g))
        return false;
    t.tok0 = r.t0;
    t.ntok = r.ntok;
    t.len = r.len;
    t.bidir = r.bidir;
    t.table = SHARED ? p.prefix_table + (int64_t)c.seq * p.max_prefix_pages
                     : p.block_table + (int64_t)c.seq * p.max_pages;
    const uint32_t rows = (uint32_t)r.ntok * g.n;
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

// A pair's place on the line: kPairCost positions that stand for its fixed cost
// (queries in, results out), then its units.
constexpr int kPairCost = 2;

// A CTA's way along its share [begin, end) of the line.
struct TileWalk {
    TileCursor c;       // the pair to look at next
    int64_t at;         // place of its unit 0
    int64_t begin, end;

    // c.unit: units of c's pair before `begin` (negative inside its fixed cost)
    __device__ TileWalk(const TileCursor& from, int64_t b, int64_t e)
        : c(from), at(b - from.unit), begin(b), end(e)
    {
    }

    // The next pair with units [u0, u1) in the share, the cursor left on it;
    // false at the end.
    template <bool SHARED>
    __device__ __forceinline__ bool next(const AttentionParams& p, const TilePlan& plan,
                                         TileSpan& t, int32_t& u0, int32_t& u1)
    {
        const int32_t entities = SHARED ? p.n_groups : p.n_seqs;
        while (at < end && c.seq < entities) {
            if (!load_span<SHARED>(p, plan, c, t)) {
                ++c.seq;
                c.sub = 0;
                continue;
            }
            u0 = (int32_t)max(begin - at, (int64_t)0);
            u1 = (int32_t)min(end - at, (int64_t)t.units);
            pair = c;
            place = at;
            at += t.units + kPairCost;
            if (++c.kvh == p.hk) {
                c.kvh = 0;
                ++c.sub;
            }
            if (u0 < u1)
                return true;
        }
        return false;
    }

    TileCursor pair;  // of the last next()
    int64_t place;    // of its unit 0
};

// The CTA's barriers and flags in shared memory.
template <int DP>
struct TileShared {
    uint64_t full[TileTraits<DP>::kSlots];
    uint64_t empty[TileTraits<DP>::kSlots];
    uint64_t tail;      // a copy of values that reaches past the sequence's end
    uint64_t q_ready[2];
    uint64_t s_full[2];
    uint64_t p_ready[2][2];
    uint64_t o_done[2];
    uint64_t drain;
    uint32_t tmem;
    int stop;           // a wait ran out: everybody leaves
    int last[2];
    int64_t sums[kTileWarps];
    int64_t found_before;  // line in front of the found entity, per key head
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
                               unsigned char* slots, TileShared<DP>& sh, TileCursor c, int64_t begin,
                               int64_t end, int lane)
{
    using R = TileTraits<DP>;
    const int boxes = kTileUnit / plan.box;
    uint32_t n = 0;      // slots filled
    uint32_t tails = 0;  // copies waited for here
    bool ok = true;
    TileWalk walk(c, begin, end);
    TileSpan t;
    int32_t u0, u1;
    while (ok && walk.next<SHARED>(p, plan, t, u0, u1)) {
        for (int32_t u = u0; ok && u < u1; ++u) {
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
                                     kv ? vmap : kmap, bar, h * 64, slot, walk.pair.kvh,
                                     page);
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
    }
    if (!ok) {
        // nothing is left in flight: the copies issued last (bounded)
        for (uint32_t i = n > R::kSlots ? n - R::kSlots : 0; i < n; ++i)
            mbar_wait(smem_addr(&sh.full[i % R::kSlots]), (i / R::kSlots) & 1);
    }
}

// ---------------------------------------------------------------------------
// Products (one warp; one thread of it issues).
// ---------------------------------------------------------------------------
template <int DP, bool SHARED>
__device__ void tile_mma_role(const AttentionParams& p, const TilePlan& plan,
                              const unsigned char* q, const unsigned char* slots,
                              TileShared<DP>& sh, TileCursor c, int64_t begin, int64_t end)
{
    using R = TileTraits<DP>;
    constexpr uint32_t kWordS = mma_word(kSubRows, kTileUnit, false);
    constexpr uint32_t kWordO = mma_word(kSubRows, DP, true);
    const uint32_t tmem = sh.tmem;
    // keys and queries: K (head_dim) contiguous, one 64-value block behind the
    // other; values: N (head_dim) contiguous, the leading offset between blocks
    const uint32_t q_low = operand_low(smem_addr(q), 16);
    const uint32_t k_low = operand_low(smem_addr(slots), 16);
    const uint32_t v_low = operand_low(smem_addr(slots), kTileUnit * 128);
    uint32_t used = 0;                   // slots consumed
    uint32_t qn[2] = {0, 0}, pn[2] = {0, 0};
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xFFFFFFFFu, wait_for(bar, parity, &sh.stop, p.err));
    };
    TileWalk walk(c, begin, end);
    TileSpan t;
    int32_t u0, u1;
    while (walk.next<SHARED>(p, plan, t, u0, u1)) {
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
            const uint32_t vb = v_low + vs * (R::kSlot >> 4);
            const uint32_t kb = k_low + ks * (R::kSlot >> 4);
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const uint32_t o = tmem + R::kO + w * DP;
                const uint32_t s = tmem + R::kS + w * kTileUnit;
                if (u >= a[w] && u < b[w]) {  // O_w (+)= P_w V
                    if (!wait(&sh.p_ready[w][0], pn[w] & 1))
                        return;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < kFirstKeys / 16; ++k)
                            tc_mma_ts(o, s + k * 8, vb + k * (2048 >> 4), kWordO,
                                      u > a[w] || k > 0);
                    }
                    __syncwarp();
                    if (!wait(&sh.p_ready[w][1], pn[w] & 1))
                        return;
                    tc_fence_after();
                    ++pn[w];
                    if (elect_one()) {
#pragma unroll
                        for (int k = kFirstKeys / 16; k < kTileUnit / 16; ++k)
                            tc_mma_ts(o, s + k * 8, vb + k * (2048 >> 4), kWordO, true);
                        tc_commit(smem_addr(&sh.o_done[w]));
                    }
                    __syncwarp();
                }
                if (u + 1 >= a[w] && u + 1 < b[w]) {  // the next S_w = Q_w K^T
                    if (u + 1 == a[w]) {
                        if (!wait(&sh.q_ready[w], qn[w] & 1))
                            return;
                        ++qn[w];
                        tc_fence_after();
                    }
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < DP / 16; ++k) {
                            const uint32_t off = ((k / 4) * (kTileUnit * 128) + (k % 4) * 32) >> 4;
                            tc_mma_ss(s, q_low + w * (R::kQ >> 4) + off, kb + off, kWordS, k > 0);
                        }
                        tc_commit(smem_addr(&sh.s_full[w]));
                    }
                    __syncwarp();
                }
            }
            if (elect_one()) {
                if (u >= u0)
                    tc_commit(smem_addr(&sh.empty[vs]));
                if (u + 1 < u1)
                    tc_commit(smem_addr(&sh.empty[ks]));
            }
            __syncwarp();
        }
    }
}

// ---------------------------------------------------------------------------
// Softmax (four warps a sub-tile, a row a thread).
// ---------------------------------------------------------------------------
__device__ __forceinline__ void sub_tile_barrier(int w)
{
    asm volatile("bar.sync %0, 128;" ::"r"(1 + w) : "memory");
}

// (token, head) of rows that a thread takes `step` apart.
struct RowStep {
    uint32_t tok, head, g, dt, dh;
    __device__ __forceinline__ RowStep(const RowDivide& d, uint32_t row, uint32_t step) : g(d.n)
    {
        tok = d(row);
        head = row - tok * g;
        dt = d(step);
        dh = step - dt * g;
    }
    __device__ __forceinline__ void next()
    {
        tok += dt;
        head += dh;
        if (head >= g) {
            head -= g;
            ++tok;
        }
    }
};

// The sub-tile's query rows into shared memory (asynchronous copies).
template <int DP>
__device__ __forceinline__ void load_q_rows(const AttentionParams& p, const RowDivide& g,
                                            const TileSpan& t, const TileCursor& c, int w,
                                            unsigned char* q, int tid)
{
    constexpr int kChunks = DP / 8;
    constexpr int kStep = 128 / kChunks;
    const int chunk = tid % kChunks;
    int row = tid / kChunks;
    const bool used = chunk < p.head_dim / 8;
    RowStep r(g, (uint32_t)c.sub * kTileRows + w * kSubRows + row, kStep);
    const __nv_bfloat16* base = static_cast<const __nv_bfloat16*>(p.q) +
                                t.tok0 * p.q_stride + (int64_t)c.kvh * g.n * p.head_dim +
                                chunk * 8;
    const uint32_t dst = smem_addr(q) + (chunk / 8) * (kSubRows * 128);
#pragma unroll 4
    for (int i = 0; i < kSubRows / kStep; ++i) {
        const bool ok = r.tok < (uint32_t)t.ntok && used;
        const __nv_bfloat16* src =
            ok ? base + (int64_t)r.tok * p.q_stride + r.head * p.head_dim
               : static_cast<const __nv_bfloat16*>(p.q);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                         dst + row * 128 + (((chunk & 7) ^ (row & 7)) << 4)),
                     "l"(src), "r"(ok ? 16u : 0u)
                     : "memory");
        row += kStep;
        r.next();
    }
}

// 64 columns of a sub-tile's results, a row a thread, divided by l: through
// shared memory, so that eight threads store a row's 128 bytes together.
template <int DP, bool SHARED>
__device__ __forceinline__ void emit_columns(const AttentionParams& p, const TilePlan& plan,
                                             const TileSpan& t, const TileCursor& c,
                                             const uint32_t (&o)[64], int col, float m, float l,
                                             unsigned char* stage, int w, int tid)
{
    const uint32_t row0 = (uint32_t)c.sub * kTileRows + w * kSubRows;
    if constexpr (SHARED) {
        const RowStep r(plan.g, row0 + tid, 1);
        if (r.tok < (uint32_t)t.ntok) {
            const int64_t at = (int64_t)(t.tok0 + r.tok) * p.hq + c.kvh * plan.g.n + r.head;
            float4* dst = reinterpret_cast<float4*>(plan.prefix_o + at * DP + col);
#pragma unroll
            for (int e = 0; e < 16; ++e)
                dst[e] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                     __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
            if (col == 0)
                *reinterpret_cast<float2*>(plan.prefix_ml + at * 2) = make_float2(m, l);
        }
    } else {
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float y[8];
#pragma unroll
            for (int x = 0; x < 8; ++x)
                y[x] = l == 0.0f ? 0.0f : __uint_as_float(o[8 * e + x]) * inv;
            *reinterpret_cast<uint4*>(stage + tid * 128 + ((e ^ (tid & 7)) << 4)) =
                Vec<__nv_bfloat16>::pack(y);
        }
        sub_tile_barrier(w);
        const int chunk = tid & 7;
        int row = tid >> 3;
        RowStep r(plan.g, row0 + row, 16);
        __nv_bfloat16* base = static_cast<__nv_bfloat16*>(p.out) +
                              ((int64_t)t.tok0 * p.hq + c.kvh * plan.g.n) * p.head_dim + col +
                              chunk * 8;
        const bool used = col + chunk * 8 < p.head_dim;
#pragma unroll
        for (int i = 0; i < kSubRows / 16; ++i) {
            const uint4 v =
                *reinterpret_cast<const uint4*>(stage + row * 128 + ((chunk ^ (row & 7)) << 4));
            if (used && r.tok < (uint32_t)t.ntok)
                *reinterpret_cast<uint4*>(base + ((int64_t)r.tok * p.hq + r.head) * p.head_dim) = v;
            row += 16;
            r.next();
        }
        sub_tile_barrier(w);
    }
}

// A row's scores from its products, in base 2: cap, then bias.
//   |s| <= cap / 2 in all rows of the warp (a cap is there for outliers): tanh
//   by its polynomial, 6 operations a pair of keys on the fp32 pipe instead of
//   2 exponential-unit operations a key (12,500 -> 1,000 clocks a unit of 128
//   keys, prompt rows with a cap of 30).
//   Keys not behind the query: |i - j| without the absolute value, one FMA.
__device__ __forceinline__ void map_row(uint32_t (&s)[kTileUnit], const ScoreMap& map, float slope,
                                        int32_t pos, int32_t key0)
{
    auto at = [&](int i) {
        return make_float2(__uint_as_float(s[i]), __uint_as_float(s[i + 1]));
    };
    auto put = [&](int i, float2 x) {
        s[i] = __float_as_uint(x.x);
        s[i + 1] = __float_as_uint(x.y);
    };
    auto both = [](float x) { return make_float2(x, x); };
    const float out = map.scale * kLog2e;
    if (map.cap > 0.0f) {
        float big = 0.0f;
#pragma unroll
        for (int i = 0; i < kTileUnit; ++i)
            big = fmaxf(big, fabsf(__uint_as_float(s[i])));
        const float in = map.scale * map.inv_cap;
        if (__all_sync(0xFFFFFFFFu, big * fabsf(in) <= 0.5f)) {
#pragma unroll
            for (int i = 0; i < kTileUnit; i += 2) {
                const float2 x = at(i);
                const float2 t = mul2(x, both(in));
                const float2 y = mul2(t, t);
                float2 q = fma2(y, both(kTanh4), both(kTanh3));
                q = fma2(q, y, both(kTanh2));
                q = fma2(q, y, both(kTanh1));
                q = fma2(q, y, both(kTanh0));
                put(i, mul2(mul2(x, both(out)), q));
            }
        } else {
#pragma unroll
            for (int i = 0; i < kTileUnit; ++i)
                s[i] = __float_as_uint(
                    soft_cap(__uint_as_float(s[i]) * map.scale, map.cap, map.inv_cap) * kLog2e);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kTileUnit; i += 2)
            put(i, mul2(at(i), both(out)));
    }
    if (__all_sync(0xFFFFFFFFu, slope == 0.0f))
        return;
    const float bias = -slope * kLog2e;
    const float gap = (float)(pos - key0);
    if (__all_sync(0xFFFFFFFFu, pos - key0 >= kTileUnit - 1)) {
        const float first = bias * gap;
#pragma unroll
        for (int i = 0; i < kTileUnit; i += 2)
            put(i, add2(at(i), fma2(both(-bias), make_float2((float)i, (float)(i + 1)),
                                    both(first))));
    } else {
#pragma unroll
        for (int i = 0; i < kTileUnit; ++i)
            s[i] = __float_as_uint(fmaf(bias, fabsf(gap - (float)i), __uint_as_float(s[i])));
    }
}

template <int DP, bool FULL, bool SHARED>
__device__ void tile_softmax_role(const AttentionParams& p, const TilePlan& plan, unsigned char* q,
                                  unsigned char* stage, TileShared<DP>& sh, const TileCursor& from,
                                  int64_t begin, int64_t end, int64_t share, int w, int tid)
{
    using R = TileTraits<DP>;
    const int lane = tid & 31;
    const uint32_t lanes = (uint32_t)(tid & ~31) << 16;  // the warp's lanes of tensor memory
    const uint32_t s_addr = sh.tmem + lanes + R::kS + w * kTileUnit;
    const uint32_t o_addr = sh.tmem + lanes + R::kO + w * DP;
    uint32_t sn = 0, on = 0;  // S tiles seen, P V products asked for

    // once a wait has run out a warp does nothing but keep the barriers
    bool dead = false;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        dead = !__all_sync(0xFFFFFFFFu, !dead && wait_for(bar, parity, &sh.stop, p.err));
        return !dead;
    };
    // the first tile's queries; later ones are asked for under the last unit of
    // the tile before
    TileWalk walk(from, begin, end);
    TileSpan next_t;
    int32_t next_u0, next_u1;
    auto next_queries = [&]() {
        const bool more = walk.next<SHARED>(p, plan, next_t, next_u0, next_u1);
        if (more)
            load_q_rows<DP>(p, plan.g, next_t, walk.pair, w, q, tid);
        return more;
    };
    bool more = next_queries();

    while (more) {
        const TileSpan t = next_t;
        const TileCursor c = walk.pair;
        const int64_t place = walk.place;
        const int32_t u0 = next_u0, u1 = next_u1;
        const int32_t a = max(t.jlo[w], u0), b = min(t.jhi[w], u1);

        // this thread's row
        const RowStep r(plan.g, (uint32_t)c.sub * kTileRows + w * kSubRows + tid, 1);
        const bool valid = r.tok < (uint32_t)t.ntok;
        int32_t pos, lo = 0, hi = t.len;
        if constexpr (SHARED) {
            bool ignore = false;
            pos = t.len - 1;
            if (FULL && valid)
                pos += clamp_length(__ldg(p.kv_lens + t.tok0 + r.tok),
                                    p.max_pages * p.map.page_size, ignore);
        } else {
            pos = t.len - t.ntok + (int32_t)r.tok;
            if (valid)
                visible_keys(pos, t.len, t.bidir, p.window, lo, hi);
            else
                hi = INT_MAX;  // nobody reads such a row
        }
        const float slope =
            FULL && p.slopes && valid ? __ldg(p.slopes + c.kvh * plan.g.n + r.head) : 0.0f;
        const float scale = FULL ? 1.0f : plan.score.scale;

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
            if (u + 1 == b) {
                // Q_w has been read for the last time
                more = next_queries();
                asked = true;
            }
            uint32_t s[kTileUnit];
#pragma unroll
            for (int i = 0; i < kTileUnit; i += 32)
                tc_load32(s + i, s_addr + i);
            tc_wait_ld();
            tc_loaded<kTileUnit>(s);

            const int32_t key0 = t.lo + u * kTileUnit;
            if constexpr (FULL)
                map_row(s, plan.score, slope, pos, key0);
            if (__any_sync(0xFFFFFFFFu, key0 < lo || hi - key0 < kTileUnit)) {
                const int32_t first = lo - key0, last = hi - key0;
#pragma unroll
                for (int i = 0; i < kTileUnit; ++i)
                    s[i] = i >= first && i < last ? s[i] : __float_as_uint(-INFINITY);
            }
            float mx[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                mx[e] = __uint_as_float(s[e]);
#pragma unroll
            for (int i = 8; i < kTileUnit - 8; i += 16)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    mx[e] = fmaxf(fmaxf(mx[e], __uint_as_float(s[i + e])),
                                  __uint_as_float(s[i + 8 + e]));
#pragma unroll
            for (int e = 0; e < 8; ++e)
                mx[e] = fmaxf(mx[e], __uint_as_float(s[kTileUnit - 8 + e]));
            const float mu = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                                   fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7]))) *
                             scale;

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
                    for (int i = 0; i < DP; i += 16) {
                        uint32_t o[16];
                        tc_load16(o, o_addr + i);
                        tc_wait_ld();
                        tc_loaded<16>(o);
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tc_store16(o_addr + i, o);
                    }
                }
            }
            const float base = m == -INFINITY ? 0.0f : -m;
            const float2 sc = make_float2(scale, scale), bs = make_float2(base, base);
            float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
            // the weights are rounded to bf16 (2^-8 of each at most), the type
            // of the values that they multiply; l keeps them in fp32
#pragma unroll
            for (int i = 0; i < kTileUnit; i += 32) {
                uint32_t pk[16];
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    float2 x = make_float2(__uint_as_float(s[i + e]), __uint_as_float(s[i + e + 1]));
                    x = fma2(x, sc, bs);
                    x.x = exp2_fast(x.x);
                    x.y = exp2_fast(x.y);
                    sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], x);
                    pk[e >> 1] = pack_bf16x2(x.x, x.y);
                }
                tc_store16(s_addr + i / 2, pk);
                if (i + 32 == kFirstKeys || i + 32 == kTileUnit) {
                    tc_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(smem_addr(&sh.p_ready[w][i + 32 == kTileUnit]));
                }
            }
            ++on;
            const float2 all = add2(sum[0], sum[1]);
            l += all.x + all.y;
        }
        if (!asked) {  // no unit of this sub-tile here
            asm volatile("cp.async.wait_all;" ::: "memory");
            more = next_queries();
        }
        const bool has = a < b && wait(&sh.o_done[w], (on - 1) & 1);
        tc_fence_after();

        // -- results -----------------------------------------------------------
        const bool whole = u0 == 0 && u1 == t.units;
        const int32_t cta0 = (int32_t)(place / share);
        const int32_t cta1 = (int32_t)((place + t.units - 1) / share);
        auto part_of = [&](int32_t x) {
            return plan.parts + ((int64_t)x * 4 + (x == cta0 ? 2 : 0) + w) * tile_part_floats(DP);
        };
        float* part = part_of(blockIdx.x);
#pragma unroll
        for (int i = 0; i < DP; i += 64) {
            uint32_t o[64];
            if (has) {
                tc_load32(o, o_addr + i);
                tc_load32(o + 32, o_addr + i + 32);
                tc_wait_ld();
                tc_loaded<64>(o);
            } else {
#pragma unroll
                for (int e = 0; e < 64; ++e)
                    o[e] = 0;
            }
            if (whole) {
                emit_columns<DP, SHARED>(p, plan, t, c, o, i, m, l, stage, w, tid);
            } else {
#pragma unroll
                for (int e = 0; e < 64; e += 4)
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
            const bool join = sh.last[w];
            sub_tile_barrier(w);  // the flag has been read
            if (join) {
                float mm = -INFINITY, ll = 0.0f;
                for (int32_t x = cta0; x <= cta1; ++x) {
                    const float mx = __ldcg(part_of(x) + kSubRows * DP + tid);
                    const float lx = __ldcg(part_of(x) + kSubRows * DP + kSubRows + tid);
                    const float mn = fmaxf(mm, mx);
                    if (mx != -INFINITY)
                        ll = (mm == -INFINITY ? 0.0f : ll * exp2_fast(mm - mn)) +
                             lx * exp2_fast(mx - mn);
                    mm = mn;
                }
#pragma unroll 1
                for (int i = 0; i < DP; i += 64) {
                    uint32_t o[64];
#pragma unroll
                    for (int e = 0; e < 64; ++e)
                        o[e] = 0;
                    for (int32_t x = cta0; x <= cta1; ++x) {
                        const float* src = part_of(x);
                        const float mx = __ldcg(src + kSubRows * DP + tid);
                        uint4 v[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            v[e] = __ldcg(reinterpret_cast<const uint4*>(
                                src + ((i / 4 + e) * kSubRows + tid) * 4));
                        const float fx = mx == -INFINITY ? 0.0f : exp2_fast(mx - mm);
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const uint32_t y[4] = {v[e].x, v[e].y, v[e].z, v[e].w};
#pragma unroll
                            for (int z = 0; z < 4; ++z)
                                o[4 * e + z] = __float_as_uint(fmaf(
                                    __uint_as_float(y[z]), fx, __uint_as_float(o[4 * e + z])));
                        }
                    }
                    emit_columns<DP, SHARED>(p, plan, t, c, o, i, mm, ll, stage, w, tid);
                }
            }
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
    unsigned char* stages = slots + R::kSlots * R::kSlot;
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
            mbar_init(smem_addr(&sh.p_ready[w][0]), 4);
            mbar_init(smem_addr(&sh.p_ready[w][1]), 4);
            mbar_init(smem_addr(&sh.o_done[w]), 1);
        }
        sh.stop = 0;
        mbar_init_fence();
    }
    pdl_wait();
    pdl_allow_dependents();

    // -- this CTA's share of the line -----------------------------------------
    // `tps` threads count an entity's tiles together
    const int32_t entities = SHARED ? p.n_groups : p.n_seqs;
    bool bad = false;
    int32_t tps = 32;
    while (tps > 1 && (int64_t)entities * tps > kTileThreads)
        tps /= 2;
    const int32_t sets = kTileThreads / tps;
    const int32_t per = (entities + sets - 1) / sets;
    const int32_t e0 = min((int32_t)threadIdx.x / tps * per, entities);
    const int32_t e1 = min(e0 + per, entities);
    auto count = [&](const Ragged& r, int32_t first, int32_t step) {
        const int32_t tiles = entity_tiles(r, plan.g);
        int64_t n = 0;
        for (int32_t i = first; i < tiles; i += step)
            n += tile_units<SHARED>(p, r, plan.g, i) + kPairCost;
        return n;
    };
    int64_t mine = 0;
    bool broken = false;  // starts of groups that do not follow one another
    if constexpr (SHARED)
        for (int32_t e = e0; e < e1; ++e) {
            const int32_t a = __ldg(p.group_start + e), b = __ldg(p.group_start + e + 1);
            broken = broken || a < 0 || b < a || b > p.n_seqs;
        }
    for (int32_t e = e0; e < e1; ++e)
        mine += count(load_entity<SHARED>(p, e, bad), threadIdx.x % tps, tps);
    __syncwarp();
    for (int o = 1; o < tps; o <<= 1)
        mine += __shfl_xor_sync(0xFFFFFFFFu, mine, o);
    const bool leads = threadIdx.x % tps == 0;
    if (!leads)
        mine = 0;
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if (lane >= o)
            upto += x;
    }
    if (lane == 31)
        sh.sums[warp] = upto;
    if (__syncthreads_or(broken)) {  // nothing is written
        if (threadIdx.x == 0 && blockIdx.x == 0)
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
    const int64_t end = min(begin + share, line);
    if (leads && begin >= (upto - mine) * p.hk && begin < upto * p.hk) {
        int64_t before = upto - mine;
        int32_t e = e0;
        bool ignore = false;
        for (; e + 1 < e1; ++e) {
            const int64_t n = count(load_entity<SHARED>(p, e, ignore), 0, 1);
            if (begin < (before + n) * p.hk)
                break;
            before += n;
        }
        sh.found.seq = e;
        sh.found_before = before;
    }
    __syncthreads();
    if (warp == 0) {  // the tile within the entity, 32 at a time
        bool ignore = false;
        const Ragged r = load_entity<SHARED>(p, sh.found.seq, ignore);
        const int32_t tiles = entity_tiles(r, plan.g);
        int64_t before = sh.found_before;
        for (int32_t i0 = 0; i0 < tiles; i0 += 32) {
            const int32_t n =
                i0 + lane < tiles ? tile_units<SHARED>(p, r, plan.g, i0 + lane) + kPairCost : 0;
            int64_t sum = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t x = __shfl_up_sync(0xFFFFFFFFu, sum, o);
                if (lane >= o)
                    sum += x;
            }
            const unsigned in = __ballot_sync(0xFFFFFFFFu, begin < (before + sum) * p.hk);
            if (in != 0) {
                if (lane == __ffs(in) - 1) {
                    const int64_t rest = begin - (before + sum - n) * p.hk;
                    sh.found.sub = i0 + lane;
                    sh.found.kvh = (int32_t)(rest / n);
                    sh.found.unit = (int32_t)(rest % n) - kPairCost;
                }
                break;
            }
            before += __shfl_sync(0xFFFFFFFFu, sum, 31);
        }
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
        tile_softmax_role<DP, FULL, SHARED>(p, plan, q + w * R::kQ, stages + w * R::kStage, sh, c,
                                            begin, end, share, w, threadIdx.x & 127);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == kMmaWarp) {
            tile_mma_role<DP, SHARED>(p, plan, q, slots, sh, c, begin, end);
            // every product and every arrival asked for has happened
            if (elect_one())
                tc_commit(smem_addr(&sh.drain));
            __syncwarp();
            mbar_wait(smem_addr(&sh.drain), 0);
            __syncwarp();
        } else if (warp == kLoadWarp) {
            tile_load_role<DP, SHARED>(p, plan, &kmap, &vmap, slots, sh, c, begin, end, lane);
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
    plan.g = make_row_divide(p.hq / p.hk);
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
