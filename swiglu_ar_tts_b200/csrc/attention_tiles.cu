// Attention over a paged KV cache (sm_100a): the tile kernel, for many query
// rows a key (prompts, chunks of prompts, a prefix under many candidates), bf16
// heads of up to 128 values, pages of a multiple of 8 slots.
//
// The formula is the row kernel's.  A tile is 256 rows ((token, head of one
// key/value head's group) pairs), two sub-tiles of 128, the M of tcgen05.mma; a
// unit is 128 keys, taken in two halves of 64.  A unit's 4 x 256 x 128 x 128
// operations are 2,048 clocks of the SM's tensor cores (2,624 with N = 64, where
// shared memory feeds an M = 128 product at 50 clocks for 32: measured), its
// 32,768 exponentials 2,048 clocks of the exponential units, its keys and values
// 64 KB.  So everything runs at once, on sixteen warps:
//   warp 9       copies: keys and values of a unit by tensor maps, page by page,
//                into a ring of slots in the 128-byte swizzle;
//   warp 10      the CTA's pieces of work (for all roles) and their queries;
//   warps 8, 11  products of sub-tile 0 and 1: S_w = Q_w K^T into tensor memory,
//                O_w += P_w V with P_w read from tensor memory;
//   warps 0-3, 4-7    softmax of sub-tile 0 and 1, a row a thread: 64 scores out
//                of tensor memory, maximum, exponentials, sum, P (bf16) back
//                over them;
//   warps 12-15  results: O out of tensor memory, divided by l, stored.
// The two halves' scores lie in columns of their own: while a half is in the
// softmax, the other half's weights are multiplied and its next scores made, so
// the softmax warps never wait for products (traced: 150 clocks between a half's
// end and the next one's first load, all of it the barrier's own latency).  A
// unit takes 3,300 clocks, 62% of them exponentials: what is left between them
// (maximum 200, loads and stores of tensor memory 140, barriers 250 of 1,650 a
// half) is latency of the two warps that a scheduler has, and there is room for
// no third in the registers.  Exponentials on the fp32 pipe (1/8 to 1/2 of them)
// measured slower, and so did weights taken with the maximum before this half's.
// One prompt of 16,384 tokens, 16 heads on 8 of 128: 900 us, 1,222 TFLOP/s at full
// clocks (73% of the measured cuBLAS rate); in repeated calls, whose clocks the
// power cap holds down, 1,000-1,050 us (75-78% of cuBLAS's rate under it).
//
// O stays in tensor memory; a row of it is scaled only when the row's maximum has
// grown by more than 2^8 since the last time (P and l carry the factor until then;
// both are floating point, so nothing is lost).  Nothing of a row depends on the
// rows beside it.  Tensor memory: S_0, S_1, O_0, O_1,
// all 512 columns, one CTA an SM.
//
// The line of units is cut into equal shares, as in the row kernel; partial
// results go through the workspace and attention_join_kernel, launched behind,
// joins them in the order of the keys.  Every wait is bounded in time.
#include <float.h>

#include "attention_common.cuh"
#include "tcgen05.cuh"

namespace arops {
namespace {

constexpr int kSubRows = 128;
constexpr int kTileRows = 2 * kSubRows;
constexpr int kTileUnit = 128;  // keys
constexpr int kTileThreads = 512;
constexpr int kTileWarps = kTileThreads / 32;
// A unit's scores are made and used in two halves of 64 keys, each in its own
// columns: while one half is in the softmax, the other's weights are multiplied
// and its next scores made.
constexpr int kHalfUnit = kTileUnit / 2;
constexpr int kMmaWarp = 8;
constexpr int kLoadWarp = 9;
constexpr int kMmaWarp1 = 11;    // of sub-tile 1; warp 10 makes pieces
constexpr int kResultWarp = 12;  // to 15

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
    static constexpr int kStage = kSubRows * DP * 2;     // results of a sub-tile
    static constexpr uint32_t kS = 0, kO = 2 * kTileUnit;  // columns: S_w at kS + 128 w
};

// A pair that CTA cta0 begins and leaves unfinished; cta1 < cta0: none.
struct TileSplit {
    int32_t tok0, ntok, sub, kvh, cta1;
};

// The cap's polynomial on raw products, in base 2: x P(x^2) with scale, cap and
// base in the coefficients.  |score| / cap is |product| * caps.  Where the cap is
// so far below the scale that the coefficients would overflow, products are
// taken times `unit` first (1 otherwise).
struct CapForm {
    float c[4];
    float caps, unit;
};

CapForm make_cap_form(const ScoreMap& m)
{
    CapForm f = {};
    float in = fmaxf(fminf(m.scale * m.inv_cap, FLT_MAX), -FLT_MAX), out = m.scale * kLog2e;
    f.caps = fabsf(in);
    f.unit = 1.0f;
    if (f.caps >= 1e5f) {
        f.unit = in;
        in = 1.0f;
        out = m.cap * kLog2e;
    }
    const float in2 = in * in;
    f.c[0] = kTanh0 * out;
    f.c[1] = kTanh1 * out * in2;
    f.c[2] = kTanh2 * out * (in2 * in2);
    f.c[3] = kTanh3 * out * (in2 * in2 * in2);
    return f;
}

struct TilePlan {
    ScoreMap score;
    CapForm cap;
    TileSplit* splits;  // one a CTA
    float* parts;
    float* prefix_o;    // shared prefixes: results go here, not to out
    float* prefix_ml;
    RowDivide g;        // query heads a key head
    int32_t box;        // keys of one tensor-map copy
    bool q_map;         // queries by tensor-map copies
};

struct TileCursor {
    int32_t seq, sub, kvh, unit;
};

// Keys of one (tile, key head) pair and of its sub-tiles: units [jlo, jhi).
struct TileSpan {
    int32_t tok0, ntok, len, bidir;
    int32_t lo, first, units;  // first seen key, rounded down to a unit and not
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
        int32_t lo, hi, first;
        ragged_range<kTileUnit>(p, r, g, (uint32_t)sub * kTileRows, kTileRows, lo, hi, first);
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
    int32_t lo[2], hi[2], first[2] = {0, 0};
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const uint32_t row0 = (uint32_t)c.sub * kTileRows + w * kSubRows;
        lo[w] = hi[w] = 0;
        if (row0 < rows) {
            if constexpr (SHARED)
                hi[w] = r.len;
            else
                ragged_range<kTileUnit>(p, r, g, row0, kSubRows, lo[w], hi[w], first[w]);
        } else if (w == 1) {
            lo[1] = lo[0];
            hi[1] = lo[0];
        }
    }
    t.lo = lo[0];
    t.first = first[0];
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

// One pair's units of a CTA's share, as the roles see it.
struct TilePiece {
    int32_t tok0, ntok, len, bidir, lo, first;
    int32_t sub, kvh;
    int32_t u0, u1;          // units of the share; u0 == u1: the end
    int32_t a[2], b[2];      // of each sub-tile: [a, b)
    int32_t cta0, cta1;      // the pair's CTAs
    int32_t whole;
    const int32_t* table;
};

constexpr int kPieces = 4;

// The CTA's barriers and flags in shared memory.
template <int DP>
struct TileShared {
    uint64_t full[TileTraits<DP>::kSlots];
    uint64_t empty[TileTraits<DP>::kSlots];
    uint64_t piece_full[kPieces];
    uint64_t piece_empty[kPieces];
    uint64_t tail;        // a copy that reaches past the sequence's end
    uint64_t q_ready[2];
    uint64_t q_free[2];   // a piece's last product with Q_w is done
    uint64_t s_full[2][2];   // [sub-tile][half]
    uint64_t p_ready[2][2];
    uint64_t o_done[2][2];
    uint64_t ml_ready[2]; // a piece's m and l are in shared memory
    uint64_t o_free[2];   // a piece's O_w, m and l have been read
    uint64_t drain[2];
    TilePiece pieces[kPieces];
    float m[2][kSubRows], l[2][kSubRows];
    uint32_t tmem;
    int stop;             // a wait ran out: everybody leaves
    int64_t sums[kTileWarps];
    int64_t found_before;  // line in front of the found entity, per key head
    TileCursor found;
};

// All of a CTA's shared memory; its operands lie on 1024-byte boundaries, which
// is where dynamic shared memory begins in a kernel without any other (checked
// by the kernel).
template <int DP>
constexpr int tile_smem()
{
    using R = TileTraits<DP>;
    return 2 * R::kQ + R::kSlots * R::kSlot + R::kStage + (int)sizeof(TileShared<DP>);
}

// Waits for `parity` of `bar`; false once anybody's wait has run out.
__device__ __noinline__ bool wait_slow(uint32_t b, uint32_t parity, int* stop, unsigned* err)
{
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

__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, int* stop, unsigned* err)
{
    const uint32_t b = smem_addr(bar);
    return mbar_try_wait(b, parity) || wait_slow(b, parity, stop, err);
}

// A warp's wait: all lanes go on together, or none does.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int* stop, unsigned* err)
{
    return __all_sync(0xFFFFFFFFu, wait_for(bar, parity, stop, err));
}

// A role's way through the pieces (a warp).
template <int DP>
struct PieceReader {
    uint32_t n = 0;
    __device__ __forceinline__ bool next(TileShared<DP>& sh, TilePiece& t, unsigned* err)
    {
        const uint32_t s = n % kPieces;
        if (!warp_wait(&sh.piece_full[s], (n / kPieces) & 1, &sh.stop, err))
            return false;
        t = sh.pieces[s];
        __syncwarp();
        if ((threadIdx.x & 31) == 0)
            mbar_arrive(smem_addr(&sh.piece_empty[s]));
        ++n;
        return t.u0 < t.u1;
    }
};

// ---------------------------------------------------------------------------
// Copies of keys and values (one warp).
// ---------------------------------------------------------------------------
template <int DP>
__device__ void tile_load_role(const AttentionParams& p, const TilePlan& plan,
                               const CUtensorMap* kmap, const CUtensorMap* vmap,
                               unsigned char* slots, TileShared<DP>& sh, int lane)
{
    using R = TileTraits<DP>;
    const int boxes = kTileUnit / plan.box;
    uint32_t n = 0;      // slots filled
    uint32_t tails = 0;  // copies waited for here
    bool ok = true;
    PieceReader<DP> reader;
    TilePiece t;
    while (ok && reader.next(sh, t, p.err)) {
        for (int32_t u = t.u0; ok && u < t.u1; ++u) {
            const int32_t key0 = t.lo + u * kTileUnit;
            const int32_t key = key0 + lane * plan.box;
            // a copy of a page that does not exist, or that nobody sees any of,
            // brings zeros
            int32_t page = (int32_t)p.map.num_pages, slot = 0;
            if (lane < boxes && key < t.len && key + plan.box > t.first) {
                int32_t pi;
                split_position(p.map, key, pi, slot);
                page = __ldg(t.table + pi);
                if (page < 0 || page >= p.map.num_pages) {
                    page = (int32_t)p.map.num_pages;
                    record_device_error(p.err, kDeviceErrBadIndexBit);
                }
            }
            const bool tail = t.len - key0 < kTileUnit;
#pragma unroll 1
            for (int kv = 0; kv < 2; ++kv) {
                const uint32_t s = n % R::kSlots;
                ok = warp_wait(&sh.empty[s], ((n / R::kSlots) & 1) ^ 1, &sh.stop, p.err);
                if (!ok)
                    break;
                unsigned char* dst = slots + s * R::kSlot;
                const bool clean = tail && kv == 1;
                const uint32_t bar = smem_addr(clean ? &sh.tail : &sh.full[s]);
                if (lane == 0)
                    mbar_arrive_expect_tx(bar, R::kSlot);
                __syncwarp();
                if (lane < boxes) {
#pragma unroll
                    for (int h = 0; h < R::kHalves; ++h)
                        tensor_load4(smem_addr(dst) + h * (kTileUnit * 128) + lane * plan.box * 128,
                                     kv ? vmap : kmap, bar, h * 64, slot, t.kvh, page);
                }
                ++n;
                if (clean) {
                    // slots behind the sequence's end may hold anything, and 0
                    // times a NaN is one: their values become zeros
                    ok = warp_wait(&sh.tail, tails & 1, &sh.stop, p.err);
                    ++tails;
                    if (!ok)
                        break;
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
// Pieces and queries (one warp).
// ---------------------------------------------------------------------------
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

// A sub-tile's 128 query rows, swizzled as a tensor-map copy leaves them: by
// such a copy where the heads of a token divide the 128 rows, else 16 bytes at
// a time.
template <int DP>
__device__ __forceinline__ void load_queries(const AttentionParams& p, const TilePlan& plan,
                                             const CUtensorMap* qmap, const TilePiece& t, int w,
                                             unsigned char* q, uint64_t* ready, int lane)
{
    using R = TileTraits<DP>;
    const uint32_t row0 = (uint32_t)t.sub * kTileRows + w * kSubRows;
    if (plan.q_map) {
        if (lane == 0) {
            mbar_arrive_expect_tx(smem_addr(ready), R::kQ);
#pragma unroll
            for (int h = 0; h < R::kHalves; ++h)
                tensor_load3(smem_addr(q) + h * (kSubRows * 128), qmap, smem_addr(ready), h * 64,
                             (int32_t)(t.kvh * plan.g.n), (int32_t)(t.tok0 + plan.g(row0)));
        }
        __syncwarp();
        return;
    }
    constexpr int kChunks = DP / 8;
    constexpr int kStep = 32 / kChunks;
    const int chunk = lane % kChunks;
    int row = lane / kChunks;
    const bool used = chunk < p.head_dim / 8;
    RowStep r(plan.g, row0 + row, kStep);
    const __nv_bfloat16* all = static_cast<const __nv_bfloat16*>(p.q);
    const __nv_bfloat16* base =
        all + t.tok0 * p.q_stride + (int64_t)t.kvh * plan.g.n * p.head_dim + chunk * 8;
    const uint32_t dst = smem_addr(q) + (chunk / 8) * (kSubRows * 128);
#pragma unroll 4
    for (int i = 0; i < kSubRows / kStep; ++i) {
        const bool ok = r.tok < (uint32_t)t.ntok && used;
        const __nv_bfloat16* src =
            ok ? base + (int64_t)r.tok * p.q_stride + r.head * p.head_dim : all;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                         dst + row * 128 + (((chunk & 7) ^ (row & 7)) << 4)),
                     "l"(src), "r"(ok ? 16u : 0u)
                     : "memory");
        row += kStep;
        r.next();
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    fence_async_proxy();
    __syncwarp();
    if (lane == 0)
        mbar_arrive(smem_addr(ready));
}

template <int DP, bool SHARED>
__device__ void tile_query_role(const AttentionParams& p, const TilePlan& plan,
                                const CUtensorMap* qmap, unsigned char* q, TileShared<DP>& sh,
                                const TileCursor& from, int64_t begin, int64_t end, int64_t share,
                                int lane)
{
    uint32_t phase = 3;  // parity of the next wait for q_free, a bit a sub-tile
    TilePiece t;
    TileWalk walk(from, begin, end);
    bool more = true;
    for (uint32_t n = 0; more; ++n) {
        TileSpan s;
        t.u0 = t.u1 = 0;
        more = walk.next<SHARED>(p, plan, s, t.u0, t.u1);
        if (more) {
            t.tok0 = s.tok0;
            t.ntok = s.ntok;
            t.len = s.len;
            t.bidir = s.bidir;
            t.lo = s.lo;
            t.first = s.first;
            t.table = s.table;
            t.sub = walk.pair.sub;
            t.kvh = walk.pair.kvh;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                t.a[i] = max(s.jlo[i], t.u0);
                t.b[i] = min(s.jhi[i], t.u1);
            }
            t.cta0 = (int32_t)(walk.place / share);
            t.cta1 = (int32_t)((walk.place + s.units - 1) / share);
            t.whole = t.u0 == 0 && t.u1 == s.units;
        } else {
            t.u0 = t.u1 = 0;
        }
        const uint32_t slot = n % kPieces;
        if (!warp_wait(&sh.piece_empty[slot], ((n / kPieces) & 1) ^ 1, &sh.stop, p.err))
            return;
        if (lane == 0) {
            sh.pieces[slot] = t;
            mbar_arrive(smem_addr(&sh.piece_full[slot]));
        }
        __syncwarp();
        if (!more)
            return;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            if (t.a[w] >= t.b[w])
                continue;
            if (!warp_wait(&sh.q_free[w], (phase >> w) & 1, &sh.stop, p.err))
                return;
            phase ^= 1u << w;
            load_queries<DP>(p, plan, qmap, t, w, q + w * TileTraits<DP>::kQ, &sh.q_ready[w],
                             lane);
        }
    }
}

// ---------------------------------------------------------------------------
// Products (one thread of one warp a sub-tile).
// ---------------------------------------------------------------------------
template <int DP>
__device__ void tile_mma_role(const AttentionParams& p, const unsigned char* q,
                              const unsigned char* slots, TileShared<DP>& sh, int w)
{
    using R = TileTraits<DP>;
    constexpr uint32_t kWordS = mma_word(kSubRows, kHalfUnit, false);
    constexpr uint32_t kWordO = mma_word(kSubRows, DP, true);
    // keys and queries: K (head_dim) contiguous, one 64-value block behind the
    // other; values: N (head_dim) contiguous, the leading offset between blocks
    const uint32_t q_low = operand_low(smem_addr(q), 16);
    const uint32_t k_low = operand_low(smem_addr(slots), 16);
    const uint32_t v_low = operand_low(smem_addr(slots), kTileUnit * 128);
    const uint32_t o = sh.tmem + R::kO + w * DP;
    const uint32_t s = sh.tmem + R::kS + w * kTileUnit;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        return wait_for(bar, parity, &sh.stop, p.err);
    };
    // The units of all pieces form one line: under the softmax of a piece's last
    // unit the next piece's first S is multiplied.  Each sub-tile has a warp:
    // one for both needed 4,000 clocks a unit for its ~600 instructions between
    // those of the softmax, the tensor cores 2,600.
    struct Unit {
        int32_t u, u1, a, b;
    };
    uint32_t pieces = 0;
    auto next_piece = [&](Unit& n) {
        const uint32_t slot = pieces % kPieces;
        if (!wait(&sh.piece_full[slot], (pieces / kPieces) & 1))
            return false;
        const TilePiece& t = sh.pieces[slot];
        n = {t.u0, t.u1, t.a[w], t.b[w]};
        mbar_arrive(smem_addr(&sh.piece_empty[slot]));
        ++pieces;
        return n.u < n.u1;
    };
    uint32_t used = 0;  // slots consumed: keys 0, values 0, keys 1, values 1, ...
    uint32_t p_phase = 0, q_phase = 0, o_phase = 1;  // parity of the next wait
    Unit cur = {0, 0, 0, 0}, nxt;
    bool have = false, more = next_piece(nxt);
    while (have || more) {
        uint32_t vs = 0, ks = 0;
        if (have) {
            vs = used % R::kSlots;
            if (!wait(&sh.full[vs], (used / R::kSlots) & 1))
                return;
            ++used;
        }
        if (more) {
            ks = used % R::kSlots;
            if (!wait(&sh.full[ks], (used / R::kSlots) & 1))
                return;
            ++used;
        }
        const uint32_t vb = v_low + vs * (R::kSlot >> 4);
        const uint32_t kb = k_low + ks * (R::kSlot >> 4);
        const bool pv = have && cur.u >= cur.a && cur.u < cur.b;
        const bool qk = more && nxt.u >= nxt.a && nxt.u < nxt.b;
        if (pv && cur.u == cur.a) {  // the piece before this one's O_w has been read
            if (!wait(&sh.o_free[w], o_phase))
                return;
            o_phase ^= 1;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (pv) {  // O_w (+)= P_w V
                if (!wait(&sh.p_ready[w][h], p_phase))
                    return;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < kHalfUnit / 16; ++k)
                    tc_mma_ts(o, s + h * kHalfUnit + k * 8,
                              vb + (h * (kHalfUnit / 16) + k) * (2048 >> 4), kWordO,
                              h > 0 || k > 0 || cur.u > cur.a);
                tc_commit(smem_addr(&sh.o_done[w][h]));
            }
            if (qk) {  // the next S_w = Q_w K^T
                if (h == 0 && nxt.u == nxt.a) {
                    if (!wait(&sh.q_ready[w], q_phase))
                        return;
                    q_phase ^= 1;
                    tc_fence_after();
                }
#pragma unroll
                for (int k = 0; k < DP / 16; ++k) {
                    const uint32_t off = ((k / 4) * (kTileUnit * 128) + (k % 4) * 32) >> 4;
                    tc_mma_ss(s + h * kHalfUnit, q_low + off,
                              kb + (h * kHalfUnit * 128 >> 4) + off, kWordS, k > 0);
                }
                tc_commit(smem_addr(&sh.s_full[w][h]));
            }
        }
        if (pv)
            p_phase ^= 1;
        if (qk && nxt.u + 1 == nxt.b)
            tc_commit(smem_addr(&sh.q_free[w]));
        if (have)
            tc_commit(smem_addr(&sh.empty[vs]));
        if (more)
            tc_commit(smem_addr(&sh.empty[ks]));
        have = more;
        cur = nxt;
        if (more && ++nxt.u >= nxt.u1)
            more = next_piece(nxt);
    }
}

// ---------------------------------------------------------------------------
// Softmax (four warps a sub-tile, a row a thread).
// ---------------------------------------------------------------------------
// Half a unit of a row's scores from its products, in base 2: cap, then bias.
//   |s| <= cap / 2 (a cap is there for outliers): tanh by its polynomial, on the
//   fp32 pipe, instead of 2 exponential-unit operations a key; scale and base are
//   in its coefficients.  The form is each score's own, so no bit depends on the
//   rows beside it; the warp skips the second one where none of its scores needs
//   it (a chunk of 256 tokens on 12 and 21 thousand keys: 119 us, 173 where every
//   half has such a score; a prompt of 16,384 tokens 1,408 and 2,417).
//   Keys not behind the query: |i - j| without the absolute value, one FMA.
__device__ __forceinline__ void map_scores(uint32_t (&s)[kHalfUnit], uint32_t s_addr,
                                           const ScoreMap& map, const CapForm& form,
                                           float slope, int32_t gap)
{
    auto at = [&](int i) {
        return make_float2(__uint_as_float(s[i]), __uint_as_float(s[i + 1]));
    };
    auto put = [&](int i, float2 x) {
        s[i] = __float_as_uint(x.x);
        s[i + 1] = __float_as_uint(x.y);
    };
    auto both = [](float x) { return make_float2(x, x); };
    const float bias = -slope * kLog2e;
    // the bias of keys e, e + 1 (e = 0, 2, .. 14); of those 16, 32, 48 on: one
    // more addition each
    const float2 step = both(-16.0f * bias);
    const bool behind = __any_sync(0xFFFFFFFFu, gap < kHalfUnit - 1);
    if (map.cap > 0.0f) {
        float big = 0.0f;
#pragma unroll
        for (int i = 0; i < kHalfUnit; i += 2)
            big = fmaxf(fmaxf(big, fabsf(__uint_as_float(s[i]))),
                        fabsf(__uint_as_float(s[i + 1])));
        const float2 c0 = both(form.c[0]), c1 = both(form.c[1]), c2 = both(form.c[2]),
                     c3 = both(form.c[3]);
        if (__any_sync(0xFFFFFFFFu, big * form.caps > 0.5f) || form.unit != 1.0f) {
            // both forms, 16 products at a time out of tensor memory and back (a
            // row's 64 with two forms each do not fit the registers); the sums as
            // below
            float2 add[8];
#pragma unroll
            for (int e = 0; e < 16; e += 2)
                add[e / 2] = behind ? both(0.0f)
                                    : make_float2(bias * (float)(gap - e),
                                                  bias * (float)(gap - e - 1));
#pragma unroll 1
            for (int c = 0; c < kHalfUnit; c += 16) {
                uint32_t raw[16];
                tc_load16(raw, s_addr + c);
                tc_wait_ld();
                tc_loaded<16>(raw);
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    const float2 p =
                        make_float2(__uint_as_float(raw[e]), __uint_as_float(raw[e + 1]));
                    const float2 x = mul2(p, both(form.unit));
                    const float2 y = mul2(x, x);
                    float2 r = fma2(x, fma2(fma2(fma2(y, c3, c2), y, c1), y, c0), add[e / 2]);
                    const float fx = soft_cap_large(p.x * map.scale, map.cap, map.inv_cap);
                    const float fy = soft_cap_large(p.y * map.scale, map.cap, map.inv_cap);
                    r.x = fabsf(p.x) * form.caps > 0.5f ? fmaf(fx, kLog2e, add[e / 2].x) : r.x;
                    r.y = fabsf(p.y) * form.caps > 0.5f ? fmaf(fy, kLog2e, add[e / 2].y) : r.y;
                    raw[e] = __float_as_uint(r.x);
                    raw[e + 1] = __float_as_uint(r.y);
                    if (!behind)
                        add[e / 2] = add2(add[e / 2], step);
                }
                tc_store16(s_addr + c, raw);
            }
            tc_wait_st();
            tc_load32(s, s_addr);
            tc_load32(s + 32, s_addr + 32);
            tc_wait_ld();
            tc_loaded<kHalfUnit>(s);
        } else if (behind) {
#pragma unroll
            for (int i = 0; i < kHalfUnit; i += 2) {
                const float2 x = at(i);
                const float2 y = mul2(x, x);
                put(i, mul2(x, fma2(fma2(fma2(y, c3, c2), y, c1), y, c0)));
            }
        } else {
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
                float2 add = make_float2(bias * (float)(gap - e), bias * (float)(gap - e - 1));
#pragma unroll
                for (int i = e; i < kHalfUnit; i += 16) {
                    const float2 x = at(i);
                    const float2 y = mul2(x, x);
                    put(i, fma2(x, fma2(fma2(fma2(y, c3, c2), y, c1), y, c0), add));
                    add = add2(add, step);
                }
            }
        }
        if (!behind)
            return;
    } else {
        const float2 out = both(map.scale * kLog2e);
#pragma unroll
        for (int i = 0; i < kHalfUnit; i += 2)
            put(i, mul2(at(i), out));
    }
    if (__all_sync(0xFFFFFFFFu, slope == 0.0f))
        return;
#pragma unroll
    for (int i = 0; i < kHalfUnit; ++i)
        s[i] = __float_as_uint(fmaf(bias, fabsf((float)gap - (float)i), __uint_as_float(s[i])));
}

template <int DP, bool FULL, bool SHARED>
__device__ void tile_softmax_role(const AttentionParams& p, const TilePlan& plan,
                                  TileShared<DP>& sh, int w, int tid)
{
    using R = TileTraits<DP>;
    const int lane = tid & 31;
    const uint32_t lanes = (uint32_t)(tid & ~31) << 16;  // the warp's lanes of tensor memory
    const uint32_t s_base = sh.tmem + lanes + R::kS + w * kTileUnit;
    const uint32_t o_addr = sh.tmem + lanes + R::kO + w * DP;
    uint32_t on = 0;     // units done: S tiles seen, P V products asked for
    uint32_t ended = 0;  // pieces with units of this sub-tile
    const float scale = FULL ? 1.0f : plan.score.scale;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        return warp_wait(bar, parity, &sh.stop, p.err);
    };
    PieceReader<DP> reader;
    for (;;) {
        int32_t key0, a, b, pos, lo = 0, hi;
        float slope = 0.0f;
        {
            TilePiece t;
            if (!reader.next(sh, t, p.err))
                return;
            key0 = t.lo;
            a = w ? t.a[1] : t.a[0];
            b = w ? t.b[1] : t.b[0];
            // this thread's row
            const RowStep r(plan.g, (uint32_t)t.sub * kTileRows + w * kSubRows + tid, 1);
            const bool valid = r.tok < (uint32_t)t.ntok;
            hi = t.len;
            if constexpr (SHARED) {
                bool ignore = false;
                pos = t.len - 1;
                if (FULL && valid)
                    pos += clamp_length(__ldg(p.kv_lens + t.tok0 + r.tok),
                                        p.max_pages * p.map.page_size, ignore);
            } else {
                pos = t.len - t.ntok + (int32_t)r.tok;
                // (nobody reads a row that does not exist, whatever query lies there;
                // no keys behind the length for it, so that masking stays rare)
                if (valid)
                    visible_keys(pos, t.len, t.bidir, p.window, lo, hi);
            }
            if (FULL && p.slopes && valid)
                slope = __ldg(p.slopes + t.kvh * plan.g.n + r.head);
        }
        if (a >= b)
            continue;
        key0 += a * kTileUnit;
        float m = -INFINITY, l = 0.0f;
        for (int32_t n = b - a; n > 0; --n) {
#pragma unroll 1
            for (int h = 0; h < 2; ++h, key0 += kHalfUnit) {
                if (!wait(&sh.s_full[w][h], on & 1))
                    return;
                tc_fence_after();
                const uint32_t s_addr = s_base + h * kHalfUnit;
                uint32_t s[kHalfUnit];
                tc_load32(s, s_addr);
                tc_load32(s + 32, s_addr + 32);
                tc_wait_ld();
                tc_loaded<kHalfUnit>(s);
                if constexpr (FULL)
                    map_scores(s, s_addr, plan.score, plan.cap, slope, pos - key0);
                if (__any_sync(0xFFFFFFFFu, key0 < lo || hi - key0 < kHalfUnit)) {
                    const int32_t first = lo - key0, last = hi - key0;
#pragma unroll
                    for (int e = 0; e < kHalfUnit; ++e)
                        s[e] = e >= first && e < last ? s[e] : __float_as_uint(-INFINITY);
                }
                float mx[4];
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    mx[x] = fmaxf(__uint_as_float(s[x]), __uint_as_float(s[4 + x]));
#pragma unroll
                for (int e = 8; e < kHalfUnit; e += 8)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        mx[x] = fmaxf(fmaxf(mx[x], __uint_as_float(s[e + x])),
                                      __uint_as_float(s[e + 4 + x]));
                const float mu = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale;

                // scale what there is only when a maximum has grown by 2^8; rows
                // beside the one that has grown keep theirs (a factor of 1), so
                // that a row's bits depend on no other row's query
                const bool grown = mu > m + 8.0f || (m == -INFINITY && mu > -INFINITY);
                if (__any_sync(0xFFFFFFFFu, grown)) {
                    float f = 1.0f;
                    if (grown) {
                        f = m == -INFINITY ? 0.0f : exp2_fast(m - mu);
                        m = mu;
                    }
                    l *= f;
                    if (h > 0 || n < b - a) {
                        if (!wait(&sh.o_done[w][h ^ 1], h > 0 ? on & 1 : (on - 1) & 1))
                            return;
                        tc_fence_after();
#pragma unroll 1
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
                // the weights are rounded to bf16 (2^-8 of each at most), the
                // type of the values that they multiply; l keeps them in fp32
                uint32_t pk[32];
#pragma unroll
                for (int e = 0; e < kHalfUnit; e += 2) {
                    float2 x = make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1]));
                    x = fma2(x, sc, bs);
                    x.x = exp2_fast(x.x);
                    x.y = exp2_fast(x.y);
                    sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], x);
                    pk[e >> 1] = pack_bf16x2(x.x, x.y);
                }
                tc_store32(s_addr, pk);
                const float2 all = add2(sum[0], sum[1]);
                l += all.x + all.y;
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_addr(&sh.p_ready[w][h]));
            }
            ++on;
        }
        if (!wait(&sh.o_free[w], (ended & 1) ^ 1))
            return;
        ++ended;
        sh.m[w][tid] = m;
        sh.l[w][tid] = l;
        __syncwarp();
        if (lane == 0)
            mbar_arrive(smem_addr(&sh.ml_ready[w]));
    }
}

// ---------------------------------------------------------------------------
// Results (four warps, a row a thread).
// ---------------------------------------------------------------------------
// All four warps agree on `ok`.
__device__ __forceinline__ bool result_agree(bool ok)
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.and.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)ok)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ void result_barrier()
{
    asm volatile("barrier.cta.sync 1, 128;" ::: "memory");
}

// 32 columns of a prefix's results, a row a thread.
template <int DP>
__device__ __forceinline__ void store_prefix(const AttentionParams& p, const TilePlan& plan,
                                             int64_t token, int head, const uint32_t (&o)[32],
                                             int col, float m, float l)
{
    const int64_t at = token * p.hq + head;
    float4* dst = reinterpret_cast<float4*>(plan.prefix_o + at * DP + col);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        dst[e] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                             __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
    if (col == 0)
        *reinterpret_cast<float2*>(plan.prefix_ml + at * 2) = make_float2(m, l);
}

// 32 values times `by` as 16 pairs of bf16.  (A row that sees no key has O = 0
// and by = 0.)
__device__ __forceinline__ void scale_pack(const uint32_t (&o)[32], float by, uint32_t (&y)[16])
{
    const float2 f = make_float2(by, by);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        const float2 x =
            mul2(make_float2(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1])), f);
        y[e] = pack_bf16x2(x.x, x.y);
    }
}

template <int DP, bool SHARED>
__device__ void tile_result_role(const AttentionParams& p, const TilePlan& plan,
                                 unsigned char* stage, TileShared<DP>& sh, int tid)
{
    using R = TileTraits<DP>;
    const int lane = tid & 31;
    const uint32_t lanes = (uint32_t)(tid & ~31) << 16;
    uint32_t on0 = 0, on1 = 0, ended0 = 0, ended1 = 0;
    TileSplit split = {0, 0, 0, 0, -1};
    PieceReader<DP> reader;
    TilePiece t;
    for (;;) {
        // the four warps leave together: one of them alone would leave the
        // others in a barrier
        const bool more = reader.next(sh, t, p.err);
        if (!result_agree(more))
            break;
        if (!t.whole && t.u0 == 0)
            split = {t.tok0, t.ntok, t.sub, t.kvh, t.cta1};
#pragma unroll 1
        for (int w = 0; w < 2; ++w) {
            const int32_t units = w ? t.b[1] - t.a[1] : t.b[0] - t.a[0];
            const bool has = units > 0;
            float m = -INFINITY, l = 0.0f;
            if (has) {
                const uint32_t done = (w ? on1 : on0) + units - 1, piece = w ? ended1 : ended0;
                if (w) {
                    on1 += units;
                    ++ended1;
                } else {
                    on0 += units;
                    ++ended0;
                }
                const bool ok = warp_wait(&sh.ml_ready[w], piece & 1, &sh.stop, p.err) &&
                                warp_wait(&sh.o_done[w][1], done & 1, &sh.stop, p.err);
                if (!result_agree(ok))
                    return;
                tc_fence_after();
                m = sh.m[w][tid];
                l = sh.l[w][tid];
            }
            const uint32_t row0 = (uint32_t)t.sub * kTileRows + w * kSubRows;
            float* part = plan.parts +
                          ((int64_t)blockIdx.x * 4 + (t.u0 == 0 ? 2 : 0) + w) *
                              tile_part_floats(DP);
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll 1
            for (int i = 0; i < DP; i += 32) {
                uint32_t o[32];
                if (has) {
                    tc_load32(o, sh.tmem + lanes + R::kO + w * DP + i);
                    tc_wait_ld();
                    tc_loaded<32>(o);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        o[e] = 0;
                }
                if (!t.whole) {
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        *reinterpret_cast<uint4*>(part + ((i + e) / 4 * kSubRows + tid) * 4) =
                            make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                } else if constexpr (SHARED) {
                    const RowStep r(plan.g, row0 + tid, 1);
                    if (r.tok < (uint32_t)t.ntok)
                        store_prefix<DP>(p, plan, t.tok0 + r.tok, t.kvh * plan.g.n + r.head, o, i,
                                         m, l);
                } else {
                    // to shared memory first, so that eight threads store a
                    // row's 128 bytes together
                    uint32_t y[16];
                    scale_pack(o, inv, y);
                    unsigned char* dst = stage + i / 64 * (kSubRows * 128) + tid * 128;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        *reinterpret_cast<uint4*>(
                            dst + (((i / 8 % 8 + e) ^ (tid & 7)) << 4)) =
                            make_uint4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
                }
            }
            if (has) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(smem_addr(&sh.o_free[w]));
            }
            if (!t.whole) {
                part[kSubRows * DP + tid] = m;
                part[kSubRows * DP + kSubRows + tid] = l;
            } else if constexpr (!SHARED) {
                result_barrier();
                const int chunk = tid & 7;
                int row = tid >> 3;
                RowStep r(plan.g, row0 + row, 16);
                const int64_t step = (int64_t)p.hq * p.head_dim;
                __nv_bfloat16* base = static_cast<__nv_bfloat16*>(p.out) + t.tok0 * step +
                                      t.kvh * plan.g.n * p.head_dim + chunk * 8;
                const unsigned char* src = stage + row * 128 + ((chunk ^ (row & 7)) << 4);
#pragma unroll 4
                for (int j = 0; j < kSubRows / 16; ++j) {
                    __nv_bfloat16* dst = base + r.tok * step + r.head * p.head_dim;
#pragma unroll
                    for (int h = 0; h < R::kHalves; ++h) {
                        const uint4 v = *reinterpret_cast<const uint4*>(
                            src + h * (kSubRows * 128) + j * 2048);
                        if (h * 64 + chunk * 8 < p.head_dim && r.tok < (uint32_t)t.ntok)
                            *reinterpret_cast<uint4*>(dst + h * 64) = v;
                    }
                    r.next();
                }
                result_barrier();
            }
        }
    }
    if (tid == 0)
        plan.splits[blockIdx.x] = split;
}

// Joins the parts of the pairs that CTAs left unfinished: a block a (CTA,
// sub-tile, 32 columns), a row a thread, the parts in their order along the
// keys: O = sum_x 2^(m_x - m) O_x, l likewise.
template <int DP, bool SHARED>
__global__ void __launch_bounds__(kSubRows)
attention_join_kernel(const __grid_constant__ AttentionParams p,
                      const __grid_constant__ TilePlan plan)
{
    pdl_wait();
    pdl_allow_dependents();
    const int32_t cta0 = blockIdx.x;
    const int w = blockIdx.y, col = blockIdx.z * 32, tid = threadIdx.x;
    const TileSplit t = plan.splits[cta0];
    if (t.cta1 < cta0)
        return;
    const RowStep r(plan.g, (uint32_t)t.sub * kTileRows + w * kSubRows + tid, 1);
    if (r.tok >= (uint32_t)t.ntok)
        return;
    auto part_of = [&](int32_t x) {
        return plan.parts + ((int64_t)x * 4 + (x == cta0 ? 2 : 0) + w) * tile_part_floats(DP);
    };
    float m = -INFINITY, l = 0.0f;
    uint32_t o[32];
#pragma unroll
    for (int e = 0; e < 32; ++e)
        o[e] = 0;
#pragma unroll 2
    for (int32_t x = cta0; x <= t.cta1; ++x) {
        const float* src = part_of(x);
        const float mx = src[kSubRows * DP + tid];
        const float lx = src[kSubRows * DP + kSubRows + tid];
        float4 v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = *reinterpret_cast<const float4*>(src + ((col / 4 + e) * kSubRows + tid) * 4);
        const float mn = fmaxf(m, mx);
        const float f = part_factor(m, mn);
        const float fx = part_factor(mx, mn);
        m = mn;
        l = l * f + lx * fx;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float y[4] = {v[e].x, v[e].y, v[e].z, v[e].w};
#pragma unroll
            for (int z = 0; z < 4; ++z)
                o[4 * e + z] = __float_as_uint(fmaf(__uint_as_float(o[4 * e + z]), f, y[z] * fx));
        }
    }
    if constexpr (SHARED) {
        store_prefix<DP>(p, plan, t.tok0 + r.tok, t.kvh * plan.g.n + r.head, o, col, m, l);
    } else {
        uint32_t y[16];
        scale_pack(o, l == 0.0f ? 0.0f : 1.0f / l, y);
        __nv_bfloat16* dst =
            static_cast<__nv_bfloat16*>(p.out) +
            ((int64_t)(t.tok0 + r.tok) * p.hq + t.kvh * plan.g.n + r.head) * p.head_dim + col;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (col + e * 8 < p.head_dim)
                *reinterpret_cast<uint4*>(dst + e * 8) =
                    make_uint4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
    }
}

template <int DP, bool FULL, bool SHARED>
__global__ void __launch_bounds__(kTileThreads, 1)
attention_tiles_kernel(const __grid_constant__ AttentionParams p,
                       const __grid_constant__ TilePlan plan,
                       const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap,
                       const __grid_constant__ CUtensorMap qmap)
{
    using R = TileTraits<DP>;
    extern __shared__ __align__(1024) unsigned char smem[];
    unsigned char* q = smem;
    unsigned char* slots = smem + 2 * R::kQ;
    unsigned char* stage = slots + R::kSlots * R::kSlot;
    TileShared<DP>& sh = *reinterpret_cast<TileShared<DP>*>(stage + R::kStage);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

    if (threadIdx.x == 0) {
        for (int i = 0; i < R::kSlots; ++i) {
            mbar_init(smem_addr(&sh.full[i]), 1);
            mbar_init(smem_addr(&sh.empty[i]), 2);  // both sub-tiles' products
        }
        for (int i = 0; i < kPieces; ++i) {
            mbar_init(smem_addr(&sh.piece_full[i]), 1);
            // read by the warps of copies, products, softmax and results
            mbar_init(smem_addr(&sh.piece_empty[i]), 1 + 2 + 8 + 4);
        }
        mbar_init(smem_addr(&sh.tail), 1);
        mbar_init(smem_addr(&sh.drain[0]), 1);
        mbar_init(smem_addr(&sh.drain[1]), 1);
        for (int w = 0; w < 2; ++w) {
            mbar_init(smem_addr(&sh.q_ready[w]), 1);
            mbar_init(smem_addr(&sh.q_free[w]), 1);
            for (int h = 0; h < 2; ++h) {
                mbar_init(smem_addr(&sh.s_full[w][h]), 1);
                mbar_init(smem_addr(&sh.p_ready[w][h]), 4);
                mbar_init(smem_addr(&sh.o_done[w][h]), 1);
            }
            mbar_init(smem_addr(&sh.ml_ready[w]), 4);
            mbar_init(smem_addr(&sh.o_free[w]), 4);
        }
        sh.stop = 0;
        mbar_init_fence();
    }
    pdl_wait();
    pdl_allow_dependents();
    if (threadIdx.x == 0)
        plan.splits[blockIdx.x].cta1 = -1;  // none so far

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
    if ((smem_addr(smem) & 1023u) != 0) {  // does not happen; the swizzle needs it
        if (threadIdx.x == 0)
            record_device_error(p.err, kDeviceErrTimeout);
        return;
    }
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

    if (warp < kMmaWarp) {
        tile_softmax_role<DP, FULL, SHARED>(p, plan, sh, warp >> 2, threadIdx.x & 127);
    } else if (warp >= kResultWarp) {
        tile_result_role<DP, SHARED>(p, plan, stage, sh, threadIdx.x & 127);
    } else {
        if (warp == kMmaWarp || warp == kMmaWarp1) {
            const int w = warp == kMmaWarp1;
            if (elect_one()) {
                tile_mma_role<DP>(p, q + w * R::kQ, slots, sh, w);
                // every product and every arrival asked for has happened
                tc_commit(smem_addr(&sh.drain[w]));
                mbar_wait(smem_addr(&sh.drain[w]), 0);
            }
        } else if (warp == kLoadWarp) {
            tile_load_role<DP>(p, plan, &kmap, &vmap, slots, sh, lane);
        } else {
            tile_query_role<DP, SHARED>(p, plan, &qmap, q, sh, c, begin, end, share, lane);
        }
    }
    __syncwarp();
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

// The queries as [token][head][value]; a copy takes 64 values of g heads of
// 128 / g tokens.
cudaError_t query_map(CUtensorMap* map, const AttentionParams& p, int g)
{
    EncodeTiled encode = encode_tiled();
    if (encode == nullptr)
        return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {(cuuint64_t)p.head_dim, (cuuint64_t)p.hq, (cuuint64_t)p.tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)p.head_dim * 2, (cuuint64_t)p.q_stride * 2};
    const cuuint32_t sizes[3] = {64, (cuuint32_t)g, (cuuint32_t)(kSubRows / g)};
    const cuuint32_t steps[3] = {1, 1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(p.q),
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
                           const CUtensorMap& vmap, const CUtensorMap& qmap, int sm_count,
                           cudaStream_t st)
{
    constexpr auto kernel = attention_tiles_kernel<DP, FULL, SHARED>;
    constexpr int kSmem = tile_smem<DP>();
    static_assert(kSmem <= (int)kMaxSmemPerCta, "shared memory of a CTA");
    // one CTA an SM: each takes all of its SM's tensor memory
    const int grid = std::min(sm_count, kMaxTileCtas);
    cudaError_t err = cudaSuccess;
    for (int attempt = 0; attempt < 2; ++attempt) {
        int ctas = 0;
        err = resident_ctas_once<kernel>(kTileThreads, kSmem, &ctas, attempt > 0);
        if (err != cudaSuccess)
            return err;
        if (ctas < 1)
            return cudaErrorNotSupported;
        err = launch(kernel, dim3(grid), dim3(kTileThreads), kSmem, st, p, plan, kmap, vmap, qmap);
        if (err != cudaErrorInvalidValue)
            break;
        cudaGetLastError();  // not kept for the caller's next call
    }
    if (err != cudaSuccess)
        return err;
    return launch(attention_join_kernel<DP, SHARED>, dim3(grid, 2, DP / 32), dim3(kSubRows), 0, st,
                  p, plan);
}

template <int DP>
cudaError_t launch_tiles_d(const AttentionParams& p, const TilePlan& plan, const CUtensorMap& kmap,
                           const CUtensorMap& vmap, const CUtensorMap& qmap, bool full,
                           int sm_count, cudaStream_t st)
{
    if (p.group_start)
        return full ? launch_tiles_f<DP, true, true>(p, plan, kmap, vmap, qmap, sm_count, st)
                    : launch_tiles_f<DP, false, true>(p, plan, kmap, vmap, qmap, sm_count, st);
    return full ? launch_tiles_f<DP, true, false>(p, plan, kmap, vmap, qmap, sm_count, st)
                : launch_tiles_f<DP, false, false>(p, plan, kmap, vmap, qmap, sm_count, st);
}

}  // namespace

// Waits are bounded by a second, and some last as long as a CTA is at one or two
// tiles: 2^23 positions are at most 65,536 units of 2 to 4 us each.  Calls whose
// tables hold more go to the row kernel, which waits for nobody.
constexpr int64_t kMaxTilePositions = 1 << 23;

bool tiles_can_run(const AttentionParams& p, arops_dtype dtype)
{
    const int64_t pages = p.group_start ? p.max_prefix_pages : p.max_pages;
    return dtype == AROPS_BF16 && p.head_dim <= 128 && p.head_dim % 8 == 0 &&
           pages * p.map.page_size <= kMaxTilePositions && p.map.page_size % 8 == 0 &&
           aligned16(p.k_pages) && aligned16(p.v_pages) &&
           aligned16(p.q) && p.q_stride % 8 == 0 && aligned16(p.out) &&
           // the tensor map's largest stride
           (int64_t)p.hk * p.map.page_size * p.head_dim * 2 < (1ll << 40);
}

size_t tile_part_bytes(int dp)
{
    return (size_t)kMaxTileCtas * (4 * tile_part_floats(dp) * sizeof(float) + 32);
}

cudaError_t launch_attention_tiles(const AttentionParams& p, float* parts, float* prefix_o,
                                   float* prefix_ml, int sm_count,
                                   cudaStream_t stream)
{
    TilePlan plan = {};
    // the plain form needs a positive factor: the largest product is then the
    // largest score
    const bool full = p.softcap > 0.0f || p.slopes != nullptr || !(p.scale > 0.0f);
    plan.score = make_score_map(p);
    if (full)
        plan.score.scale = p.scale;
    plan.cap = make_cap_form(plan.score);
    plan.parts = parts;
    plan.splits = reinterpret_cast<TileSplit*>(
        parts + (size_t)kMaxTileCtas * 4 * tile_part_floats(p.head_dim <= 64 ? 64 : 128));
    plan.prefix_o = prefix_o;
    plan.prefix_ml = prefix_ml;
    plan.g = make_row_divide(p.hq / p.hk);
    plan.box = box_slots(p.map.page_size);
    // whole tokens in the 128 rows of a sub-tile, and strides that a map can hold
    const int g = p.hq / p.hk;
    plan.q_map = kSubRows % g == 0 && p.q_stride < (1ll << 38);
    CUtensorMap kmap, vmap, qmap = {};
    cudaError_t err = pool_map(&kmap, p.k_pages, p, plan.box);
    if (err == cudaSuccess)
        err = pool_map(&vmap, p.v_pages, p, plan.box);
    if (err == cudaSuccess && plan.q_map)
        err = query_map(&qmap, p, g);
    if (err != cudaSuccess)
        return err;
    return p.head_dim <= 64
               ? launch_tiles_d<64>(p, plan, kmap, vmap, qmap, full, sm_count, stream)
               : launch_tiles_d<128>(p, plan, kmap, vmap, qmap, full, sm_count, stream);
}

}  // namespace arops
