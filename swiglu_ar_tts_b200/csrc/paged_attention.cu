// Attention over a paged KV cache (sm_100a): the row kernel, for few query rows
// a key (decode steps, candidates of a prompt, a handful of tokens), every
// type, head width, page size and alignment.
//
//   out_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = 2^(s_ij - m_i),  m_i = max_j s_ij
// (s in base 2) over the keys j that query i sees, in one pass over the keys
// with a running maximum: when m grows, the sums so far are scaled by
// 2^(m_old - m_new).  Every key and value is read once for all rows of a tile,
// 4 D operations a (row, key): up to ~200 rows a key, memory bounds it.
//
// Rows: a tile is 16 rows, (token, head of one key/value head's group) pairs in
// token order, the M of mma.m16n8.  Decode fills 2 of them (16 query heads on 8
// key heads), five candidates of a shared prompt 10; the products cost a tenth
// of the bytes' time either way.
//
// Keys: a unit is 64 keys, 16 a warp.  Each warp copies its 16 keys and values
// into its own ring of shared-memory stages (cp.async, 16-byte chunks swizzled
// by chunk ^ (key & 7) so that ldmatrix meets no bank twice), multiplies, keeps
// its own m, l and O in registers, and never waits for another warp until the
// tile's keys are done.  tcgen05 is not used here: its smallest tile is 128
// rows (the tile kernel has it); 16-row mma.sync leaves the memory bound alone.
//
// Split: all units of all (tile, key head) pairs form one line, cut into equal
// shares, one a CTA, from the lengths on the device (no plan on the host; the
// cut depends on the lengths alone).  A CTA whose share covers only part of a
// pair's keys writes (m, l, O) to the workspace; the last of the pair's CTAs to
// arrive joins the parts in their order along the keys, so arrival changes no
// bit.  No CTA waits for another.
#include "attention_common.cuh"

namespace arops {
namespace {

constexpr int kRowWarps = 4;
constexpr int kRowThreads = 32 * kRowWarps;
constexpr int kUnit = 64;   // keys of a unit
constexpr int kBlock = 16;  // of which a warp takes
constexpr int kRows = 16;   // rows of a tile

// A pair's place on the line is kRowPairCost positions for its fixed cost (its
// queries, the joins, its results: that of about as many units), then its units.
constexpr int kRowPairCost = 2;

// Least share of a CTA: with fewer units a share, a pair has more parts to join
// than the units take (5 candidates on 1,100 positions: 24.5, 20.1, 18.3, 21.1,
// 21.7 us with 1, 2, 3, 4, 6).
constexpr int kMinUnits = 3;

__host__ __device__ constexpr int padded_head_dim(int d)
{
    return d <= 64 ? 64 : d <= 128 ? 128 : 256;
}

// Floats of one partial result: O, then m and l.
__host__ __device__ constexpr int part_floats(int dp)
{
    return kRows * dp + 2 * kRows;
}

// Largest grid: the workspace holds two partial results a CTA.
constexpr int kMaxRowCtas = 640;

struct RowPlan {
    ScoreMap score;
    int32_t* counters;
    float* parts;
    RowDivide g;           // query heads a key head
    int32_t seqs_a_tile;   // shared prefixes: sequences of a tile (g <= 16)
    int32_t tiles_a_seq;   // shared prefixes: tiles of a sequence's heads (g > 16)
    int32_t min_units;     // of a CTA's share
    bool vec_q, vec_out;   // 16-byte q rows, 8/16-byte output groups
    // Shared prefixes whose keys the tile kernel has already taken: O and (m, l)
    // of every (sequence, head).  Null: this kernel takes them.
    const float* prefix_o;
    const float* prefix_ml;
};

// ---------------------------------------------------------------------------
// Tensor-core products of a 16-row tile with a warp's 16 keys.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void mma_bf16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_tf32(float* c, const uint32_t* a, uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// x as the sum of two tf32 numbers (11 significant bits each), by integer
// operations: conversions run at an eighth of their rate.  The first is rounded
// (half away from zero, as a conversion would); what is left, 12 bits and exact,
// is cut to 11: 2^-23 of x is left out.  A NaN whose first part the rounding
// carries into the sign is one in the second.
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo)
{
    hi = (__float_as_uint(x) + 0x1000u) & 0xFFFFE000u;
    lo = __float_as_uint(x - __uint_as_float(hi)) & 0xFFFFE000u;
}

__device__ __forceinline__ void ldmatrix4(uint32_t* r, uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

__device__ __forceinline__ void ldmatrix4_trans(uint32_t* r, uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes)
{
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ void cp_async_commit()
{
    asm volatile("cp.async.commit_group;" ::: "memory");
}

template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t shared_address(const void* p)
{
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

template <typename T, int DP>
struct RowTraits {
    static constexpr int kE = (int)sizeof(T);
    static constexpr int kRowBytes = DP * kE;             // of a key in shared memory
    static constexpr int kChunks = kRowBytes / 16;
    static constexpr int kHalf = kBlock * kRowBytes;      // a warp's keys (or values)
    static constexpr int kStage = 2 * kHalf;
    // Stages of a warp's ring and CTAs an SM.  A warp asks for its next stage when
    // it has used one, so kStages - 1 of them are on their way while it waits and
    // one fewer while it multiplies: with two stages that is none, and other
    // warps' copies fill the time (bf16 heads of 128: at most 96 KB an SM, above
    // the ~64 KB that 44 GB/s an SM need at ~1 us of latency).  Three CTAs of two
    // stages, the third to fill the other two's changes of sequence, measured 344
    // us against 354 for two of three (256 sequences of 60-4,100 keys).
    static constexpr int kStages = kStage == 8192 ? 2 : 3;
    static constexpr int kCtas = kStage <= 4096 ? 4 : kStage <= 8192 ? 3 : 1;
    static constexpr int kSteps = kE == 2 ? DP / 16 : DP / 8;  // of the first product
    static constexpr int kQWords = kE == 2 ? 4 : 8;            // a lane's fragment words a step
    static constexpr int kQBytes = kSteps * 32 * kQWords * 4;
    static constexpr int kRing = kRowWarps * kStages * kStage;
    static constexpr int kSmem = kRing + kQBytes;
};

// Where a CTA's walk along the line of units stands.
struct Cursor {
    int32_t seq;   // first sequence of the tile
    int32_t sub;   // tile within the sequence
    int32_t kvh;   // key head
    int32_t unit;  // units of the pair before the share (negative: in its fixed cost)
};

// Keys of one (tile, key head) pair.  Lane m < 16 holds member m's length in
// shared-prefix tiles (units: prefix first, then each member's own).
struct TileKeys {
    int32_t tok0;    // first token of the entity (a sequence, or a tile's members)
    int32_t lo, hi;  // keys [lo, hi) of the sequence (the prefix), lo a multiple of kUnit
    int32_t seen;    // the first of them that a row sees
    int32_t len;     // sequence length, or prefix length
    int32_t ntok;    // query tokens, or members
    int32_t bidir;
    int32_t group;
    int32_t own_len, own_lo, own_end;  // lane m: member m's length, first key, running unit count
    int32_t prefix_units;
    int32_t units;   // >= 1
};

__device__ __forceinline__ int32_t ragged_tiles(const Ragged& r, const RowDivide& g)
{
    return (int32_t)(((uint32_t)r.ntok * g.n + kRows - 1) / kRows);
}

// -- shared prefixes ---------------------------------------------------------
struct Member {
    int32_t group;        // -1: of no group
    int32_t index, count; // within the group
    int32_t prefix;
};

// The group of sequence s by bisection (one thread).
__device__ __forceinline__ Member find_member(const AttentionParams& p, int32_t s, bool& bad)
{
    int32_t lo = 0, hi = p.n_groups;
    while (hi - lo > 1) {
        const int32_t mid = (lo + hi) / 2;
        if (__ldg(p.group_start + mid) <= s)
            lo = mid;
        else
            hi = mid;
    }
    Member m;
    const int64_t a = __ldg(p.group_start + lo), b = __ldg(p.group_start + lo + 1);
    const bool ok = a >= 0 && a <= s && s < b && b <= p.n_seqs;
    m.group = ok ? lo : -1;
    m.index = ok ? (int32_t)(s - a) : 0;
    m.count = ok ? (int32_t)(b - a) : 0;
    m.prefix = ok ? clamp_length(__ldg(p.prefix_lens + lo), p.max_prefix_pages * p.map.page_size,
                                 bad)
                  : 0;
    return m;
}

__device__ __forceinline__ int32_t own_length(const AttentionParams& p, int32_t s, bool& bad)
{
    return clamp_length(__ldg(p.kv_lens + s), p.max_pages * p.map.page_size, bad);
}

// First key of the prefix, and of the member's own keys, that the window leaves
// (..._first: of its unit).
__device__ __forceinline__ int32_t prefix_seen(const AttentionParams& p, int32_t prefix,
                                               int32_t own)
{
    int32_t lo, hi;
    visible_keys(prefix + own - 1, prefix + own, 0, p.window, lo, hi);
    return min(lo, prefix);
}

__device__ __forceinline__ int32_t prefix_first(const AttentionParams& p, int32_t prefix,
                                                int32_t own)
{
    return prefix_seen(p, prefix, own) & ~(kUnit - 1);
}

__device__ __forceinline__ int32_t own_seen(const AttentionParams& p, int32_t prefix, int32_t own)
{
    int32_t lo, hi;
    visible_keys(prefix + own - 1, prefix + own, 0, p.window, lo, hi);
    return max(lo - prefix, 0);
}

__device__ __forceinline__ int32_t own_first(const AttentionParams& p, int32_t prefix, int32_t own)
{
    return own_seen(p, prefix, own) & ~(kUnit - 1);
}

// What sequence s adds to the line (per key head): its own units, once a tile of
// its heads, and, if it is its tile's first member, the prefix's and the fixed
// cost.
__device__ __forceinline__ int64_t member_units(const AttentionParams& p, const RowPlan& plan,
                                                int32_t s, const Member& m, bool& bad)
{
    if (m.group < 0)
        return 0;
    const int32_t own = own_length(p, s, bad);
    int64_t n = units_between<kUnit>(own_first(p, m.prefix, own), own);
    if (m.index % plan.seqs_a_tile == 0) {
        int32_t lo = prefix_first(p, m.prefix, own);
        int64_t rest = 0;
        const int32_t members = min(plan.seqs_a_tile, m.count - m.index);
        if (p.window > 0)
            for (int32_t i = 1; i < members; ++i)
                lo = min(lo, prefix_first(p, m.prefix, own_length(p, s + i, bad)));
        rest = plan.prefix_o ? 0 : units_between<kUnit>(lo, m.prefix);
        // a tile without any key still has a unit: it writes zeros
        if (rest == 0 && n == 0) {
            bool any = false;
            for (int32_t i = 1; i < members && !any; ++i) {
                const int32_t l = own_length(p, s + i, bad);
                any = units_between<kUnit>(own_first(p, m.prefix, l), l) > 0;
            }
            rest = any ? 0 : 1;
        }
        n += rest + kRowPairCost;
    }
    return n * plan.tiles_a_seq;
}

// What sequence s adds to the line, for one key head.
template <bool SHARED>
__device__ __forceinline__ int64_t sequence_units(const AttentionParams& p, const RowPlan& plan,
                                                  int32_t s, bool& bad)
{
    if constexpr (SHARED) {
        const Member m = find_member(p, s, bad);
        return member_units(p, plan, s, m, bad);
    } else {
        const Ragged r = load_ragged(p, s, bad);
        const int32_t tiles = ragged_tiles(r, plan.g);
        int64_t n = 0;
        for (int32_t i = 0; i < tiles; ++i) {
            int32_t lo, hi, seen;
            ragged_range<kUnit>(p, r, plan.g, i * kRows, kRows, lo, hi, seen);
            n += max(1, units_between<kUnit>(lo, hi)) + kRowPairCost;
        }
        return n;
    }
}

// The keys of the tile at the cursor; every warp of the CTA computes them, each
// for itself.  False: the sequence at the cursor starts no tile.
template <bool SHARED>
__device__ __forceinline__ bool load_tile(const AttentionParams& p, const RowPlan& plan,
                                          const Cursor& c, TileKeys& k, int lane)
{
    bool bad = false;
    if constexpr (SHARED) {
        const Member m = find_member(p, c.seq, bad);
        if (m.group < 0 || m.index % plan.seqs_a_tile != 0)
            return false;
        const int32_t members = min(plan.seqs_a_tile, m.count - m.index);
        k.tok0 = c.seq;
        k.ntok = members;
        k.len = m.prefix;
        k.group = m.group;
        k.bidir = 0;
        k.own_len = lane < members ? own_length(p, c.seq + lane, bad) : 0;
        k.own_lo = own_first(p, m.prefix, k.own_len);
        int32_t lo = lane < members ? prefix_seen(p, m.prefix, k.own_len) : INT_MAX;
        int32_t n = lane < members ? units_between<kUnit>(k.own_lo, k.own_len) : 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            lo = min(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t x = __shfl_up_sync(0xFFFFFFFFu, n, o);
            if (lane >= o)
                n += x;
        }
        k.own_end = n;
        k.seen = lo;
        lo &= ~(kUnit - 1);
        k.lo = lo;
        k.hi = m.prefix;
        k.prefix_units = plan.prefix_o ? 0 : units_between<kUnit>(lo, m.prefix);
        k.units = max(1, k.prefix_units + __shfl_sync(0xFFFFFFFFu, n, 31));
        return true;
    } else {
        const Ragged r = load_ragged(p, c.seq, bad);
        if (c.sub >= ragged_tiles(r, plan.g))
            return false;
        k.tok0 = r.t0;
        k.ntok = r.ntok;
        k.len = r.len;
        k.bidir = r.bidir;
        k.group = -1;
        k.own_len = k.own_lo = k.own_end = 0;
        ragged_range<kUnit>(p, r, plan.g, c.sub * kRows, kRows, k.lo, k.hi, k.seen);
        k.prefix_units = max(1, units_between<kUnit>(k.lo, k.hi));
        k.units = k.prefix_units;
        return true;
    }
}

// A warp's 16 keys of one unit.
struct KeyBlock {
    const int32_t* table;
    int32_t key0, end;  // keys [key0, min(key0 + 16, end)) of the table's positions,
    int32_t seen;       // those before `seen` left out
    int32_t shift;      // position in the sequence = key + shift
    int32_t member;     // the only member whose rows see them; -1: all rows
};

template <bool SHARED>
__device__ __forceinline__ KeyBlock key_block(const AttentionParams& p, const Cursor& c,
                                              const TileKeys& k, int32_t unit, int warp)
{
    KeyBlock b;
    if constexpr (SHARED) {
        const bool own = unit >= k.prefix_units;
        const int32_t u = unit - k.prefix_units;
        const int member =
            own ? __popc(__ballot_sync(0xFFFFFFFFu, k.own_end <= u) & 0xFFFFu) : 0;
        const int32_t before = __shfl_sync(0xFFFFFFFFu, k.own_end, max(member - 1, 0));
        const int32_t lo = __shfl_sync(0xFFFFFFFFu, k.own_lo, member & 31);
        const int32_t len = __shfl_sync(0xFFFFFFFFu, k.own_len, member & 31);
        if (own) {
            b.table = p.block_table + (int64_t)(c.seq + member) * p.max_pages;
            b.key0 = lo + (u - (member > 0 ? before : 0)) * kUnit + warp * kBlock;
            b.end = member < k.ntok ? len : 0;
            b.seen = own_seen(p, k.len, len);
            b.shift = k.len;
            b.member = member;
            return b;
        }
        b.table = p.prefix_table + (int64_t)k.group * p.max_prefix_pages;
    } else {
        b.table = p.block_table + (int64_t)c.seq * p.max_pages;
    }
    b.key0 = k.lo + unit * kUnit + warp * kBlock;
    b.end = k.hi;
    b.seen = k.seen;
    b.shift = 0;
    b.member = -1;
    return b;
}

// Element offset of the lane's key (lane & 15) in the pools, -1 for none.
__device__ __forceinline__ int64_t key_offset(const AttentionParams& p, const KeyBlock& b, int kvh,
                                              int lane, bool& bad)
{
    const int32_t key = b.key0 + (lane & (kBlock - 1));
    if (key < b.seen || key >= b.end)
        return -1;
    int32_t pi, slot;
    split_position(p.map, key, pi, slot);
    const int64_t page = __ldg(b.table + pi);
    if (page < 0 || page >= p.map.num_pages) {
        bad = true;
        return -1;
    }
    return ((page * p.hk + kvh) * p.map.page_size + slot) * p.head_dim;
}

// Byte of element e of key row `row` in a swizzled half stage.
template <typename T, int DP>
__device__ __forceinline__ uint32_t swizzled(int row, int e)
{
    const int byte = e * (int)sizeof(T);
    return row * RowTraits<T, DP>::kRowBytes + (((byte >> 4) ^ (row & 7)) << 4) + (byte & 15);
}

// Copies a warp's 16 keys and values into a stage; what no key fills is zero.
template <typename T, int DP, bool VEC>
__device__ __forceinline__ void load_block(const AttentionParams& p, unsigned char* stage,
                                           int64_t off, int lane)
{
    using R = RowTraits<T, DP>;
    const T* kp = static_cast<const T*>(p.k_pages);
    const T* vp = static_cast<const T*>(p.v_pages);
    if constexpr (VEC) {
        const uint32_t dst = shared_address(stage);
        const int used = p.head_dim * R::kE / 16;
#pragma unroll
        for (int n = 0; n < kBlock * R::kChunks / 32; ++n) {
            const int idx = n * 32 + lane;
            const int row = idx / R::kChunks, chunk = idx % R::kChunks;
            const int64_t o = __shfl_sync(0xFFFFFFFFu, off, row);
            const bool ok = o >= 0 && chunk < used;
            const int64_t e = ok ? o + chunk * (16 / R::kE) : 0;
            const uint32_t d = dst + row * R::kRowBytes + ((chunk ^ (row & 7)) << 4);
            cp_async16(d, kp + e, ok ? 16u : 0u);
            cp_async16(d + R::kHalf, vp + e, ok ? 16u : 0u);
        }
    } else {
        for (int row = 0; row < kBlock; ++row) {
            const int64_t o = __shfl_sync(0xFFFFFFFFu, off, row);
            for (int e = lane; e < DP; e += 32) {
                const bool ok = o >= 0 && e < p.head_dim;
                T* k = reinterpret_cast<T*>(stage + swizzled<T, DP>(row, e));
                T* v = reinterpret_cast<T*>(stage + R::kHalf + swizzled<T, DP>(row, e));
                store_elem(k, ok ? load_elem(kp + o + e) : 0.0f);
                store_elem(v, ok ? load_elem(vp + o + e) : 0.0f);
            }
        }
    }
}

// The tile's query rows as mma fragments in shared memory, a lane's words of a
// step side by side; rows and columns that do not exist are zero.
template <typename T, int DP>
__device__ __forceinline__ void store_q(uint32_t* frag, int row, int e, float x, float y)
{
    if constexpr (sizeof(T) == 2) {  // elements e, e + 1 (e even)
        const int step = e / 16, w = (row >> 3) + 2 * ((e >> 3) & 1);
        frag[(step * 32 + (row & 7) * 4 + ((e >> 1) & 3)) * 4 + w] = pack_bf16x2(x, y);
    } else {
        const int step = e / 8, w = (row >> 3) + 2 * ((e >> 2) & 1);
        uint32_t* f = frag + (step * 32 + (row & 7) * 4) * 8 + w;
        uint32_t hi, lo;
        split_tf32(x, hi, lo);
        f[(e & 3) * 8] = hi;
        f[(e & 3) * 8 + 4] = lo;
        split_tf32(y, hi, lo);
        f[((e + 1) & 3) * 8] = hi;
        f[((e + 1) & 3) * 8 + 4] = lo;
    }
}

struct RowOf {
    int32_t token;  // -1: no such row
    int32_t head;
    int32_t index;  // token or member within the entity
};

// (token, head) of a row of the tile: rows run over an entity's tokens, g heads each.
__device__ __forceinline__ RowOf row_of(const TileKeys& k, const RowPlan& plan, const Cursor& c,
                                        int row)
{
    RowOf r;
    const uint32_t at = (uint32_t)c.sub * kRows + row;
    r.index = (int32_t)plan.g(at);
    r.head = (int32_t)(c.kvh * plan.g.n + at - r.index * plan.g.n);
    r.token = r.index < k.ntok ? k.tok0 + r.index : -1;
    return r;
}

template <typename T>
__device__ __forceinline__ void store_group(T* dst, const float* f, int n, bool vec);

template <>
__device__ __forceinline__ void store_group(float* dst, const float* f, int n, bool vec)
{
    if (vec) {
        *reinterpret_cast<float4*>(dst) = make_float4(f[0], f[1], f[2], f[3]);
    } else {
        for (int i = 0; i < n; ++i)
            dst[i] = f[i];
    }
}

template <>
__device__ __forceinline__ void store_group(__nv_bfloat16* dst, const float* f, int n, bool vec)
{
    if (vec) {
        *reinterpret_cast<uint2*>(dst) =
            make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
    } else {
        for (int i = 0; i < n; ++i)
            store_elem(dst + i, f[i]);
    }
}

// Four values of a row: the prefix's part joined, divided by l, stored.  A row
// that sees no key has l == 0 and gets zeros.
template <typename T, int DP, bool SHARED>
__device__ __forceinline__ void store_result(const AttentionParams& p, const RowPlan& plan,
                                             const RowOf& r, int e, float* sum, float m, float l)
{
    const int64_t row = (int64_t)r.token * p.hq + r.head;
    if (SHARED && plan.prefix_o) {
        const float2 ml = __ldcg(reinterpret_cast<const float2*>(plan.prefix_ml) + row);
        const float4 o = __ldcg(reinterpret_cast<const float4*>(plan.prefix_o + row * DP + e));
        const float mm = fmaxf(m, ml.x);
        const float f = part_factor(m, mm);
        const float fp = part_factor(ml.x, mm);
        l = l * f + ml.y * fp;
        sum[0] = sum[0] * f + o.x * fp;
        sum[1] = sum[1] * f + o.y * fp;
        sum[2] = sum[2] * f + o.z * fp;
        sum[3] = sum[3] * f + o.w * fp;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int x = 0; x < 4; ++x)
        sum[x] = l == 0.0f ? 0.0f : sum[x] * inv;
    store_group<T>(static_cast<T*>(p.out) + row * p.head_dim + e, sum, min(4, p.head_dim - e),
                   plan.vec_out);
}

// Joins the parts of CTAs cta0 .. cta1 in their order: 2^(m_x - m) O_x summed
// over x, likewise l.  Latency is all that counts here (parts come out of L2,
// instructions too: this runs once a CTA at most), so it is short code with
// eight parts on their way.
template <typename T, int DP, bool SHARED>
__device__ void join_parts(const AttentionParams& p, const RowPlan& plan, const RowOf* row_at,
                           int32_t cta0, int32_t cta1, float (*row_m)[kRows],
                           float (*row_l)[kRows], float* weights)
{
    constexpr int kMost = 64;  // parts whose weights fit in shared memory
    constexpr int kBatch = 8;  // parts a thread asks for at once
    auto part_of = [&](int32_t x) {
        return plan.parts + ((int64_t)x * 2 + (x == cta0 ? 1 : 0)) * part_floats(DP);
    };
    const int row = threadIdx.x % kRows, lead = threadIdx.x / kRows;
    constexpr int kLeads = kRowThreads / kRows;
    // every row's m and l: kLeads threads a row, then theirs joined
    const bool few = cta1 - cta0 < kMost;
    float m = -INFINITY, l = 0.0f;
    for (int32_t x = cta0 + lead; x <= cta1; x += kLeads) {
        const bool in = row_at[row].token >= 0;
        const float* src = part_of(x) + kRows * DP + row;
        const float mx = in ? __ldcg(src) : -INFINITY;
        const float lx = in ? __ldcg(src + kRows) : 0.0f;
        if (few)
            weights[(x - cta0) * kRows + row] = mx;
        const float mn = fmaxf(m, mx);
        l = l * part_factor(m, mn) + lx * part_factor(mx, mn);
        m = mn;
    }
    float* lead_m = weights + kMost * kRows;
    float* lead_l = lead_m + kRowThreads;
    lead_m[threadIdx.x] = m;
    lead_l[threadIdx.x] = l;
    __syncthreads();
    if (threadIdx.x < kRows) {
        m = -INFINITY;
        l = 0.0f;
#pragma unroll
        for (int i = 0; i < kLeads; ++i)
            m = fmaxf(m, lead_m[i * kRows + row]);
#pragma unroll
        for (int i = 0; i < kLeads; ++i)
            l += lead_l[i * kRows + row] * part_factor(lead_m[i * kRows + row], m);
        row_m[0][row] = m;
        row_l[0][row] = l;
    }
    __syncthreads();
    if (few)
        for (int i = threadIdx.x; i < (cta1 - cta0 + 1) * kRows; i += kRowThreads)
            weights[i] = part_factor(weights[i], row_m[0][i % kRows]);
    __syncthreads();
#pragma unroll 1
    for (int idx = threadIdx.x; idx < kRows * DP / 4; idx += kRowThreads) {
        const int at = idx / (DP / 4), e = idx % (DP / 4) * 4;
        const RowOf r = row_at[at];
        if (r.token < 0 || e >= p.head_dim)
            continue;
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
        for (int32_t x = cta0; x <= cta1; x += kBatch) {
            float4 v[kBatch];
            float f[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                const int32_t y = min(x + j, cta1);
                const float* src = part_of(y);
                v[j] = __ldcg(reinterpret_cast<const float4*>(src) + idx);
                f[j] = few ? weights[(y - cta0) * kRows + at]
                           : __ldcg(src + kRows * DP + at);
            }
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
                if (!few)
                    f[j] = part_factor(f[j], row_m[0][at]);
                if (x + j > cta1)
                    f[j] = 0.0f;
                sum[0] = fmaf(v[j].x, f[j], sum[0]);
                sum[1] = fmaf(v[j].y, f[j], sum[1]);
                sum[2] = fmaf(v[j].z, f[j], sum[2]);
                sum[3] = fmaf(v[j].w, f[j], sum[3]);
            }
        }
        store_result<T, DP, SHARED>(p, plan, r, e, sum, row_m[0][at], row_l[0][at]);
    }
}

template <typename T, int DP, bool VEC, bool FULL, bool SHARED>
__global__ void __launch_bounds__(kRowThreads, RowTraits<T, DP>::kCtas)
attention_rows_kernel(const __grid_constant__ AttentionParams p,
                      const __grid_constant__ RowPlan plan)
{
    using R = RowTraits<T, DP>;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int64_t warp_sums[kRowWarps];
    __shared__ Cursor found;
    __shared__ float row_m[kRowWarps][kRows], row_l[kRowWarps][kRows];
    __shared__ RowOf row_at[kRows];
    __shared__ int last_flag;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int quad = lane & 3;
    unsigned char* ring = smem + warp * R::kStages * R::kStage;
    uint32_t* qfrag = reinterpret_cast<uint32_t*>(smem + R::kRing);

    pdl_wait();
    pdl_allow_dependents();

    // -- this CTA's share of the line of units --------------------------------
    bool bad = false;
    const int32_t per = (p.n_seqs + kRowThreads - 1) / kRowThreads;
    const int32_t s_begin = min((int64_t)threadIdx.x * per, (int64_t)p.n_seqs);
    const int32_t s_end = min(s_begin + per, p.n_seqs);
    // (kept in shared memory as far as it reaches, for the search below)
    int64_t* counted = reinterpret_cast<int64_t*>(smem);
    const bool keeps = p.n_seqs <= (int)(R::kRing / sizeof(int64_t));
    int64_t mine = 0;
    for (int32_t s = s_begin; s < s_end; ++s) {
        const int64_t n = sequence_units<SHARED>(p, plan, s, bad);
        if (keeps)
            counted[s] = n;
        mine += n;
    }
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if (lane >= o)
            upto += x;
    }
    if (lane == 31)
        warp_sums[warp] = upto;
    bool broken = false;
    if constexpr (SHARED) {
        // starts that are not non-decreasing would cut tiles in two ways
        for (int32_t i = threadIdx.x; i < p.n_groups; i += kRowThreads) {
            const int32_t a = __ldg(p.group_start + i), b = __ldg(p.group_start + i + 1);
            broken = broken || a < 0 || a > b || b > p.n_seqs;
        }
    }
    if (__syncthreads_or(broken)) {
        if (threadIdx.x == 0 && blockIdx.x == 0)
            record_device_error(p.err, kDeviceErrBadIndexBit);
        return;
    }
    int64_t total = 0;
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w) {
        if (w < warp)
            upto += warp_sums[w];
        total += warp_sums[w];
    }
    if (bad && blockIdx.x == 0)
        record_device_error(p.err, kDeviceErrBadIndexBit);
    const int64_t line = total * p.hk;
    int64_t share = (line + gridDim.x - 1) / gridDim.x;
    if (share < plan.min_units)
        share = plan.min_units;
    const int64_t begin = (int64_t)blockIdx.x * share;
    if (begin >= line)
        return;
    const int64_t end = min(begin + share, line);
    {
        int64_t before = upto - mine;
        if (begin >= before * p.hk && begin < upto * p.hk) {
            bool ignore = false;
            auto count = [&](int32_t x) {
                return keeps ? counted[x] : sequence_units<SHARED>(p, plan, x, ignore);
            };
            int32_t s = s_begin;
            int64_t n = 0;
            for (;; ++s) {
                n = count(s);
                if (begin < (before + n) * p.hk)
                    break;
                before += n;
            }
            Cursor c;
            c.seq = s;
            c.sub = 0;
            int64_t tile_line = n;
            if constexpr (SHARED) {
                // back to the tile's first member, then into the tile of its heads
                const Member m = find_member(p, s, ignore);
                const int32_t in_tile = m.index % plan.seqs_a_tile;
                c.seq = s - in_tile;
                const int32_t end = c.seq + min(plan.seqs_a_tile, m.count - m.index + in_tile);
                tile_line = 0;
                for (int32_t x = c.seq; x < end; ++x) {
                    const int64_t u = x == s ? n : count(x);
                    if (x < s)
                        before -= u;
                    tile_line += u;
                }
                tile_line /= plan.tiles_a_seq;
                c.sub = (int32_t)((begin / p.hk - before) / tile_line);
                before += c.sub * tile_line;
            } else {
                const Ragged r = load_ragged(p, s, ignore);
                if (ragged_tiles(r, plan.g) > 1)
                    for (;; ++c.sub) {
                        int32_t lo, hi, seen;
                        ragged_range<kUnit>(p, r, plan.g, c.sub * kRows, kRows, lo, hi, seen);
                        tile_line = max(1, units_between<kUnit>(lo, hi)) + kRowPairCost;
                        if (begin < (before + tile_line) * p.hk)
                            break;
                        before += tile_line;
                    }
            }
            const int64_t rest = begin - before * p.hk;
            c.kvh = (int32_t)(rest / tile_line);
            c.unit = (int32_t)(rest % tile_line) - kRowPairCost;
            found = c;
        }
    }
    __syncthreads();
    Cursor c = found;
    int64_t at = begin - c.unit;  // place of the pair's unit 0 on the line

    while (at < end && c.seq < p.n_seqs) {
        TileKeys k;
        if (!load_tile<SHARED>(p, plan, c, k, lane)) {
            ++c.seq;
            c.sub = 0;
            continue;
        }
        const int32_t u0 = (int32_t)max(begin - at, (int64_t)0);
        const int32_t u1 = (int32_t)min(end - at, (int64_t)k.units);
        auto next_pair = [&]() {
            at += k.units + kRowPairCost;
            if (++c.kvh == p.hk) {
                c.kvh = 0;
                ++c.sub;
                if (SHARED && c.sub >= plan.tiles_a_seq) {
                    c.sub = 0;
                    c.seq += k.ntok;
                }
            }
        };
        if (u0 >= u1) {
            next_pair();
            continue;
        }

        // -- the tile's queries, and this lane's two rows ----------------------
        __syncthreads();  // the last pair's use of shared memory is over
        // keys and values first: their way is the longest.  Stages are filled
        // ahead; a page is looked up one block before its copy.
        bool bad_page = false;
        int32_t issue = u0;
        KeyBlock nb = key_block<SHARED>(p, c, k, u0, warp);
        int64_t noff = key_offset(p, nb, c.kvh, lane, bad_page);
        auto issue_next = [&]() {
            if (issue < u1) {
                load_block<T, DP, VEC>(p, ring + (issue - u0) % R::kStages * R::kStage, noff, lane);
                ++issue;
                if (issue < u1) {
                    nb = key_block<SHARED>(p, c, k, issue, warp);
                    noff = key_offset(p, nb, c.kvh, lane, bad_page);
                }
            }
            cp_async_commit();
        };
#pragma unroll 1
        for (int i = 0; i < R::kStages - 1; ++i)
            issue_next();

        if (threadIdx.x < kRows)
            row_at[threadIdx.x] = row_of(k, plan, c, threadIdx.x);
        __syncthreads();
        if (plan.vec_q) {
            constexpr int kPer = 16 / R::kE;
            const int used = p.head_dim / kPer;
            for (int idx = threadIdx.x; idx < kRows * R::kChunks; idx += kRowThreads) {
                const int row = idx / R::kChunks, chunk = idx % R::kChunks;
                const RowOf r = row_at[row];
                uint4 v = make_uint4(0, 0, 0, 0);
                if (r.token >= 0 && chunk < used)
                    v = __ldg(reinterpret_cast<const uint4*>(
                        static_cast<const T*>(p.q) + r.token * p.q_stride +
                        (int64_t)r.head * p.head_dim + chunk * kPer));
                float f[kPer];
                Vec<T>::unpack(v, f);
#pragma unroll
                for (int e = 0; e < kPer; e += 2)
                    store_q<T, DP>(qfrag, row, chunk * kPer + e, f[e], f[e + 1]);
            }
        } else {
            for (int idx = threadIdx.x; idx < kRows * DP / 2; idx += kRowThreads) {
                const int row = idx / (DP / 2), e = idx % (DP / 2) * 2;
                const RowOf r = row_at[row];
                float x = 0.0f, y = 0.0f;
                if (r.token >= 0) {
                    const T* src = static_cast<const T*>(p.q) + r.token * p.q_stride +
                                   (int64_t)r.head * p.head_dim;
                    x = e < p.head_dim ? load_elem(src + e) : 0.0f;
                    y = e + 1 < p.head_dim ? load_elem(src + e + 1) : 0.0f;
                }
                store_q<T, DP>(qfrag, row, e, x, y);
            }
        }
        int32_t pos[2], lo[2], hi[2], member[2];
        float slope[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const RowOf r = row_at[(lane >> 2) + 8 * i];
            member[i] = r.index;
            if constexpr (SHARED) {
                const int32_t own = __shfl_sync(0xFFFFFFFFu, k.own_len, r.index & 31);
                pos[i] = k.len + own - 1;
                visible_keys(pos[i], k.len + own, 0, p.window, lo[i], hi[i]);
            } else {
                pos[i] = k.len - k.ntok + r.index;
                visible_keys(pos[i], k.len, k.bidir, p.window, lo[i], hi[i]);
            }
            if (r.token < 0)
                hi[i] = lo[i];
            slope[i] = FULL && p.slopes && r.token >= 0 ? __ldg(p.slopes + r.head) : 0.0f;
        }
        __syncthreads();

        // -- this warp's 16 keys of every unit ---------------------------------
        float o[DP / 8][4];
#pragma unroll
        for (int n = 0; n < DP / 8; ++n)
            o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.0f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
        for (int32_t u = u0; u < u1; ++u) {
            cp_async_wait<R::kStages - 2>();
            __syncwarp();
            const KeyBlock b = key_block<SHARED>(p, c, k, u, warp);
            const unsigned char* ks = ring + (u - u0) % R::kStages * R::kStage;
            const unsigned char* vs = ks + R::kHalf;

            // scores: rows (lane / 4, + 8), keys t * 8 + 2 quad + {0, 1}
            float s[2][4];
#pragma unroll
            for (int t = 0; t < 2; ++t)
                s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.0f;
            if constexpr (sizeof(T) == 2) {
                const int row = (lane & 7) + ((lane >> 4) << 3);
                const uint32_t kbase = shared_address(ks) + row * R::kRowBytes;
#pragma unroll
                for (int step = 0; step < R::kSteps; ++step) {
                    const uint4 q4 = reinterpret_cast<const uint4*>(qfrag)[step * 32 + lane];
                    const uint32_t a[4] = {q4.x, q4.y, q4.z, q4.w};
                    uint32_t kb[4];
                    ldmatrix4(kb, kbase + (((2 * step + ((lane >> 3) & 1)) ^ (row & 7)) << 4));
                    mma_bf16(s[0], a, kb[0], kb[1]);
                    mma_bf16(s[1], a, kb[2], kb[3]);
                }
            } else {
                // the tensor cores cut every sum off instead of rounding it: the
                // small products have a sum of their own, so that the large
                // one is cut once a step
                float rest[2][4];
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    rest[t][0] = rest[t][1] = rest[t][2] = rest[t][3] = 0.0f;
#pragma unroll 4
                for (int step = 0; step < R::kSteps; ++step) {
                    const uint4* qf = reinterpret_cast<const uint4*>(qfrag) + (step * 32 + lane) * 2;
                    const uint4 h4 = qf[0], l4 = qf[1];
                    const uint32_t ah[4] = {h4.x, h4.y, h4.z, h4.w};
                    const uint32_t al[4] = {l4.x, l4.y, l4.z, l4.w};
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const int row = t * 8 + (lane >> 2);
                        uint32_t h0, l0, h1, l1;
                        split_tf32(*reinterpret_cast<const float*>(
                                       ks + swizzled<T, DP>(row, step * 8 + quad)), h0, l0);
                        split_tf32(*reinterpret_cast<const float*>(
                                       ks + swizzled<T, DP>(row, step * 8 + 4 + quad)), h1, l1);
                        mma_tf32(rest[t], al, h0, h1);
                        mma_tf32(rest[t], ah, l0, l1);
                        mma_tf32(s[t], ah, h0, h1);
                    }
                }
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        s[t][e] += rest[t][e];
            }

            // softmax: what a row does not see is -inf
            map_scores<FULL>(s, plan.score, slope, pos, b.key0 + b.shift + 2 * quad);
            const int32_t end = b.end + b.shift;
            float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = e >> 1;
                    const int32_t j = b.key0 + b.shift + t * 8 + 2 * quad + (e & 1);
                    bool seen = j >= lo[i] && j < min(hi[i], end);
                    if (SHARED && b.member >= 0)
                        seen = seen && member[i] == b.member;
                    s[t][e] = seen ? s[t][e] : -INFINITY;
                    mx[i] = fmaxf(mx[i], s[t][e]);
                }
            float f[2];
            bool grew = false;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xFFFFFFFFu, mx[i], 1));
                mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xFFFFFFFFu, mx[i], 2));
                const float mn = fmaxf(m[i], mx[i]);
                grew = grew || mn > m[i];
                f[i] = m[i] == -INFINITY ? 0.0f : exp2_fast(m[i] - mn);
                m[i] = mn;
            }
            if (__any_sync(0xFFFFFFFFu, grew)) {
#pragma unroll
                for (int n = 0; n < DP / 8; ++n) {
                    o[n][0] *= f[0];
                    o[n][1] *= f[0];
                    o[n][2] *= f[1];
                    o[n][3] *= f[1];
                }
                l[0] *= f[0];
                l[1] *= f[1];
            }
            const float m0 = m[0] == -INFINITY ? 0.0f : m[0];
            const float m1 = m[1] == -INFINITY ? 0.0f : m[1];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[t][e] = exp2_fast(s[t][e] - (e < 2 ? m0 : m1));
                    l[e >> 1] += s[t][e];
                }

            // weights times values
            if constexpr (sizeof(T) == 2) {
                // the weights are rounded to bf16 (2^-8 of each at most), the
                // type of the values that they multiply; l keeps them in fp32
                const uint32_t a[4] = {pack_bf16x2(s[0][0], s[0][1]), pack_bf16x2(s[0][2], s[0][3]),
                                       pack_bf16x2(s[1][0], s[1][1]), pack_bf16x2(s[1][2], s[1][3])};
                const int row = lane & 15;
                const uint32_t vbase = shared_address(vs) + row * R::kRowBytes;
#pragma unroll
                for (int n = 0; n < DP / 16; ++n) {
                    uint32_t vb[4];
                    ldmatrix4_trans(vb, vbase + (((2 * n + (lane >> 4)) ^ (row & 7)) << 4));
                    mma_bf16(o[2 * n], a, vb[0], vb[1]);
                    mma_bf16(o[2 * n + 1], a, vb[2], vb[3]);
                }
            } else {
                // the sum over keys has no order: key 2 quad takes the place of
                // k = quad and key 2 quad + 1 that of k = quad + 4, so that the
                // scores are the fragments as they lie
                uint32_t ah[2][4], al[2][4];
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    split_tf32(s[t][0], ah[t][0], al[t][0]);
                    split_tf32(s[t][2], ah[t][1], al[t][1]);
                    split_tf32(s[t][1], ah[t][2], al[t][2]);
                    split_tf32(s[t][3], ah[t][3], al[t][3]);
                }
#pragma unroll
                for (int n = 0; n < DP / 8; ++n) {
                    // these 16 keys' sum, then added to O with rounding
                    float add[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const int row = t * 8 + 2 * quad;
                        uint32_t h0, l0, h1, l1;
                        split_tf32(*reinterpret_cast<const float*>(
                                       vs + swizzled<T, DP>(row, n * 8 + (lane >> 2))), h0, l0);
                        split_tf32(*reinterpret_cast<const float*>(
                                       vs + swizzled<T, DP>(row + 1, n * 8 + (lane >> 2))), h1, l1);
                        mma_tf32(add, al[t], h0, h1);
                        mma_tf32(add, ah[t], l0, l1);
                        mma_tf32(add, ah[t], h0, h1);
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        o[n][e] += add[e];
                }
            }
            __syncwarp();  // every lane has read the stage that the next copy fills
            issue_next();
        }
        cp_async_wait<0>();
        if (bad_page)
            record_device_error(p.err, kDeviceErrBadIndexBit);

        // -- join the warps ----------------------------------------------------
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 1);
            l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 2);
            if (quad == 0) {
                row_m[warp][(lane >> 2) + 8 * i] = m[i];
                row_l[warp][(lane >> 2) + 8 * i] = l[i];
            }
        }
        __syncthreads();
        float* joined = reinterpret_cast<float*>(smem);  // [warp][row][DP] over the rings
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int row = (lane >> 2) + 8 * i;
            float mm = -INFINITY;
#pragma unroll
            for (int w = 0; w < kRowWarps; ++w)
                mm = fmaxf(mm, row_m[w][row]);
            const float f = part_factor(m[i], mm);
            if (row_at[row].token < 0)
                continue;
            float* dst = joined + (warp * kRows + row) * DP + 2 * quad;
#pragma unroll
            for (int n = 0; n < DP / 8; ++n)
                *reinterpret_cast<float2*>(dst + n * 8) =
                    make_float2(o[n][2 * i] * f, o[n][2 * i + 1] * f);
        }
        __syncthreads();

        const bool whole = u0 == 0 && u1 == k.units;
        // the pair's first unit on the line, its first and last CTA
        const int32_t cta0 = (int32_t)(at / share);
        const int32_t cta1 = (int32_t)((at + k.units - 1) / share);
        float* part = plan.parts +
                      ((int64_t)blockIdx.x * 2 + (u0 == 0 ? 1 : 0)) * part_floats(DP);
        for (int idx = threadIdx.x; idx < kRows * DP / 4; idx += kRowThreads) {
            const int row = idx / (DP / 4), e = idx % (DP / 4) * 4;
            const RowOf r = row_at[row];
            if (r.token < 0)
                continue;
            float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f}, ll = 0.0f, mm = -INFINITY;
#pragma unroll
            for (int w = 0; w < kRowWarps; ++w)
                mm = fmaxf(mm, row_m[w][row]);
#pragma unroll
            for (int w = 0; w < kRowWarps; ++w) {
                const float4 x =
                    *reinterpret_cast<const float4*>(joined + (w * kRows + row) * DP + e);
                sum[0] += x.x;
                sum[1] += x.y;
                sum[2] += x.z;
                sum[3] += x.w;
                ll += row_l[w][row] * part_factor(row_m[w][row], mm);
            }
            if (whole) {
                if (e >= p.head_dim)
                    continue;
                store_result<T, DP, SHARED>(p, plan, r, e, sum, mm, ll);
            } else {
                *reinterpret_cast<float4*>(part + row * DP + e) =
                    make_float4(sum[0], sum[1], sum[2], sum[3]);
                if (e == 0) {
                    part[kRows * DP + row] = mm;
                    part[kRows * DP + kRows + row] = ll;
                }
            }
        }

        // -- join the CTAs: the last to arrive does ---------------------------
        if (!whole) {
            __syncthreads();
            if (threadIdx.x == 0) {
                const int32_t n = cta1 - cta0 + 1;
                // releases what the barrier brought together, acquires the others'
                int32_t old;
                asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;"
                             : "=r"(old)
                             : "l"(plan.counters + cta0)
                             : "memory");
                if (old < 0 || old >= n)
                    record_device_error(p.err, AROPS_DEVICE_ERR_WORKSPACE);
                last_flag = old == n - 1;
                if (last_flag)
                    plan.counters[cta0] = 0;
            }
            __syncthreads();
            if (last_flag)
                join_parts<T, DP, SHARED>(p, plan, row_at, cta0, cta1, row_m, row_l,
                                          reinterpret_cast<float*>(smem));
        }

        next_pair();
    }
}

template <typename T, int DP, bool VEC, bool FULL, bool SHARED>
cudaError_t launch_rows(const AttentionParams& p, const RowPlan& plan, int sm_count,
                        cudaStream_t st)
{
    using R = RowTraits<T, DP>;
    constexpr auto kernel = attention_rows_kernel<T, DP, VEC, FULL, SHARED>;
    cudaError_t err = cudaSuccess;
    for (int attempt = 0; attempt < 2; ++attempt) {
        int ctas = 0;
        err = resident_ctas_once<kernel>(kRowThreads, R::kSmem, &ctas, attempt > 0);
        if (err != cudaSuccess)
            return err;
        const int64_t grid =
            std::min<int64_t>((int64_t)sm_count * std::max(ctas, 1), kMaxRowCtas);
        err = launch(kernel, dim3((unsigned)grid), dim3(kRowThreads), R::kSmem, st, p, plan);
        if (err != cudaErrorInvalidValue)
            return err;
        cudaGetLastError();  // not kept for the caller's next call
    }
    return err;
}

template <typename T, int DP, bool VEC>
cudaError_t launch_rows_v(const AttentionParams& p, const RowPlan& plan, int sm_count,
                          cudaStream_t st)
{
    const bool full = p.softcap > 0.0f || p.slopes != nullptr;
    if (p.group_start)
        return full ? launch_rows<T, DP, VEC, true, true>(p, plan, sm_count, st)
                    : launch_rows<T, DP, VEC, false, true>(p, plan, sm_count, st);
    return full ? launch_rows<T, DP, VEC, true, false>(p, plan, sm_count, st)
                : launch_rows<T, DP, VEC, false, false>(p, plan, sm_count, st);
}

template <typename T>
cudaError_t launch_rows_t(const AttentionParams& p, RowPlan plan, int sm_count, cudaStream_t st)
{
    constexpr int E = Vec<T>::N;
    const bool vec = p.head_dim % E == 0 && aligned16(p.k_pages) && aligned16(p.v_pages);
    plan.vec_q = p.head_dim % E == 0 && aligned16(p.q) && p.q_stride % E == 0;
    plan.vec_out = p.head_dim % 4 == 0 && aligned16(p.out);
    const int dp = padded_head_dim(p.head_dim);
    if (dp == 64)
        return vec ? launch_rows_v<T, 64, true>(p, plan, sm_count, st)
                   : launch_rows_v<T, 64, false>(p, plan, sm_count, st);
    if (dp == 128)
        return vec ? launch_rows_v<T, 128, true>(p, plan, sm_count, st)
                   : launch_rows_v<T, 128, false>(p, plan, sm_count, st);
    if constexpr (sizeof(T) == 2)
        return vec ? launch_rows_v<T, 256, true>(p, plan, sm_count, st)
                   : launch_rows_v<T, 256, false>(p, plan, sm_count, st);
    return cudaErrorNotSupported;  // refused by the entry points
}

}  // namespace

size_t attention_counter_bytes()
{
    return kCounterBytes;
}

// Which calls go to the tile kernel, by their rows (tokens times query heads a
// key head).  It passes over the keys once for up to 256 rows, the row kernel
// once for 16; its fixed cost is the higher one (a prompt of 60 tokens: row 7.9
// against tile 13.6 us; 200: 16.9 / 17.4; 400: 31.9 / 19.1; 1,000: 65 / 26).
//   Ragged batches (rows a sequence, row against tile kernel): 64 sequences on
//   1,000 positions 16: 62 against 76 us, 24: 103 / 76; 8 on 4,000 16: 38 / 47,
//   24: 54 / 47; 200 on 300 16: 72 / 87, 24: 115 / 88; one on 8,000 96: 43 / 37.
//   Prefixes (rows a group): 8 groups on 2,000 positions 48: 78 / 82, 64: 95 / 90,
//   128: 164 / 129; one on 2,000 128: 37 / 57, 510: 93 / 85.
// The rule sees the call's rows alone, and one kernel takes all of it.  So the
// shortest prompts lose up to 6 us, 20 groups of 64 rows on 500 positions 7 (134 /
// 141), and a call of decode steps and prompts pays for the side that is in the
// minority (255 steps and a prompt of 1,500 tokens: 271 us; apart 185 and 33).
bool many_rows(const AttentionParams& p)
{
    const int64_t rows = p.tokens * (p.hq / p.hk);
    if (p.group_start)
        return rows >= 64 * (int64_t)p.n_groups && rows >= 512;
    return rows > kRows * (int64_t)p.n_seqs && rows >= 96;
}

// The two kernels' partial results share a region: the second launch of a call
// waits for the first.  With shared prefixes the prefix's results of every
// (sequence, head) follow.
size_t attention_workspace_bytes(int64_t tokens, int hq, int head_dim, bool shared_prefix)
{
    const int dp = padded_head_dim(head_dim);
    size_t parts = (size_t)kMaxRowCtas * 2 * part_floats(dp) * sizeof(float);
    if (dp > 128 || tokens * hq < 96)  // too few rows for the tile kernel
        return kCounterBytes + parts;
    return kCounterBytes + std::max(parts, tile_part_bytes(dp)) +
           (shared_prefix ? (size_t)tokens * hq * (dp + 2) * sizeof(float) : 0);
}

cudaError_t launch_attention(const AttentionParams& p, arops_dtype dtype, void* workspace,
                             cudaStream_t stream)
{
    DeviceInfo di;
    cudaError_t err = current_device_info(&di);
    if (err != cudaSuccess)
        return err;
    const int dp = padded_head_dim(p.head_dim);
    RowPlan plan = {};
    plan.score = make_score_map(p);
    plan.counters = static_cast<int32_t*>(workspace);
    plan.parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + kCounterBytes);
    const int g = p.hq / p.hk;
    plan.g = make_row_divide(g);
    plan.seqs_a_tile = std::max(1, kRows / g);
    plan.tiles_a_seq = (int32_t)ceil_div(g, kRows);
    plan.min_units = kMinUnits;

    // The tile kernel takes all of a ragged batch, or the prefixes of a shared
    // one (a window cuts prefixes row by row: the row kernel leaves out what
    // nobody sees).
    if (many_rows(p) && tiles_can_run(p, dtype) && !(p.group_start && p.window > 0)) {
        float* prefix_o = nullptr;
        float* prefix_ml = nullptr;
        if (p.group_start) {
            const size_t parts = std::max((size_t)kMaxRowCtas * 2 * part_floats(dp) * sizeof(float),
                                          tile_part_bytes(dp));
            prefix_o = reinterpret_cast<float*>(reinterpret_cast<char*>(plan.parts) + parts);
            prefix_ml = prefix_o + (size_t)p.tokens * p.hq * dp;
        }
        err = launch_attention_tiles(p, plan.parts, prefix_o, prefix_ml, di.sm_count, stream);
        if (err != cudaSuccess || !p.group_start)
            return err;
        plan.prefix_o = prefix_o;
        plan.prefix_ml = prefix_ml;
    }
    if (dtype == AROPS_BF16)
        return launch_rows_t<__nv_bfloat16>(p, plan, di.sm_count, stream);
    return launch_rows_t<float>(p, plan, di.sm_count, stream);
}

}  // namespace arops
