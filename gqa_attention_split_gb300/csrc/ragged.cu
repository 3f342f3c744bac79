// Attention over ragged batches on the 5th-generation tensor cores: packed
// prompts, and drafted token trees on top of the KV cache; and appending
// packed tokens to the cache.
//
//   O = softmax(scale * Q K^T over the visible keys) V,   lse = ln sum exp(.)
//
// Both calls stream the same two sources of keys per row of the batch: the
// context in the cache (decode_tree only; every slot below context_lens[b] is
// visible), then the row's own packed tokens (prefill_packed: a causal limit
// or all of them; decode_tree: the bits of a mask, or a line). A key that a
// query does not see never reaches its result, whatever K and V hold there.
//
// Layout of the work. The G query heads of a KV head are folded into the rows
// of the matrix products: a group of rows is tok = floor(128 / G) consecutive
// tokens x G heads (token-major, one TMA box {64, G, tok} per 64 columns), so
// a causal diagonal is only tok tokens wide and a short prompt or a small
// tree still fills rows. A work item is up to two groups that read the same
// K/V tiles of 128 keys.
//
// Roles of a CTA (one per SM, persistent): warp 0 TMA, warp 1 issues every
// tcgen05.mma, warp 2 finds the work items from the prefix sums on the device
// (the host never waits for them) and passes them on through a ring in shared
// memory, warp 3 repairs V tiles whose keys not every row may see, two
// warpgroups run the online softmax, one query row per thread. S and O live in
// tensor memory, P is written over its S columns and read from there by the P V
// product.
//
// What bounds it. A group's tile is a chain: S seen, softmax (1150 to 1250 cycles:
// exponentials, sums and packing at the rate of the fp32 and special function
// pipes, which the other group's sums share), P V and the next S (1024 cycles of
// tensor work at d = 128, 512 at 64), and 600 of hand-overs (commit to waiting warps
// 250, each wait of the issuing thread about 100 even when its barrier is complete).
// Two groups take turns at the tensor cores, so a pair of tiles takes 3090 cycles at
// d = 128 and 2630 at d = 64, where the products alone would take 2048 and 1024:
// packed 32K tokens 1.45-1.48 PFLOP/s, 0.78-0.79 of the measured bf16 rate. A long
// context under few queries is bound by HBM, a short one by latencies: launch 1 us,
// prefix sums to first tile 4, per tile 1.5, end of an item 2, merge 2 to 5.
// Measured and slower on the same box (packed 8K batch / packed 32K, against
// 174 / 4300 us at that point): steps of 64 keys with two S buffers per group
// (208 / 5930: S products of N = 64 run at 0.6 of the rate); one S buffer for
// both groups with P in columns of its own (194 / 4750: the next S is not ready
// in time); P handed over in halves (191 / 4600); a worker per group with its own
// items and K/V ring, as two CTAs per SM (230 / 5110: their products interleave
// and both wait) or in one CTA with a lock around the issue (203 / 4600); the end
// of an item behind the next item's first tile (188 / 4350); O through TMA boxes
// (172 / 4300). Against 154 / 3920, with O divided by the sum of the unrounded
// weights: half of a tile's exponentials against the maximum so far, beside the
// search for the new one (167 / 4290); two threads to a query row, 16 softmax warps
// (178 / 4420, and 164 / 4160 with nothing exchanged between the two: the pipes, not
// latency, are the softmax's limit); scalar in place of packed fp32 arithmetic (164 /
// 4310); S products a tile ahead from a second issuing warp, P in columns of its own
// (200 / 3990); the barriers of an issue polled by one lane each (152 / 3920, but a
// batch of 8 trees 145 against 135).

#include <cuda_runtime.h>
#include <math.h>

#include <type_traits>

#include "gqa_attn.h"
#include "plan.cuh"
#include "ptx.cuh"
#include "runtime.cuh"
#include "tcgen05.cuh"

namespace gqa {
namespace ragged {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMaxTreeTokens = 128;  // drafted tokens of a row: one tile of keys
constexpr int BM = kPrefillBlockM;   // rows of a group
constexpr int BN = kPrefillBlockN;   // keys of a tile
constexpr int kThreads = 384;
constexpr int kRingSlots = 4;        // K/V tiles in flight
constexpr int kItemSlots = 4;        // work items known ahead
constexpr int kSchedSeqs = 1024;     // sequences whose schedule is kept in shared memory
constexpr int kTreeCtas = 152;       // most CTAs of a decode_tree launch (workspace size)
// decode_tree: rows are not cut where the cache holds at most this many tiles with the drafts' own
// (512 slots), which saves the merge (8 units of 2 tiles 8.1 us against 10.2 cut, 4 tiles 10.5
// against 11.0, 5 tiles 12.0 against 11.2, 9 tiles 18.4 against 11.7). The host goes by the size
// of the cache, since the lengths are on the device: short contexts in a larger cache are cut.
constexpr int kWholeTiles = 5;
constexpr uint32_t kBoxBytes = BM * 128;       // 128 rows x 64 bf16
constexpr uint32_t kStageBytes = 32 * 64;      // a warp's output stage: 32 rows x 64 B
constexpr uint32_t kTmemCols = 512;            // S_0, S_1, O_0, O_1
// rescale O only when the running maximum (base 2) grew by more than this: P <= 2^8
constexpr float kRescaleThreshold = 8.f;

// kPrompts: items are blocks of 2 * tok tokens of a sequence, all of its keys.
// kTreePair: items are blocks of 2 * tok drafted tokens, a range of the keys.
// kTreeAlt: all drafted tokens of a row fit in one group; the two softmax
// groups take alternate K/V tiles and are merged in the epilogue (28/4 heads,
// 5 drafts, contexts of 64 to 9100: 19.0 us against 19.9 as kTreePair, whose
// second group would be empty).
enum Mode { kPrompts, kTreePair, kTreeAlt };

struct Params {
    const uint16_t* v;            // packed V, read again only for values that are not finite
    uint16_t* o;                  // [total_q, H_q, d]
    float* lse;                   // [total_q, H_q] or null
    // decode_tree: partial results, two slots per CTA. O is laid out
    // [slot][d / 4][part_rows][4] so that a warp, one row per lane, reads and
    // writes 512 contiguous bytes at a time.
    float *part_o, *part_lse;     // lse: [slot][part_rows]
    int4* part_info;              // [CTA]: the unit that begins there (see schedule_tree)
    const int32_t *cu_q, *cu_k, *ctx;
    const uint32_t* mask;         // [total_q, mask_words] or null
    unsigned* status;
    int64_t v_st, v_sh;
    int B, H_q, H_kv, G, total_q, total_k, S_max, max_tokens, mask_words, causal;
    int max_blocks;   // kPrompts: blocks of all rows under any valid prefix sums
    int tok;          // tokens of a group
    int team;         // decode_tree: CTAs that share a range of keys, one per token block
    int n_teams, part_rows;
    int whole;        // decode_tree: no (row, KV head) is cut
    float scale_log2;
    int inject_timeout;  // test hook: block 0 withholds its first Q copy
};

// One work item: tiles j0 .. j0 + n - 1 of a row's tile list (the context's
// tiles, c_t of them, then its own tokens') against one or two groups of rows.
struct __align__(16) Item {
    int n;       // tiles, the larger of n0 and n1; -1: no more items
    int n0, n1;  // tiles of group 0 and 1 (kTreeAlt: unused)
    int j0;
    int kvh, b;
    int dst;     // partial slot, or -1: the item is the whole row, write O and lse
    int ctx;     // context length
    int q_row;   // packed index of the row's first token
    int tok0;    // first token of group 0, counted in the row
    int T;       // tokens of the row
    int c_t;     // context tiles
    int k_row;   // packed index of the row's first own key
    int off;     // own key of token 0 (keys minus queries)
    int n_own;   // own keys
    int pad;
};
static_assert(sizeof(Item) == 64, "four 16-byte copies");

__device__ __forceinline__ int clampi(int x, int lo, int hi) { return min(max(x, lo), hi); }
__device__ __forceinline__ int cdiv(int a, int b) { return (a + b - 1) / b; }

// First packed token and token count of row b under prefix sums cu (null:
// every row has total / B tokens). Bad prefix sums are clamped: the row stays
// inside [0, total), and bad is set.
__device__ __forceinline__ void row_range(const int32_t* cu, int B, int total, int b, int& first,
                                          int& count, bool& bad) {
    if (!cu) {
        count = total / B;
        first = b * count;
        return;
    }
    const int a = cu[b], e = cu[b + 1];
    first = clampi(a, 0, total);
    const int last = clampi(e, first, total);
    count = last - first;
    bad = bad || first != a || last != e;
}

__device__ __forceinline__ void tree_row(const Params& p, int b, int& first, int& T, int& ctx,
                                         bool& bad) {
    row_range(p.cu_q, p.B, p.total_q, b, first, T, bad);
    if (T > p.max_tokens) {
        T = p.max_tokens;
        bad = true;
    }
    const int c = p.ctx[b];
    ctx = clampi(c, 0, p.S_max);
    bad = bad || ctx != c;
}

// Tiles that each block of a row's drafted tokens runs: the context's and one
// for the drafted tokens.
__device__ __forceinline__ int tree_tiles(int T, int ctx) {
    return T > 0 ? cdiv(ctx, BN) + 1 : 0;
}

// ---- limits of an item, as every role needs them

// Own keys visible to token t (kPrompts).
__device__ __forceinline__ int token_limit(const Params& p, const Item& w, int t) {
    return p.causal ? clampi(w.off + t + 1, 0, w.n_own) : w.n_own;
}
// Own keys that every row of group g sees / that some row of it sees.
template <int kMode>
__device__ __forceinline__ int group_first(const Params& p, const Item& w, int g) {
    return kMode == kPrompts ? token_limit(p, w, w.tok0 + g * p.tok) : 0;
}
template <int kMode>
__device__ __forceinline__ int group_last(const Params& p, const Item& w, int g) {
    return kMode == kPrompts ? token_limit(p, w, min(w.T, w.tok0 + (g + 1) * p.tok) - 1) : w.n_own;
}
// Keys of tile jj that some row of group g sees (1..128).
template <int kMode>
__device__ __forceinline__ int tile_keys(const Params& p, const Item& w, int jj, int g) {
    if (kMode != kPrompts && jj < w.c_t) return min(BN, w.ctx - jj * BN);
    return clampi(group_last<kMode>(p, w, g) - (jj - w.c_t) * BN, 0, BN);
}
// The same value in every lane, in a form that the compiler knows to be so:
// loop bounds and ring positions derived from it stay in uniform registers,
// where the descriptors of the matrix instructions have to be.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// Leading tiles of an item that every row of group g (and of the groups before
// it) sees whole: no mask, no repair, all 128 keys.
template <int kMode>
__device__ __forceinline__ int plain_tiles(const Params& p, const Item& w, int g) {
    const int whole = (kMode == kPrompts ? group_first<kMode>(p, w, g) : w.ctx) / BN;
    return clampi(whole - w.j0, 0, w.n);
}
// The keys of V tile jj that the P V products read are [0, end). Those from
// `seen` on are not visible to every row, those from `keys` on to none.
struct Repair {
    int seen, keys, end;
};
template <int kMode>
__device__ __forceinline__ Repair repair_of(const Params& p, const Item& w, int jj) {
    const int last = kMode == kPrompts && w.n1 > 0 ? 1 : 0;  // the group that sees more
    Repair r;
    r.keys = tile_keys<kMode>(p, w, jj, last);
    r.end = (r.keys + 15) & ~15;
    r.seen = kMode != kPrompts && jj < w.c_t
                 ? r.keys
                 : clampi(group_first<kMode>(p, w, 0) - (jj - w.c_t) * BN, 0, r.keys);
    return r;
}

// ---- shared memory

template <int D>
struct Geo {
    static_assert(D == 64 || D == 128, "head dim");
    static constexpr int kBoxes = D / 64;
    static constexpr uint32_t kTileBytes = kBoxes * kBoxBytes;
    static constexpr uint32_t kQOff = 0;  // two groups
    static constexpr uint32_t kRingOff = 2 * kTileBytes;
    static constexpr uint32_t kStageOff = kRingOff + kRingSlots * kTileBytes;  // 8 warps
    static constexpr uint32_t kXchOff = kStageOff + 8 * kStageBytes;  // float4 [2][128]
    static constexpr uint32_t kSeqOff = kXchOff + 2 * BM * 16;        // int2 [kSchedSeqs]
    static constexpr uint32_t kItemOff = kSeqOff + kSchedSeqs * 8;
    static constexpr uint32_t kBarOff = kItemOff + kItemSlots * 64;
    static constexpr int kSmemBytes = 1024 + kBarOff + 512;
    static_assert(kSmemBytes <= 232448, "more dynamic shared memory than one CTA may have");
};
// An item, read from its slot in shared memory each time it is written here:
// the softmax warps keep few of its fields in registers over a tile loop.
__device__ __forceinline__ Item read_item(uint32_t addr) {
    Item w;
    int4* q = reinterpret_cast<int4*>(&w);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm volatile("ld.shared.v4.s32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(q[i].x), "=r"(q[i].y), "=r"(q[i].z), "=r"(q[i].w)
                     : "r"(addr + i * 16));
    return w;
}

__device__ __forceinline__ uint32_t col_s_of(int g) { return uint32_t(g) * 128u; }
__device__ __forceinline__ uint32_t col_o_of(int g) { return 256u + uint32_t(g) * 128u; }

enum Bar {
    bQFull = 0,                            // Q of an item landed
    bQEmpty,                               // the item's last S products completed
    bSlotFull,                             // x kRingSlots
    bSlotEmpty = bSlotFull + kRingSlots,   // x kRingSlots
    bSFull = bSlotEmpty + kRingSlots,      // x2: S_g ready
    bPFull = bSFull + 2,                   // x2: P_g ready (4 warps)
    bODone = bPFull + 2,                   // x2: O_g final
    bItemFull = bODone + 2,                // x kItemSlots
    bItemEmpty = bItemFull + kItemSlots,   // x kItemSlots (kItemReaders)
    bFixAsk = bItemEmpty + kItemSlots,     // x2: the repair warp may start on a tile
    bFixDone = bFixAsk + 2,                // x2
    bXch = bFixDone + 2,                   // kTreeAlt: m, l of both groups written (8 warps)
    bXchDone,                              // kTreeAlt: both O read (8 warps)
    bDrain,
    kNumBars
};
static_assert(kNumBars * 8 + 8 <= 512, "barrier area");
constexpr int kItemReaders = 3 + 8;  // TMA, MMA and repair warps, 8 softmax warps

// ---- the scheduling warp

struct Publisher {
    uint8_t* items;
    uint64_t* bars;
    unsigned* status;
    int count = 0;
    __device__ bool put(const Item& w, int lane) {
        const int s = count % kItemSlots;
        if (count >= kItemSlots &&
            !__all_sync(0xffffffffu,
                        mbar_wait_bounded(smem_u32(&bars[bItemEmpty + s]),
                                          ((count / kItemSlots) - 1) & 1, status)))
            return false;
        if (lane == 0) {
            *reinterpret_cast<Item*>(items + s * sizeof(Item)) = w;
            mbar_arrive(smem_u32(&bars[bItemFull + s]));
        }
        __syncwarp();
        ++count;
        return true;
    }
};

// kPrompts. A block's cost is the number of keys it sees, so a sequence's
// blocks are numbered by levels (key position of the block / block length) and
// the launch runs the levels from the highest down over all sequences, in
// snake order over the CTAs: heaviest first, found from the prefix sums by
// counting, without sorting, so that every CTA finds its own items alone. All KV
// heads run together even where their K and V are larger than L2: one group of
// heads after another, each within L2, ends on heavy items several times (one
// sequence of 64K tokens, 16/8 heads: 11.9 ms in groups, 10.8 this way).
__device__ __forceinline__ void schedule_prompts(const Params& p, int2* seqs, Publisher& pub,
                                                 int lane) {
    const int block = 2 * p.tok;
    bool bad = false;
    auto levels = [&](int b) {  // x: lowest level, y: blocks
        int q0, T, k0, n;
        row_range(p.cu_q, p.B, p.total_q, b, q0, T, bad);
        if (p.cu_k) row_range(p.cu_k, p.B, p.total_k, b, k0, n, bad);
        else n = T;
        return make_int2((p.causal ? max(n - T, 0) : n) / block, cdiv(T, block));
    };
    // More sequences than the table holds: the blocks run in the sequences'
    // order instead, found through the block counts of `chunk` sequences each
    // (counting through all levels for every item takes B / 32 rounds a step;
    // 20000 sequences of 1 to 4 tokens: 171 ms that way, 2.8 this way). There are
    // many items then, so their order matters little for the balance.
    const bool in_order = p.B > kSchedSeqs;
    const int chunk = cdiv(p.B, kSchedSeqs);
    int* before_chunk = reinterpret_cast<int*>(seqs);  // blocks before chunk c
    int top = 0, blocks;
    // (64 bits, and no work at all above max_blocks: rows of bad prefix sums may overlap,
    // and then have more blocks together than there are tokens)
    int64_t sum = 0;
    if (in_order) {
#pragma unroll 1
        for (int c0 = 0; c0 < kSchedSeqs; c0 += 32) {
            int64_t n = 0;
            const int first = min(p.B, (c0 + lane) * chunk);
#pragma unroll 4
            for (int b = first; b < min(p.B, first + chunk); ++b) n += levels(b).y;
            int64_t incl = n;
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            before_chunk[c0 + lane] = int(min(sum + incl - n, int64_t(p.max_blocks)));
            sum += __shfl_sync(0xffffffffu, incl, 31);
        }
    } else {
#pragma unroll 1
        for (int b = lane; b < p.B; b += 32) {
            const int2 s = levels(b);
            seqs[b] = s;
            sum += s.y;
            if (s.y > 0) top = max(top, p.causal ? s.x + s.y - 1 : s.x);
        }
        top = __reduce_max_sync(0xffffffffu, top);
        // (at most 32 rows of 2^30 blocks a lane: the low 26 bits and the rest)
        const unsigned low = __reduce_add_sync(0xffffffffu, unsigned(sum) & 0x3ffffffu);
        const unsigned high = __reduce_add_sync(0xffffffffu, unsigned(sum >> 26));
        sum = (int64_t(high) << 26) + low;
    }
    blocks = sum <= p.max_blocks ? int(sum) : 0;
    if (bad && blockIdx.x == 0) atomicOr(p.status, kStatusBadSeqlen);
    __syncwarp();
    auto above = [&](int l) {  // blocks on levels > l
        int c = 0;
#pragma unroll 1
        for (int b = lane; b < p.B; b += 32) {
            const int2 s = seqs[b];
            c += p.causal ? clampi(s.x + s.y - 1 - l, 0, s.y) : (s.x > l ? s.y : 0);
        }
        return __reduce_add_sync(0xffffffffu, c);
    };
    const int64_t total = int64_t(blocks) * p.H_kv;
    const int ctas = gridDim.x;
    int hint = top;
    for (int it = 0;; ++it) {
        const int64_t R = int64_t(it) * ctas + ((it & 1) ? ctas - 1 - int(blockIdx.x) : blockIdx.x);
        if (R >= total) break;
        const int rank = int(R / p.H_kv);  // of the block, whose KV heads follow one another
        int b = 0, i = 0;
        if (in_order) {
            int c = 0;  // the last chunk with at most `rank` blocks before it
            for (int step = kSchedSeqs / 2; step > 0; step >>= 1)
                if (before_chunk[c + step] <= rank) c += step;
            int k = rank - before_chunk[c];
            b = c * chunk;
            for (int b0 = b;; b0 += 32) {
                const int y = b0 + lane < min(p.B, (c + 1) * chunk) ? levels(b0 + lane).y : 0;
                int incl = y;
                for (int o = 1; o < 32; o <<= 1) {
                    const int z = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += z;
                }
                const unsigned hit = __ballot_sync(0xffffffffu, incl > k);
                if (hit || b0 + 32 >= (c + 1) * chunk) {
                    const int src = hit ? __ffs(hit) - 1 : 0;
                    b = b0 + src;
                    i = __shfl_sync(0xffffffffu, y - 1 - (k - (incl - y)), src);
                    break;
                }
                k -= __shfl_sync(0xffffffffu, incl, 31);
            }
        } else {
            int lo = 0, hi = hint;  // the lowest level with at most `rank` blocks above it
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (above(mid) <= rank) hi = mid;
                else lo = mid + 1;
            }
            hint = lo;
            int k = rank - above(lo);  // the k-th block of this level
#pragma unroll 1
            for (int b0 = 0; b0 < p.B; b0 += 32) {
                int c = 0;
                int2 s = make_int2(0, 0);
                if (b0 + lane < p.B) {
                    s = seqs[b0 + lane];
                    c = p.causal ? (lo >= s.x && lo < s.x + s.y) : (s.x == lo ? s.y : 0);
                }
                int sum = c;
                for (int o = 1; o < 32; o <<= 1) {
                    const int x = __shfl_up_sync(0xffffffffu, sum, o);
                    if (lane >= o) sum += x;
                }
                const unsigned hit = __ballot_sync(0xffffffffu, sum > k);
                if (hit) {
                    const int src = __ffs(hit) - 1;
                    b = b0 + src;
                    i = __shfl_sync(0xffffffffu, p.causal ? lo - s.x : k - (sum - c), src);
                    break;
                }
                k -= __shfl_sync(0xffffffffu, sum, 31);
            }
        }
        Item w{};
        w.kvh = int(R % p.H_kv);
        w.b = b;
        w.dst = -1;
        row_range(p.cu_q, p.B, p.total_q, b, w.q_row, w.T, bad);
        w.k_row = w.q_row;
        w.n_own = w.T;
        if (p.cu_k) row_range(p.cu_k, p.B, p.total_k, b, w.k_row, w.n_own, bad);
        w.off = w.n_own - w.T;
        w.tok0 = i * block;
        w.n0 = cdiv(group_last<kPrompts>(p, w, 0), BN);
        w.n1 = w.tok0 + p.tok < w.T ? cdiv(group_last<kPrompts>(p, w, 1), BN) : 0;
        w.n = max(w.n0, w.n1);
        if (!pub.put(w, lane)) return;
    }
    Item end{};
    end.n = -1;
    pub.put(end, lane);
}

// decode_tree. CTAs work in teams of as many as the longest row can have
// blocks of drafted tokens. The members of a team run the same tiles of a row
// at the same time: its blocks against one KV head (K and V then come from L2
// for all but one), and where a row has fewer blocks, several KV heads. Such a
// set of KV heads is a unit. How the units are cut into the teams' shares:
//  - whole: not at all, unit u goes to team u mod n_teams (short caches);
//  - even: every unit into equal parts of at most `even` tiles, the tiles of all
//    units over the teams, when there are no more parts than teams: one part each;
//  - else all units in one line, cut every `per` steps: however ragged the
//    contexts are, every team streams the same number of keys, at the price of
//    a second and third item where a share crosses into the next unit. A unit
//    is its tiles long and kItemCost steps before them, about what an item's
//    first loads and its end cost.
// A unit that is cut leaves partial results for the merge. (A batch of
// 8 rows with contexts of 17 to 31007 and 1 to 64 drafts: 143 us, without the
// item cost 167, with one KV head in every unit 162.)
constexpr int kItemCost = 2;

// The CTA that holds the first part of a block of a unit describes it for the
// merge in part_info: x the packed index of the block's first token, y the rows
// of the block (tokens x G), z the KV head, w the number of parts (0: nothing to
// merge); the other parts are those of the same member of the next teams.
template <int kMode>
__device__ __forceinline__ void schedule_tree(const Params& p, Publisher& pub, int lane) {
    bool bad = false;
    const int team = blockIdx.x / p.team, member = blockIdx.x % p.team;
    struct Row {
        int q0, T, ctx, tiles;
        int blocks, heads, units;  // blocks of tokens; KV heads of a unit; units
    };
    auto load_row = [&](int b) {
        Row r{0, 0, 0, 0, 1, 1, 0};
        if (b >= p.B) return r;
        tree_row(p, b, r.q0, r.T, r.ctx, bad);
        r.tiles = tree_tiles(r.T, r.ctx);
        if (r.tiles == 0) return r;
        r.units = p.H_kv;
        if (p.team > 1) {
            r.blocks = cdiv(r.T, 2 * p.tok);
            r.heads = p.team / r.blocks;
            r.units = cdiv(p.H_kv, r.heads);
        }
        return r;
    };
    const Row row_0 = load_row(lane);  // the first 32 rows stay in registers
    auto row_of = [&](int b0) { return b0 == 0 ? row_0 : load_row(b0 + lane); };
    int even = 0, per = 1, end = 0, x = 0;  // this team's share [x, end) of the line
    if (p.whole) {
        x = team;
        end = 0x7fffffff;
    } else {
        int tiles = 0, units = 0, parts = 0;
#pragma unroll 1
        for (int b0 = 0; b0 < p.B; b0 += 32) {
            const Row r = row_of(b0);
            tiles += r.tiles * r.units;
            units += r.units;
        }
        tiles = __reduce_add_sync(0xffffffffu, tiles);
        const int steps = tiles + __reduce_add_sync(0xffffffffu, units) * kItemCost;
        const int most = max(1, cdiv(tiles, p.n_teams));
        per = max(1, cdiv(steps, p.n_teams));
#pragma unroll 1
        for (int b0 = 0; b0 < p.B; b0 += 32) {
            const Row r = row_of(b0);
            parts += cdiv(r.tiles, most) * r.units;
        }
        if (__reduce_add_sync(0xffffffffu, parts) <= p.n_teams) even = most;
        const int64_t begin = int64_t(team) * per;
        x = even ? team : int(min(begin, int64_t(steps)));
        end = even ? team + 1 : int(min(int64_t(steps), begin + per));
    }
    if (!p.whole && lane == 0) p.part_info[blockIdx.x] = make_int4(0, 0, 0, 0);
    int before = 0;  // steps of the rows before b0
#pragma unroll 1
    for (int b0 = 0; b0 < p.B && x < end; b0 += 32) {
        const Row mine = row_of(b0);
        // steps of a unit in the line: 1, its parts, or the item cost and its tiles
        const int len = mine.tiles == 0 ? 0
                        : p.whole       ? 1
                        : even          ? cdiv(mine.tiles, even)
                                        : mine.tiles + kItemCost;
        int sum = len * mine.units;  // inclusive prefix sum over the lanes
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += y;
        }
        const int all = __shfl_sync(0xffffffffu, sum, 31);
#pragma unroll 1
        while (x < end && x < before + all) {
            const int src = __ffs(__ballot_sync(0xffffffffu, before + sum > x)) - 1;
            auto of = [&](int v) { return __shfl_sync(0xffffffffu, v, src); };
            const int tiles = of(mine.tiles), blocks = of(mine.blocks), heads = of(mine.heads);
            const int unit = of(len);
            const int at = x - (before + of(sum) - unit * of(mine.units));
            const int i = at % unit;  // step of the unit
            Item w{};
            w.b = b0 + src;
            w.kvh = at / unit * heads + member / blocks;
            w.n = tiles;
            int parts = 1;
            if (p.whole) {
                x += p.n_teams;
            } else if (even) {
                // (below 2^32: a row has less than 2^24 tiles and kTreeCtas parts)
                w.j0 = int(unsigned(tiles) * unsigned(i) / unsigned(unit));
                w.n = int(unsigned(tiles) * unsigned(i + 1) / unsigned(unit)) - w.j0;
                parts = unit;
                ++x;
            } else {
                const int start = x - i + kItemCost;  // of the unit's tiles in the line
                w.j0 = max(0, i - kItemCost);
                w.n = min(tiles, end - start) - w.j0;  // (0: the share ends in the item cost)
                parts = (start + tiles - 1) / per - start / per + 1;
                x += min(unit - i, end - x);
            }
            w.q_row = w.k_row = of(mine.q0);
            w.T = w.n_own = of(mine.T);
            w.ctx = of(mine.ctx);
            w.c_t = tiles - 1;
            w.tok0 = member % blocks * 2 * p.tok;
            w.n0 = w.n;
            w.n1 = w.tok0 + p.tok < w.T ? w.n : 0;
            if (w.n <= 0 || member >= blocks * heads || w.kvh >= p.H_kv) continue;
            // slot 2c + 1 holds the first part of a unit, 2c another one
            w.dst = parts == 1 ? -1 : 2 * int(blockIdx.x) + (w.j0 == 0);
            if (parts > 1 && w.j0 == 0 && lane == 0)
                p.part_info[blockIdx.x] = make_int4(
                    w.q_row + w.tok0, min(w.T - w.tok0, 2 * p.tok) * p.G, w.kvh, parts);
            if (!pub.put(w, lane)) return;
        }
        before += all;
    }
    // (block 0 has read every row by now: above, or, when no row is cut, in this walk)
    if (bad && blockIdx.x == 0) atomicOr(p.status, kStatusBadSeqlen);
    Item stop{};
    stop.n = -1;
    pub.put(stop, lane);
}

// ---- softmax of one tile of scores

struct RowState {
    float m, l, lb;  // running maximum (base 2), sums of p and of bf16(p)
};

// P = 2^(s - m) over the tile, written as bf16 pairs over S (the operand type of
// the P V product) and left in pk; returns the factor that O has to be scaled by
// (1: left as it is). lse comes from l, the sum of the unrounded p, O from lb, that
// of the rounded ones (rounded_sum): O is then a weighted mean of the V rows,
// whose weights are off by half a bf16 step at most, and what all weights are off
// by together drops out.
__device__ __forceinline__ float softmax_tile(const float (&sv)[BN], RowState& st,
                                              float scale_log2, uint64_t c2, uint32_t s_addr,
                                              uint32_t (&pk)[2][32]) {
    float mm[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) mm[i] = fmaxf(sv[i], sv[8 + i]);
#pragma unroll
    for (int c = 16; c < BN; c += 16)
#pragma unroll
        for (int i = 0; i < 8; ++i) mm[i] = fmax3(mm[i], sv[c + i], sv[c + 8 + i]);
    const float mx = fmax3(fmax3(mm[0], mm[1], mm[2]), fmax3(mm[3], mm[4], mm[5]),
                           fmaxf(mm[6], mm[7]));
    const float m_new = fmaxf(st.m, mx * scale_log2);
    const bool need = m_new > st.m + kRescaleThreshold;
    const float corr = need ? fast_exp2(st.m - m_new) : 1.f;
    if (need) st.m = m_new;
    // a row that has seen no key yet keeps m = -inf and p = 0
    const float m_sub = st.m == -INFINITY ? 0.f : st.m;
    const uint64_t n2 = f2pack(-m_sub, -m_sub);
    uint64_t s2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
    for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const int c = half * 64 + 2 * i;
            float x0, x1;
            f2unpack(ffma2(f2pack(sv[c], sv[c + 1]), c2, n2), x0, x1);
            const float e0 = fast_exp2(x0), e1 = fast_exp2(x1);
            s2[i & 3] = fadd2(s2[i & 3], f2pack(e0, e1));
            pk[half][i] = pack_bf16x2(e0, e1);
        }
        tc::tmem_st32(s_addr + half * 32, pk[half]);
    }
    float t[8];
#pragma unroll
    for (int u = 0; u < 4; ++u) f2unpack(s2[u], t[2 * u], t[2 * u + 1]);
    st.l = st.l * corr + (((t[0] + t[1]) + (t[2] + t[3])) + ((t[4] + t[5]) + (t[6] + t[7])));
    st.lb *= corr;
    return corr;
}

// Sum of a tile's rounded p. Two mixed-precision additions for every pair of keys,
// for which the softmax has no free pipe: 5 to 8% of the time wherever they stand
// (packed 8K batch / packed 32K / d = 64 chunks / ragged trees, us). Ahead of the wait
// for the next S 166 / 4190 / 80 / 143; right behind the hand-over of P 168 / 4250 /
// 83 / 147 (kTreeAlt does that: the other spills, 21 us for 19 on short drafts); beside
// the exponentials 167 / 4230 / 85 / 148; widened by shift and mask and added in
// pairs there 173 / 4440 / 85 / 156; as products with ones on mma.sync 202 / 5680 /
// 103 / 199. O divided by l needs none, 153 / 3960 / 75 / 135, but its error is up to
// 1.2 times the bound of a weighted mean on short rows, and equal V rows do not come
// out as they are.
__device__ __forceinline__ float rounded_sum(const uint32_t (&pk)[2][32]) {
    float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 64; ++i) {
        t[2 * (i & 1)] = add_f32_bf16_lo(t[2 * (i & 1)], pk[i >> 5][i & 31]);
        t[2 * (i & 1) + 1] = add_f32_bf16_hi(t[2 * (i & 1) + 1], pk[i >> 5][i & 31]);
    }
    return (t[0] + t[1]) + (t[2] + t[3]);
}

// ---- output: 64 bytes of each of a warp's 32 rows, through shared memory so
// that four neighbouring lanes write one row's 64 bytes.
struct RowPtrs {
    uint8_t* p[4];  // rows lane / 4 + 8 * i of the warp (null: not written)
    __device__ RowPtrs(uint8_t* own, int lane) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            p[i] = reinterpret_cast<uint8_t*>(
                __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(own),
                            i * 8 + (lane >> 2)));
    }
};
__device__ __forceinline__ void store_rows(uint32_t stage, int lane, const uint4 (&v)[4],
                                           const RowPtrs& rows, int byte) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        st_shared_v4(stage + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4), v[i]);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = i * 8 + (lane >> 2);
        const uint4 x = ld_shared_v4(stage + r * 64 + (((lane & 3) ^ ((r >> 1) & 3)) << 4));
        if (rows.p[i]) *reinterpret_cast<uint4*>(rows.p[i] + byte + (lane & 3) * 16) = x;
    }
    __syncwarp();
}

template <int D, int kMode>
__global__ void __launch_bounds__(kThreads, 1)
    ragged_kernel(const __grid_constant__ CUtensorMap tmap_q,
                  const __grid_constant__ CUtensorMap tmap_k,
                  const __grid_constant__ CUtensorMap tmap_v,
                  const __grid_constant__ CUtensorMap tmap_kc,
                  const __grid_constant__ CUtensorMap tmap_vc, const Params p) {
    using Gm = Geo<D>;
    constexpr uint32_t kTileBytes = Gm::kTileBytes;
    constexpr bool kTree = kMode != kPrompts, kAlt = kMode == kTreeAlt;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Gm::kBarOff);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kNumBars);
    // set once a repaired V tile held a value that is not finite; never cleared
    volatile uint32_t* odd_values = tmem_slot + 1;
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    // (through uniform(): with the roles chosen by a value that the compiler
    // knows to be the same in a warp, addresses and descriptors are computed on
    // the uniform path; causal 8K 861 -> 820 us)
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        mbar_init(bar(bQFull), 1);
        mbar_init(bar(bQEmpty), 1);
        for (int s = 0; s < kRingSlots; ++s) {
            mbar_init(bar(bSlotFull + s), 1);
            mbar_init(bar(bSlotEmpty + s), 1);
        }
        for (int g = 0; g < 2; ++g) {
            mbar_init(bar(bSFull + g), 1);
            mbar_init(bar(bPFull + g), 4);
            mbar_init(bar(bODone + g), 1);
            mbar_init(bar(bFixAsk + g), 1);
            mbar_init(bar(bFixDone + g), 1);
        }
        for (int s = 0; s < kItemSlots; ++s) {
            mbar_init(bar(bItemFull + s), 1);
            mbar_init(bar(bItemEmpty + s), kItemReaders);
        }
        mbar_init(bar(bXch), 8);
        mbar_init(bar(bXchDone), 8);
        mbar_init(bar(bDrain), 1);
        *odd_values = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tc::tmem_alloc(smem_u32(tmem_slot), kTmemCols);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (threadIdx.x == 0) {
        tma_prefetch_desc(&tmap_q);
        tma_prefetch_desc(&tmap_k);
        tma_prefetch_desc(&tmap_v);
        if (kTree) {
            tma_prefetch_desc(&tmap_kc);
            tma_prefetch_desc(&tmap_vc);
        }
    }
    // Nothing above touches global memory: it overlaps the previous kernel.
    grid_launch_dependents();
    grid_wait_primary();
    const uint32_t tmem = uniform(*tmem_slot);
    const int wg = warp >> 2;

    auto ring_wait = [&](int r) {
        return mbar_wait_bounded(bar(bSlotFull + r % kRingSlots), (r / kRingSlots) & 1, p.status);
    };

    if (wg == 0) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 104;" ::: "memory");
      // The item loops run on whole warps (see uniform()); lane 0 issues.
      auto wait_item = [&](int it) {
          return bool(__all_sync(0xffffffffu,
                                 mbar_wait_bounded(bar(bItemFull + it % kItemSlots),
                                                   (it / kItemSlots) & 1, p.status)));
      };
      auto item_at = [&](int it) {
          const Item w = read_item(smem_u32(smem + Gm::kItemOff + (it % kItemSlots) * sizeof(Item)));
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(bItemEmpty + it % kItemSlots));
          return w;
      };
      if (warp == 0) {
        // ------------------------------------------------------ TMA producer
        // A context streams through L2 once (for all members of a team at the same
        // time): it leaves room for what is read again, code and partial results
        // among it.
        const uint64_t once = l2_policy_evict_first();
        int r = 0, q_loads = 0;  // ring items and Q loads before this item
        int issued = 0;          // ring items this lane issued
        bool withheld = false;
        for (int it = 0;; ++it) {
            if (!wait_item(it)) break;
            const Item w = item_at(it);
            const int n = uniform(w.n);
            if (n < 0) break;
            if (n == 0) continue;  // no key: nothing to load
            bool alive = true;
            // Test hook: block 0 withholds its first Q copy, so every wait on
            // it runs out and reports kStatusTimeout (nothing faults or hangs).
            withheld = p.inject_timeout && blockIdx.x == 0 && q_loads == 0;
            if (lane == 0) {
                if (q_loads > 0)
                    alive = mbar_wait_bounded(bar(bQEmpty), (q_loads - 1) & 1, p.status);
                if (alive && !withheld) {
                    const int groups = !kAlt && w.tok0 + p.tok < w.T ? 2 : 1;
                    mbar_arrive_expect_tx(bar(bQFull), groups * Gm::kBoxes * p.G * p.tok * 128);
                    for (int g = 0; g < groups; ++g)
                        for (int hh = 0; hh < Gm::kBoxes; ++hh)
                            tma_load(smem_u32(smem + Gm::kQOff + g * kTileBytes) + hh * kBoxBytes,
                                     &tmap_q, hh * 64, w.kvh * p.G, w.q_row + w.tok0 + g * p.tok,
                                     bar(bQFull));
                }
#pragma unroll 1
                for (int i = 0; i < 2 * n && alive; ++i) {  // K_0, V_0, K_1, V_1, ...
                    const int ri = r + i, s = ri % kRingSlots;
                    if (ri >= kRingSlots)
                        alive = mbar_wait_bounded(bar(bSlotEmpty + s), ((ri / kRingSlots) - 1) & 1,
                                                  p.status);
                    if (!alive) break;
                    const int jj = w.j0 + (i >> 1);
                    const uint32_t dst = smem_u32(smem + Gm::kRingOff + s * kTileBytes);
                    mbar_arrive_expect_tx(bar(bSlotFull + s), kTileBytes);
                    for (int hh = 0; hh < Gm::kBoxes; ++hh) {
                        if (kTree && jj < w.c_t)
                            tma_load_3d(dst + hh * kBoxBytes, (i & 1) ? &tmap_vc : &tmap_kc,
                                        hh * 64, jj * BN, w.b * p.H_kv + w.kvh,
                                        bar(bSlotFull + s), once);
                        else
                            tma_load(dst + hh * kBoxBytes, (i & 1) ? &tmap_v : &tmap_k, hh * 64,
                                     w.k_row + (jj - w.c_t) * BN, w.kvh, bar(bSlotFull + s));
                    }
                    issued = ri + 1;
                }
            }
            if (!withheld) ++q_loads;
            if (!__all_sync(0xffffffffu, alive) || withheld) break;
            r += 2 * n;
        }
        // Every copy still in flight lands before the CTA exits.
        if (lane == 0) {
            if (q_loads > 0) mbar_wait_bounded(bar(bQFull), (q_loads - 1) & 1, p.status);
            for (int i = max(0, issued - kRingSlots); i < issued; ++i) ring_wait(i);
        }
      } else if (warp == 1) {
        // -------------------------------------------------------- MMA issuer
        const uint32_t idesc_s = tc::idesc_bf16_f32(BM, BN, false);
        const uint32_t idesc_pv = tc::idesc_bf16_f32(BM, D, true);
        auto slot_addr = [&](int i) {
            return smem_u32(smem + Gm::kRingOff + (i % kRingSlots) * kTileBytes);
        };
        const uint64_t qdesc0 = tc::sdesc_sw128(smem_u32(smem + Gm::kQOff), 16, 1024);
        const uint64_t qdesc1 = tc::sdesc_sw128(smem_u32(smem + Gm::kQOff + kTileBytes), 16, 1024);
        // S_g = Q K^T with K in ring item ri (kTreeAlt: both groups hold the same rows)
        auto issue_s = [&](int g, int ri) {
            const uint64_t qdesc = !kAlt && g ? qdesc1 : qdesc0;
            const uint64_t kdesc = tc::sdesc_sw128(slot_addr(ri), 16, 1024);
            const uint32_t qlo = uint32_t(qdesc), qhi = uint32_t(qdesc >> 32);
            const uint32_t klo = uint32_t(kdesc), khi = uint32_t(kdesc >> 32);
            const uint32_t dst = tmem + col_s_of(g);
            tc::mma_ss_lo<0>(dst, qlo, qhi, klo, khi, idesc_s);
#pragma unroll
            for (int kk = 1; kk < D / 16; ++kk) {
                const uint32_t o = ((kk >> 2) * kBoxBytes + (kk & 3) * 32) >> 4;
                tc::mma_ss_lo<1>(dst, qlo + o, qhi, klo + o, khi, idesc_s);
            }
            tc::commit(bar(bSFull + g));
        };
        // O_g (+)= P_g V over the first `keys` keys, V in ring item ri
        auto issue_pv = [&](int g, int ri, bool first, auto keys) {
            const uint64_t vdesc = tc::sdesc_sw128(slot_addr(ri), kBoxBytes, 1024);
            const uint32_t vlo = uint32_t(vdesc), vhi = uint32_t(vdesc >> 32);
            const uint32_t dst = tmem + col_o_of(g), src = tmem + col_s_of(g);
            tc::mma_ts_lo(dst, src, vlo, vhi, idesc_pv, first ? 0u : 1u);
#pragma unroll
            for (int ks = 1; ks < BN / 16; ++ks)
                if (ks * 16 < keys)
                    tc::mma_ts_lo(dst, src + ks * 8, vlo + uint32_t((ks * 2048) >> 4), vhi,
                                  idesc_pv, 1u);
        };
        constexpr std::integral_constant<int, BN> kAllKeys{};
        int r = 0, qi = 0;   // ring items and items with tiles before this item
        int t0 = 0, t1 = 0;  // tiles of group 0 and 1 before this item (their S and P phases)
        int asked = 0, fixed = 0;
        for (int it = 0;; ++it) {
            if (!wait_item(it)) break;
            const Item w = item_at(it);
            const int n = uniform(w.n);
            if (n < 0) break;
            if (n == 0) continue;
            const int n0 = kAlt ? (n + 1) >> 1 : uniform(w.n0), n1 = kAlt ? n >> 1 : uniform(w.n1);
            // tiles before `plain` need no repair and count with all their keys;
            // the last tile of a group (kPrompts), the context's last and the
            // drafted tokens' tile (decode_tree) may count with fewer
            const int plain = uniform(plain_tiles<kMode>(p, w, 0));
            const int j_own = uniform(w.c_t - w.j0);
            const int k0 = uniform(kMode == kPrompts ? tile_keys<kMode>(p, w, n0 - 1, 0) : w.n_own);
            const int k1 = uniform(kMode == kPrompts ? tile_keys<kMode>(p, w, n1 - 1, 1)
                                                     : w.ctx - (w.c_t - 1) * BN);
            auto keys_of = [&](int j, int g) {
                if (kMode == kPrompts) return j + 1 < (g ? n1 : n0) ? BN : (g ? k1 : k0);
                return j < plain ? BN : (j < j_own ? k1 : k0);
            };
            // The repair of V tile j may start once V tile j - 2, which had its
            // ring slot, has been seen here; at most two are asked for at a time.
            auto ask = [&](int j) {
                if (j >= plain && j < n) mbar_arrive(bar(bFixAsk + (asked++ & 1)));
            };
            auto repaired = [&](int j) {
                if (j < plain) return true;
                const int f = fixed++;
                return mbar_wait_bounded(bar(bFixDone + (f & 1)), (f >> 1) & 1, p.status);
            };
            bool alive = true;
            // Tiles that both groups run whole and that are not a group's last:
            // no conditions between the issues, which are on the critical path.
            const int fast = kAlt ? 0 : min(plain, min(n0, n1) - 1);
            if (lane == 0) {
                if (fast <= 0) {
                    ask(0);
                    ask(1);
                }
                alive = mbar_wait_bounded(bar(bQFull), qi & 1, p.status) && ring_wait(r);
            }
            if (lane == 0 && alive) {
              tc::fence_after_sync();
              if constexpr (kAlt) {
                issue_s(0, r);
                tc::commit(bar(bSlotEmpty + r % kRingSlots));
                if (n > 1) {
                    alive = ring_wait(r + 2);
                    if (alive) {
                        tc::fence_after_sync();
                        issue_s(1, r + 2);
                        tc::commit(bar(bSlotEmpty + (r + 2) % kRingSlots));
                    }
                }
                if (n <= 2) tc::commit(bar(bQEmpty));
#pragma unroll 1
                for (int j = 0; j < n && alive; ++j) {
                    const int g = j & 1, rv = r + 2 * j + 1;
                    alive = ring_wait(rv) && (j + 2 >= n || ring_wait(rv + 3)) && repaired(j);
                    if (!alive) break;
                    ask(j + 2);
                    alive = mbar_wait_bounded(bar(bPFull + g), ((g ? t1 : t0) + (j >> 1)) & 1,
                                              p.status);
                    if (!alive) break;
                    tc::fence_after_sync();
                    issue_pv(g, rv, j < 2, keys_of(j, 0));
                    tc::commit(bar(bSlotEmpty + rv % kRingSlots));
                    if (j + 2 < n) {
                        issue_s(g, rv + 3);  // K_{j+2}
                        tc::commit(bar(bSlotEmpty + (rv + 3) % kRingSlots));
                        if (j + 3 == n) tc::commit(bar(bQEmpty));
                    } else {
                        tc::commit(bar(bODone + g));
                    }
                }
              } else {
                // The last group that reads K_t / V_t is group 1 while it has tiles.
                auto last_user = [&](int t) { return t < n1 ? 1 : 0; };
                if (n0 > 0) issue_s(0, r);
                if (n1 > 0) issue_s(1, r);
                tc::commit(bar(bSlotEmpty + r % kRingSlots));
                if (n == 1) tc::commit(bar(bQEmpty));
                int j = 0;
#pragma unroll 1
                for (; j < fast && alive; ++j) {
                    const int rv = r + 2 * j + 1;  // V_j; K_{j+1} follows it
                    alive = ring_wait(rv) && ring_wait(rv + 1);
                    if (alive) alive = mbar_wait_bounded(bar(bPFull), (t0 + j) & 1, p.status);
                    if (!alive) break;
                    tc::fence_after_sync();
                    issue_pv(0, rv, j == 0, kAllKeys);
                    issue_s(0, rv + 1);
                    alive = mbar_wait_bounded(bar(bPFull + 1), (t1 + j) & 1, p.status);
                    if (!alive) break;
                    tc::fence_after_sync();
                    issue_pv(1, rv, j == 0, kAllKeys);
                    tc::commit(bar(bSlotEmpty + rv % kRingSlots));
                    issue_s(1, rv + 1);
                    tc::commit(bar(bSlotEmpty + (rv + 1) % kRingSlots));
                    if (j + 2 == n) tc::commit(bar(bQEmpty));
                }
                if (j > 0 && alive) {
                    ask(j);
                    ask(j + 1);
                }
#pragma unroll 1
                for (; j < n && alive; ++j) {
                    const int rv = r + 2 * j + 1;
                    alive = ring_wait(rv) && (j + 1 == n || ring_wait(rv + 1)) && repaired(j);
                    if (alive) ask(j + 2);
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        if (!alive) break;
                        const int n_g = g ? n1 : n0;
                        if (j >= n_g) continue;
                        alive = mbar_wait_bounded(bar(bPFull + g), ((g ? t1 : t0) + j) & 1,
                                                  p.status);
                        if (!alive) break;
                        tc::fence_after_sync();
                        issue_pv(g, rv, j == 0, keys_of(j, g));
                        if (g == last_user(j)) tc::commit(bar(bSlotEmpty + rv % kRingSlots));
                        if (j + 1 < n_g) {
                            issue_s(g, rv + 1);
                            if (g == last_user(j + 1)) {
                                tc::commit(bar(bSlotEmpty + (rv + 1) % kRingSlots));
                                if (j + 2 == n) tc::commit(bar(bQEmpty));
                            }
                        } else {
                            tc::commit(bar(bODone + g));
                        }
                    }
                }
              }
            }
            if (!__all_sync(0xffffffffu, alive)) break;
            ++qi;
            t0 += n0;
            t1 += n1;
            r += 2 * n;
        }
        // No product may still run when the tensor memory is freed.
        if (lane == 0) {
            tc::commit(bar(bDrain));
            mbar_wait_bounded(bar(bDrain), 0, p.status);
        }
      } else if (warp == 2) {
        // --------------------------------------------------------- scheduler
        Publisher pub{smem + Gm::kItemOff, bars, p.status};
        if constexpr (kTree)
            schedule_tree<kMode>(p, pub, lane);
        else
            schedule_prompts(p, reinterpret_cast<int2*>(smem + Gm::kSeqOff), pub, lane);
      } else {
        // ------------------------------------------------------------ repair
        // P is 0 at a key that a row does not see, but 0 * NaN is not: in the
        // tiles that reach past the first row's last key, V rows that nobody
        // sees are set to 0, and values that are not finite among the others
        // are too; the rows that do see those add them in the epilogue.
        bool alive = true;
        int r = 0, f = 0;
        for (int it = 0; alive; ++it) {
            if (!wait_item(it)) break;
            const Item w = item_at(it);
            if (w.n < 0) break;
            for (int j = plain_tiles<kMode>(p, w, 0); j < w.n && alive; ++j) {
                const Repair fix = repair_of<kMode>(p, w, w.j0 + j);
                const int ri = r + 2 * j + 1;
                alive = __all_sync(0xffffffffu,
                                   mbar_wait_bounded(bar(bFixAsk + (f & 1)), (f >> 1) & 1,
                                                     p.status)) &&
                        __all_sync(0xffffffffu, ring_wait(ri));
                if (!alive) break;
                const uint32_t tile = smem_u32(smem + Gm::kRingOff + (ri % kRingSlots) * kTileBytes);
                // Four 16-byte pieces a lane at a time; a piece without a halfword
                // whose exponent is all ones (x has none if no lane of
                // ~x & (0x7f80, 0x7f80) is 0) is left as it is.
                constexpr int kPieces = Gm::kBoxes * 8;  // pieces of a row
                auto at = [&](int i) {
                    const int row = i / kPieces, piece = i % kPieces;
                    return tile + (piece >> 3) * kBoxBytes + row * 128 + (piece & 7) * 16;
                };
                bool odd = false;
                const int scan_end = fix.keys * kPieces;
#pragma unroll 1
                for (int i0 = fix.seen * kPieces + lane; i0 < scan_end; i0 += 128) {
                    uint4 x[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        x[u] = i0 + 32 * u < scan_end ? ld_shared_v4(at(i0 + 32 * u))
                                                      : make_uint4(0, 0, 0, 0);
                    uint32_t hit = 0;
                    auto test = [&](uint32_t v) {
                        const uint32_t z = ~v & 0x7f807f80u;
                        hit |= (z - 0x00010001u) & ~z & 0x80008000u;
                    };
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        test(x[u].x);
                        test(x[u].y);
                        test(x[u].z);
                        test(x[u].w);
                    }
                    if (!hit) continue;
#pragma unroll 1
                    for (int u = 0; u < 4; ++u) {
                        if (i0 + 32 * u >= scan_end) break;
                        uint4 y = ld_shared_v4(at(i0 + 32 * u));
                        auto clean = [&](uint32_t v) {
                            if ((v & 0x7f80u) == 0x7f80u) v &= 0xffff0000u;
                            if ((v & 0x7f800000u) == 0x7f800000u) v &= 0xffffu;
                            return v;
                        };
                        const uint4 z = make_uint4(clean(y.x), clean(y.y), clean(y.z), clean(y.w));
                        if (z.x != y.x || z.y != y.y || z.z != y.z || z.w != y.w) {
                            st_shared_v4(at(i0 + 32 * u), z);
                            odd = true;
                        }
                    }
                }
#pragma unroll 1
                for (int i = scan_end + lane; i < fix.end * kPieces; i += 32)
                    st_shared_v4(at(i), make_uint4(0, 0, 0, 0));
                if (odd) *odd_values = 1;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(bFixDone + (f & 1)));
                ++f;
            }
            r += 2 * w.n;
        }
      }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;" ::: "memory");
        // ------------------------------------------------ softmax warpgroups
        const int g = wg - 1;
        const int quad = warp & 3;  // tensor-memory lanes 32 * quad .. + 31
        const int row = quad * 32 + lane;
        const int row_tok = row / p.G, row_head = row % p.G;
        const uint32_t lane_base = tmem + (uint32_t(quad * 32) << 16);
        const uint32_t col_s = col_s_of(g), col_o = col_o_of(g);
        const uint32_t stage = smem_u32(smem + Gm::kStageOff + (g * 4 + quad) * kStageBytes);
        float4* xch = reinterpret_cast<float4*>(smem + Gm::kXchOff);
        const uint64_t c2 = f2pack(p.scale_log2, p.scale_log2);
        bool alive = true;
        int tt = 0;              // tiles this group finished: its S phases
        int done0 = 0, done1 = 0;  // O_0, O_1 phases (kTreeAlt reads both, else its own)
        int xk = 0;
        auto wait_all = [&](int b, int phase) {
            return bool(__all_sync(0xffffffffu, mbar_wait_bounded(bar(b), phase & 1, p.status)));
        };
        for (int it = 0;; ++it) {
            // the warp gives the item's slot back when it is done with the item
            auto done_with_item = [&] {
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(bItemEmpty + it % kItemSlots));
            };
            alive = wait_all(bItemFull + it % kItemSlots, it / kItemSlots);
            if (!alive) break;
            const uint32_t item_addr =
                smem_u32(smem + Gm::kItemOff + (it % kItemSlots) * sizeof(Item));
            const Item w = read_item(item_addr);
            if (uniform(w.n) < 0) break;
            const int tok0 = kAlt ? w.tok0 : w.tok0 + g * p.tok;
            const int count = uniform(min(p.tok, w.T - tok0));  // tokens of this group
            if (count <= 0) {
                done_with_item();
                continue;
            }
            const int ng = uniform(kAlt ? (w.n + 1 - g) >> 1 : (g ? w.n1 : w.n0));
            // some row of this warp is valid
            const bool act = __any_sync(0xffffffffu, row_tok < count);
            if (kMode == kPrompts && ng == 0) {  // queries that see no key
                if (row_tok < count) {
                    const size_t orow = (size_t(w.q_row) + tok0 + row_tok) * p.H_q +
                                        w.kvh * p.G + row_head;
                    uint4* dst = reinterpret_cast<uint4*>(p.o + orow * D);
#pragma unroll 1
                    for (int i = 0; i < D / 8; ++i) dst[i] = make_uint4(0, 0, 0, 0);
                    if (p.lse) p.lse[orow] = -INFINITY;
                }
                done_with_item();
                continue;
            }
            // Keys of tile i that this row sees, for the tiles from `plain` on:
            // c < last - 128 i. The drafted tokens' tile goes by the bits.
            const int plain = uniform(plain_tiles<kMode>(p, w, kTree ? 0 : g));
            const int last = (kTree ? w.ctx : token_limit(p, w, tok0 + row_tok)) - w.j0 * BN;
            const int own_tile = kTree ? uniform(w.c_t - w.j0) : 0;
            uint32_t bits[4] = {0, 0, 0, 0};  // drafted tokens this row sees
            if (kTree && own_tile < w.n && row_tok < count) {
                const int t = tok0 + row_tok;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int rest = w.T - 32 * i;  // tokens from this word on
                    if (rest <= 0) break;
                    const uint32_t live = rest >= 32 ? 0xffffffffu : (1u << rest) - 1u;
                    const int upto = t + 1 - 32 * i;
                    bits[i] = live & (p.mask ? p.mask[(size_t(w.q_row) + t) * p.mask_words + i]
                                      : upto >= 32 ? 0xffffffffu
                                      : upto <= 0  ? 0u
                                                   : (1u << upto) - 1u);
                }
            }
            RowState st{-INFINITY, 0.f, 0.f};
            uint32_t pk[2][32];  // the last tile's P, not in lb yet
#pragma unroll 1
            for (int i = 0; i < ng && alive; ++i) {
                if (!kAlt && act && i > 0) st.lb += rounded_sum(pk);
                alive = wait_all(bSFull + g, tt + i);
                if (!alive) break;
                if (act) {
                    tc::fence_after_sync();
                    float sv[BN];
#pragma unroll
                    for (int c = 0; c < BN / 32; ++c) {
                        uint32_t x[32];
                        tc::tmem_ld32(lane_base + col_s + c * 32, x);
#pragma unroll
                        for (int e = 0; e < 32; ++e) sv[c * 32 + e] = __uint_as_float(x[e]);
                    }
                    tc::tmem_wait_ld();
                    const int j = kAlt ? 2 * i + g : i;
                    if (j >= plain) {
                        if (kTree && j >= own_tile) {
#pragma unroll
                            for (int c = 0; c < BN; ++c)
                                sv[c] = (bits[c >> 5] >> (c & 31)) & 1 ? sv[c] : -INFINITY;
                        } else {
                            const int lim = last - j * BN;
#pragma unroll
                            for (int c = 0; c < BN; ++c) sv[c] = c < lim ? sv[c] : -INFINITY;
                        }
                    }
                    const float corr = softmax_tile(sv, st, p.scale_log2, c2, lane_base + col_s, pk);
                    // O is complete here: this tile's S product was issued after
                    // the previous P V of the group, and they complete in order.
                    if (i > 0 && __any_sync(0xffffffffu, corr != 1.f)) {
                        const uint64_t corr2 = f2pack(corr, corr);
#pragma unroll
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t x[32];
                            tc::tmem_ld32(lane_base + col_o + c * 32, x);
                            tc::tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                float a0, a1;
                                f2unpack(fmul2(f2pack(__uint_as_float(x[2 * e]),
                                                      __uint_as_float(x[2 * e + 1])),
                                               corr2),
                                         a0, a1);
                                x[2 * e] = __float_as_uint(a0);
                                x[2 * e + 1] = __float_as_uint(a1);
                            }
                            tc::tmem_st32(lane_base + col_o + c * 32, x);
                        }
                    }
                    tc::tmem_wait_st();
                    tc::fence_before_sync();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(bPFull + g));
                if (kAlt && act) st.lb += rounded_sum(pk);
            }
            if (!alive) break;
            if (!kAlt && act && ng > 0) st.lb += rounded_sum(pk);
            tt += ng;

            // ---- epilogue. Every read of O completes before this warp's next
            // P arrive, which is what lets the next item overwrite O.
            float f0 = 1.f, f1 = 0.f;  // weights of O_0 and O_1 (kTreeAlt)
            const Item e = read_item(item_addr);
            const bool two = kAlt && uniform(e.n) > 1;
            if constexpr (kAlt) {
                xch[g * BM + row] = make_float4(st.m, st.l, st.lb, 0.f);
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(bXch));
                alive = wait_all(bXch, xk);
                if (!alive) break;
                const float4 a = xch[row], b = xch[BM + row];  // group 1 without tiles: -inf, 0, 0
                const float m = fmaxf(a.x, b.x), ms = m == -INFINITY ? 0.f : m;
                f0 = fast_exp2(a.x - ms);
                f1 = fast_exp2(b.x - ms);
                st.m = m;
                st.l = f0 * a.y + f1 * b.y;
                st.lb = f0 * a.z + f1 * b.z;
            }
            // (what does not need O comes before the wait for it)
            const int t = (kAlt ? e.tok0 : e.tok0 + g * p.tok) + row_tok;
            const bool valid = row_tok < p.tok && t < e.T;
            const bool own = e.j0 + e.n > e.c_t;  // the item has the row's own tokens
            const size_t orow = (size_t(e.q_row) + t) * p.H_q + e.kvh * p.G + row_head;
            const bool direct = !kTree || uniform(e.dst) < 0;
            // row of the item's token block
            const int prow = (t - e.tok0) * p.G + row_head;
            const RowPtrs rows(
                valid && direct ? reinterpret_cast<uint8_t*>(p.o + orow * D) : nullptr, lane);
            // the sums are 0 only for a row that saw no key (and NaN stays NaN)
            const float inv = st.lb == 0.f ? 0.f : 1.f / st.lb;
            if (valid && (!kAlt || g == 0)) {
                const float lse = st.l == 0.f ? -INFINITY : (st.m + log2f(st.l)) * kLn2;
                if (!direct)
                    p.part_lse[size_t(e.dst) * p.part_rows + prow] = lse;
                else if (p.lse)
                    p.lse[orow] = lse;
            }
            if constexpr (kAlt) {
                alive = wait_all(bODone, done0) && (!two || wait_all(bODone + 1, done1));
                done1 += two;
            } else {
                alive = wait_all(bODone + g, done0);
            }
            if (!alive) break;
            ++done0;
            if (act) {
                tc::fence_after_sync();
                const bool odd = *odd_values != 0 && own;
                const int c_begin = kAlt ? g * (D / 64) : 0;
                const int c_end = kAlt ? (g + 1) * (D / 64) : D / 32;
#pragma unroll 1
                for (int c = c_begin; c < c_end; ++c) {
                    uint32_t x[32];
                    tc::tmem_ld32(lane_base + (kAlt ? col_o_of(0) : col_o) + c * 32, x);
                    if constexpr (kAlt) {
                        if (two) {
                            uint32_t y[32];
                            tc::tmem_ld32(lane_base + col_o_of(1) + c * 32, y);
                            tc::tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                x[i] = __float_as_uint(f0 * __uint_as_float(x[i]) +
                                                       f1 * __uint_as_float(y[i]));
                        }
                    }
                    tc::tmem_wait_ld();
                    if (odd && valid) {
                        // values that are not finite among the keys that not every
                        // row sees: those that this row sees are added here
                        const int k_end = kTree ? e.n_own : token_limit(p, e, t);
#pragma unroll 1
                        for (int k = kTree ? 0 : group_first<kMode>(p, e, 0); k < k_end; ++k) {
                            if (kTree) {
                                const uint32_t word = k < 32 ? bits[0] : k < 64 ? bits[1]
                                                    : k < 96 ? bits[2] : bits[3];
                                if (!((word >> (k & 31)) & 1)) continue;
                            }
                            const uint16_t* vr = p.v + (int64_t(e.k_row) + k) * p.v_st +
                                                 e.kvh * p.v_sh + c * 32;
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                const uint32_t bf = vr[i];
                                if ((bf & 0x7f80u) == 0x7f80u)
                                    x[i] = __float_as_uint(__uint_as_float(x[i]) +
                                                           __uint_as_float(bf << 16));
                            }
                        }
                    }
                    if (direct) {
                        uint4 v[4];
                        uint32_t* u = reinterpret_cast<uint32_t*>(v);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            u[i] = pack_bf16x2(__uint_as_float(x[2 * i]) * inv,
                                               __uint_as_float(x[2 * i + 1]) * inv);
                        store_rows(stage, lane, v, rows, c * 64);
                    } else if (valid) {
                        float4* dst = reinterpret_cast<float4*>(p.part_o) +
                                      (size_t(e.dst) * (D / 4) + c * 8) * p.part_rows + prow;
#pragma unroll
                        for (int h = 0; h < 8; ++h)
                            dst[size_t(h) * p.part_rows] =
                                make_float4(__uint_as_float(x[4 * h]) * inv,
                                            __uint_as_float(x[4 * h + 1]) * inv,
                                            __uint_as_float(x[4 * h + 2]) * inv,
                                            __uint_as_float(x[4 * h + 3]) * inv);
                    }
                }
            }
            if constexpr (kAlt) {
                // both groups have read O_0, O_1 and xch
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(bXchDone));
                alive = wait_all(bXchDone, xk);
                if (!alive) break;
                ++xk;
            }
            done_with_item();
        }
    }

    tc::fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, kTmemCols);
    }
}

// Folds the partial results of every unit that was cut, in key order:
//   lse = ln sum_i exp(lse_i),  O = sum_i exp(lse_i - lse) O_i.
// A warp takes 32 rows (one per lane) x 16 columns and kMergeBatch parts at a
// time with all their loads in flight. A unit cut into no more parts than that is
// merged by the 8 warps of a block for all columns at once; of more parts, two
// warps take 16 columns each and four a quarter of the parts each. Bound by the
// loads' latency. What it adds to a call in a graph: 7 drafts on 333 tokens 2.4 us,
// 26 drafts on 8K tokens (8 units in 17 parts, 14 MB) 5.6, a batch of 8 trees in 2 to
// 4 parts (23 MB) 12.3, two wide trees of 16 query heads to a KV head 19. (Every unit
// merged the second way: the batch 144.1 us in all, like this 143.4.)
constexpr int kMergeThreads = 256;
constexpr int kMergeBatch = 4;

template <int D>
__global__ void __launch_bounds__(kMergeThreads, 2) merge_kernel(const Params p) {
    __shared__ int list[kTreeCtas];       // CTAs that begin a unit that was cut
    __shared__ int4 infos[kTreeCtas];     // their part_info
    __shared__ int counts[kMergeThreads / 32];
    __shared__ float4 acc_s[kMergeThreads / 32][5][32];  // per warp: 4 x 4 columns; maximum, sum
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_launch_dependents();
    grid_wait_primary();
    const int ctas = p.n_teams * p.team;
    static_assert(kTreeCtas <= kMergeThreads, "one thread per CTA of the launch");
    const int4 mine_info =
        int(threadIdx.x) < ctas ? p.part_info[threadIdx.x] : make_int4(0, 0, 0, 0);
    const bool cut = mine_info.w > 0;
    const unsigned votes = __ballot_sync(0xffffffffu, cut);
    if (lane == 0) counts[warp] = __popc(votes);
    __syncthreads();
    int n = 0, mine = __popc(votes & ((1u << lane) - 1));
    for (int i = 0; i < kMergeThreads / 32; ++i) {
        if (i < warp) mine += counts[i];
        n += counts[i];
    }
    if (cut) {
        list[mine] = threadIdx.x;
        infos[mine] = mine_info;
    }
    __syncthreads();
    const int chunks = cdiv(p.part_rows, 32);
    constexpr int kPartWarps = kMergeThreads / 64;
    const int col_warp = warp & 1, part_warp = warp >> 1;
    for (int task = blockIdx.x; task < n * chunks * (D / 32); task += gridDim.x) {
        const int nth = task / (chunks * (D / 32)), c = list[nth];
        const int chunk = task / (D / 32) % chunks, quarter = task % (D / 32);
        const int4 info = infos[nth];
        const int r = chunk * 32 + lane, parts = info.w;
        // (these are the same for the whole block)
        const bool few = parts <= kMergeBatch;
        if (chunk * 32 >= info.y || (few && quarter > 0)) continue;
        // first group of 4 columns
        const int col4 = few ? warp * 4 : quarter * 8 + col_warp * 4;
        const bool valid = r < info.y && col4 < D / 4;
        // part i is that of CTA c + i * team: slot 2c + 1 for the first, 2c for the others
        auto slot = [&](int i) { return size_t(2 * (c + i * p.team) + (i == 0)); };
        float mx = -INFINITY, sum = 0.f;
        float4 acc[4];
        auto add = [&](float w, const float4* v) {
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                acc[h].x += w * v[h].x;
                acc[h].y += w * v[h].y;
                acc[h].z += w * v[h].z;
                acc[h].w += w * v[h].w;
            }
        };
        auto scale = [&](float f) {
            sum *= f;
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                acc[h].x *= f;
                acc[h].y *= f;
                acc[h].z *= f;
                acc[h].w *= f;
            }
        };
        // exp(lse - mx), 0 for a part that saw no key (-inf), whatever mx is
        auto weight = [&](float lse) {
            return lse == -INFINITY ? 0.f : exp2f((lse - mx) * kLog2e);
        };
#pragma unroll
        for (int h = 0; h < 4; ++h) acc[h] = make_float4(0.f, 0.f, 0.f, 0.f);
        const int step = few ? 1 : kPartWarps;
        for (int i0 = few ? 0 : part_warp; i0 < parts; i0 += step * kMergeBatch) {
            float lse[kMergeBatch];
            float4 v[kMergeBatch][4];
#pragma unroll
            for (int u = 0; u < kMergeBatch; ++u) {
                const int i = i0 + u * step;
                lse[u] = -INFINITY;
                if (i < parts && valid) {
                    lse[u] = p.part_lse[slot(i) * p.part_rows + r];
                    const float4* src = reinterpret_cast<const float4*>(p.part_o) +
                                        (slot(i) * (D / 4) + col4) * p.part_rows + r;
#pragma unroll
                    for (int h = 0; h < 4; ++h) v[u][h] = src[size_t(h) * p.part_rows];
                } else {
#pragma unroll
                    for (int h = 0; h < 4; ++h) v[u][h] = make_float4(0.f, 0.f, 0.f, 0.f);
                }
            }
            float m = mx;
#pragma unroll
            for (int u = 0; u < kMergeBatch; ++u) m = fmaxf(m, lse[u]);
            const float f = mx == -INFINITY ? 0.f : exp2f((mx - m) * kLog2e);
            mx = m;
            scale(f);
#pragma unroll
            for (int u = 0; u < kMergeBatch; ++u) {
                const float w = weight(lse[u]);
                sum += w;
                add(w, v[u]);
            }
        }
        if (!few) {
#pragma unroll
            for (int h = 0; h < 4; ++h) acc_s[warp][h][lane] = acc[h];
            acc_s[warp][4][lane] = make_float4(mx, sum, 0.f, 0.f);
            __syncthreads();
            if (part_warp == 0 && valid) {
                const float own = mx;
                for (int k = 1; k < kPartWarps; ++k)
                    mx = fmaxf(mx, acc_s[2 * k + col_warp][4][lane].x);
                scale(own == -INFINITY ? 0.f : exp2f((own - mx) * kLog2e));
#pragma unroll
                for (int k = 1; k < kPartWarps; ++k) {
                    const float4 ms = acc_s[2 * k + col_warp][4][lane];
                    const float w = weight(ms.x);
                    float4 v[4];
#pragma unroll
                    for (int h = 0; h < 4; ++h) v[h] = acc_s[2 * k + col_warp][h][lane];
                    sum += w * ms.y;
                    add(w, v);
                }
            }
            __syncthreads();  // acc_s is free again
        }
        if (valid && (few || part_warp == 0)) {
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            const size_t orow = (size_t(info.x) + r / p.G) * p.H_q + info.z * p.G + r % p.G;
            uint4* out = reinterpret_cast<uint4*>(p.o + orow * D + col4 * 4);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float4 a = acc[2 * h], b = acc[2 * h + 1];
                out[h] = make_uint4(pack_bf16x2(a.x * inv, a.y * inv),
                                    pack_bf16x2(a.z * inv, a.w * inv),
                                    pack_bf16x2(b.x * inv, b.y * inv),
                                    pack_bf16x2(b.z * inv, b.w * inv));
            }
            if (col4 == 0 && p.lse) p.lse[orow] = sum == 0.f ? -INFINITY : mx + logf(sum);
        }
    }
}

// ------------------------------------------------------------------ host side

template <typename... A>
cudaError_t launch(void (*kern)(A...), unsigned grid, int threads, size_t smem,
                   cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    // The grid may start while the previous kernel of the stream finishes; it
    // reads no global memory before griddepcontrol.wait.
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

struct Maps {
    CUtensorMap q, k, v, kc, vc;
};

template <int D, int kMode>
int launch_ragged(const Maps& m, const Params& p, int ctas, cudaStream_t stream) {
    auto kern = ragged_kernel<D, kMode>;
    static std::atomic<uint64_t> attr_done{0};
    const int dev = current_device();
    if (device_attrs_pending(attr_done, dev)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Geo<D>::kSmemBytes) != cudaSuccess)
            return GQA_ERR_CUDA;
        device_attrs_mark(attr_done, dev);
    }
    return launch(kern, unsigned(ctas), kThreads, Geo<D>::kSmemBytes, stream, m.q, m.k, m.v, m.kc,
                  m.vc, p) == cudaSuccess
               ? GQA_OK
               : GQA_ERR_CUDA;
}

// Tensor maps of the packed operands: Q in boxes of tok tokens x G heads, K
// and V in boxes of 128 tokens of one head.
bool packed_maps(Maps& m, const Params& p, const uint16_t* q, const uint16_t* k, const uint16_t* v,
                 int d, int64_t q_st, int64_t q_sh, int64_t k_st, int64_t k_sh, int64_t v_st,
                 int64_t v_sh) {
    // a dimension of size 1 has no stride of its own
    auto fix = [](int64_t s, int64_t n) { return n > 1 ? uint64_t(s) : uint64_t(8); };
    if (encode_tmap_3d_bf16_strided(&m.q, q, d, p.H_q, p.total_q, fix(q_sh, p.H_q),
                                    fix(q_st, p.total_q), p.G, p.tok) != cudaSuccess)
        return false;
    m.k = m.v = m.kc = m.vc = m.q;  // never read unless set
    if (p.total_k == 0) return true;
    return encode_tmap_3d_bf16_strided(&m.k, k, d, p.total_k, p.H_kv, fix(k_st, p.total_k),
                                       fix(k_sh, p.H_kv), BN, 1) == cudaSuccess &&
           encode_tmap_3d_bf16_strided(&m.v, v, d, p.total_k, p.H_kv, fix(v_st, p.total_k),
                                       fix(v_sh, p.H_kv), BN, 1) == cudaSuccess;
}

// CTAs of a decode_tree launch work in teams of one per block of 2 * tok
// drafted tokens.
struct TreePlan {
    int tok, team, part_rows;
    bool alt;
};
TreePlan tree_plan(int G, int max_tokens) {
    TreePlan t;
    t.tok = BM / G;
    t.alt = max_tokens <= t.tok;
    t.team = t.alt ? 1 : (max_tokens + 2 * t.tok - 1) / (2 * t.tok);
    t.part_rows = (max_tokens < 2 * t.tok ? max_tokens : 2 * t.tok) * G;
    return t;
}

bool bad_strides(int64_t st, int64_t sh, int64_t tokens, int heads) {
    // TMA strides are multiples of 16 bytes below 2^40
    const int64_t lim = int64_t(1) << 39;
    if (heads > 1 && (sh <= 0 || sh >= lim)) return true;
    return tokens > 1 && (st <= 0 || st >= lim);
}
bool odd_strides(int64_t st, int64_t sh, int64_t tokens, int heads) {
    return ((tokens > 1 ? st : 0) | (heads > 1 ? sh : 0)) & 7;
}

int check_common(const void* q, const void* k, const void* v, const void* o, const void* lse,
                 int B, int H_q, int H_kv, int d, float scale) {
    if (B < 0 || B > 65535 || H_q <= 0 || H_kv <= 0) return GQA_ERR_INVALID_ARG;
    // scale > 0: the row maximum is taken over the raw scores
    if (H_q % H_kv != 0 || !isfinite(scale) || !(scale > 0.f)) return GQA_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return GQA_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) ||
        (reinterpret_cast<uintptr_t>(lse) & 3u))
        return GQA_ERR_MISALIGNED;
    return GQA_OK;
}

// ------------------------------------------------------------ cache append

struct AppendParams {
    uint16_t *kc, *vc;
    const uint16_t *k, *v;
    const int32_t *cu, *starts, *index;
    unsigned* status;
    int64_t k_st, k_sh, v_st, v_sh;
    int B, H_kv, d, S_max, total, total_new;
};

// One warp per entry: K and V of one token, every head, four 16-byte pieces of
// each a lane at a time with all their loads in flight. A copy, bound by HBM (a
// packed step of 7205 tokens, 59 MB: 11.5 us against 8.7 at the copy rate) or,
// for a few tokens, by the chain launch, prefix sums, start, copy (2.7 us in a graph).
constexpr int kAppendWarps = 8;

template <int D>
__global__ void __launch_bounds__(kAppendWarps * 32) append_kernel(const AppendParams p) {
    grid_launch_dependents();
    grid_wait_primary();
    const int lane = threadIdx.x & 31;
    const int e = blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
    bool bad = false;
    if (blockIdx.x == 0 && p.cu) {  // bad prefix sums are reported by the first block
#pragma unroll 1
        for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
            int first, n;
            row_range(p.cu, p.B, p.total, b, first, n, bad);
        }
    }
    // the entry's row: the last b with cu[b] <= e, by 32 probes at a time
    int b = 0, i = 0;
    bool mine = e < p.total;
    if (!p.cu) {
        const int per = p.total / p.B;
        if (mine) {
            b = e / per;
            i = e - b * per;
        }
    } else if (mine) {
        int lo = 0, hi = p.B;  // cu[lo] <= e (or lo = 0), the answer below hi
        while (hi - lo > 1) {
            const int step = cdiv(hi - lo, 32);
            const int at = lo + lane * step;
            const unsigned le = __ballot_sync(0xffffffffu, at < hi && p.cu[at] <= e);
            const int k = le ? 31 - __clz(le) : 0;
            lo += k * step;
            hi = min(hi, lo + step);
        }
        b = lo;
        int first, n;
        bool dummy = false;
        row_range(p.cu, p.B, p.total, b, first, n, dummy);
        i = e - first;
        mine = i >= 0 && i < n;  // (else it lies before the first or behind the last row)
    }
    if (mine) {
        const int64_t slot = int64_t(p.starts[b]) + i;
        const int src = p.index ? p.index[e] : e;
        if (slot < 0 || slot >= p.S_max || src < 0 || src >= p.total_new) {
            bad = true;
        } else {
            constexpr int kPieces = D / 8, kBatch = 4;
            const uint16_t* k_src = p.k + src * p.k_st;
            const uint16_t* v_src = p.v + src * p.v_st;
            const size_t base = (size_t(b) * p.H_kv * p.S_max + slot) * D;
            const size_t head = size_t(p.S_max) * D;
            const int n = p.H_kv * kPieces;
#pragma unroll 1
            for (int v0 = lane; v0 < n; v0 += 32 * kBatch) {
                uint4 kx[kBatch], vx[kBatch];
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const int v = v0 + 32 * u;
                    if (v >= n) break;
                    const int h = v / kPieces, c = v % kPieces * 8;
                    kx[u] = *reinterpret_cast<const uint4*>(k_src + h * p.k_sh + c);
                    vx[u] = *reinterpret_cast<const uint4*>(v_src + h * p.v_sh + c);
                }
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const int v = v0 + 32 * u;
                    if (v >= n) break;
                    const size_t dst = base + v / kPieces * head + v % kPieces * 8;
                    *reinterpret_cast<uint4*>(p.kc + dst) = kx[u];
                    *reinterpret_cast<uint4*>(p.vc + dst) = vx[u];
                }
            }
        }
    }
    if (bad) atomicOr(p.status, kStatusBadSeqlen);
}

}  // namespace ragged
}  // namespace gqa

using namespace gqa;

extern "C" int gqa_attn_prefill_packed(const uint16_t* q, const uint16_t* k, const uint16_t* v,
                                       uint16_t* o, float* lse, const int32_t* cu_q,
                                       const int32_t* cu_k, int B, int H_q, int H_kv, int d,
                                       int total_q, int total_k, int64_t q_stride_t,
                                       int64_t q_stride_h, int64_t k_stride_t,
                                       int64_t k_stride_h, int64_t v_stride_t,
                                       int64_t v_stride_h, int causal, float scale,
                                       cudaStream_t stream) {
    using namespace ragged;
    const int rc = check_common(q, k, v, o, lse, B, H_q, H_kv, d, scale);
    if (rc != GQA_OK) return rc;
    if (!cu_q || total_q < 0 || total_k < 0 || (total_q > 0 && (!q || !o)) ||
        (total_k > 0 && (!k || !v)) || (!cu_k && total_k != total_q))
        return GQA_ERR_INVALID_ARG;
    if (H_q / H_kv > 128) return GQA_ERR_UNSUPPORTED;
    if (bad_strides(q_stride_t, q_stride_h, total_q, H_q) ||
        bad_strides(k_stride_t, k_stride_h, total_k, H_kv) ||
        bad_strides(v_stride_t, v_stride_h, total_k, H_kv))
        return GQA_ERR_INVALID_ARG;
    if (odd_strides(q_stride_t, q_stride_h, total_q, H_q) ||
        odd_strides(k_stride_t, k_stride_h, total_k, H_kv) ||
        odd_strides(v_stride_t, v_stride_h, total_k, H_kv) ||
        (reinterpret_cast<uintptr_t>(cu_q) & 3u) ||
        (reinterpret_cast<uintptr_t>(cu_k) & 3u))
        return GQA_ERR_MISALIGNED;
    if (B == 0 || total_q == 0) return GQA_OK;
    const int sms = num_sms();
    Params p{};
    p.v = v; p.o = o; p.lse = lse;
    p.cu_q = cu_q; p.cu_k = cu_k;
    p.status = status_word();
    if (!p.status || sms <= 0) return GQA_ERR_CUDA;
    p.v_st = v_stride_t; p.v_sh = v_stride_h;
    p.B = B; p.H_q = H_q; p.H_kv = H_kv; p.G = H_q / H_kv; p.total_q = total_q; p.total_k = total_k;
    p.causal = causal != 0;
    p.tok = BM / p.G;
    p.scale_log2 = scale * kLog2e;
    p.inject_timeout = take_injected_timeout() ? 1 : 0;
    // at most this many blocks, however the tokens are spread over the rows
    const int64_t blocks = int64_t(total_q) / (2 * p.tok) + (B < total_q ? B : total_q);
    const int ctas = int(blocks * H_kv < sms ? blocks * H_kv : sms);
    p.max_blocks = int(blocks);  // (below 2^31: total_q / 2 + 65535 at most)
    Maps m;
    if (!packed_maps(m, p, q, k, v, d, q_stride_t, q_stride_h, k_stride_t, k_stride_h, v_stride_t,
                     v_stride_h))
        return GQA_ERR_CUDA;
    return d == 128 ? launch_ragged<128, kPrompts>(m, p, ctas, stream)
                    : launch_ragged<64, kPrompts>(m, p, ctas, stream);
}

extern "C" size_t gqa_attn_decode_tree_workspace_size(int H_q, int H_kv, int d, int max_tokens) {
    if (H_q <= 0 || H_kv <= 0 || H_q % H_kv || (d != 64 && d != 128) || max_tokens < 1 ||
        max_tokens > ragged::kMaxTreeTokens || H_q / H_kv > 16)
        return 0;
    const ragged::TreePlan t = ragged::tree_plan(H_q / H_kv, max_tokens);
    // a description and two slots per CTA: fp32 O and lse of part_rows rows
    return size_t(ragged::kTreeCtas) * (16 + size_t(2) * t.part_rows * (d + 1) * 4);
}

extern "C" int gqa_attn_decode_tree(
    const uint16_t* q, const uint16_t* k_new, const uint16_t* v_new, const uint16_t* k_cache,
    const uint16_t* v_cache, uint16_t* o, float* lse, const int32_t* cu_seqlens,
    const int32_t* context_lens, const int32_t* tree_mask, int mask_words, int B, int H_q,
    int H_kv, int d, int total, int max_tokens, int S_max, int64_t q_stride_t,
    int64_t q_stride_h, int64_t k_stride_t, int64_t k_stride_h, int64_t v_stride_t,
    int64_t v_stride_h, float scale, void* workspace, size_t workspace_bytes,
    cudaStream_t stream) {
    using namespace ragged;
    const int rc = check_common(q, k_new, v_new, o, lse, B, H_q, H_kv, d, scale);
    if (rc != GQA_OK) return rc;
    const bool empty = B == 0 || total == 0;  // nothing to do: the tensors may be null
    if ((!empty && (!q || !k_new || !v_new || !k_cache || !v_cache || !o || !context_lens)) ||
        total < 0 || S_max < 1 || max_tokens < 1 || (B > 0 && !cu_seqlens && total % B != 0) ||
        (B > 0 && !cu_seqlens && total / B > max_tokens) ||
        (tree_mask && int64_t(mask_words) * 32 < max_tokens))
        return GQA_ERR_INVALID_ARG;
    if (H_q / H_kv > 16 || max_tokens > kMaxTreeTokens ||
        int64_t(B) * H_kv * S_max >= (int64_t(1) << 31))
        return GQA_ERR_UNSUPPORTED;
    if (bad_strides(q_stride_t, q_stride_h, total, H_q) ||
        bad_strides(k_stride_t, k_stride_h, total, H_kv) ||
        bad_strides(v_stride_t, v_stride_h, total, H_kv))
        return GQA_ERR_INVALID_ARG;
    if (odd_strides(q_stride_t, q_stride_h, total, H_q) ||
        odd_strides(k_stride_t, k_stride_h, total, H_kv) ||
        odd_strides(v_stride_t, v_stride_h, total, H_kv) || !aligned16(k_cache) ||
        !aligned16(v_cache) ||
        ((reinterpret_cast<uintptr_t>(cu_seqlens) | reinterpret_cast<uintptr_t>(context_lens) |
          reinterpret_cast<uintptr_t>(tree_mask)) & 3u))
        return GQA_ERR_MISALIGNED;
    if (!empty && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
        workspace_bytes < gqa_attn_decode_tree_workspace_size(H_q, H_kv, d, max_tokens)))
        return GQA_ERR_WORKSPACE;
    if (empty) return GQA_OK;
    const int sms = num_sms();
    const TreePlan plan = tree_plan(H_q / H_kv, max_tokens);
    Params p{};
    p.v = v_new; p.o = o; p.lse = lse;
    p.cu_q = cu_seqlens; p.ctx = context_lens;
    p.mask = reinterpret_cast<const uint32_t*>(tree_mask);
    p.status = status_word();
    if (!p.status || sms <= 0) return GQA_ERR_CUDA;
    p.v_st = v_stride_t; p.v_sh = v_stride_h;
    p.B = B; p.H_q = H_q; p.H_kv = H_kv; p.G = H_q / H_kv; p.total_q = total; p.total_k = total;
    p.S_max = S_max; p.max_tokens = max_tokens; p.mask_words = mask_words;
    p.causal = 1;
    p.tok = plan.tok; p.team = plan.team; p.part_rows = plan.part_rows;
    p.scale_log2 = scale * kLog2e;
    p.inject_timeout = take_injected_timeout() ? 1 : 0;
    // no more teams than there can be tiles, or units that are not cut
    const int64_t row_tiles = (int64_t(S_max) + BN - 1) / BN + 1;
    p.whole = row_tiles <= kWholeTiles;
    const int64_t shares = int64_t(B) * H_kv * (p.whole ? 1 : row_tiles);
    const int most = (sms < kTreeCtas ? sms : kTreeCtas) / plan.team;
    p.n_teams = int(shares < most ? shares : most < 1 ? 1 : most);
    const int ctas = p.n_teams * plan.team;
    p.part_info = static_cast<int4*>(workspace);
    p.part_o = reinterpret_cast<float*>(p.part_info + kTreeCtas);
    p.part_lse = p.part_o + size_t(2) * ctas * p.part_rows * d;
    Maps m;
    if (!packed_maps(m, p, q, k_new, v_new, d, q_stride_t, q_stride_h, k_stride_t, k_stride_h,
                     v_stride_t, v_stride_h) ||
        encode_tmap_3d_bf16(&m.kc, k_cache, d, S_max, uint64_t(B) * H_kv, 64, BN,
                            CU_TENSOR_MAP_SWIZZLE_128B) != cudaSuccess ||
        encode_tmap_3d_bf16(&m.vc, v_cache, d, S_max, uint64_t(B) * H_kv, 64, BN,
                            CU_TENSOR_MAP_SWIZZLE_128B) != cudaSuccess)
        return GQA_ERR_CUDA;
    int rl;
    if (d == 128)
        rl = plan.alt ? launch_ragged<128, kTreeAlt>(m, p, ctas, stream)
                      : launch_ragged<128, kTreePair>(m, p, ctas, stream);
    else
        rl = plan.alt ? launch_ragged<64, kTreeAlt>(m, p, ctas, stream)
                      : launch_ragged<64, kTreePair>(m, p, ctas, stream);
    if (rl != GQA_OK || p.whole || p.n_teams == 1) return rl;
    const int64_t tasks = int64_t(ctas) * ((p.part_rows + 31) / 32) * (d / 32);
    const unsigned grid = unsigned(tasks < 2 * kTreeCtas ? tasks : 2 * kTreeCtas);
    return launch(d == 128 ? merge_kernel<128> : merge_kernel<64>, grid, kMergeThreads, 0, stream,
                  p) == cudaSuccess
               ? GQA_OK
               : GQA_ERR_CUDA;
}

extern "C" int gqa_attn_cache_append(uint16_t* k_cache, uint16_t* v_cache, const uint16_t* k_new,
                                     const uint16_t* v_new, const int32_t* cu_seqlens,
                                     const int32_t* starts, const int32_t* index, int B,
                                     int H_kv, int d, int S_max, int total, int total_new,
                                     int64_t k_stride_t, int64_t k_stride_h, int64_t v_stride_t,
                                     int64_t v_stride_h, cudaStream_t stream) {
    using namespace ragged;
    const bool empty = B == 0 || total == 0;
    if ((!empty && (!k_cache || !v_cache || !starts)) || B < 0 || B > 65535 || H_kv <= 0 ||
        S_max < 1 || total < 0 || total_new < 0 || (total_new > 0 && (!k_new || !v_new)) ||
        (!index && total > total_new) || (B > 0 && !cu_seqlens && total % B != 0))
        return GQA_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return GQA_ERR_UNSUPPORTED;
    if (int64_t(B) * H_kv * S_max >= (int64_t(1) << 31)) return GQA_ERR_UNSUPPORTED;
    if (bad_strides(k_stride_t, k_stride_h, total_new, H_kv) ||
        bad_strides(v_stride_t, v_stride_h, total_new, H_kv))
        return GQA_ERR_INVALID_ARG;
    if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_new) || !aligned16(v_new) ||
        odd_strides(k_stride_t, k_stride_h, total_new, H_kv) ||
        odd_strides(v_stride_t, v_stride_h, total_new, H_kv) ||
        ((reinterpret_cast<uintptr_t>(cu_seqlens) | reinterpret_cast<uintptr_t>(starts) |
          reinterpret_cast<uintptr_t>(index)) & 3u))
        return GQA_ERR_MISALIGNED;
    if (empty) return GQA_OK;
    unsigned* status = status_word();
    if (!status) return GQA_ERR_CUDA;
    const AppendParams p{k_cache, v_cache, k_new, v_new, cu_seqlens, starts, index, status,
                         k_stride_t, k_stride_h, v_stride_t, v_stride_h, B, H_kv, d, S_max,
                         total, total_new};
    return launch(d == 128 ? append_kernel<128> : append_kernel<64>,
                  unsigned((total + kAppendWarps - 1) / kAppendWarps), kAppendWarps * 32, 0,
                  stream, p) == cudaSuccess
               ? GQA_OK
               : GQA_ERR_CUDA;
}
