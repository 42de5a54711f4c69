// Attention of each request's block rows through a window: the last tokens
// before each row, and a few first ones that stay visible, of a shared prefix
// and the request's own tokens in the quantised cache.
//
// Mathematics.  As in block_attention.cu: row m (a block row of a query head)
// against tokens j, with 8-bit codes k~, v~ and scales ks, vs, has scores
// s_j = c ks_j (q . k~_j) in log2 units, and with any reference r
//   O = sum_j 2^(s_j - r) v_j,   l = sum_j 2^(s_j - r),   out = O / l,
//   lse = ln 2 (r + log2 l).
// q after a power of two per row and the codes are exact in fp16, scales and
// all sums are fp32, and P = 2^(s_j - r) (2^12 vs_j) is rounded once to fp16 (2^-11);
// for fp16 results, whose own rounding is no larger, its rest is rounded to a second
// fp16 and multiplied too, so that P counts to 2^-22.
// The reference is an integer that moves only when a P passes fp16's range.
//
// A row sees at most window + sinks tokens, so that an item (a request's kv head
// and up to 8 N rows of it) is short, and what bounds a call is reading the codes.
// The products therefore put tokens on their long side: a warp takes 16 tokens
// at a time, S^T = K Q^T and O^T = V^T P^T as 16 x 8 x 16 products whose first
// operand is the codes, converted in registers once for all the item's rows, and
// whose second one is N blocks of 8 rows.  (128-row tensor-core tiles would be
// filled to a sixteenth by 8 rows, and need the codes in shared memory as fp16.)
// Each warp walks its own tokens: every 4th chunk of 16 of the item, and of a
// cluster's share; copies by cp.async into a ring of its own, no barrier in the
// loop.  At the end the warps' parts meet in shared memory, and a cluster's
// through its distributed shared memory: one launch, no workspace.
//
// Layouts.  Lane (g, t) = (lane / 4, lane % 4).
//   S^T: the lane holds tokens g and g + 8 against rows 2 t and 2 t + 1.  Its part of the
//     keys is 16 codes of either token at a time, dimensions 16 t .. 16 t + 15 of each
//     64; the order of dimensions inside the sum is free, and q is laid out alike.
//   P^T goes from S^T's layout to a second operand's by a transposing move of 8 x 8 fp16.
//   O^T: the lane's part of the values is dimensions g DP/8 .. of tokens 2 t, 2 t + 1,
//     2 t + 8 and 2 t + 9; codes of two tokens are interleaved by byte permutations
//     before they are converted, so that it ends up with DP/8 consecutive dimensions
//     of rows 2 t and 2 t + 1.
// In shared memory 16-byte pieces of a chunk are permuted so that neither read
// meets itself in a bank.
//
// What bounds it.  With 8 rows an item, memory: 64 single tokens of 64 heads over 4,100 of
// their up to 20,000 tokens in 82 us (5.8 TB/s, 85% of a copy's rate).  With more, the
// issue of instructions, of which the half-rate integer pipe has half: some 320 a chunk for 16 rows (64
// of them conversions) and 1,250 a warp and item for its start and its joining; 256
// blocks of 1 to 6 rows of 32 heads over 1,040 tokens in 121 us (4.3 TB/s).  What
// counted on the way: bounds looked at only where a chunk is an edge (209 -> 167 us for
// those blocks), queries in shared memory and row blocks that do not exist left out
// (142), what the loop does not need out of its registers (130), divisions by
// multiplication and a joining without any (118; 121 with items in the order of packed
// rows).  Two chunks a step, for two chains of products at once, took 193 us: the loop
// leaves the instruction cache.  8, 12 or 16 warps an SM make no difference.
#include <type_traits>

#include <cooperative_groups.h>

#include "attention_common.cuh"
#include "tc_primitives.cuh"

namespace dspark {
namespace {

namespace cg = cooperative_groups;
using namespace tc;

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kChunk = 16;          // tokens of a warp's step
constexpr uint32_t kNoChunk = 0xffffffffu, kBadChunk = 0xfffffffeu;
constexpr int kMaxCluster = 8;
constexpr float kUnset = -1e30f;    // the reference before the first token: below all that count

// Division of numbers below 2^31 by a fixed one: x / d = (2 x m / 2^32) / 2^s with s = ceil(log2 d),
// m = ceil(2^(31 + s) / d).
struct Divider {
    uint32_t d, m, s;
    explicit Divider(int by = 1) : d((uint32_t)by), s(0) {
        while ((1ull << s) < d) ++s;
        m = (uint32_t)(((1ull << (31 + s)) + d - 1) / d);
    }
    __device__ __forceinline__ int div(int x) const { return (int)(__umulhi(2u * (uint32_t)x, m) >> s); }
    __device__ __forceinline__ int div(int x, int &rest) const {
        const int y = div(x);
        rest = x - y * (int)d;
        return y;
    }
};

struct WindowArgs {
    AttentionArgs a;
    Divider by_cluster, by_heads, by_group, by_page;     // the last: chunks a page
    bool listed;        // items in the order of packed rows (see slot_of), or one for each request and head, of which
                        // more row blocks follow in a loop
    float requests_a_slot;
    int cluster;        // blocks an item's tokens are split over
};

// N blocks of 8 rows a warp: blocks of 4 warps that an SM holds, and chunks of a warp under way
template <int DP, int N>
struct Shape {
    static constexpr int kAcc = DP / 64 * N;       // sixteens of a lane's sums
    static constexpr int kBlocks = kAcc <= 4 ? 4 : 3;
    static constexpr int kStages = 3;
};
template <int DP>
struct Slot {
    static constexpr uint32_t kV = kChunk * DP, kScales = 2 * kChunk * DP, kBytes = kScales + 128;
};
// Shared memory: the ring, in whose place the parts meet at the end; the queries
template <int DP, int N>
struct Smem {
    static constexpr uint32_t kRing = kWarps * Shape<DP, N>::kStages * Slot<DP>::kBytes;
    static constexpr uint32_t kJoin = (kWarps + 1) * 8 * N * (DP + 4) * 4;
    static constexpr uint32_t kQ = kRing > kJoin ? kRing : kJoin;
    static constexpr uint32_t kBytes = kQ + N * (DP / 32) * 512;
};

// (offsets that are known go into the instruction)
template <uint32_t kDst, uint32_t kSrc>
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %3], 16;" ::"r"(dst), "l"(src), "n"(kDst), "n"(kSrc) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}
// d += a b of 16 x 16 by 16 x 8 fp16
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
template <uint32_t kAt = 0>
__device__ __forceinline__ uint4 lds128(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4 + %5];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at), "n"(kAt));
    return v;
}
template <uint32_t kAt = 0>
__device__ __forceinline__ uint2 lds64(uint32_t at) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2 + %3];" : "=r"(v.x), "=r"(v.y) : "r"(at), "n"(kAt));
    return v;
}
template <uint32_t kAt = 0>
__device__ __forceinline__ float lds32(uint32_t at) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1 + %2];" : "=f"(v) : "r"(at), "n"(kAt));
    return v;
}

// Calls f with the numbers 0 .. n - 1 as constants.
template <int n, int i = 0, typename F>
__device__ __forceinline__ void each(F &&f) {
    if constexpr (i < n) {
        f(std::integral_constant<int, i>{});
        each<n, i + 1>(f);
    }
}

// Where 16-byte piece `c` of token `tok` is in a chunk.  DP = 128: a token a line of 128
// bytes; DP = 64: two.  The permutations keep apart, by banks, pieces t of tokens
// 2 p and 2 p + 1 (keys) and pieces of tokens 2 t (or 2 t + 1) that 8 lanes read at once (values).
template <int DP>
__device__ __forceinline__ uint32_t piece_at(uint32_t tok, uint32_t c) {
    if constexpr (DP == 128) return tok * 128u + ((c ^ (tok & 6u) ^ ((tok & 1u) << 2)) << 4);
    return (tok >> 1) * 128u + ((((tok & 1u) << 2 | c) ^ (tok & 6u)) << 4);
}

// The chunks of 16 tokens that an item's rows can see: of the prefix the first
// ones and the window's, of the request's own tokens the same.
struct Chunks {
    int n0, n1, n2, total;            // chunks of the prefix's first tokens, and of its window's, of the own first tokens
    int first1, first3;               // where the windows' begin
    __device__ __forceinline__ void find(int prefix, int sinks, int low, int end) {
        auto up = [](int x) { return (int)(((unsigned)x + kChunk - 1) / kChunk); };
        const int s = min(sinks, end);
        n0 = up(min(s, prefix));
        first1 = max(n0, low / kChunk);
        n1 = low < prefix ? max(0, up(min(end, prefix)) - first1) : 0;
        n2 = up(max(s - prefix, 0));
        first3 = max(n2, max(low - prefix, 0) / kChunk);
        total = n0 + n1 + n2 + max(0, up(max(end - prefix, 0)) - first3);
    }
    // chunk i: its number in its list; whether that is the own tokens'
    __device__ __forceinline__ int at(int i, bool &own) const {
        own = i >= n0 + n1;
        if (!own) return i < n0 ? i : first1 + i - n0;
        i -= n0 + n1;
        return i < n2 ? i : first3 + i - n2;
    }
};

// What one row sees: tokens in [low, end), and those before `sinks` (if before `end`);
// with a mask word the block's tokens by their bits.
struct RowRange {
    int low, end;
};
// An item as a warp sees it.  In shared memory, as the loop over chunks needs every register.
struct View {
    Chunks chunks;
    int low_min, low_max, end_min, end_max;     // of the rows' ranges
    int ctx;                                    // tokens before the block
    int m0, rows;                               // the item's rows: their first of the request's head's, how many
    int n, b, head;
    int64_t first;                              // packed row of the request's first
};

// Row blocks of requests of any lengths, each of `rows` rows: request b's first one has number
// row0[b] group / rows + b, which leaves at least as many numbers as it has blocks up to the next request's.
__device__ __forceinline__ int64_t slot_of(int64_t row0, int b, int group, int rows) {
    return (int64_t)((uint64_t)row0 * (uint64_t)group / (uint64_t)rows) + b;
}
// the largest b whose first number is `slot` or less, by the whole warp: 32 probes around `guess`, which nearly
// always hold it, else 32 a round; -1: none
__device__ __forceinline__ int find_slot(const int64_t *__restrict__ row0, int B, int64_t slot, int group, int rows, int guess,
                                         int lane) {
    int lo = max(min(guess - 16, B - 32), 0), n = B;
    const unsigned near = __ballot_sync(0xffffffffu, lo + lane < B && slot_of(row0[lo + lane], lo + lane, group, rows) <= slot);
    if (near != 0 && (near != 0xffffffffu || lo + 32 >= B)) return lo + 31 - __clz(near);
    lo = 0;
    while (true) {
        const int step = (n + 31) / 32, i = lane * step;
        const unsigned hits = __ballot_sync(0xffffffffu, i < n && slot_of(row0[lo + i], lo + i, group, rows) <= slot);
        if (hits == 0) return -1;
        const int k = 31 - __clz(hits);
        lo += k * step;
        n = min(step, n - k * step);
        if (step == 1) return lo;
    }
}

template <typename T, int kFormat, int DP, int N>
__global__ void __launch_bounds__(kThreads, Shape<DP, N>::kBlocks)
window_kernel(const __grid_constant__ WindowArgs w) {
    using Sl = Slot<DP>;
    constexpr int kStages = Shape<DP, N>::kStages, kRows = 8 * N, kHalves = DP / 64;
    constexpr int kCols = DP / 8;                 // dimensions of a lane's rows
    constexpr int kParts = std::is_same_v<T, __half> ? 2 : 1;   // fp16 parts of P
    constexpr int kPieces = DP / 16, kPer = 32 / kPieces;   // pieces of a token; tokens a copy takes at once
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ View views[kWarps];
    __shared__ RowRange ranges[kRows];
    __shared__ uint64_t words[kRows];
    __shared__ float2 stats[kWarps + 1][kRows];   // (r, l) of the warps, and of the block
    __shared__ float weights[kWarps][kRows];      // of the warps' parts in the block's
    __shared__ float lacks[kRows];                // what the rows' queries lack
    __shared__ int64_t row_place[kRows];          // of the rows' results, in heads

    const AttentionArgs &a = w.a;
    const dspark_kv_cache &c = a.cache;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int D = c.head_dim, H = c.n_kv_heads, group = a.n_q_heads / H;
    int split;
    int item = w.by_cluster.div((int)blockIdx.x, split);
    const int parts = w.cluster * kWarps, part = split * kWarps + warp;     // the warp takes every parts-th chunk
    const bool tree = a.row_mask != nullptr, causal = !tree && a.mask == DSPARK_MASK_CAUSAL;
    const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * kStages) * Sl::kBytes;
    View &view = views[warp];
    int m0;
    {
        int head, b;
        const int slot = w.by_heads.div(item, head);
        if (w.listed) {
            b = find_slot(a.rows.row0, a.rows.B, slot, group, kRows, (int)((float)slot * w.requests_a_slot), lane);
            if (b < 0) b = 0;
        } else {
            b = slot;
        }
        const Request q = load_request(a, b);
        if (lane == 0) view.b = b, view.head = head, view.first = q.first, view.n = q.n;
        // (no row0 that is no good may lead past a request's rows)
        const int64_t at = w.listed && q.rows_ok ? (slot - slot_of(q.first, b, group, kRows)) * kRows : 0;
        m0 = at >= 0 && at < (int64_t)q.n * group ? (int)at : q.n * group;
        if (blockIdx.x == 0)
            for (int i = threadIdx.x; i < a.rows.B; i += kThreads) {
                const Request x = load_request(a, i);
                if (!x.rows_ok || (x.n > 0 && !x.len_ok)) atomicOr(c.flags, kFlagBadLength);
            }
        if (!q.rows_ok || (q.n > 0 && !q.len_ok)) {     // no rows, or rows of NaN
            if (m0 == 0 && split == 0)
                for (int64_t i = threadIdx.x; i < (int64_t)q.n * group * (D / 8); i += kThreads) {
                    const int m = (int)(i / (D / 8)), blk = m / group;
                    const int64_t place = (q.first + blk) * a.n_q_heads + head * group + (m - blk * group);
                    reinterpret_cast<uint4 *>(static_cast<T *>(a.out) + place * D)[i - (int64_t)m * (D / 8)] =
                        make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
                    if (i == (int64_t)m * (D / 8) && a.lse) a.lse[place] = __int_as_float(0x7fffffff);
                }
            return;
        }
        if (lane == 0) view.ctx = a.prefix_len + q.len - q.n;
    }
    if (D != DP) {      // columns that no copy fills
        for (uint32_t i = threadIdx.x; i < Smem<DP, N>::kRing / 16; i += kThreads)
            reinterpret_cast<uint4 *>(smem)[i] = make_uint4(0, 0, 0, 0);
        __syncthreads();
    }
    __syncwarp();

#pragma unroll 1
    while (m0 < view.n * group) {
        // ---- what the rows see, a lane each
        int mine;
        {
            const int n = view.n, ctx = view.ctx, rows = min(kRows, n * group - m0);
            const int blk = w.by_group.div(m0 + min(lane, rows - 1));
            RowRange r{max(ctx + blk - a.window + 1, 0), causal ? ctx + blk + 1 : ctx + n};
            uint64_t word = 0;
            if (tree) {
                word = a.row_mask[view.first + blk];
                if (n < 64) word &= (1ull << n) - 1;
                r.low = max(ctx - max(a.window - __popcll(word), 0), 0);
            }
            if (warp == 0 && lane < kRows) ranges[lane] = r, words[lane] = word;
            const int low_min = __reduce_min_sync(0xffffffffu, r.low), low_max = __reduce_max_sync(0xffffffffu, r.low);
            const int end_min = tree ? ctx : __reduce_min_sync(0xffffffffu, r.end), end_max = __reduce_max_sync(0xffffffffu, r.end);
            Chunks chunks;
            chunks.find(a.prefix_len, a.sinks, low_min, end_max);
            mine = chunks.total > part ? (chunks.total - part + parts - 1) / parts : 0;
            if (lane == 0) {
                view.chunks = chunks;
                view.low_min = low_min, view.low_max = low_max, view.end_min = end_min, view.end_max = end_max;
                view.m0 = m0, view.rows = rows;
            }
            __syncwarp();
        }
        // ---- the warp's chunks: the tokens of chunk i that some row may see, [from, to), and where it begins
        auto bounds = [&](int i, int &pos0, int &from, int &to) {
            bool own;
            const int chunk = view.chunks.at(part + i * parts, own);
            pos0 = chunk * kChunk + (own ? a.prefix_len : 0);
            to = min(own ? view.end_max : min(a.prefix_len, view.end_max), pos0 + kChunk) - pos0;
            from = pos0 < a.sinks ? 0 : max(view.low_min - pos0, 0);
        };
        // Chunk i's number in the cache, in 16 head rows; bits (of the lanes' chunks) of those that some row sees only
        // in part or not at all.
        auto look = [&](int i, uint32_t &place, uint32_t &edges) {
            place = kNoChunk;
            bool edge = false;
            if (i < mine) {
                bool own;
                int in_page;
                const int chunk = view.chunks.at(part + i * parts, own), page_slot = w.by_page.div(chunk, in_page);
                const int page = own ? a.rows.block_table[(int64_t)view.b * a.rows.max_pages + page_slot] : a.prefix_pages[page_slot];
                place = page < 0 || page >= c.n_pages ? kBadChunk
                                                      : ((uint32_t)page * (uint32_t)H + (uint32_t)view.head) * w.by_page.d + (uint32_t)in_page;
                int pos0, from, to;
                bounds(i, pos0, from, to);
                edge = !(from == 0 && to == kChunk && pos0 + kChunk <= view.end_min &&
                         (pos0 >= view.low_max || pos0 + kChunk <= a.sinks));
            }
            edges = __ballot_sync(0xffffffffu, edge);
        };
        uint32_t places, edges, places_next = kNoChunk, edges_next = 0;    // of 32 chunks, a lane each, and of the next 32
        look(lane, places, edges);
        uint32_t slot_edge = 0, slot_bad = 0;   // bits of the ring's chunks that are an edge, and of those that have no page
        const int col = lane % kPieces, tok0 = lane / kPieces;
        // (the permutation repeats every 8 tokens: tokens tok0 + 4 j at DP = 128 have two, tok0 + 8 j at 64 one)
        const uint32_t put0 = piece_at<DP>((uint32_t)tok0, (uint32_t)col), put1 = piece_at<DP>((uint32_t)(tok0 + kPer), (uint32_t)col);
        const float *const scales = (lane < 4 ? c.k_scale : c.v_scale) + (lane & 3) * 4;
        auto copy = [&](uint32_t dst, uint64_t place, auto width) {
            const uint64_t at = place * (uint64_t)(kChunk * width) + (uint32_t)(tok0 * width + col * 16);
            const unsigned char *k = static_cast<const unsigned char *>(c.k) + at, *v = static_cast<const unsigned char *>(c.v) + at;
            if (lane < 8) cp_async16<Sl::kScales, 0>(dst + (uint32_t)lane * 16u, scales + place * kChunk);
            if (D != DP && col * 16 >= D) return;
            const uint32_t to0 = dst + put0, to1 = dst + put1;
            each<kChunk / kPer>([&](auto j) {
                constexpr uint32_t kTo = (decltype(j)::value >> 1) * 2 * kPer * DP;
                const uint32_t to = decltype(j)::value & 1 ? to1 : to0;
                if constexpr (std::is_same_v<decltype(width), int>) {
                    cp_async16<kTo, 0>(to, k + j * kPer * width);
                    cp_async16<kTo + Sl::kV, 0>(to, v + j * kPer * width);
                } else {
                    cp_async16<kTo, decltype(j)::value * kPer * DP>(to, k);
                    cp_async16<kTo + Sl::kV, decltype(j)::value * kPer * DP>(to, v);
                }
            });
        };
        auto load = [&](int i, uint32_t s) {
            if (i < mine) {
                if ((i & 31) == 0) {
                    if (i) places = places_next, edges = edges_next;
                    if (i + 32 < mine) look(i + 32 + lane, places_next, edges_next);
                }
                const uint32_t place = __shfl_sync(0xffffffffu, places, i & 31), bit = 1u << s;
                slot_edge = (edges >> (i & 31) & 1u) || place >= kBadChunk ? slot_edge | bit : slot_edge & ~bit;
                if (place < kBadChunk) {
                    slot_bad &= ~bit;
                    if (D == DP) copy(ring + s * Sl::kBytes, place, std::integral_constant<int, DP>{});
                    else copy(ring + s * Sl::kBytes, place, D);
                } else {
                    slot_bad |= bit;
                    if (lane == 0) atomicOr(c.flags, kFlagBadPage);
                }
            }
            cp_async_commit();
        };
#pragma unroll 1
        for (int i = 0; i < kStages - 1; ++i) load(i, (uint32_t)i);

        // ---- the queries, a block of 8 rows a warp: row g, dimensions 64 h + 16 t + 0 .. 15, in fp16 after a power of
        // two; what lane (g, t) needs of them for two products lies together
        for (int n = warp; n < N; n += kWarps) {
            const int r = 8 * n + g;
            int of;
            const int blk = w.by_group.div(m0 + r, of);
            const T *src = static_cast<const T *>(a.q) + (view.first + blk) * a.q_stride + (int64_t)(view.head * group + of) * D;
            uint4 in[2 * kHalves];
#pragma unroll
            for (int i = 0; i < 2 * kHalves; ++i) {
                const int d = 64 * (i >> 1) + 16 * t + 8 * (i & 1);
                in[i] = r < view.rows && d < D ? __ldg(reinterpret_cast<const uint4 *>(src + d)) : make_uint4(0, 0, 0, 0);
            }
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < 2 * kHalves; ++i) {
                // (two values a word: the 16-bit types' bits order like their values)
                const uint32_t m2 = 0x7fff7fffu, u = __vmaxu2(__vmaxu2(in[i].x & m2, in[i].y & m2), __vmaxu2(in[i].z & m2, in[i].w & m2));
                const float2 x = pair_to_float<T>(u);
                top = max(top, max(__float_as_uint(x.x), __float_as_uint(x.y)));
            }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int e2 = max((int)(top >> 23) - 127, -110);
            float mul = 1.f, f = 1.f;         // the largest element goes to [2^7, 2^8)
            if (top >= 0x7f800000u) mul = __int_as_float(0x7fffffff);
            else if (top != 0) {
                mul = __uint_as_float((uint32_t)(127 + 7 - e2) << 23);
                f = __uint_as_float((uint32_t)(127 - 7 + e2) << 23);
            }
            if (t == 0) lacks[r] = f;
#pragma unroll
            for (int i = 0; i < 2 * kHalves; ++i) {
                const uint32_t u[4] = {in[i].x, in[i].y, in[i].z, in[i].w};
                uint32_t h[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 x = pair_to_float<T>(u[e]);
                    h[e] = half_pair(x.x * mul, x.y * mul);
                }
                reinterpret_cast<uint4 *>(smem + Smem<DP, N>::kQ)[(n * 2 * kHalves + i) * 32 + lane] = make_uint4(h[0], h[1], h[2], h[3]);
            }
        }
        __syncthreads();

        // ---- the loop over chunks
        float o[N][DP / 16][4];
        float ref[N][2], l[N][2], lack[N][2];  // of rows 2 t and 2 t + 1 of each block
#pragma unroll
        for (int n = 0; n < N; ++n) {
#pragma unroll
            for (int i = 0; i < DP / 16; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
            ref[n][0] = ref[n][1] = kUnset;
            l[n][0] = l[n][1] = 0.f;
            lack[n][0] = lacks[8 * n + 2 * t], lack[n][1] = lacks[8 * n + 2 * t + 1];
        }
        const float up = a.scale * kLog2e;
        const uint32_t q_at = smem_u32(smem) + Smem<DP, N>::kQ + (uint32_t)lane * 16u;
        // places in a chunk of what the lane reads: keys of tokens g and g + 8 (8 lines on), its pieces 64 dimensions
        // apart; values of tokens 2 t, 2 t + 1 and of those 8 on
        uint32_t get_k[kHalves], get_v[2];
#pragma unroll
        for (int h = 0; h < kHalves; ++h) get_k[h] = piece_at<DP>((uint32_t)g, (uint32_t)(4 * h + t));
#pragma unroll
        for (int j = 0; j < 2; ++j)
            get_v[j] = Sl::kV + (DP == 128 ? piece_at<DP>((uint32_t)(2 * t + j), (uint32_t)g)
                                           : piece_at<DP>((uint32_t)(2 * t + j), (uint32_t)g >> 1) + ((uint32_t)g & 1u) * 8u);
        // (of the N blocks of rows the first M exist)
        auto walk = [&](auto blocks) {
            constexpr int M = decltype(blocks)::value;
            uint32_t s = 0;
#pragma unroll 1
            for (int i = 0; i < mine; ++i) {
                cp_async_wait<kStages - 2>();
                __syncwarp();
                load(i + kStages - 1, s == 0 ? kStages - 1 : s - 1);    // to the place that the chunk before has left
                const uint32_t src = ring + s * Sl::kBytes;
                const bool edge = slot_edge >> s & 1u;
                // scores
                float x[M][4];
#pragma unroll
                for (int n = 0; n < M; ++n) x[n][0] = x[n][1] = x[n][2] = x[n][3] = 0.f;
                each<kHalves>([&](auto hc) {
                    constexpr int h = decltype(hc)::value;
                    const uint4 lo = lds128(src + get_k[h]), hi = lds128<8 * DP>(src + get_k[h]);
                    const uint32_t kl[4] = {lo.x, lo.y, lo.z, lo.w}, kh[4] = {hi.x, hi.y, hi.z, hi.w};
                    each<2>([&](auto kc) {
                        constexpr int k = 2 * decltype(kc)::value;
                        __half2 f[4], e[4];
                        decode4<kFormat>(kl[k], f[0], f[1]);
                        decode4<kFormat>(kh[k], e[0], e[1]);
                        decode4<kFormat>(kl[k + 1], f[2], f[3]);
                        decode4<kFormat>(kh[k + 1], e[2], e[3]);
                        each<M>([&](auto nc) {
                            constexpr int n = decltype(nc)::value;
                            const uint4 u = lds128<(n * 2 * kHalves + 2 * h + (k >> 1)) * 512>(q_at);
                            mma16816(x[n], as_u32(f[0]), as_u32(e[0]), as_u32(f[1]), as_u32(e[1]), u.x, u.y);
                            mma16816(x[n], as_u32(f[2]), as_u32(e[2]), as_u32(f[3]), as_u32(e[3]), u.z, u.w);
                        });
                    });
                });
                // scales of tokens g and g + 8; one whose value scale (or page) is no number carries its NaN in the
                // key's alone: where it is masked, its zero weight must not become 0 times NaN
                float vs[2];
                const uint32_t scale_at = src + (uint32_t)g * 4u;
                each<2>([&](auto ec) {
                    constexpr int e = decltype(ec)::value;
                    const float kv = lds32<Sl::kScales + e * 32>(scale_at), vv = lds32<Sl::kScales + 64 + e * 32>(scale_at);
                    const bool good = vv <= 3.4028235e38f;
                    const float ks = good ? kv * up : __int_as_float(0x7fffffff);
                    vs[e] = good ? fminf(vv * kVUp, 3.4028235e38f) : 0.f;
#pragma unroll
                    for (int n = 0; n < M; ++n) x[n][2 * e] *= ks, x[n][2 * e + 1] *= ks;
                });
                if (edge) {     // scores that the row does not see: -inf
                    const bool bad = slot_bad >> s & 1u;
                    const int ctx = view.ctx;
                    int pos0, from, to;
                    bounds(i, pos0, from, to);
                    // what lies where no token is must not meet a weight of 0
#pragma unroll 1
                    for (int j = tok0; j < kChunk; j += kPer)
                        if (bad || j < from || j >= to)
                            st_shared_v4(src + Sl::kV + piece_at<DP>((uint32_t)j, (uint32_t)col), make_uint4(0, 0, 0, 0));
                    __syncwarp();
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int tok = g + 8 * e, pos = pos0 + tok;
                        const bool there = tok >= from && tok < to;
                        if (!there || bad) vs[e] = 0.f;
#pragma unroll
                        for (int n = 0; n < M; ++n)
#pragma unroll
                            for (int f = 0; f < 2; ++f) {
                                const RowRange r = ranges[8 * n + 2 * t + f];
                                bool sees = there && pos < r.end && (pos >= r.low || pos < a.sinks);
                                if (tree && pos >= ctx) sees = tok < to && (words[8 * n + 2 * t + f] >> (pos - ctx) & 1);
                                float &y = x[n][2 * e + f];
                                y = !sees ? -INFINITY : bad ? __int_as_float(0x7fffffff) : y;
                            }
                    }
                }
                // softmax terms and what they weigh the values' codes with; whether one of these, or a sum, passes its
                // bound
                uint32_t pk[M][kParts][2];
                float sum[M][2];
#pragma unroll 1
                for (bool again = false;; again = true) {
                    uint32_t past = 0;
                    float most = 0.f;
#pragma unroll
                    for (int n = 0; n < M; ++n) {
                        float p[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) p[e] = fast_exp2(fmaf(x[n][e], lack[n][e & 1], -ref[n][e & 1]));
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float x0 = p[2 * e] * vs[e], x1 = p[2 * e + 1] * vs[e];
                            pk[n][0][e] = half_pair(x0, x1);
                            if constexpr (kParts == 2) {
                                const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&pk[n][0][e]));
                                pk[n][1][e] = half_pair(x0 - h.x, x1 - h.y);
                            }
                        }
                        static_assert(kPast + 0x0400u == 0x8000u, "");
                        past |= __vmaxu2(pk[n][0][0], pk[n][0][1]) + 0x04000400u;       // kPast and more: a half's top bit
                        sum[n][0] = p[0] + p[2];
                        sum[n][1] = p[1] + p[3];
                        most = max3(most, sum[n][0], sum[n][1]);
                    }
                    if (again || !__any_sync(0xffffffffu, (past & 0x80008000u) || most > kSumMost)) break;
                    // the references move to the chunk's largest terms, where these lie above
                    const float v0 = fmaxf(fast_log2(vs[0]), kVLeast), v1 = fmaxf(fast_log2(vs[1]), kVLeast);
#pragma unroll
                    for (int n = 0; n < M; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float top = fmaxf(x[n][e] * lack[n][e] + v0, x[n][e + 2] * lack[n][e] + v1);
#pragma unroll
                            for (int d = 4; d < 32; d *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                            if (top == -INFINITY || !(top > ref[n][e] + kPeak)) continue;
                            const float r = ceilf(top) - kPeak;           // P <= 2^7
                            const float f = scale_down(1.f, ref[n][e] - r);
                            l[n][e] = scale_down(l[n][e], ref[n][e] - r);
                            ref[n][e] = r;
#pragma unroll
                            for (int k = 0; k < DP / 16; ++k) o[n][k][e] *= f, o[n][k][e + 2] *= f;
                        }
                }
#pragma unroll
                for (int n = 0; n < M; ++n) {
                    l[n][0] += sum[n][0];
                    l[n][1] += sum[n][1];
#pragma unroll
                    for (int i = 0; i < kParts; ++i) {
                        pk[n][i][0] = transpose8x8(pk[n][i][0]);
                        pk[n][i][1] = transpose8x8(pk[n][i][1]);
                    }
                }
                // outputs
                uint32_t vw[4][DP / 32];
                each<4>([&](auto jc) {
                    constexpr int j = decltype(jc)::value;
                    const uint32_t at = src + get_v[j & 1];
                    if constexpr (DP == 128) {
                        const uint4 v = lds128<(j >> 1) * 8 * DP>(at);
                        vw[j][0] = v.x, vw[j][1] = v.y, vw[j][2] = v.z, vw[j][3] = v.w;
                    } else {
                        const uint2 v = lds64<(j >> 1) * 8 * DP>(at);
                        vw[j][0] = v.x, vw[j][1] = v.y;
                    }
                });
#pragma unroll
                for (int k = 0; k < DP / 16; ++k) {
                    const uint32_t pick = (k & 1) ? 0x7362u : 0x5140u;
                    __half2 a0, a1, a2, a3;
                    decode4<kFormat>(__byte_perm(vw[0][k >> 1], vw[1][k >> 1], pick), a0, a1);
                    decode4<kFormat>(__byte_perm(vw[2][k >> 1], vw[3][k >> 1], pick), a2, a3);
#pragma unroll
                    for (int n = 0; n < M; ++n)
#pragma unroll
                        for (int i = 0; i < kParts; ++i)
                            mma16816(o[n][k], as_u32(a0), as_u32(a1), as_u32(a2), as_u32(a3), pk[n][i][0], pk[n][i][1]);
                }
                s = s + 1 == kStages ? 0 : s + 1;
            }
        };
        if (N == 3 && view.rows <= 8) walk(std::integral_constant<int, 1>{});
        else if (N > 1 && view.rows <= 8 * (N - 1)) walk(std::integral_constant<int, N == 1 ? 1 : N - 1>{});
        else walk(std::integral_constant<int, N>{});
        cp_async_wait<0>();

        // ---- the warps' parts join: [warp][row][dimension], the rows 4 floats apart from a power of two
        __syncthreads();
        float *parts_o = reinterpret_cast<float *>(smem);
        constexpr int kPitch = DP + 4;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            if (8 * n >= view.rows) break;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float sum = l[n][e];
#pragma unroll
                for (int d = 4; d < 32; d *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                const int row = 8 * n + 2 * t + e;
                if (g == 0) stats[warp][row] = make_float2(ref[n][e], sum);
                float *to = parts_o + (warp * kRows + row) * kPitch + g * kCols;
#pragma unroll
                for (int k = 0; k < DP / 16; k += 2)
                    *reinterpret_cast<float4 *>(to + 2 * k) = make_float4(o[n][k][e], o[n][k][e + 2], o[n][k + 1][e], o[n][k + 1][e + 2]);
            }
        }
        __syncthreads();
        // what a part's row counts in the join of `count` parts, whose references and sums `stat` gives (a part that
        // saw nothing: kUnset and 0, and its output is 0)
        auto weigh = [&](int count, auto stat, float &top, float &total, auto put) {
            top = kUnset;
            for (int i = 0; i < count; ++i) top = fmaxf(top, stat(i).x);
            total = 0.f;
            for (int i = 0; i < count; ++i) {
                const float2 st = stat(i);
                put(i, scale_down(1.f, st.x - top));
                total += scale_down(st.y, st.x - top);
            }
        };
        auto finish = [&](int r, float top, float total) {     // what a row's sums are multiplied by
            if (a.lse) a.lse[row_place[r]] = total == 0.f ? -INFINITY : kLn2 * (top + log2f(total));
            return total == 0.f ? 0.f : kVDown / total;
        };
        const int rows = view.rows;
        if (threadIdx.x < rows) {
            const int r = threadIdx.x;
            int of;
            const int blk = w.by_group.div(view.m0 + r, of);
            row_place[r] = (view.first + blk) * a.n_q_heads + view.head * group + of;
            float top, total, f[kWarps];
            weigh(kWarps, [&](int k) { return stats[k][r]; }, top, total, [&](int k, float x) { f[k] = x; });
            stats[kWarps][r] = make_float2(top, total);
            const float by = w.cluster == 1 ? finish(r, top, total) : 1.f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) weights[k][r] = f[k] * by;
        }
        __syncthreads();
        auto add = [](float4 &sum, const float4 &x, float f) { sum.x += x.x * f, sum.y += x.y * f, sum.z += x.z * f, sum.w += x.w * f; };
        auto store = [&](int r, int d, const float4 &x) {
            *reinterpret_cast<uint2 *>(static_cast<T *>(a.out) + row_place[r] * D + d) =
                make_uint2(float_to_pair<T>(x.x, x.y), float_to_pair<T>(x.z, x.w));
        };
        // a thread takes four dimensions of every kAtOnce-th row
        constexpr int kAtOnce = kThreads / (DP / 4);
        const int d = (int)threadIdx.x % (DP / 4) * 4;
        float *block_o = parts_o + kWarps * kRows * kPitch;
        for (int r = (int)threadIdx.x / (DP / 4); r < rows; r += kAtOnce) {
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < kWarps; ++k) add(sum, *reinterpret_cast<const float4 *>(parts_o + (k * kRows + r) * kPitch + d), weights[k][r]);
            if (w.cluster > 1) *reinterpret_cast<float4 *>(block_o + r * kPitch + d) = sum;
            else if (d < D) store(r, d, sum);
        }
        if (w.cluster > 1) {
            cg::cluster_group cluster = cg::this_cluster();
            cluster.sync();
            for (int r = split * kAtOnce + (int)threadIdx.x / (DP / 4); r < rows; r += w.cluster * kAtOnce) {
                float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
                float top, total;
                weigh(w.cluster, [&](int k) { return *cluster.map_shared_rank(&stats[kWarps][r], k); }, top, total,
                      [&](int k, float f) {
                          add(sum, *reinterpret_cast<const float4 *>(cluster.map_shared_rank(block_o, k) + r * kPitch + d), f);
                      });
                const float by = d == 0 ? finish(r, top, total) : total == 0.f ? 0.f : kVDown / total;
                sum.x *= by, sum.y *= by, sum.z *= by, sum.w *= by;
                if (d < D) store(r, d, sum);
            }
            cluster.sync();     // before another block's memory goes, or is written again
        }
        m0 = w.listed ? view.n * group : view.m0 + kRows;
        if (m0 >= view.n * group) break;
        __syncthreads();        // the ring, the ranges and the queries are the next rows'
        if (D != DP) {
            for (uint32_t i = threadIdx.x; i < Smem<DP, N>::kRing / 16; i += kThreads)
                reinterpret_cast<uint4 *>(smem)[i] = make_uint4(0, 0, 0, 0);
            __syncthreads();
        }
    }
}

// tokens of a request that its rows see at most (of an average block)
int64_t seen_tokens(const AttentionArgs &a) {
    const int64_t own = (int64_t)a.rows.max_pages * a.cache.page_size + a.prefix_len;
    const int64_t seen = (int64_t)a.window + a.sinks + a.rows.n_rows / a.rows.B;
    return own < seen ? own : seen;
}

template <typename T, int kFormat, int DP, int N>
cudaError_t launch_n(WindowArgs &w, cudaStream_t s) {
    static PerDeviceOnce once;
    auto *kernel = window_kernel<T, kFormat, DP, N>;
    constexpr size_t bytes = Smem<DP, N>::kBytes;
    cudaError_t e = once.run([&] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes); });
    if (e != cudaSuccess) return e;
    const AttentionArgs &a = w.a;
    const int group = a.n_q_heads / a.cache.n_kv_heads;
    // a row a request is what decoding has: no list is needed then (and none is looked through)
    w.listed = a.rows.n_rows > a.rows.B;
    // an item's tokens go to a cluster of up to 8 blocks while there are fewer blocks than SMs hold and a warp has
    // four chunks or more
    const int64_t items = w.listed ? (int64_t)a.rows.n_rows * group / (8 * N) + a.rows.B : a.rows.B;
    w.requests_a_slot = (float)a.rows.B / (float)items;
    int64_t blocks = items * a.cache.n_kv_heads;
    const int64_t chunks = seen_tokens(a) / kChunk;
    w.cluster = 1;
    while (w.cluster < kMaxCluster && blocks * w.cluster * 2 <= (int64_t)kNumSMs * Shape<DP, N>::kBlocks && chunks >= w.cluster * 2 * kWarps * 4)
        w.cluster *= 2;
    blocks *= w.cluster;
    w.by_cluster = Divider(w.cluster);
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = s;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)w.cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, w);
}

template <typename T, int kFormat, int DP>
cudaError_t launch_dp(WindowArgs &w, cudaStream_t s) {
    const int group = w.a.n_q_heads / w.a.cache.n_kv_heads;
    const int64_t rows = ((int64_t)w.a.rows.n_rows + w.a.rows.B - 1) / w.a.rows.B * group;
    if (rows <= 8) return launch_n<T, kFormat, DP, 1>(w, s);
    if (rows <= 16) return launch_n<T, kFormat, DP, 2>(w, s);
    return launch_n<T, kFormat, DP, 3>(w, s);
}

template <typename T>
cudaError_t launch_t(WindowArgs &w, cudaStream_t s) {
    const bool e4m3 = w.a.cache.format == DSPARK_KV_E4M3;
    if (w.a.cache.head_dim <= 64)
        return e4m3 ? launch_dp<T, DSPARK_KV_E4M3, 64>(w, s) : launch_dp<T, DSPARK_KV_INT8, 64>(w, s);
    return e4m3 ? launch_dp<T, DSPARK_KV_E4M3, 128>(w, s) : launch_dp<T, DSPARK_KV_INT8, 128>(w, s);
}

template <typename T>
cudaError_t launch_rows(const AttentionArgs &a, cudaStream_t s) {
    WindowArgs w{a, Divider(), Divider(a.cache.n_kv_heads), Divider(a.n_q_heads / a.cache.n_kv_heads),
                 Divider(a.cache.page_size / kChunk), false, 0.f, 1};
    return launch_t<T>(w, s);
}

}  // namespace

#ifdef DSPARK_WINDOW_F16
cudaError_t launch_window_rows_f16(const AttentionArgs &a, cudaStream_t s) { return launch_rows<__half>(a, s); }
#else
// Blocks with many rows of a kv head go to the 128-row tiles of the tensor cores (window_blocks.cu) when there is
// enough to do: those start later (55 us before the first result) and an item costs them more, then a tile less.
// Measured, rows a kv head x requests, window 1,024, D = 128 (here / there, us): 64 x 64 111 / 152, 128 x 64 196 / 167,
// 256 x 64 358 / 187, 512 x 64 692 / 307, 128 x 8 34 / 89, 256 x 8 62 / 76, 512 x 8 104 / 82, 1,024 x 1 34 / 70;
// window 128: 256 x 64 154 / 111, window 8,000: 128 x 32 594 / 361.
static bool may_be_many(int B, int n_rows, int n_q_heads, int n_kv_heads) {
    return ((int64_t)n_rows + B - 1) / B * (n_q_heads / n_kv_heads) >= 128;
}
size_t window_ws_bytes(int B, int n_rows, int n_q_heads, int n_kv_heads, int head_dim) {
    return may_be_many(B, n_rows, n_q_heads, n_kv_heads) ? window_blocks_ws_bytes(B, n_rows, n_q_heads, n_kv_heads, head_dim) : 0;
}

cudaError_t launch_window_attention(const AttentionArgs &a, cudaStream_t s) {
    if (may_be_many(a.rows.B, a.rows.n_rows, a.n_q_heads, a.cache.n_kv_heads) &&
        (double)a.rows.n_rows * a.n_q_heads * (double)(seen_tokens(a) + 256) >= 40e6)
        return launch_window_blocks(a, s);
    return a.dt == DSPARK_BF16 ? launch_rows<__nv_bfloat16>(a, s) : launch_window_rows_f16(a, s);
}
#endif

}  // namespace dspark
