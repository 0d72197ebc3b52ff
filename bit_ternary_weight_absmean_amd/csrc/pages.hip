// The pages of a cache: giving sequences pages for new tokens, sharing and dropping them, bringing the pages in use
// together, and copying pages (bt_pages_grow, _fork, _compact, _copy).
//
// State: table [B, W] (the pages of each sequence, in order; -1 behind them), length [B] in tokens, refs [P] (how many
// tables hold a page; 0: free) and a bound `first` below which every page is in use. All of it is on the device and
// read there, so that a step that changes it can be captured and replayed. Every entry taken from it or from the
// caller's lists is checked against the arrays before it is used as an index.
//
// Determinism: free pages are taken lowest index first, in the order of the sequences; the only atomics add and take
// minima of integers, whose order does not matter. Counts rise in one launch and fall in a later one (fork), so a
// page is seen to reach 0 exactly when it is free.
//
// Bound by launches and, where pages are copied, by their bytes (each read once and written once).
#include "bt_internal.h"
#include "pages.h"
#include "wave.h"

namespace bt {
namespace {

constexpr int kPlan = 1024;         // threads of the one workgroup that hands out pages
constexpr int kPlanWaves = kPlan / 64;
constexpr int kCopyBytes = 16384;   // of a page, by one workgroup at a time

__device__ inline int pages_for(int64_t tokens, int shift) { return (int)((tokens + (1 << shift) - 1) >> shift); }
__device__ inline int rank_in(uint64_t mask)
{
    return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
}

struct Range {
    int from, n;
};
// The new tokens of sequence b, kept inside [0, T) whatever the offsets say.
__device__ inline Range new_tokens(const PagesArgs &a, int b)
{
    const int from = min(max(a.q_start[b], 0), a.T);
    return {from, min(max(a.q_start[b + 1], from), a.T) - from};
}

__device__ inline int length_of(const PagesArgs &a, int b)
{
    return (int)min((int64_t)max(a.length[b], 0), (int64_t)a.W << a.page_shift);
}

// Sum over the workgroup of v, and the sum over the threads before this one.
__device__ inline int block_scan(int v, int *lds, int &total)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int sum = v;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int up = __shfl_up(sum, d);
        sum += lane >= d ? up : 0;
    }
    __syncthreads();  // lds may still be read from before
    if (lane == 63)
        lds[wave] = sum;
    __syncthreads();
    int before = 0;
    total = 0;
    for (int w = 0; w < kPlanWaves; ++w) {
        before += w < wave ? lds[w] : 0;
        total += lds[w];
    }
    return before + sum - v;
}

// Copies one piece of page src to page dst: four pieces of 16 bytes for each of 256 threads, all read before the first is
// written. (Not an array: the compiler put one into LDS, and a compaction took a quarter longer.)
__device__ inline void copy_piece(const PagesArgs &a, int64_t src, int64_t dst, int layer, int piece)
{
    const char *from = a.pool + layer * a.layer_stride + src * a.page_bytes;
    char *to = a.pool + layer * a.layer_stride + dst * a.page_bytes;
    const int64_t lo = (int64_t)piece * kCopyBytes, hi = min(lo + kCopyBytes, a.page_bytes);
    constexpr int U = kCopyBytes / 16 / 256;
    v4i x[U];
#pragma unroll
    for (int u = 0; u < U; ++u)  // past the end: the last piece again, not stored
        x[u] = *reinterpret_cast<const v4i *>(from + min(lo + (u * 256 + (int)threadIdx.x) * 16, hi - 16));
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t at = lo + (u * 256 + threadIdx.x) * 16;
        if (at < hi)
            *reinterpret_cast<v4i *>(to + at) = x[u];
    }
}

template <typename Pair>
__device__ inline void copy_pages(const PagesArgs &a, int64_t count, Pair pair)
{
    const int pieces = (int)((a.page_bytes + kCopyBytes - 1) / kCopyBytes);
    const int64_t per = (int64_t)a.layers * pieces;
    for (int64_t task = blockIdx.x; task < count * per; task += gridDim.x) {
        const int64_t i = task / per;
        const int rest = (int)(task % per);
        int64_t src, dst;
        if (pair(i, src, dst))
            copy_piece(a, src, dst, rest / pieces, rest % pieces);
    }
}

unsigned copy_grid(const PagesArgs &a, int64_t count)
{
    const int64_t tasks = count * a.layers * ((a.page_bytes + kCopyBytes - 1) / kCopyBytes);
    return (unsigned)(tasks < 1 ? 1 : tasks > 4096 ? 4096 : tasks);
}

// ---------------------------------------------------------------------------------- grow
//
// One workgroup hands out the pages: what every sequence needs, the free pages in order, who gets them. Up to 1024
// sequences it keeps all of it in registers and LDS and writes the tables, the counts and the tokens' places itself
// (each reading of memory behind another costs about 0.7 us here: first lengths, then the last pages' numbers and the
// counts from `first` on, then the last pages' counts); the second launch copies pages. For more sequences, or more
// than 2048 tokens, that launch also fills in the tables or the places. 8 sequences and 256 with a token each and 300 new
// ones: 7.0 and 7.6 us, and 2.3 and 4.3 for the copies. (The way for more sequences costs 1.5 us more for 8, 3 for 256.)
//
// Who needs a copy of a shared last page is told by the counts before the call, for all sequences at once: each of its
// holders that grows gets one, also where none stays, and the page is free after the call. To leave it to one of them, the
// holders of every page would have to be put in order behind those that are refused: a chain more, to save one copy.
//
// Workspace: [0] pages handed out, [1] pages copied, then per sequence the end of its demand (inclusive sum) and
// the page slot it starts at, then the list of copied pages (from, to), then the free pages.

struct GrowSpace {
    int *counts, *end, *slot, *from, *to, *free;
};
__device__ __host__ inline GrowSpace grow_space(int *ws, int64_t B)
{
    return {ws, ws + 4, ws + 4 + B, ws + 4 + 2 * B, ws + 4 + 3 * B, ws + 4 + 4 * B};
}

constexpr int kTokensHere = 2 * kPlan;  // places filled in by the one workgroup

// First index i in [0, n) with x[i] > v (n: none); x does not fall.
template <typename P>
__device__ inline int first_above(P x, int n, int v)
{
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (x[mid] > v)
            hi = mid;
        else
            lo = mid + 1;
    }
    return lo;
}

// Need of a sequence: pages, the slot of the first of them (-1: none to be had, or nothing asked), and the page that is
// copied into it (-1: none).
struct Need {
    int pages, slot, from;
};
__device__ inline Need need_of(const PagesArgs &a, int b, int n, int len)
{
    Need x = {0, -1, -1};
    const int have = pages_for(len, a.page_shift), want = pages_for((int64_t)len + n, a.page_shift);
    if (n > 0 && want <= a.W) {
        if (len & ((1 << a.page_shift) - 1)) {
            const int tail = a.table[(int64_t)b * a.W + have - 1];
            if (tail >= 0 && tail < a.P && a.refs[tail] > 1)
                x.from = tail;
        }
        x.pages = want - have + (x.from >= 0);
        x.slot = have - (x.from >= 0);
    }
    return x;
}

// The first `asked` free pages from `base` on, in order, as put(k, page); how many were found. The first step's counts are
// given (they were loaded before it was known how many pages are wanted).
constexpr int kPer = 8, kStep = kPlan * kPer;
__device__ inline void load_refs(const PagesArgs &a, int base, int (&refs)[kPer])
{
    const int mine = base + (int)(threadIdx.x >> 6) * 64 * kPer + (int)(threadIdx.x & 63);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        refs[i] = mine + i * 64 < a.P ? a.refs[mine + i * 64] : 1;
}
template <typename Put>
__device__ inline int free_pages(const PagesArgs &a, int base, int asked, int (&refs)[kPer], int *lds, Put put)
{
    const int lane = threadIdx.x & 63, wave = uniform((int)(threadIdx.x >> 6));
    int found = 0;
    while (base < a.P && found < asked) {
        uint64_t free[kPer];
        int n = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            free[i] = __ballot(refs[i] == 0);
            n += __popcll(free[i]);
        }
        __syncthreads();  // lds may still be read from before
        if (lane == 0)
            lds[wave] = n;
        __syncthreads();
        int at = found;
        for (int w = 0; w < kPlanWaves; ++w) {
            at += w < wave ? lds[w] : 0;
            found += lds[w];
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int k = at + rank_in(free[i]);
            if ((free[i] >> lane & 1) && k < asked)
                put(k, base + wave * 64 * kPer + i * 64 + lane);
            at += __popcll(free[i]);
        }
        base += kStep;
        if (base < a.P && found < asked)
            load_refs(a, base, refs);
    }
    return found;
}

// `first` after `taken` of the pages that were asked for are handed out; freed: the lowest page that may be free now.
__device__ inline void set_first(const PagesArgs &a, const int *free, int taken, int found, int freed)
{
    *a.first = min(taken > 0 ? free[taken - 1] + 1 : found > 0 ? free[0] : a.P, freed);
}

// The place and number of new token t of sequence b, whose new pages are free[start ..] from slot on.
struct Token {
    int row, at;
};
__device__ inline Token place_token(const PagesArgs &a, int b, int t, int from, int len, int slot, int start, int end,
                                    const int *free)
{
    const int at = len + t - from;
    if (slot < 0)
        return {-1, at};
    const int p = at >> a.page_shift;
    // what this call writes to the table is taken from the list
    const int page = p >= slot && start + p - slot < end ? free[start + p - slot] : a.table[(int64_t)b * a.W + p];
    return {page < 0 || page >= a.P ? -1 : page << a.page_shift | (at & ((1 << a.page_shift) - 1)), at};
}

__global__ __launch_bounds__(kPlan) void k_pages_plan_small(PagesArgs a)
{
    __shared__ int lds[kPlanWaves], s_end[kPlan], s_slot[kPlan], s_from[kPlan], s_to[kPlan], s_len[kPlan];
    __shared__ int freed;
    const GrowSpace ws = grow_space(a.ws, a.B);
    const int b = threadIdx.x;
    const int base = min(max(*a.first, 0), a.P);
    int refs[kPer];
    Need x = {0, -1, -1};
    Range r = {0, 0};
    int len = 0;
    if (b < a.B) {
        r = new_tokens(a, b);
        len = length_of(a, b);
    }
    load_refs(a, base, refs);
    if (b < a.B)
        x = need_of(a, b, r.n, len);
    if (b == 0)
        freed = a.P;
    int asked;
    const int before = block_scan(x.pages, lds, asked), end = before + x.pages;
    const int found = free_pages(a, base, asked, refs, lds, [&](int k, int page) { ws.free[k] = page; });
    const bool fits = x.slot >= 0 && (x.pages == 0 || end <= found);
    const bool copy = fits && x.from >= 0;
    s_end[b] = end;
    s_slot[b] = fits ? x.slot : -1;
    s_from[b] = b < a.B ? r.from : a.T;
    s_to[b] = r.from + r.n;
    s_len[b] = len;
    int taken, copies;
    block_scan(fits ? x.pages : 0, lds, taken);
    const int at = block_scan(copy ? 1 : 0, lds, copies);  // (its barriers: the lists are there for all of the workgroup)
    if (b < a.B) {
        a.granted[b] = fits ? r.n : 0;
        if (fits)
            a.length[b] = len + r.n;
    }
    if (copy) {
        ws.from[at] = x.from;
        ws.to[at] = ws.free[before];
        atomicSub(a.refs + x.from, 1);
        atomicMin(&freed, x.from);  // perhaps free now
    }
    for (int k = b; k < taken; k += kPlan) {
        const int q = first_above(s_end, a.B, k), page = ws.free[k];
        a.table[(int64_t)q * a.W + s_slot[q] + k - (q ? s_end[q - 1] : 0)] = page;
        a.refs[page] = 1;
    }
    if (a.T <= kTokensHere) {
        for (int t = b; t < a.T; t += kPlan) {
            Token k = {-1, -1};
            const int q = first_above(s_from, a.B, t) - 1;  // the last sequence that starts at or before t
            if (q >= 0 && t >= s_from[q] && t < s_to[q])
                k = place_token(a, q, t, s_from[q], s_len[q], s_slot[q], q ? s_end[q - 1] : 0, s_end[q], ws.free);
            a.rows[t] = k.row;
            a.positions[t] = k.at;
        }
    } else if (b < a.B) {
        ws.end[b] = s_end[b];
        ws.slot[b] = s_slot[b];
    }
    __syncthreads();
    if (b == 0) {
        ws.counts[0] = taken;
        ws.counts[1] = copies;
        if (asked > 0)
            set_first(a, ws.free, taken, found, freed);
    }
}

__global__ __launch_bounds__(kPlan) void k_pages_plan(PagesArgs a)
{
    __shared__ int lds[kPlanWaves];
    __shared__ int freed;
    const GrowSpace ws = grow_space(a.ws, a.B);
    const int tid = threadIdx.x;
    if (tid == 0)
        freed = a.P;
    // what every sequence needs
    int asked = 0;
    for (int c = 0; c < a.B; c += kPlan) {
        const int b = c + tid;
        Need x = {0, -1, -1};
        if (b < a.B)
            x = need_of(a, b, new_tokens(a, b).n, length_of(a, b));
        int total;
        const int before = block_scan(x.pages, lds, total);
        if (b < a.B) {
            ws.end[b] = asked + before + x.pages;
            ws.slot[b] = x.slot;
        }
        asked += total;
    }
    const int base = asked > 0 ? min(max(*a.first, 0), a.P) : a.P;
    int refs[kPer];
    load_refs(a, base, refs);
    const int found = free_pages(a, base, asked, refs, lds, [&](int k, int page) { ws.free[k] = page; });
    __syncthreads();  // the lists, for all of the workgroup
    // who gets them: those whose demand ends within what was found
    int taken = 0, copies = 0;
    for (int c = 0; c < a.B; c += kPlan) {
        const int b = c + tid;
        int need = 0, copy = 0, from = 0, to = 0;
        if (b < a.B) {
            const int end = ws.end[b], slot = ws.slot[b], n = new_tokens(a, b).n;
            need = end - (b ? ws.end[b - 1] : 0);
            const bool fits = slot >= 0 && (need == 0 || end <= found);
            a.granted[b] = fits ? n : 0;
            if (fits) {
                const int len = length_of(a, b);
                copy = slot < pages_for(len, a.page_shift);
                if (copy) {
                    from = a.table[(int64_t)b * a.W + slot];
                    to = ws.free[end - need];
                    atomicSub(a.refs + from, 1);
                    atomicMin(&freed, from);
                }
                a.length[b] = len + n;
            } else {
                ws.slot[b] = -1;
                need = 0;
            }
        }
        int total;
        const int at = copies + block_scan(copy, lds, total);
        if (copy) {
            ws.from[at] = from;
            ws.to[at] = to;
        }
        copies += total;
        block_scan(need, lds, total);
        taken += total;
    }
    __syncthreads();
    if (tid == 0) {
        ws.counts[0] = taken;
        ws.counts[1] = copies;
        if (asked > 0)
            set_first(a, ws.free, taken, found, freed);
    }
}

// tables, tokens: whether the tables and the places are left to this launch
__global__ __launch_bounds__(256) void k_pages_grow(PagesArgs a, int tables, int tokens)
{
    __shared__ int s_end[kPlan];
    const GrowSpace ws = grow_space(a.ws, a.B);
    const int copies = ws.counts[1];
    copy_pages(a, copies, [&](int64_t i, int64_t &src, int64_t &dst) {
        src = ws.from[i];
        dst = ws.to[i];
        return true;
    });
    const int id = blockIdx.x * 256 + threadIdx.x, step = gridDim.x * 256;
    if (tables)
        for (int k = id; k < ws.counts[0]; k += step) {
            const int b = first_above(ws.end, a.B, k);
            if (b >= a.B)
                continue;
            const int start = b ? ws.end[b - 1] : 0, page = ws.free[k];
            a.table[(int64_t)b * a.W + ws.slot[b] + k - start] = page;
            a.refs[page] = 1;
        }
    if (tokens) {
        // the sequences' ends nearby where they fit
        const bool near = a.B <= kPlan;
        if (near) {
            for (int i = threadIdx.x; i < a.B; i += 256)
                s_end[i] = a.q_start[i + 1];
            __syncthreads();
        }
        for (int t = id; t < a.T; t += step) {
            const int b = near ? first_above(s_end, a.B, t) : first_above(a.q_start + 1, a.B, t);
            Token k = {-1, -1};
            if (b < a.B) {
                const Range r = new_tokens(a, b);
                if (t >= r.from && t < r.from + r.n)
                    k = place_token(a, b, t, r.from, length_of(a, b) - a.granted[b], ws.slot[b], b ? ws.end[b - 1] : 0,
                                    ws.end[b], ws.free);
            }
            a.rows[t] = k.row;
            a.positions[t] = k.at;
        }
    }
}

// ---------------------------------------------------------------------------------- fork
//
// Counts go up first, for all pages that are taken, and down only then, for all that are given up. Tables of up to kCells
// entries in one launch of one workgroup, with a barrier between the two; larger ones in two launches of one workgroup
// per sequence, the first of which also keeps the rows as they will be in the workspace (the new lengths, the new rows).
// Bound by the chain parent, length, entry, count: 8 sequences of up to 9 pages 5.9 us (two launches: 3.1 and 3.4, and a beam
// step called from the host 21.3 us instead of 18), 256 of up to 64 pages 2.1 and 3.8.

constexpr int kCells = 8 * kPlan;

__device__ inline bool fork_source(const PagesArgs &a, int b, int &p)
{
    p = a.parent[b];
    return p >= 0 && p < a.B;
}

// `first` to the lowest of the workgroup's pages, by one lane of each wave.
__device__ inline void lower_first(const PagesArgs &a, uint32_t lowest)
{
    lowest = wave_reduce_bits(lowest, [](uint32_t x, uint32_t y) { return x < y ? x : y; });
    if ((threadIdx.x & 63) == 0 && lowest != UINT32_MAX)
        atomicMin(a.first, (int)lowest);
}

__global__ __launch_bounds__(kPlan) void k_fork_small(PagesArgs a)
{
    constexpr int U = kCells / kPlan;
    const uint32_t cells = (uint32_t)a.B * a.W;
    int page[U], old[U], now[U];  // what the cell will hold; pages of its sequence before and after (0, 0: it stays)
    int len = -1;                 // of sequence threadIdx.x
    if ((int)threadIdx.x < a.B) {
        int p;
        const bool from = fork_source(a, threadIdx.x, p);
        if (!(from && p == (int)threadIdx.x))
            len = from ? length_of(a, p) : 0;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t c = u * kPlan + threadIdx.x;
        page[u] = -1;
        old[u] = now[u] = 0;
        if (c < cells) {
            const int b = (int)(c / (uint32_t)a.W), i = (int)(c - (uint32_t)b * (uint32_t)a.W);
            int p;
            const bool from = fork_source(a, b, p);
            if (!(from && p == b)) {
                old[u] = pages_for(length_of(a, b), a.page_shift) - i;
                now[u] = (from ? pages_for(length_of(a, p), a.page_shift) : 0) - i;
                if (now[u] > 0) {
                    page[u] = a.table[(int64_t)p * a.W + i];
                    if (page[u] >= 0 && page[u] < a.P)
                        atomicAdd(a.refs + page[u], 1);
                }
            }
        }
    }
    __threadfence();
    __syncthreads();
    uint32_t lowest = UINT32_MAX;  // of the pages that nothing holds any more
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t c = u * kPlan + threadIdx.x;
        if (old[u] > 0) {
            const int was = a.table[c];
            if (was >= 0 && was < a.P && atomicSub(a.refs + was, 1) == 1)
                lowest = min(lowest, (uint32_t)was);
        }
        if (old[u] > 0 || now[u] > 0)
            a.table[c] = page[u];
    }
    lower_first(a, lowest);
    if (len >= 0)
        a.length[threadIdx.x] = len;
}

__global__ __launch_bounds__(256) void k_fork_take(PagesArgs a)
{
    const int b = blockIdx.x;
    int p;
    const bool from = fork_source(a, b, p);
    if (from && p == b)
        return;
    const int len = from ? length_of(a, p) : 0, n = pages_for(len, a.page_shift);
    int *rows = a.ws + a.B + (int64_t)b * a.W;
    for (int i = threadIdx.x; i < n; i += 256) {
        const int page = a.table[(int64_t)p * a.W + i];
        rows[i] = page;
        if (page >= 0 && page < a.P)
            atomicAdd(a.refs + page, 1);
    }
    if (threadIdx.x == 0)
        a.ws[b] = len;
}

__global__ __launch_bounds__(256) void k_fork_give(PagesArgs a)
{
    const int b = blockIdx.x;
    int p;
    if (fork_source(a, b, p) && p == b)
        return;
    const int old = pages_for(length_of(a, b), a.page_shift), len = a.ws[b], n = pages_for(len, a.page_shift);
    const int *rows = a.ws + a.B + (int64_t)b * a.W;
    int *table = a.table + (int64_t)b * a.W;
    uint32_t lowest = UINT32_MAX;  // of the pages that this sequence was the last to hold
    for (int i = threadIdx.x; i < max(old, n); i += 256) {
        if (i < old) {
            const int page = table[i];
            if (page >= 0 && page < a.P && atomicSub(a.refs + page, 1) == 1)
                lowest = min(lowest, (uint32_t)page);
        }
        table[i] = i < n ? rows[i] : -1;
    }
    lower_first(a, lowest);
    __syncthreads();  // all have read the length
    if (threadIdx.x == 0)
        a.length[b] = len;
}

// ------------------------------------------------------------------------------- compact
//
// With L pages in use, the k-th one at or past L goes to the k-th free one below L. A page in use has a rank (how
// many are in use before it), a free page i has i - rank free ones before it: segments of pages need no more than
// the counts of those before them. The pages that move are those with the last ranks. Up to eight segments are listed in one
// launch, every workgroup going over all counts (4096 pages: 6.1 us; with a launch that counts 2 to 3 more); bound by the
// copies: 64 sequences of up to 40 pages in four layers of 43520 bytes 39 us (237 MB read and written; 6.0 TB/s, more
// than a large copy's 5.2 since part of the pool is in the last cache from the call before).
// Workspace: [0] L, [1] moves, then counts of the segments, then for each free page below L (in order) its index, for
// each rank its page (those that move), for each page its rank (those that move; -1).

constexpr int kSegment = 4096;

struct CompactSpace {
    int *counts, *segment, *hole, *mover, *rank;
};
__device__ __host__ inline CompactSpace compact_space(int *ws, int64_t P)
{
    int *segment = ws + 4, *hole = segment + (P + kSegment - 1) / kSegment;
    return {ws, segment, hole, hole + P, hole + 2 * P};
}

__global__ __launch_bounds__(kPlan) void k_compact_count(PagesArgs a)
{
    __shared__ int lds[kPlanWaves];
    const int base = blockIdx.x * kSegment;
    int n = 0;
#pragma unroll
    for (int i = 0; i < kSegment / kPlan; ++i) {
        const int page = base + i * kPlan + (int)threadIdx.x;
        n += page < a.P && a.refs[page] > 0;
    }
    int total;
    block_scan(n, lds, total);
    if (threadIdx.x == 0)
        compact_space(a.ws, a.P).segment[blockIdx.x] = total;
}

// counted: whether a launch before counted the segments; otherwise (few of them) every workgroup goes over all counts
__global__ __launch_bounds__(kPlan) void k_compact_list(PagesArgs a, int counted)
{
    __shared__ int lds[kPlanWaves];
    const CompactSpace ws = compact_space(a.ws, a.P);
    const int segments = (a.P + kSegment - 1) / kSegment, base = blockIdx.x * kSegment;
    int live = 0, rank = 0, total;
    if (counted) {
        for (int i = threadIdx.x; i < segments; i += kPlan) {
            live += ws.segment[i];
            rank += i < (int)blockIdx.x ? ws.segment[i] : 0;
        }
    } else {
#pragma unroll 4
        for (int i = threadIdx.x; i < a.P; i += kPlan) {
            const int used = a.refs[i] > 0;
            live += used;
            rank += i < base ? used : 0;
        }
    }
    block_scan(live, lds, total);
    live = total;
    block_scan(rank, lds, total);
    rank = total;
    if (live == 0 && blockIdx.x == 0 && threadIdx.x == 0)
        ws.counts[0] = ws.counts[1] = 0;
    for (int i = 0; i < kSegment / kPlan; ++i) {
        const int page = base + i * kPlan + (int)threadIdx.x;
        const int used = page < a.P && a.refs[page] > 0;
        const int r = rank + block_scan(used, lds, total);
        rank += total;
        if (page >= a.P)
            continue;
        if (page < live && !used)
            ws.hole[page - r] = page;
        if (page >= live) {
            ws.rank[page] = used ? r : -1;
            if (used)
                ws.mover[r] = page;
        }
        if (page == live - 1) {
            ws.counts[0] = live;
            ws.counts[1] = live - r - used;
        }
    }
}

__global__ __launch_bounds__(256) void k_compact_move(PagesArgs a)
{
    const CompactSpace ws = compact_space(a.ws, a.P);
    const int live = ws.counts[0], moves = ws.counts[1], stay = live - moves;
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
    for (int64_t i = id; i < (int64_t)a.B * a.W; i += step) {
        const int page = a.table[i];
        if (page >= live && page < a.P) {
            const int r = ws.rank[page];
            if (r >= stay && r < live)
                a.table[i] = ws.hole[r - stay];
        }
    }
    for (int64_t i = id; i < moves; i += step) {
        const int src = ws.mover[stay + i], dst = ws.hole[i];
        a.refs[dst] = a.refs[src];
        a.refs[src] = 0;
    }
    if (id == 0)
        *a.first = live;
    copy_pages(a, moves, [&](int64_t i, int64_t &src, int64_t &dst) {
        src = ws.mover[stay + i];
        dst = ws.hole[i];
        return true;
    });
}

// ---------------------------------------------------------------------------------- copy

__global__ __launch_bounds__(256) void k_pages_copy(PagesArgs a, const int *src, const int *dst, int64_t n)
{
    copy_pages(a, n, [&](int64_t i, int64_t &from, int64_t &to) {
        from = src[i];
        to = dst[i];
        return from >= 0 && from < a.P && to >= 0 && to < a.P && from != to;
    });
}

}  // namespace

size_t pages_workspace_bytes(int64_t B, int64_t W, int64_t P)
{
    const int64_t grow = 4 + 4 * B + P, fork = B + B * W;
    const int64_t compact = 4 + (P + kSegment - 1) / kSegment + 3 * P;
    const int64_t most = grow > fork ? grow : fork;
    return (size_t)(4 * (most > compact ? most : compact));
}

hipError_t launch_pages_grow(const PagesArgs &a, hipStream_t s)
{
    const bool small = a.B <= kPlan, tokens = !small || a.T > kTokensHere;
    if (small)
        k_pages_plan_small<<<1, kPlan, 0, s>>>(a);
    else
        k_pages_plan<<<1, kPlan, 0, s>>>(a);
    if (hipError_t e = hipGetLastError())
        return e;
    const int64_t places = tokens ? ((int64_t)a.T + 255) / 256 : 1;
    const unsigned copies = copy_grid(a, a.B), all = places > 4096 ? 4096u : (unsigned)(places < 1 ? 1 : places);
    k_pages_grow<<<copies > all ? copies : all, 256, 0, s>>>(a, !small, tokens);
    return hipGetLastError();
}

hipError_t launch_pages_fork(const PagesArgs &a, hipStream_t s)
{
    if (a.B <= kPlan && (int64_t)a.B * a.W <= kCells) {
        k_fork_small<<<1, kPlan, 0, s>>>(a);
        return hipGetLastError();
    }
    k_fork_take<<<(unsigned)a.B, 256, 0, s>>>(a);
    if (hipError_t e = hipGetLastError())
        return e;
    k_fork_give<<<(unsigned)a.B, 256, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_pages_compact(const PagesArgs &a, hipStream_t s)
{
    const unsigned segments = (unsigned)((a.P + kSegment - 1) / kSegment);
    const bool counted = segments > 8;
    if (counted) {
        k_compact_count<<<segments, kPlan, 0, s>>>(a);
        if (hipError_t e = hipGetLastError())
            return e;
    }
    k_compact_list<<<segments, kPlan, 0, s>>>(a, counted);
    if (hipError_t e = hipGetLastError())
        return e;
    const int64_t cells = ((int64_t)a.B * a.W + 255) / 256;
    const unsigned copies = copy_grid(a, a.P / 2), all = cells > 4096 ? 4096u : (unsigned)(cells < 1 ? 1 : cells);
    k_compact_move<<<copies > all ? copies : all, 256, 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_pages_copy(const PagesArgs &a, const int *src, const int *dst, int64_t n, hipStream_t s)
{
    k_pages_copy<<<copy_grid(a, n), 256, 0, s>>>(a, src, dst, n);
    return hipGetLastError();
}

}  // namespace bt
