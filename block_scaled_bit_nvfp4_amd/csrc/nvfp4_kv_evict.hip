// nvfp4_kv_evict.hip -- cuts sequences of the paged cache to a budget: which tokens of
// each head stay, and their move to the front (gfx950).
//
// Select, a workgroup per sequence and head: a candidate's key is its weight, as a whole
// number in the order of the weights, and then its position, the lower the larger, so that
// no two are equal and the ones that stay are those from one key, the border, on.  The
// keys are counted by their top 12 bits; the bin that holds the border usually holds few,
// whose ranks are found by comparing all of them with all; only where it holds many (equal
// weights) the next 12 bits are counted.  Then one walk in order writes the kept positions
// and moves their weights.  Up to 8192, 16384 or 32768 positions, by the bound, stay in
// registers throughout.  Bound by its chain of dependent steps, 10.6 us for 4607 positions, and
// by a CU's issue where there are many: of 25 us for 32768 of eight heads, 13 are 2.5e5 vector
// instructions of waves on eight CUs.
//
// Move: a kept token's slot is never past its old one, and both rise together.  So one
// workgroup can move a stretch of tokens at a time, all reads before all writes, and the
// places that it overwrites are behind everything it has yet to read.  The bytes of a
// unit are split over workgroups so that no two share any: a piece of the keys' codes, a
// part of the values' rows, either side's scales.  What bounds it: three dependent loads
// for a stretch (the kept position, its page, the bytes), so that a stretch is 4096 tokens
// (9 us for 4096 of 4607), and for many sequences the lines that hold something that is
// kept, twice the bytes themselves (64 sequences of 1 to 8191 to 2048: 96 us, 282 MB read
// of 274 in such lines, 144 written, 4.4 TB/s).  512 threads: with 256 these take 2 and 9 us
// more, with 1024 0.3 less and 23 more.
#include "nvfp4_kv.h"

namespace nvfp4 {

constexpr int kSelectThreads = 1024, kSelectWaves = kSelectThreads / kLanes;
constexpr int kDigitBits = 12, kBins = 1 << kDigitBits;
constexpr int kRanked = 512;                                      // keys that are compared with one another
constexpr int kMoveThreads = 512, kMoveTokens = 4096;            // tokens of a stretch
// A head's workgroups are put on one XCD, whose cache then serves the lines that its value
// parts share (64 sequences 115 us, both launches, with the parts one after another 123;
// 4096 of 4607 tokens 19.1 against 21.8).
constexpr int kXcds = 8;
constexpr int kMostParts = 32, kValueParts = 5;    // workgroups that move a head's tokens; those of its values

struct EvictArgs {
    KvView kv;
    const float *weights;
    float *weights_out;
    int64_t width;
    int *kept, *left;
    int budget, first, recent;
};

// Whole numbers in the order of the weights: NaN 0, then -infinity to infinity, -0 as 0.
__device__ __forceinline__ uint32_t weight_order(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return x != x ? 0u : b & 0x80000000u ? ~b : b | 0x80000000u;
}

// The inclusive sum over the lanes up to this one.
__device__ __forceinline__ int sum_upto(int v) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < kLanes; d <<= 1) {
        const int y = __shfl_up(v, d);
        v += lane >= d ? y : 0;
    }
    return v;
}

// HELD: positions that a thread holds.
template <int HELD>
__global__ void __launch_bounds__(kSelectThreads, HELD == 8 ? 8 : 4) kv_evict_select_kernel(EvictArgs a) {
    constexpr int kStripes = HELD / 4;                 // a thread holds four positions in a row of each
    constexpr int kStripe = 4 * kSelectThreads, kBlock = HELD * kSelectThreads;
    constexpr int kCells = kStripes * kSelectWaves;
    __shared__ int bins[kBins];
    __shared__ unsigned long long ranked[kRanked];
    __shared__ int totals[kCells];                     // [stripe][wave]
    __shared__ int chosen, above, inside, found;
    __shared__ unsigned long long at_border;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int s = blockIdx.x / a.kv.heads;
    const int length = a.kv.past[s];
    const float *w = a.weights + int64_t(blockIdx.x) * a.width;
    float *out = a.weights_out + int64_t(blockIdx.x) * a.width;
    int *kept = a.kept + int64_t(blockIdx.x) * a.budget;
    const int held = max(length, 0);
    const int lo = a.first, hi = held - a.recent;      // the candidates
    const bool many = held > kBlock;
    const auto position = [&](int base, int i) { return base + i / 4 * kStripe + 4 * tid + i % 4; };
    const auto read = [&](int base, float (&x)[HELD]) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < kStripes; ++j) {
            const int i = position(base, 4 * j);
            if (i + 4 <= held) {
                typedef float F4 __attribute__((ext_vector_type(4), aligned(4)));
                const F4 v = *reinterpret_cast<const F4 *>(w + i);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[4 * j + e] = v[e];
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) x[4 * j + e] = i + e < held ? w[i + e] : 0.0f;
            }
        }
    };
    // the orders of the weights from 1 on, 0 for what is no candidate
    uint32_t o[HELD];
    const auto load = [&](int base) __attribute__((always_inline)) {
        float x[HELD];
        read(base, x);
#pragma unroll
        for (int i = 0; i < HELD; ++i) {
            const int p = position(base, i);
            o[i] = p >= lo && p < hi ? weight_order(x[i]) + 1 : 0u;
        }
    };
    if (held > a.budget && held <= a.kv.capacity) load(0);
    // every position has a page, or the sequence stays as it is
    bool whole = held <= a.kv.capacity;
    if (whole) {
        const int pages = int(ceil_div(held, int64_t(1) << a.kv.page_shift));
        for (int p = tid; p < pages; p += kSelectThreads) {
            const int entry = a.kv.table[int64_t(s) * a.kv.width + p];
            whole &= entry >= 0 && entry < a.kv.pages;
        }
    }
    for (int i = tid; i < kBins; i += kSelectThreads) bins[i] = 0;
    if (tid == 0) found = 0;
    whole = __syncthreads_and(whole);
    if (!whole || held <= a.budget) {
        for (int i = tid; i < a.budget; i += kSelectThreads) kept[i] = whole && i < held ? i : -1;
        if (whole && out != w)
            for (int i = tid; i < held; i += kSelectThreads) out[i] = w[i];
        return;
    }
    int want = a.budget - a.first - a.recent;          // of the candidates that stay
    // f(order, position) for each candidate; a lone block is in registers already
    const auto each = [&](auto f) __attribute__((always_inline)) {
        for (int base = 0; base < held; base += kBlock) {
            if (many) load(base);
#pragma unroll
            for (int i = 0; i < HELD; ++i)
                if (base + i / 4 * kStripe < held && o[i]) f(o[i], position(base, i));
        }
    };
    // The bin of the want-th largest from the counts, then `want` within it.
    const auto choose = [&]() {
        __syncthreads();
        // a thread's four bins from the top, and how many are above them
        const int top = kBins - 1 - 4 * tid;
        const int n0 = bins[top], n1 = bins[top - 1], n2 = bins[top - 2], n3 = bins[top - 3];
        const int own = n0 + n1 + n2 + n3, upto = sum_upto(own);
        if (lane == 63) totals[wave] = upto;
        __syncthreads();
        int before = upto - own;
#pragma unroll
        for (int v = 0; v < kSelectWaves; ++v) before += v < wave ? totals[v] : 0;
        if (before < want && before + own >= want) {
            int b = top, n = n0;
            if (before + n < want) { before += n; n = n1; --b; }
            if (before + n < want) { before += n; n = n2; --b; }
            if (before + n < want) { before += n; n = n3; --b; }
            chosen = b;
            above = before;
            inside = n;
        }
        __syncthreads();
        want -= above;
    };
    const auto key_of = [](uint32_t order, int p) { return static_cast<unsigned long long>(order) << 32 | (0xFFFFFFFFu - uint32_t(p)); };
    unsigned long long border = ~0ull;
    if (want > 0) {
        each([&](uint32_t order, int) { atomicAdd(&bins[order >> (32 - kDigitBits)], 1); });
        choose();
        unsigned long long prefix = chosen;
        int shift = 64 - kDigitBits;
        while (inside > kRanked) {                     // weights alike in their top bits: further down the key
            for (int i = tid; i < kBins; i += kSelectThreads) bins[i] = 0;
            __syncthreads();
            const int next = max(shift - kDigitBits, 0), bits = shift - next;
            each([&](uint32_t order, int p) {
                const unsigned long long k = key_of(order, p);
                if (k >> shift == prefix) atomicAdd(&bins[int(k >> next) & ((1 << bits) - 1)], 1);
            });
            choose();
            prefix = prefix << bits | unsigned(chosen);
            shift = next;
        }
        each([&](uint32_t order, int p) {
            const unsigned long long k = key_of(order, p);
            if (k >> shift == prefix) ranked[atomicAdd(&found, 1)] = k;
        });
        __syncthreads();
        if (tid < inside) {
            const unsigned long long mine = ranked[tid];
            int rank = 0;
            for (int j = 0; j < inside; ++j) rank += ranked[j] > mine;
            if (rank == want - 1) at_border = mine;
        }
        __syncthreads();
        border = at_border;
    }
    const uint32_t border_order = uint32_t(border >> 32);
    const int border_position = int(0xFFFFFFFFu - uint32_t(border));
    // In order, a block of positions at a time, reads before writes (slots are never past
    // positions, so that what a block writes is behind the next one).
    int at = 0;
    for (int base = 0; base < held; base += kBlock) {
        if (many) load(base);
        uint32_t stay = 0;
        int upto[kStripes];
#pragma unroll
        for (int j = 0; j < kStripes; ++j) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = 4 * j + e, p = position(base, i);
                stay |= uint32_t(o[i] > border_order || (o[i] == border_order && p <= border_position) || (o[i] == 0 && p < held)) << i;
            }
            upto[j] = sum_upto(__popc(stay >> 4 * j & 15u));
            if (lane == 63) totals[j * kSelectWaves + wave] = upto[j];
        }
        float x[HELD];                                 // again, where the orders were
        read(base, x);
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();
        // the totals before each one, two cells a lane
        const int t0 = 2 * lane < kCells ? totals[2 * lane] : 0, t1 = 2 * lane < kCells ? totals[2 * lane + 1] : 0;
        const int sums = sum_upto(t0 + t1);
#pragma unroll
        for (int j = 0; j < kStripes; ++j) {
            const int cell = j * kSelectWaves + wave;
            const int upto_cell = __shfl(cell & 1 ? sums : sums - t1, cell >> 1);      // with the cell's own
            const int of_cell = __shfl(cell & 1 ? t1 : t0, cell >> 1);
            int slot = at + upto_cell - of_cell + upto[j] - __popc(stay >> 4 * j & 15u);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (stay >> (4 * j + e) & 1) {
                    kept[slot] = position(base, 4 * j + e);
                    out[slot] = x[4 * j + e];
                    ++slot;
                }
        }
        at += __shfl(sums, 63);
        __syncthreads();
    }
}

// Copies BYTES per thread and token.
template <int BYTES>
struct Moved;
template <> struct Moved<1> { typedef uint8_t type; };
template <> struct Moved<2> { typedef uint16_t type; };
template <> struct Moved<4> { typedef uint32_t type; };
template <> struct Moved<8> { typedef u32x2 type; };
template <> struct Moved<16> { typedef u32x4 type; };

// Moves the tokens of one head: COLUMNS items of BYTES of each, item c of the token at
// place r of a unit at offset(r, c) of the unit's `unit_bytes`.
template <int BYTES, int COLUMNS, class Offset>
__device__ __forceinline__ void move_tokens(const EvictArgs &a, int s, int head, const int *kept, uint8_t *plane,
                                            int unit_bytes, Offset offset) {
    typedef typename Moved<BYTES>::type T;
    constexpr int kTokens = kMoveThreads / COLUMNS, kMost = BYTES == 16 ? 8 : 16;      // registers hold no more
    constexpr int kDeep = kMoveTokens / kTokens < kMost ? kMoveTokens / kTokens : kMost;
    const int column = threadIdx.x % COLUMNS, lane_token = threadIdx.x / COLUMNS;
    const KvView &v = a.kv;
    const int *const pages = v.table + int64_t(s) * v.width;
    const auto place = [&](int page, int pos) {
        return reinterpret_cast<T *>(plane + v.unit_of(page, head, pos) * unit_bytes + offset(pos & (kKvUnit - 1), column));
    };
    const int last = kept[a.budget - 1];
    for (int base = 0; base < a.budget; base += kDeep * kTokens) {
        int from[kDeep], page[kDeep];
        T x[kDeep];
#pragma unroll
        for (int k = 0; k < kDeep; ++k) from[k] = kept[min(base + k * kTokens + lane_token, a.budget - 1)];
        if (last < a.budget) return;                     // nothing was cut
#pragma unroll
        for (int k = 0; k < kDeep; ++k) page[k] = pages[from[k] >> v.page_shift];
        // those of the slots past the budget read the last one's, and write nothing
#pragma unroll
        for (int k = 0; k < kDeep; ++k) x[k] = *place(page[k], from[k]);
#pragma unroll
        for (int k = 0; k < kDeep; ++k) page[k] = pages[min(base + k * kTokens + lane_token, a.budget - 1) >> v.page_shift];
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kDeep; ++k) {
            const int slot = base + k * kTokens + lane_token;
            if (slot < a.budget && from[k] != slot) *place(page[k], slot) = x[k];
        }
    }
}

template <int D, int BITS, int SIDE>
__device__ __forceinline__ void move_side(const EvictArgs &a, int s, int head, const int *kept, int part) {
    typedef KvSide<D, BITS> S;
    if (part == 0) {
        if constexpr (SIDE == 0)
            move_tokens<S::kBlocks, 1>(a, s, head, kept, a.kv.scales[0], S::kUnitScales,
                                       [](int r, int) { return S::key_scale(r, 0); });
        else
            move_tokens<1, S::kBlocks>(a, s, head, kept, a.kv.scales[1], S::kUnitScales,
                                       [](int r, int c) { return S::value_scale(r, c); });
        return;
    }
    const int p = part - 1;
    if constexpr (SIDE == 0) {
        if (p < S::kPieces)
            move_tokens<S::kPiece, 1>(a, s, head, kept, a.kv.codes[0], S::kUnitCodes,
                                      [p](int r, int) { return S::key_code(r, p * S::kPiece); });
    } else {
        if (p < 4)
            move_tokens<S::kPart, 4>(a, s, head, kept, a.kv.codes[1], S::kUnitCodes,
                                     [p](int r, int c) { return S::value_code(r, (4 * p + c) * S::kPart); });
    }
}

template <int D>
__global__ void __launch_bounds__(kMoveThreads) kv_evict_move_kernel(EvictArgs a, int k_bits, int v_bits, int key_parts, int parts) {
    const int part = int(blockIdx.x / kXcds) % parts, row = int(blockIdx.x / (kXcds * parts)) * kXcds + int(blockIdx.x % kXcds);
    if (row >= a.kv.seqs * a.kv.heads) return;
    const int head = row % a.kv.heads, s = row / a.kv.heads;
    const int *kept = a.kept + int64_t(row) * a.budget;
    if (part == 0 && head == 0 && threadIdx.x == 0) {
        const int held = a.kv.past[s];
        a.left[s] = kept[a.budget - 1] >= 0 ? a.budget : held;
    }
    if (part < key_parts) {
        if (k_bits == 8) move_side<D, 8, 0>(a, s, head, kept, part);
        else move_side<D, 4, 0>(a, s, head, kept, part);
    } else {
        if (v_bits == 8) move_side<D, 8, 1>(a, s, head, kept, part - key_parts);
        else move_side<D, 4, 1>(a, s, head, kept, part - key_parts);
    }
}

}  // namespace nvfp4

using namespace nvfp4;

NVFP4_API int nvfp4_kv_evict(const nvfp4_kv_cache *cache, const nvfp4_kv_batch *batch, int budget, int first,
                             int recent, const float *weights, float *weights_out, int64_t width, int32_t *kept,
                             int32_t *left, hipStream_t stream) {
    EvictArgs a;
    if (int st = kv_check(cache, batch, a.kv)) return st;
    if (!weights || !weights_out || !kept || !left) return NVFP4_EINVAL;
    if (budget < 1 || first < 0 || recent < 0 || int64_t(first) + recent > budget) return NVFP4_EINVAL;
    const int64_t rows = int64_t(batch->seqs) * cache->heads;
    if (rows > kMaxGrid / (kMoveThreads * kMostParts) || budget > (int64_t(1) << 30) / rows) return NVFP4_ESHAPE;
    if (width < a.kv.capacity || width > (int64_t(1) << 40)) return NVFP4_ESHAPE;
    if (!aligned(weights, 4) || !aligned(weights_out, 4) || !aligned(kept, 4) || !aligned(left, 4)) return NVFP4_EALIGN;
    a.weights = weights;
    a.weights_out = weights_out;
    a.width = width;
    a.kept = kept;
    a.left = left;
    a.budget = budget;
    a.first = first;
    a.recent = recent;
    // The fewest positions a thread that the bound allows: with eight two workgroups fit a CU
    // (4607 positions 10.6 us, with 32 a thread 18; 9000 positions 15 with 16, 19.6 with 32),
    // but what does not stay in registers is read several times (32768 positions 25 us with
    // 32 a thread, 32 with 8 or 16).  The lengths are on the device, so a bound far above
    // them has its price: both launches for 4607 positions take 19.4 us, under a bound of
    // 131072 26.7; 9000 positions 25.7 and 30.5.
    const unsigned groups = unsigned(rows);
    const int held = ceil_div(batch->max_context, kSelectThreads);
    if (held <= 8) kv_evict_select_kernel<8><<<groups, kSelectThreads, 0, stream>>>(a);
    else if (held <= 16) kv_evict_select_kernel<16><<<groups, kSelectThreads, 0, stream>>>(a);
    else kv_evict_select_kernel<32><<<groups, kSelectThreads, 0, stream>>>(a);
    if (int st = launch_status()) return st;
    const int kb = cache->k_format == NVFP4_KV_MXFP8 ? 8 : 4, vb = cache->v_format == NVFP4_KV_MXFP8 ? 8 : 4;
    return kv_dim(cache->head_dim, [&](auto dim) {
        constexpr int D = decltype(dim)::value;
        static_assert(1 + KvSide<D, 8>::kPieces + kValueParts <= kMostParts);
        const int key_parts = 1 + (kb == 8 ? KvSide<D, 8>::kPieces : KvSide<D, 4>::kPieces);
        kv_evict_move_kernel<D><<<unsigned(ceil_div(rows, int64_t(kXcds)) * kXcds * (key_parts + kValueParts)), kMoveThreads, 0, stream>>>(
            a, kb, vb, key_parts, key_parts + kValueParts);
        return launch_status();
    });
}
