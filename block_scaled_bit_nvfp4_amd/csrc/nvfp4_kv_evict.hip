// nvfp4_kv_evict.hip -- cuts sequences of the paged cache to a budget: which tokens of
// each head stay, and their move to the front (gfx950).
//
// Select, a workgroup per sequence and head: the candidates' weights, as whole numbers
// in their order, are counted by digits from the top, which finds the weight of the last
// one that stays and how many of its equals stay with it; then one walk in order writes
// the kept positions and moves their weights.
//
// Move: a kept token's slot is never past its old one, and both rise together.  So one
// workgroup can move a stretch of tokens at a time, all reads before all writes, and the
// places that it overwrites are behind everything it has yet to read.  The bytes of a
// unit are split over workgroups so that no two share any: a piece of the keys' codes, a
// part of the values' rows, either side's scales.
#include "nvfp4_kv.h"

namespace nvfp4 {

constexpr int kSelectThreads = 1024, kSelectWaves = kSelectThreads / kLanes;
constexpr int kDigitBits = 8, kDigits = 1 << kDigitBits;
constexpr int kMoveThreads = 1024;
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

// Sums over the workgroup of each wave's `n` (the same in its lanes): of the waves
// before this one, and of all.
__device__ __forceinline__ int waves_before(int n, int (&sh)[kSelectWaves], int &all) {
    const int wave = threadIdx.x / kLanes;
    if ((threadIdx.x & 63) == 0) sh[wave] = n;
    __syncthreads();
    int before = 0;
    all = 0;
#pragma unroll
    for (int w = 0; w < kSelectWaves; ++w) {
        const int x = sh[w];
        before += w < wave ? x : 0;
        all += x;
    }
    __syncthreads();
    return before;
}

__global__ void __launch_bounds__(kSelectThreads) kv_evict_select_kernel(EvictArgs a) {
    __shared__ int digits[kDigits];
    __shared__ int waves[kSelectWaves], waves2[kSelectWaves];
    __shared__ int chosen, above;
    const int tid = threadIdx.x, lane = tid & 63;
    const int s = blockIdx.x / a.kv.heads;
    const int length = a.kv.past[s];
    const float *w = a.weights + int64_t(blockIdx.x) * a.width;
    float *out = a.weights_out + int64_t(blockIdx.x) * a.width;
    int *kept = a.kept + int64_t(blockIdx.x) * a.budget;
    const int held = max(length, 0);
    // every position has a page, or the sequence stays as it is
    bool whole = held <= a.kv.capacity;
    if (whole) {
        const int pages = int(ceil_div(held, int64_t(1) << a.kv.page_shift));
        for (int p = tid; p < pages; p += kSelectThreads) {
            const int entry = a.kv.table[int64_t(s) * a.kv.width + p];
            whole &= entry >= 0 && entry < a.kv.pages;
        }
    }
    whole = __syncthreads_and(whole);
    if (!whole || held <= a.budget) {
        for (int i = tid; i < a.budget; i += kSelectThreads) kept[i] = whole && i < held ? i : -1;
        if (whole && out != w)
            for (int i = tid; i < held; i += kSelectThreads) out[i] = w[i];
        return;
    }
    // Among the candidates lo .. hi - 1 `take` stay: those of a larger order than
    // `border`, and the first `equals` of that order.
    const int lo = a.first, hi = held - a.recent;
    const int take = a.budget - a.first - a.recent;
    uint32_t border = 0;
    int want = take;
    for (int shift = 32 - kDigitBits; shift >= 0; shift -= kDigitBits) {
        for (int i = tid; i < kDigits; i += kSelectThreads) digits[i] = 0;
        __syncthreads();
        for (int i = lo + tid; i < hi; i += kSelectThreads) {
            const uint32_t o = weight_order(w[i]);
            if (shift == 32 - kDigitBits || (o ^ border) >> (shift + kDigitBits) == 0)
                atomicAdd(&digits[o >> shift & (kDigits - 1)], 1);
        }
        __syncthreads();
        if (tid < kLanes) {
            // a lane's four digits from the top; the lanes' sums before it
            const int top = kDigits - 1 - 4 * lane;
            int mine = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) mine += digits[top - j];
            int upto = mine;
#pragma unroll
            for (int d = 1; d < kLanes; d <<= 1) {
                const int y = __shfl_up(upto, d);
                upto += lane >= d ? y : 0;
            }
            int before = upto - mine;
            if (want > 0 && before < want && upto >= want) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int n = digits[top - j];
                    if (before < want && before + n >= want) {
                        chosen = top - j;
                        above = before;
                    }
                    before += n;
                }
            }
            if (want == 0 && lane == 0) {
                chosen = kDigits - 1;
                above = 0;
            }
        }
        __syncthreads();
        border |= uint32_t(chosen) << shift;
        want -= above;
        __syncthreads();
    }
    const int equals = want;
    // In order: a stretch of positions at a time, reads before writes (slots are never
    // past positions, so that what a stretch writes is behind the next one).
    int at = 0, same = 0;
    for (int first = 0; first < held; first += kSelectThreads) {
        const int i = first + tid;
        const bool in = i < held, candidate = in && i >= lo && i < hi;
        const float x = in ? w[i] : 0.0f;
        const uint32_t o = weight_order(x);
        const bool equal = candidate && o == border;
        const unsigned long long equal_lanes = __ballot(equal);
        int all_equal;
        const int rank = same + waves_before(__popcll(equal_lanes), waves2, all_equal) +
                         __popcll(equal_lanes & ((1ull << lane) - 1));
        const bool stay = in && (!candidate || o > border || (equal && rank < equals));
        const unsigned long long lanes = __ballot(stay);
        int all;
        const int slot = at + waves_before(__popcll(lanes), waves, all) + __popcll(lanes & ((1ull << lane) - 1));
        if (stay) {
            kept[slot] = i;
            out[slot] = x;
        }
        at += all;
        same += all_equal;
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
    constexpr int kDeep = 4;
    constexpr int kTokens = kMoveThreads / COLUMNS;
    const int column = threadIdx.x % COLUMNS, lane_token = threadIdx.x / COLUMNS;
    const KvView &v = a.kv;
    const auto place = [&](int pos) {
        const int page = v.table[int64_t(s) * v.width + (pos >> v.page_shift)];
        return reinterpret_cast<T *>(plane + v.unit_of(page, head, pos) * unit_bytes + offset(pos & (kKvUnit - 1), column));
    };
    for (int base = 0; base < a.budget; base += kDeep * kTokens) {
        int from[kDeep];
        T x[kDeep];
#pragma unroll
        for (int k = 0; k < kDeep; ++k) {
            const int i = base + k * kTokens + lane_token;
            from[k] = i < a.budget ? kept[i] : -1;
            if (from[k] == i) from[k] = -1;              // it stays where it is
        }
#pragma unroll
        for (int k = 0; k < kDeep; ++k)
            if (from[k] >= 0) x[k] = *place(from[k]);
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kDeep; ++k)
            if (from[k] >= 0) *place(base + k * kTokens + lane_token) = x[k];
    }
}

template <int D, int BITS, int SIDE>
__device__ __forceinline__ void move_side(const EvictArgs &a, int s, int head, const int *kept, int part) {
    typedef KvSide<D, BITS> S;
    if (part == 0) {
        move_tokens<1, S::kBlocks>(a, s, head, kept, a.kv.scales[SIDE], S::kUnitScales,
                                   [](int r, int c) { return SIDE == 0 ? S::key_scale(r, c) : S::value_scale(r, c); });
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
    const int row = blockIdx.x / parts, part = blockIdx.x % parts;
    const int head = row % a.kv.heads, s = row / a.kv.heads;
    const int *kept = a.kept + int64_t(row) * a.budget;
    const int last = kept[a.budget - 1];
    if (part == 0 && head == 0 && threadIdx.x == 0) {
        const int held = a.kv.past[s];
        a.left[s] = last >= 0 ? a.budget : held;
    }
    if (last < a.budget) return;                         // nothing was cut
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
    kv_evict_select_kernel<<<unsigned(rows), kSelectThreads, 0, stream>>>(a);
    if (int st = launch_status()) return st;
    const int kb = cache->k_format == NVFP4_KV_MXFP8 ? 8 : 4, vb = cache->v_format == NVFP4_KV_MXFP8 ? 8 : 4;
    return kv_dim(cache->head_dim, [&](auto dim) {
        constexpr int D = decltype(dim)::value;
        static_assert(1 + KvSide<D, 8>::kPieces + kValueParts <= kMostParts);
        const int key_parts = 1 + (kb == 8 ? KvSide<D, 8>::kPieces : KvSide<D, 4>::kPieces);
        kv_evict_move_kernel<D><<<unsigned(rows * (key_parts + kValueParts)), kMoveThreads, 0, stream>>>(
            a, kb, vb, key_parts, key_parts + kValueParts);
        return launch_status();
    });
}
