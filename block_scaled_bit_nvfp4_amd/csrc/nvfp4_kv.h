// nvfp4_kv.h -- the paged key/value cache of nvfp4_kv_append, nvfp4_kv_read and
// nvfp4_kv_attention: its layout as compile-time facts, and the device helpers
// the three share.  Internal to the library; the public definition of the
// layout is in nvfp4.h.
#pragma once

#include "nvfp4_host.h"

namespace nvfp4 {

constexpr int kKvUnit = 16;            // tokens of a unit
constexpr int kKvMaxPages = 1 << 30;
constexpr int kKvMaxPositions = 1 << 30;   // that a sequence's table names
constexpr int64_t kMaxGrid = int64_t(1) << 32;   // threads along one extent of a grid stay below this

// One side (keys or values) of a unit at head dimension D and BITS per code.
template <int D, int BITS>
struct KvSide {
    static constexpr int kRow = D * BITS / 8;            // code bytes of a token
    static constexpr int kUnitCodes = kKvUnit * kRow;
    static constexpr int kBlocks = D / kMxBlock;         // scale bytes of a token
    static constexpr int kUnitScales = kKvUnit * kBlocks;
    // keys: [piece][token][kPiece]; a lane's load is one piece
    static constexpr int kPiece = kRow / 4 < 16 ? kRow / 4 : 16;
    static constexpr int kPieces = kRow / kPiece;
    static constexpr int kPieceDims = kPiece * 8 / BITS;
    // values: [slot][quad][row][token of the slot][kPart]; a lane's load is one
    // row's slot
    static constexpr int kPart = kRow / 16;              // bytes of a token in a row
    static constexpr int kSlot = 4 * kPart < 16 ? 4 * kPart : 16;
    static constexpr int kSlotTokens = kSlot / kPart;
    static constexpr int kSlots = 4 / kSlotTokens;

    // Offset in the unit of byte `b` of token `r`'s codes.
    static __device__ __forceinline__ int key_code(int r, int b) {
        return (b / kPiece) * (kKvUnit * kPiece) + r * kPiece + b % kPiece;
    }
    static __device__ __forceinline__ int value_code(int r, int b) {
        const int t = r & 3;
        return (((t / kSlotTokens * 4 + (r >> 2)) * 16 + b / kPart) * kSlotTokens + t % kSlotTokens) * kPart +
               b % kPart;
    }
    // Offset in the unit of the scale byte of token `r`'s block `b`.
    static __device__ __forceinline__ int key_scale(int r, int b) { return r * kBlocks + b; }
    static __device__ __forceinline__ int value_scale(int r, int b) { return ((r >> 2) * kBlocks + b) * 4 + (r & 3); }
};

// The cache and the batch as the kernels take them.
struct KvView {
    uint8_t *codes[2], *scales[2];       // keys, values
    int pages, page_shift, heads;        // tokens of a page: 1 << page_shift
    const int *table, *offsets, *past;
    int width, seqs, tokens;
    int capacity;                        // tokens that the table can name: width << page_shift

    // Sequence s's rows are [begin, end) of the new tokens and start at position
    // `past` of the sequence; whatever the arrays hold, 0 <= begin <= end <=
    // tokens and 0 <= past <= capacity.
    __device__ __forceinline__ void sequence(int s, int &begin, int &end, int &before) const {
        begin = min(max(offsets[s], 0), tokens);
        end = min(max(offsets[s + 1], begin), tokens);
        before = min(max(past[s], 0), capacity);
    }
    // The page of sequence s's position `pos` in two steps, for loads ahead of their
    // use: the table's entry (any one where `pos` is past the table), then the page, or
    // -1 where there is none.
    __device__ __forceinline__ int entry_at(int s, int pos) const {
        return table[int64_t(s) * width + (min(max(pos, 0), capacity - 1) >> page_shift)];
    }
    // The entry as a scalar load, for `s` and `pos` that are the same in the whole wave.
    __device__ __forceinline__ int entry_at_scalar(int s, int pos) const {
        const int at = __builtin_amdgcn_readfirstlane(min(max(pos, 0), capacity - 1) >> page_shift);
        typedef __attribute__((address_space(4))) const int32_t Constant;
        return ((Constant *)(table + int64_t(__builtin_amdgcn_readfirstlane(s)) * width))[at];
    }
    __device__ __forceinline__ int page_in(int entry, int pos) const {
        return pos >= 0 && pos < capacity && entry >= 0 && entry < pages ? entry : -1;
    }
    // The unit (of a head's units in the whole pool) of position `pos` in page `p`.
    __device__ __forceinline__ int64_t unit_of(int p, int head, int pos) const {
        const int shift = page_shift - 4;
        return ((int64_t(p) * heads + head) << shift) + ((pos & ((1 << page_shift) - 1)) >> 4);
    }
};

// The number of i in 0..n-1 with key(i) <= x, for keys that do not decrease,
// found by a whole wave (x the same in its lanes): one load latency for each 64
// keys, where a binary search would take one for each halving.
template <class Key>
__device__ __forceinline__ int wave_count_le(int n, int64_t x, Key key) {
    const int lane = threadIdx.x & 63;
    for (int base = 0;; base += kLanes) {
        const bool le = base + lane < n && key(base + lane) <= x;
        const int c = __popcll(__ballot(le));
        if (c < kLanes) return base + c;
    }
}

// Host: the checks that the three entry points share.  Fills `v`.
int kv_check(const nvfp4_kv_cache *cache, const nvfp4_kv_batch *batch, KvView &v);

// f(KvSide-style tag) dispatch helpers.
template <int V>
struct IntC {
    static constexpr int value = V;
};
template <class F>
int kv_dim(int dim, F f) {
    switch (dim) {
        case 64: return f(IntC<64>());
        case 128: return f(IntC<128>());
        default: return f(IntC<256>());
    }
}
template <class F>
int kv_bits(int format, F f) {
    return format == NVFP4_KV_MXFP8 ? f(IntC<8>()) : f(IntC<4>());
}

}  // namespace nvfp4
