// nvfp4_attn.h -- what the attention kernels over the paged cache share: their
// arguments, the map from workgroups to rows and keys, the loads and decodes of a
// 16-token unit as matrix operands, and the softmax state.  Internal to the
// library.
//
// Both kernels compute S^T = K Q^T with keys as the rows of the A operand and query
// rows as the columns of B, and O^T = V^T P^T.  The accumulator of the first product
// then holds, in one lane, several keys of one query row: row sums and rescales
// need no other lane, and the exponentials, rounded to bf16, are the B operand of the
// second product as they stand (the order of keys in that contraction is chosen to
// match, and the cache's value layout with it).
//
// That rounding, at most 2^-8 of a weight, is chosen for the one matrix instruction that
// it takes: the remainders as a second operand would double those of the second
// product, which bound chunks. The outputs are divided by the sum of the weights as
// rounded, so that it does not shift them. Against 64-bit arithmetic the outputs are 0.0017
// to 0.0023 off (2-norm), of which 0.0016 is their own rounding to bf16. Everything
// else, scores, references, sums, parts and the log-sum-exp, is fp32.
#pragma once

#include <atomic>

#include "nvfp4_kv.h"

namespace nvfp4 {

constexpr int kMaxSplits = 256;     // splits of the key axis (the join's threads)
constexpr int kNarrowRows = 16;     // rows of the narrow kernel's tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNegInf = -__builtin_inff();

// The weights' reference is moved only when a lane's weights of a tile sum to more
// than this: they stay far inside fp32 with bf16's relative rounding unchanged, and
// most tiles neither look for their maximum nor rescale.
constexpr float kMaxSum = 1024.0f;

// How a kernel cuts the work: rows of a tile, keys of a split (a multiple of 128),
// how many splits at most, how tiles are found (0: by the offsets; else so many tile
// indexes per sequence), and its first part row in the workspace.
struct AttnCut {
    int rows, keys, splits, tiles_per_seq, first_row;
};

// Where a row's parts are: part row first + z * stride of each of `pieces` splits z.
struct RowInfo {
    int first, stride, pieces, unused;
};

struct AttnArgs {
    KvView kv;
    const uint16_t *q;
    uint16_t *out;
    float *lse;
    const unsigned long long *tree;
    int64_t q_stride, out_stride;
    int q_heads, group;
    int window;
    float scale_log2;      // scale * log2(e)
    int narrow_rows;       // sequences of at most so many rows (new tokens x group) are the narrow kernel's
    bool reused;           // whether several tiles read a sequence's keys
    AttnCut cut[2];        // the narrow kernel's, the wide kernel's
    RowInfo *info;         // [tokens * q_heads]; NULL where no tile is split
    int part_rows;
    float *part_o;         // [part_rows][D], relative to 2^m
    float *part_ml;        // [part_rows][4]: m (base 2), l, lr, unused
};

// One workgroup's rows: rows (token, head of the group) of one sequence, token
// major, in tiles; tile t of sequence s has the index
// floor(offsets[s] * group / rows) + s + t, so that it is found without a prefix sum
// over the sequences (some indexes have no tile).  Where short sequences stand among
// long ones, the narrow kernel has a few indexes for each sequence instead.
struct RowTile {
    int s;                 // sequence
    int begin;             // its first token row
    int n;                 // its new tokens
    int past;
    int row0, rows;        // first row of the tile, and the sequence's rows
    int lo, hi;            // the keys that some row of the tile may see: lo <= j < hi
    int inner_lo, inner_hi;  // the keys that every row sees (by position)
    bool some;             // whether the item has a tile
};

__device__ __forceinline__ RowTile row_tile(const AttnArgs &a, int cls, int item) {
    const KvView &v = a.kv;
    const int tile_rows = a.cut[cls].rows, each = a.cut[cls].tiles_per_seq;
    RowTile r;
    // The item's sequence is the last one whose first item is not past it; the
    // lanes load 64 sequences' facts at once, so the whole search costs one
    // memory latency for each 64 sequences.
    const int lane = threadIdx.x & 63;
    int first_item = -1, end = 0;
    r.s = r.begin = r.past = 0;
    for (int base = 0; base < v.seqs; base += kLanes) {
        const int s = min(base + lane, v.seqs - 1);
        int begin, stop, past;
        v.sequence(s, begin, stop, past);
        const int item0 = each > 0 ? s * each : int(int64_t(begin) * a.group / tile_rows) + s;
        const int c = __popcll(__ballot(base + lane < v.seqs && item0 <= item));
        if (c == 0) break;
        r.s = base + c - 1;
        first_item = __builtin_amdgcn_readlane(item0, c - 1);
        r.begin = __builtin_amdgcn_readlane(begin, c - 1);
        end = __builtin_amdgcn_readlane(stop, c - 1);
        r.past = __builtin_amdgcn_readlane(past, c - 1);
        if (c < kLanes) break;
    }
    r.n = end - r.begin;
    r.rows = r.n * a.group;
    r.row0 = (item - first_item) * tile_rows;
    r.some = first_item >= 0 && r.row0 < r.rows && (r.rows > a.narrow_rows) == (cls == 1);
    const int first = r.some ? r.row0 / a.group : 0;
    const int last = r.some ? min(r.row0 + tile_rows, r.rows) - 1 : 0;
    const int i1 = last / a.group;
    r.lo = a.window > 0 ? max(0, r.past + first + 1 - a.window) : 0;
    r.hi = min(a.tree ? r.past + r.n : r.past + i1 + 1, v.capacity);
    r.inner_lo = a.window > 0 ? max(0, r.past + i1 + 1 - a.window) : 0;
    r.inner_hi = min(a.tree ? r.past : r.past + first + 1, v.capacity);
    return r;
}

// The keys lo .. hi - 1 of split z of a tile, in `splits` in all: lo is a multiple of
// 64 plus whole splits, and the last split takes what is left.  Its parts' first row in
// the workspace, and whether there is work (split 0 has it always: rows that see
// nothing are written too).
struct KeyRange {
    int lo, hi, splits, part;
    bool some;
};
__device__ __forceinline__ KeyRange key_range(const AttnArgs &a, int cls, const RowTile &r, int item, int head, int z) {
    const AttnCut &c = a.cut[cls];
    KeyRange k;
    const int base = r.lo & ~63;
    const int all = max(r.hi - base, 0);
    k.splits = min((all + c.keys - 1) / c.keys, c.splits);
    k.lo = base + z * c.keys;
    k.hi = z + 1 >= k.splits ? r.hi : k.lo + c.keys;
    k.part = c.first_row + ((item * a.kv.heads + head) * c.splits + z) * c.rows;
    k.some = z == 0 || z < k.splits;
    return k;
}

// Eight codes -> the bf16 operand, times the power of two in `unit`'s exponent.
__device__ __forceinline__ bf16x8 codes8(uint32_t lo, uint32_t hi, float unit) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, unit, false);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, unit, true);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, unit, false);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, unit, true);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}
__device__ __forceinline__ bf16x8 codes4(uint32_t w, float unit) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, unit, 0);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, unit, 1);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, unit, 2);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, unit, 3);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Byte `i` of `w` as the fp32 whose exponent field it is.
__device__ __forceinline__ float unit_of_byte(uint32_t w, int i) {
    return __uint_as_float(__builtin_amdgcn_ubfe(w, 8 * i, 8) << 23);
}

// A load of BYTES per lane into words.
template <int BYTES>
__device__ __forceinline__ void load_words(const uint8_t *p, uint32_t *w) {
    if constexpr (BYTES == 16) {
        const u32x4 t = *reinterpret_cast<const u32x4 *>(p);
        w[0] = t[0]; w[1] = t[1]; w[2] = t[2]; w[3] = t[3];
    } else if constexpr (BYTES == 8) {
        const u32x2 t = *reinterpret_cast<const u32x2 *>(p);
        w[0] = t[0]; w[1] = t[1];
    } else if constexpr (BYTES == 4) {
        w[0] = *reinterpret_cast<const uint32_t *>(p);
    } else {
        w[0] = *reinterpret_cast<const uint16_t *>(p);
    }
}

// Two elements (2 jp, 2 jp + 1 of a row's D / 16) of token i of a lane's quad.
template <int D, int BITS>
__device__ __forceinline__ uint32_t value_pair(const uint32_t *w, int i, int jp, float unit) {
    if constexpr (BITS == 8) {
        const uint32_t x = w[i * (D / 64) + jp / 2];
        return jp & 1 ? as_u32(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, unit, true))
                      : as_u32(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, unit, false));
    } else {
        const int byte = i * (D / 32) + jp;
        const uint32_t x = w[byte / 4];
        switch (byte & 3) {
            case 0: return as_u32(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, unit, 0));
            case 1: return as_u32(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, unit, 1));
            case 2: return as_u32(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, unit, 2));
            default: return as_u32(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, unit, 3));
        }
    }
}

// Clears token i's codes of a lane's quad.
template <int D, int BITS>
__device__ __forceinline__ void clear_token(uint32_t *w, int i) {
    constexpr int kBits = D / 16 * BITS;             // of a token
#pragma unroll
    for (int k = 0; k < 4 * kBits / 32; ++k) {
        const int from = i * kBits - 32 * k, to = from + kBits;
        if (to <= 0 || from >= 32) continue;
        w[k] &= ~((to >= 32 ? ~0u : (1u << to) - 1u) & (from <= 0 ? ~0u : ~0u << from));
    }
}

// Low and high halves of a pair of words side by side.
__device__ __forceinline__ uint32_t low_halves(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x05040100u); }
__device__ __forceinline__ uint32_t high_halves(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x07060302u); }

typedef short s16x4 __attribute__((ext_vector_type(4)));

// s_waitcnt operands: for all loads from memory, for all of shared memory's.
constexpr int kWaitLoads = 0x0F70, kWaitLds = 0xC07F;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    bf16x2 v;
    v[0] = static_cast<__bf16>(a);
    v[1] = static_cast<__bf16>(b);
    return as_u32(v);
}

__device__ __forceinline__ float piece_weight(float mz, float m) {
    return mz == kNegInf ? (m == kNegInf ? 1.0f : 0.0f) : exp2_fast(mz - m);
}

// What a row that has no maximum yet adds to its sum in a tile where it sees keys:
// their scores are all minus infinity (an infinite query) or NaN.  A row that sees
// nothing keeps a sum of zero, and zeros are its output; such a one divides zeros by a
// sum of zero weights and is NaN.  A maximum found later clears the mark.
__device__ __forceinline__ float no_maximum(float m, bool sees) { return m == kNegInf && sees ? 1.0f : 0.0f; }

// log(sum of exponentials) from a base-2 maximum and the sum relative to it.
__device__ __forceinline__ float lse_of(float m, float l) {
    if (m == kNegInf) return l == 0.0f ? kNegInf : __builtin_nanf("");
    return (m + __builtin_amdgcn_logf(l)) * kLn2;
}

int wide_rows(int dim);            // rows of the wide kernel's tile

// Raises a kernel's limit of dynamic shared memory, once per device (by several
// threads at once, it may be twice).
template <auto KERNEL>
bool raise_lds(int bytes) {
    constexpr int kDevices = 64;
    static std::atomic<bool> done[kDevices];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kDevices) return false;
    if (done[dev].load(std::memory_order_acquire)) return true;
    if (hipFuncSetAttribute(reinterpret_cast<const void *>(KERNEL), hipFuncAttributeMaxDynamicSharedMemorySize,
                            bytes) != hipSuccess)
        return false;
    done[dev].store(true, std::memory_order_release);
    return true;
}

// `tiles`: tile indexes.
int launch_attn_narrow(const AttnArgs &a, int64_t tiles, int dim, int k_format, int v_format, hipStream_t stream);
int launch_attn_wide(const AttnArgs &a, int64_t tiles, int dim, int k_format, int v_format, hipStream_t stream);
// Joins the splits; `many`: a workgroup per row, for rows in many splits.
int launch_attn_join(const AttnArgs &a, bool many, int dim, hipStream_t stream);

}  // namespace nvfp4
