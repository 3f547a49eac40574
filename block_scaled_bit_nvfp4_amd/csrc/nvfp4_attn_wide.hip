// nvfp4_attn_wide.hip -- attention of many query rows over the paged cache
// (prefill chunks, wide verifies) on gfx950.
//
// A workgroup of eight waves walks the keys in tiles of kKeys = 8192 / D.  Keys and
// values are decoded to bf16 once per workgroup, into shared memory and as whole
// operands of v_mfma_f32_32x32x16_bf16: the waves read them with conflict-free
// 16-byte loads, and the cache's byte order makes each thread's share of the decode
// one load and a few stores.  The stores do conflict, those of values by their stride
// of 16 bytes, those of 4-bit keys by their two pieces a kilobyte apart: 10 % of shared
// memory's busy cycles, with 4-bit keys at heads of 128 and 256 17 to 18 %.
//
// The two waves of a SIMD work in opposite phases, a barrier between phases: while
// one multiplies (the values of tile i - 1 by its weights, then the keys of tile i by
// its queries), the other takes tile i's softmax and decodes its share of the tiles
// to come, so that the matrix and the vector pipe of a SIMD both stay busy.  Keys are
// decoded two tiles ahead, values one, into rings of two, between the matrix
// instructions; codes are loaded one tile before that.
//
// At D <= 128 a wave owns 32 rows.  At D = 256 two waves own 32 rows together,
// each half the elements: they add their halves of the scores through shared
// memory, take the same softmax, and each keeps half of the output.
//
// Measured: 2048 tokens of 40 heads of 128 over 32768 keys 1220 us, 1091 TFLOP/s (1190
// to 1280 us from card to card; a large library product of matrices reaches 1270
// TFLOP/s, at a clock that both lower); 512 tokens of 32 heads over 8192 keys 79 us,
// of which the splits' parts and their join take 15.  Per tile and CU 1.75 us at 128, bound by the matrix instructions; 2.5 us at
// 64, by the exponentials, of which there are twice as many for each product; 1.2 us for
// half the rows at 256, by the decode and the phases' starts.
#include "nvfp4_attn.h"

namespace nvfp4 {

typedef float floatx16 __attribute__((ext_vector_type(16)));

template <int D>
struct WideShape {
    static constexpr int kWaves = 8;
    static constexpr int kThreads = kWaves * kLanes;
    static constexpr int kHalves = D == 256 ? 2 : 1;   // waves that share 32 rows
    static constexpr int kRows = 32 * kWaves / kHalves;
    static constexpr int kKeys = 8192 / D;             // of a tile
    static constexpr int kUnits = kKeys / kKvUnit;
    static constexpr int kBlocks32 = kKeys / 32;
    static constexpr int kDimSteps = D / 16;           // MFMAs of a 32-key block's scores
    static constexpr int kDimBlocks = D / 32;          // accumulators of the output
    static constexpr int kSide = kKeys * D * 2;        // bytes of a tile's keys (and of its values): 16 KiB
    static constexpr int kMarks = kKeys * (D / kMxBlock);
    static constexpr int kRing = 2;
    // shared memory: keys, values, marks, and the halves' scores
    static constexpr int kValuesAt = kRing * kSide;
    static constexpr int kMarksAt = 2 * kRing * kSide;
    static constexpr int kScoresAt = kMarksAt + kRing * kMarks;
    static constexpr int kUsed = kScoresAt + (kHalves == 2 ? kWaves * kLanes * 64 : 0);
    static constexpr int kOut = kWaves * 32 * (64 + 4) * 4;            // the rows on their way out, over all that
    static constexpr int kLds = kUsed > kOut ? kUsed : kOut;
};

// One thread's share of a tile between its load and its store to shared memory: 16
// elements of one key, and 8 elements of a value row of two keys (D = 64: 4
// elements of four).  A wave's items are all of one unit.
template <int D, int KB, int VB>
struct WideStage {
    typedef WideShape<D> W;
    typedef KvSide<D, KB> KS;
    typedef KvSide<D, VB> VS;
    static constexpr int kItems = W::kThreads / W::kUnits;           // of a unit, keys or values
    static_assert(kItems == kKvUnit * D / 16 && kItems % kLanes == 0, "a key item per thread, a unit per wave");
    static constexpr int kTokens = D == 64 ? 4 : 2, kDims = 16 / kTokens;
    static constexpr int kParts = D / 16 / kDims;                    // of a value row
    static_assert(kItems == kKvUnit / kTokens * 16 * kParts, "a value item per thread");
    static constexpr int kValueWords = 16 * VB / 32;
    // an item's value bytes stand together unless a slot, or a row's part, splits them
    static constexpr int kRun = VS::kSlotTokens >= kTokens && kParts == 1 ? kValueWords * 4 : kDims * VB / 8;
    static constexpr int kRunTokens = kRun * 8 / (kDims * VB);

    uint32_t k[KB / 2], ks, v[kValueWords], vs;
    // offsets of the item's bytes in its unit, and of its operands in a ring slot
    uint32_t k_at, ks_at, v_at, vs_at, k_to, v_to;
    int token, block;              // the value item's first token in the tile, and its block

    __device__ __forceinline__ WideStage() {
        const int i = threadIdx.x % kItems, unit = threadIdx.x / kItems;
        // keys; in 16-byte pieces of 4-bit codes, two items of a piece side by side
        const bool two = KB == 4 && KS::kPiece == 16;
        const int r = two ? (i >> 1) & 15 : i & 15, part = two ? (i >> 5) * 2 + (i & 1) : i >> 4;
        k_at = KS::key_code(r, part * 2 * KB);
        ks_at = KS::key_scale(r, part / 2);
        k_to = (((unit >> 1) * W::kDimSteps + part) * kLanes + (unit & 1) * 16 + r) * 16;
        // values: quad (half + 2 * upper), pair of its tokens, row, part of the row
        const int row = i & 15, quad = D == 64 ? i >> 4 : ((i >> 4) & 1) * 2 + ((i >> 6) & 1);
        const int pair = D == 64 ? 0 : (i >> 5) & 1, piece = D == 64 ? 0 : i >> 7;
        const int t0 = quad * 4 + pair * 2;
        v_at = VS::value_code(t0, row * VS::kPart + piece * (kDims * VB / 8));
        vs_at = VS::value_scale(t0, row * VS::kBlocks / 16);
        // operand (unit, dim block, half, row): eight keys, the quad's four at
        // 8 * (quad / 2) bytes
        v_to = ((unit * W::kDimBlocks + piece * kDims / 2) * kLanes + (quad & 1) * 32 + row) * 16 + (quad >> 1) * 8 + pair * 4;
        token = unit * kKvUnit + t0;
        block = row * VS::kBlocks / 16;
    }

    // `unit`: the pool's unit that this wave's items are of.
    __device__ __forceinline__ void load_keys(const KvView &kv, int64_t unit) {
        load_words<2 * KB>(kv.codes[0] + unit * KS::kUnitCodes + k_at, k);
        ks = (kv.scales[0] + unit * KS::kUnitScales)[ks_at];
    }
    __device__ __forceinline__ void load_values(const KvView &kv, int64_t unit) {
        const uint8_t *base = kv.codes[1] + unit * VS::kUnitCodes;
        // runs of tokens of a quad: in slots of their own, or one row's parts apart
#pragma unroll
        for (int n = 0; n < kValueWords * 4 / kRun; ++n) {
            constexpr uint32_t kNext = VS::kSlotTokens >= kTokens ? VS::kPart : 4 * 16 * VS::kSlot;
            load_words<kRun>(base + v_at + n * kNext, v + n * kRun / 4);
        }
        load_words<kTokens>(kv.scales[1] + unit * VS::kUnitScales + vs_at, &vs);
    }
    // In an edge tile: values of keys outside lo..hi - 1 or without a page, and NaN
    // blocks, become zeros, the latter marked.
    __device__ __forceinline__ void clear_values(uint8_t *marks, int key, int lo, int hi, unsigned some) {
#pragma unroll
        for (int i = 0; i < kTokens; ++i) {
            const int pos = key + token + i;
            const bool held = ((some >> (token / kKvUnit)) & 1) && pos >= lo && pos < hi;
            const bool nan = ((vs >> (8 * i)) & 0xFFu) == 0xFFu;
            marks[(token + i) * VS::kBlocks + block] = held && nan ? 1 : 0;
            if (held && !nan) continue;
            vs &= ~(0xFFu << (8 * i));
#pragma unroll
            for (int w = 0; w < kValueWords; ++w) {
                // the bits of word w that are token i's
                constexpr int kBits = kDims * VB;
                const int from = i * kBits - 32 * w, to = from + kBits;
                const uint32_t mine = to <= 0 || from >= 32 ? 0u
                                      : (to >= 32 ? ~0u : (1u << to) - 1u) & (from <= 0 ? ~0u : ~0u << from);
                v[w] &= ~mine;
            }
        }
    }
    // The decode to the operands of ring slots in steps of a few instructions,
    // which stand between matrix instructions: the values' pairs of elements, each
    // converted, then paired over tokens and stored; and the keys' two halves.
    uint32_t held[4];
    static constexpr int kValueSteps = kDims, kKeySteps = 4;
    __device__ __forceinline__ void store_value_step(uint8_t *slot, int n) {
        const int jp = n / 2;
        if (n % 2 == 0) {
#pragma unroll
            for (int i = 0; i < kTokens; ++i) held[i] = value_pair<16 * kDims, VB>(v, i, jp, unit_of_byte(vs, i));
            return;
        }
        uint8_t *at = slot + v_to + jp * kLanes * 16;
        if constexpr (kTokens == 4) {
            *reinterpret_cast<u32x2 *>(at) = u32x2{low_halves(held[0], held[1]), low_halves(held[2], held[3])};
            *reinterpret_cast<u32x2 *>(at + 16 * 16) = u32x2{high_halves(held[0], held[1]), high_halves(held[2], held[3])};
        } else {
            *reinterpret_cast<uint32_t *>(at) = low_halves(held[0], held[1]);
            *reinterpret_cast<uint32_t *>(at + 16 * 16) = high_halves(held[0], held[1]);
        }
    }
    __device__ __forceinline__ void store_key_step(uint8_t *slot, int n) {
        const float scale = __uint_as_float(ks << 23);
        const int half = n / 2;
        // words 2 (n mod 2) and the next of the operand
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int pair = 2 * (n % 2) + i;      // of the half's eight elements
            uint32_t x;
            if constexpr (KB == 8)
                x = as_u32(i ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(k[2 * half + n % 2], scale, true)
                             : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(k[2 * half + n % 2], scale, false));
            else if (pair == 0) x = as_u32(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(k[half], scale, 0));
            else if (pair == 1) x = as_u32(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(k[half], scale, 1));
            else if (pair == 2) x = as_u32(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(k[half], scale, 2));
            else x = as_u32(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(k[half], scale, 3));
            held[pair] = x;
        }
        if (n % 2 == 1) reinterpret_cast<u32x4 *>(slot + k_to)[32 * half] = u32x4{held[0], held[1], held[2], held[3]};
    }
    __device__ __forceinline__ void store_values(uint8_t *slot) {
#pragma unroll
        for (int n = 0; n < kValueSteps; ++n) store_value_step(slot, n);
    }
    __device__ __forceinline__ void store_keys(uint8_t *slot) {
#pragma unroll
        for (int n = 0; n < kKeySteps; ++n) store_key_step(slot, n);
    }
};

// The table's entries of the tile at `key`: lane u (u < units) that of its unit u.
// They are made pages a tile later: a test here would wait for the load, and with
// it for every load before it.
__device__ __forceinline__ int wide_entries(const KvView &kv, int s, int key) {
    return kv.entry_at(s, key + (threadIdx.x & 63) * kKvUnit);
}
template <int D>
__device__ __forceinline__ int wide_pages(const KvView &kv, int entries, int key, int end) {
    const int u = threadIdx.x & 63, pos = key + u * kKvUnit;
    const bool ok = (u < WideShape<D>::kUnits) & (pos < end) & (pos < kv.capacity) & (entries >= 0) & (entries < kv.pages);
    return ok ? entries : -1;
}

// A barrier of the workgroup that orders shared memory only: global loads stay in
// flight across it.
__device__ __forceinline__ void phase_barrier() {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
    __builtin_amdgcn_sched_barrier(0);
}

// Orders a wave's own accesses to shared memory.
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
}

template <int D, int KB, int VB>
__global__ void __launch_bounds__(WideShape<D>::kThreads) attn_wide_kernel(AttnArgs a) {
    typedef WideShape<D> W;
    constexpr int kSteps = W::kDimSteps / W::kHalves, kDims = W::kDimBlocks / W::kHalves;    // a wave's own
    extern __shared__ __align__(16) uint8_t lds[];
    const int lane = threadIdx.x & 63, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // heads first: the tiles of a head, which read the same keys, meet in few
    // XCDs' caches; a sequence's last tiles, which have the most keys, go first
    const int item = int(gridDim.x / a.kv.heads) - 1 - int(blockIdx.x / a.kv.heads);
    const int head = blockIdx.x % a.kv.heads, z = blockIdx.y;
    const RowTile tile = row_tile(a, 1, item);
    if (!tile.some) return;
    const KeyRange keys = key_range(a, 1, tile, item, head, z);
    if (!keys.some) return;

    // Waves w and w + 4 share a SIMD and are in opposite phases; at D = 256 waves
    // 2 k and 2 k + 1 share rows.
    const int late = wave >> 2, half = W::kHalves == 2 ? wave & 1 : 0;
    const int row = tile.row0 + (wave / W::kHalves) * 32 + (lane & 31);
    const bool in = row < tile.rows;
    const int i = in ? row / a.group : 0;
    const int token = tile.begin + i, qhead = head * a.group + (in ? row - i * a.group : 0);
    const int pos = tile.past + i;
    const int klo = a.window > 0 ? max(0, pos + 1 - a.window) : 0;
    const int khi = in ? (a.tree ? tile.past : pos + 1) : 0;
    const unsigned long long tree = in && a.tree ? a.tree[token] : 0ull;
    bf16x8 q[kSteps];
    {
        const uint16_t *src = a.q + token * a.q_stride + qhead * D + half * kSteps * 16 + 8 * h;
#pragma unroll
        for (int m = 0; m < kSteps; ++m) {
            u32x4 w = {0, 0, 0, 0};
            if (in) w = *reinterpret_cast<const u32x4 *>(src + 16 * m);
            q[m] = __builtin_bit_cast(bf16x8, w);
        }
    }
    if (a.info && z == 0 && in && h == 0 && half == 0)
        a.info[int64_t(token) * a.q_heads + qhead] = RowInfo{keys.part + (row - tile.row0), W::kRows, keys.splits, 0};
    floatx16 o[kDims], s[W::kBlocks32];
    uint32_t p[W::kBlocks32][8];
    unsigned long long seen = 0;           // in an edge tile, bit 16 b + e where score e of block b is allowed
#pragma unroll
    for (int d = 0; d < kDims; ++d) o[d] = floatx16{};
    // Weights are 2^(score - sub); l is their sum, lr the sum of the weights as
    // rounded to bf16, which normalises the output.  lr comes from the smallest
    // matrix instruction, whose sixteen 4 x 4 products give each lane the sum of its
    // own four weights (dot2 runs on the matrix pipe as well, and waits for it: 60
    // cycles each beside a busy one).
    float sub = kNegInf, l = 0.0f;
    floatx4 lr = {0, 0, 0, 0};
    const s16x4 ones = {0x3F80, 0x3F80, 0x3F80, 0x3F80};
    const float scale = a.scale_log2;
    // rows that see nothing never have a maximum, and need none
    if (!in) sub = 0.0f;

    // The matrix phase: the values of one tile by its weights, added to the output,
    // then the scores of the next (its keys, rows, by the queries, columns).
    // kAhead operands are in flight, in an order that the compiler is kept to: left
    // to itself it waits for each pair.
    const auto multiply = [&](int value_slot, int key_slot, auto first_tag, auto between) {
        constexpr int kValues = decltype(first_tag)::value != 0 ? 0 : W::kUnits * kDims;
        constexpr int kAll = kValues + W::kBlocks32 * kSteps, kAhead = 8;
        const bf16x8 *vop = reinterpret_cast<const bf16x8 *>(lds + W::kValuesAt + value_slot * W::kSide) + half * kDims * kLanes + lane;
        const bf16x8 *kop = reinterpret_cast<const bf16x8 *>(lds + key_slot * W::kSide) + half * kSteps * kLanes + lane;
        const auto operand = [&](int n) {
            if (n < kValues) return vop[(n / kDims * W::kDimBlocks + n % kDims) * kLanes];
            n -= kValues;
            return kop[(n % W::kBlocks32 * W::kDimSteps + n / W::kBlocks32) * kLanes];
        };
        bf16x8 ahead[kAhead];
#pragma unroll
        for (int n = 0; n < kAhead; ++n) ahead[n] = operand(n);
        __builtin_amdgcn_sched_barrier(0);
        if (kValues > 0) {
            // meanwhile: the sum of the rounded weights, each lane's own
#pragma unroll
            for (int w = 0; w < 4 * W::kUnits; w += 2)
                lr = __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(ones, __builtin_bit_cast(s16x4, u32x2{p[w >> 3][w & 7], p[w >> 3][(w & 7) + 1]}), lr, 0, 0, 0);
        }
#pragma unroll
        for (int b = 0; b < W::kBlocks32; ++b) s[b] = floatx16{};
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int n = 0; n < kAll; ++n) {
            if (n < kValues) {
                const int u = n / kDims;
                const uint32_t *w = &p[u >> 1][4 * (u & 1)];
                o[n % kDims] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(ahead[n % kAhead], __builtin_bit_cast(bf16x8, u32x4{w[0], w[1], w[2], w[3]}), o[n % kDims], 0, 0, 0);
            } else {
                const int b = (n - kValues) % W::kBlocks32, m = (n - kValues) / W::kBlocks32;
                s[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(ahead[n % kAhead], q[m], s[b], 0, 0, 0);
            }
            if (n + kAhead < kAll) ahead[n % kAhead] = operand(n + kAhead);
            between(n);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // In an edge tile NaN blocks, left out of the values, reach the rows that see
    // their keys: the product of the marks with the allowed keys tells which.
    unsigned nan_rows = 0;                 // bit e: accumulator element e is NaN
    const auto spread_nan = [&](int slot) {
        static_assert(W::kMarks == 256, "a word of marks per lane");
        const uint8_t *marks = lds + W::kMarksAt + slot * W::kMarks;
        if (!__any(reinterpret_cast<const uint32_t *>(marks)[lane] != 0)) return;
        const int block = (lane & 15) * (D / kMxBlock) / 16;
#pragma unroll 1
        for (int u = 0; u < W::kUnits; ++u) {
            const unsigned now = unsigned(seen >> (8 * u));
            u32x4 mark, on;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                mark[e] = on[e] = 0;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int at = 2 * e + k, t = 8 * (at >> 2) + 4 * h + (at & 3);
                    mark[e] |= (marks[(u * kKvUnit + t) * (D / kMxBlock) + block] ? 0x3F80u : 0u) << (16 * k);
                    on[e] |= ((now >> at) & 1 ? 0x3F80u : 0u) << (16 * k);
                }
            }
            const floatx16 n = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, mark), __builtin_bit_cast(bf16x8, on), floatx16{}, 0, 0, 0);
#pragma unroll
            for (int e = 0; e < 16; ++e) nan_rows |= unsigned(n[e] > 0.0f) << e;
        }
    };
    // scores -> weights, and the running maximum and sums
    const auto softmax = [&](int key, unsigned some, bool edge) {
        if (edge) {
            const int last = min(khi, tile.hi);
            seen = 0;
#pragma unroll
            for (int b = 0; b < W::kBlocks32; ++b) {
                const int base = key + b * 32 + 4 * h;
                unsigned ok = 0;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int at = base + 8 * (e >> 2) + (e & 3);
                    ok |= unsigned((at >= klo) & (at < last)) << e;
                }
                if (a.tree) {
                    const int drafted = min(min(tile.n, 64), tile.hi - tile.past);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int t = base + 8 * (e >> 2) + (e & 3) - tile.past;
                        ok |= (unsigned((t >= 0) & (t < drafted)) & unsigned(tree >> (t & 63))) << e;
                    }
                }
                ok &= (((some >> (2 * b)) & 1) ? 0xFFu : 0u) | (((some >> (2 * b + 1)) & 1) ? 0xFF00u : 0u);
#pragma unroll
                for (int e = 0; e < 16; ++e) s[b][e] = (ok >> e) & 1u ? s[b][e] : kNegInf;
                seen |= static_cast<unsigned long long>(ok) << (16 * b);
            }
        }
        // The weights, against the reference that earlier tiles left.  It moves up
        // only where their sum shows a weight too large (or none was set), so most
        // tiles never look for their maximum.
        float sum[4];
        const auto exponentials = [&](float ref) {
#pragma unroll
            for (int b = 0; b < W::kBlocks32; ++b)
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    const float x = exp2_fast(__builtin_fmaf(s[b][e], scale, -ref));
                    const float y = exp2_fast(__builtin_fmaf(s[b][e + 1], scale, -ref));
                    float &to = sum[e / 2 % 4];        // four chains: one would wait for itself
                    to = b == 0 && e < 8 ? x + y : to + (x + y);
                    p[b][e / 2] = pack_bf16(x, y);
                }
            return (sum[0] + sum[1]) + (sum[2] + sum[3]);
        };
        float total = exponentials(sub == kNegInf ? 0.0f : sub);
        if (__any(sub == kNegInf || total > kMaxSum)) {
            float top = kNegInf;
#pragma unroll
            for (int b = 0; b < W::kBlocks32; ++b)
#pragma unroll
                for (int e = 0; e < 16; ++e) top = fmaxf(top, s[b][e]);
            top *= scale;
            top = fmaxf(top, __shfl_xor(top, 32));
            const float m = fmaxf(sub, top);
            const float by = m == sub ? 1.0f : exp2_fast(sub - m);
            sub = m;
            l = l * by + no_maximum(m, !edge || seen != 0);
            lr *= by;
#pragma unroll
            for (int d = 0; d < kDims; ++d) o[d] *= by;
            total = exponentials(sub == kNegInf ? 0.0f : sub);
        }
        l += total;
    };

    const unsigned all = (1u << W::kUnits) - 1;
    const auto valid = [&](int pages) { return unsigned(__ballot(pages >= 0)) & all; };
    const auto is_edge = [&](int key, unsigned some) {
        return (key < tile.inner_lo) | (key + W::kKeys > min(tile.inner_hi, keys.hi)) | (some != all);
    };
    const int tiles = (max(keys.hi - keys.lo, 0) + W::kKeys - 1) / W::kKeys;
    if (tiles > 0) {
        WideStage<D, KB, VB> stage;
        const auto key_at = [&](int t) { return keys.lo + t * W::kKeys; };
        const auto entries_at = [&](int t) { return wide_entries(a.kv, tile.s, key_at(t)); };
        const auto pages_of = [&](int entries, int t) { return wide_pages<D>(a.kv, entries, key_at(t), keys.hi); };
        const int my_unit = wave * kLanes / WideStage<D, KB, VB>::kItems;
        const auto unit_in = [&](int pages, int t) {
            return a.kv.unit_of(max(__builtin_amdgcn_readlane(pages, my_unit), 0), head, key_at(t) + my_unit * kKvUnit);
        };
        const auto values_slot = [&](int slot) { return lds + W::kValuesAt + slot * W::kSide; };
        const auto marks_slot = [&](int slot) { return lds + W::kMarksAt + slot * W::kMarks; };
        // Tile t's keys and values are in slot t mod 2.  some0, some1, ..: which
        // units of tiles t, t + 1, .. have pages; unit: the wave's unit of tile
        // t + 2, whose keys are loaded; the values of tile t + 1 are.
        const int entries0 = entries_at(0), entries1 = entries_at(1), entries2 = entries_at(2);
        int entries = entries_at(3);              // of tile t + 3
        int pages = pages_of(entries0, 0);
        unsigned some0 = valid(pages), some1, some2;
        int64_t unit = unit_in(pages, 0);
        stage.load_keys(a.kv, unit);
        stage.load_values(a.kv, unit);
        bool edge = is_edge(key_at(0), some0);
        stage.store_keys(lds);
        if (edge) stage.clear_values(marks_slot(0), key_at(0), tile.lo, tile.hi, some0);
        stage.store_values(values_slot(0));
        pages = pages_of(entries1, 1);
        some1 = valid(pages);
        unit = unit_in(pages, 1);
        stage.load_keys(a.kv, unit);
        stage.load_values(a.kv, unit);
        stage.store_keys(lds + W::kSide);
        pages = pages_of(entries2, 2);
        some2 = valid(pages);
        unit = unit_in(pages, 2);
        stage.load_keys(a.kv, unit);
        phase_barrier();
        if (late) phase_barrier();
        // D = 256: the halves of the scores meet
        floatx4 *const shared = reinterpret_cast<floatx4 *>(lds + W::kScoresAt) + lane;
        const auto give_scores = [&] {
            if constexpr (W::kHalves == 2)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    shared[(wave * 4 + e) * kLanes] = floatx4{s[0][4 * e], s[0][4 * e + 1], s[0][4 * e + 2], s[0][4 * e + 3]};
        };
        const auto take_scores = [&] {
            if constexpr (W::kHalves == 2)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const floatx4 x = shared[((wave ^ 1) * 4 + e) * kLanes];
#pragma unroll
                    for (int k = 0; k < 4; ++k) s[0][4 * e + k] += x[k];
                }
        };
        multiply(0, 0, IntC<1>(), [](int) {});
        give_scores();
        phase_barrier();
        for (int t = 0; t < tiles; ++t) {
            const int slot = t & 1;
            // The page numbers of tile t + 3 first: their load is older than those
            // that follow, and waiting for it later would be waiting for them.
            // Nothing here asks whether the tiles to come exist: past the last
            // one, loads go to some page and stores to slots that nobody reads.
            pages = pages_of(entries, t + 3);
            entries = entries_at(t + 4);
            take_scores();
            softmax(key_at(t), some0, edge);
            if (edge) spread_nan(slot);
            edge = is_edge(key_at(t + 1), some1);
            if (edge) stage.clear_values(marks_slot(slot ^ 1), key_at(t + 1), tile.lo, tile.hi, some1);
            some0 = some1;
            some1 = some2;
            some2 = valid(pages);
            const int64_t unit1 = unit_in(pages, t + 3);
            phase_barrier();
            // Tile t's values and tile t + 1's keys (after the last tile: unused
            // scores of old keys); meanwhile tile t + 1's values and tile t + 2's
            // keys are decoded, and the next ones' codes loaded.
            __builtin_amdgcn_s_setprio(1);
            multiply(slot, slot ^ 1, IntC<0>(), [&](int n) {
                typedef WideStage<D, KB, VB> S;
                constexpr int kKeysFrom = S::kValueSteps, kLoadsFrom = kKeysFrom + S::kKeySteps;
                if (n < kKeysFrom) stage.store_value_step(values_slot(slot ^ 1), n);
                else if (n < kLoadsFrom) stage.store_key_step(lds + slot * W::kSide, n - kKeysFrom);
                else if (n == kLoadsFrom) stage.load_values(a.kv, unit);
                else if (n == kLoadsFrom + 1) stage.load_keys(a.kv, unit1);
            });
            __builtin_amdgcn_s_setprio(0);
            give_scores();
            unit = unit1;
            phase_barrier();
        }
        if (!late) phase_barrier();
    }

    if (nan_rows != 0) {
#pragma unroll
        for (int e = 0; e < 16; ++e)
#pragma unroll
            for (int d = 0; d < kDims; ++d) o[d][e] = (nan_rows >> e) & 1 ? __builtin_nanf("") : o[d][e];
    }
    l += __shfl_xor(l, 32);
    const float norm = lr[0] + __shfl_xor(lr[0], 32);
    if (in && h == 0 && half == 0) {
        if (keys.splits > 1)
            *reinterpret_cast<float4 *>(a.part_ml + int64_t(keys.part + (row - tile.row0)) * 4) = float4{sub, l, norm, 0.0f};
        else if (a.lse)
            a.lse[int64_t(token) * a.q_heads + qhead] = lse_of(sub, l);
    }
    // Lane (h, row) holds value rows r = 8 x + 4 h + y, each D / 16 elements in a row
    // of the cache: element 2 d + jj of it in accumulator d's 8 jj + 4 x + y.  They
    // go out through shared memory, 64 elements of the wave's rows at a time, so that
    // 16 lanes write 64 elements of a row together (a lane's own 16 bytes at a time made
    // four times the requests: 512 tokens over 8192 keys 82.3 us, so 77.3).
    constexpr int kRowDims = D / 16, kOwn = kRowDims / W::kHalves;     // of a value row; this wave's of them
    constexpr int kPass = 64 / (8 * kOwn), kStride = 64 + 4;
    const int first = half * kOwn;
    const bool whole = keys.splits <= 1;
    const float inv = !whole ? 1.0f : sub == kNegInf && l == 0.0f ? 0.0f : 1.0f / norm;
    float *const rows = reinterpret_cast<float *>(lds) + wave * 32 * kStride;
    __syncthreads();
#pragma unroll
    for (int x0 = 0; x0 < 2; x0 += kPass) {
#pragma unroll
        for (int x = x0; x < x0 + kPass; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y)
#pragma unroll
                for (int d = 0; d < kDims; d += 2) {
                    const int e = 4 * x + y;
                    *reinterpret_cast<float4 *>(rows + (lane & 31) * kStride + (8 * (x - x0) + 4 * h + y) * kOwn + 2 * d) =
                        float4{o[d][e] * inv, o[d][8 + e] * inv, o[d + 1][e] * inv, o[d + 1][8 + e] * inv};
                }
        wave_fence();
        const int c = (lane & 15) * 4, at = (8 * x0 + c / kOwn) * kRowDims + first + c % kOwn;
#pragma unroll
        for (int n = 0; n < 8; ++n) {
            const int r = 4 * n + (lane >> 4);
            const float4 v = *reinterpret_cast<const float4 *>(rows + r * kStride + c);
            const int t = __shfl(token, r), qh = __shfl(qhead, r), mine = wave / W::kHalves * 32 + r;
            if (tile.row0 + mine >= tile.rows) continue;
            if (whole)
                *reinterpret_cast<u32x2 *>(a.out + t * a.out_stride + qh * D + at) = u32x2{pack_bf16(v.x, v.y), pack_bf16(v.z, v.w)};
            else
                *reinterpret_cast<float4 *>(a.part_o + int64_t(keys.part + mine) * D + at) = v;
        }
        wave_fence();
    }
}

int wide_rows(int dim) { return kv_dim(dim, [](auto d) { return WideShape<decltype(d)::value>::kRows; }); }

int launch_attn_wide(const AttnArgs &a, int64_t tiles, int dim, int k_format, int v_format, hipStream_t stream) {
    return kv_dim(dim, [&](auto d) {
        return kv_bits(k_format, [&](auto k) {
            return kv_bits(v_format, [&](auto v) {
                constexpr int D = decltype(d)::value, K = decltype(k)::value, V = decltype(v)::value;
                typedef WideShape<D> W;
                const int64_t groups = tiles * a.kv.heads;
                if (groups >= kMaxGrid / W::kThreads) return NVFP4_ESHAPE;
                if (!raise_lds<attn_wide_kernel<D, K, V>>(W::kLds)) return NVFP4_EHIP;
                attn_wide_kernel<D, K, V><<<dim3(unsigned(groups), unsigned(a.cut[1].splits)), W::kThreads, W::kLds,
                                            stream>>>(a);
                return launch_status();
            });
        });
    });
}

}  // namespace nvfp4
