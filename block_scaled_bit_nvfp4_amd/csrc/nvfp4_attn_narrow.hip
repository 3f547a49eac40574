// nvfp4_attn_narrow.hip -- attention of few query rows over the paged cache
// (decode, speculative verify) on gfx950, and the join of split rows.
//
// A workgroup owns 16 rows and a range of keys; its waves take 32-key tiles in turn,
// each with its own softmax state, and meet at the end.  The work is bound by the
// cache's bytes, so the codes and scales of a wave's next tile go to shared memory by
// direct loads while it works on one: they take no registers, and three workgroups
// of a CU keep 100 KB in flight.  A tile's codes are then read once, decoded in
// registers straight to operands of v_mfma_f32_16x16x32_bf16; sixteen rows are
// the least that instruction takes, so a group of one to sixteen query heads costs the
// same.  A tile's 230 vector and 18 matrix instructions take about half a microsecond of
// a SIMD, a third of the time that its bytes take, so that the masks of edge tiles, the
// search for the maximum and NaN have branches of their own.
//
// Measured: one token over 131008 keys of 8 heads of 128 (277 MB) 45 us, 6.2 TB/s,
// and 5 us for the join; 64 tokens over 8192 keys each 146 us (5.8 TB/s), over 1 to
// 8192 keys 84 us (4.4 TB/s: the last workgroups run alone); over 1037 keys of one
// sequence 9.6 us, of which 7 are the two launches.
#include "nvfp4_attn.h"

namespace nvfp4 {

constexpr int kTileKeys = 32;      // keys of a wave's tile: two units
constexpr int kNarrowWaves = 4, kNarrowThreads = kNarrowWaves * kLanes;

template <int D, int KB, int VB>
struct NarrowShape {
    typedef KvSide<D, KB> KS;
    typedef KvSide<D, VB> VS;
    static constexpr int kPerSimd = D == 256 ? 2 : D == 128 ? 3 : 4;                 // waves, by registers
    // a tile in shared memory: [key codes][value codes][scales]
    static constexpr int kValuesAt = 2 * KS::kUnitCodes, kScalesAt = kValuesAt + 2 * VS::kUnitCodes;
    static constexpr int kScaleBytes = 16 * D / 32, kScaleLoads = D == 256 ? 2 : 1;      // of a unit and side; of all four
    static constexpr int kTileBytes = kScalesAt + kScaleLoads * kLanes * 4;
    // the waves' outputs meet in parts of at most 8 elements of each value row
    static constexpr int kRowDims = D / 16, kPart = kRowDims < 8 ? kRowDims : 8;
    static constexpr int kCols = 16 * kPart + 4;       // floats of one row's part, padded against bank conflicts
    static constexpr int kMeet = kNarrowWaves * kNarrowRows * kCols * 4;
    static constexpr int kTiles = kNarrowWaves * kTileBytes;
    static constexpr int kStatesAt = kTiles > kMeet ? kTiles : kMeet;
    static constexpr int kLds = kStatesAt + 3 * kNarrowWaves * kNarrowRows * 4;
};

typedef __attribute__((address_space(1))) const void GlobalBytes;
typedef __attribute__((address_space(3))) void LdsBytes;

// The operands of one 32-key tile.
template <int D, int KB, int VB>
struct NarrowTile {
    typedef KvSide<D, KB> KS;
    typedef KvSide<D, VB> VS;
    static constexpr int kLoads = KS::kPieces / 4;
    uint32_t k[2][kLoads][KS::kPiece / 4];
    uint32_t v[2][VS::kSlots * VS::kSlot / 4];
    uint32_t ks[2][(KS::kBlocks + 3) / 4], vs[2];

    __device__ __forceinline__ void load(const uint8_t *keys, const uint8_t *values, const uint8_t *scales) {
        const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const uint8_t *kc = keys + u * KS::kUnitCodes + lane * KS::kPiece;
#pragma unroll
            for (int j = 0; j < kLoads; ++j) load_words<KS::kPiece>(kc + j * kLanes * KS::kPiece, k[u][j]);
            load_words<KS::kBlocks>(scales + u * KS::kUnitScales + r * KS::kBlocks, ks[u]);
            const uint8_t *vc = values + u * VS::kUnitCodes + lane * VS::kSlot;
#pragma unroll
            for (int j = 0; j < VS::kSlots; ++j) load_words<VS::kSlot>(vc + j * kLanes * VS::kSlot, &v[u][j * (VS::kSlot / 4)]);
            load_words<4>(scales + (2 + u) * VS::kUnitScales + (g * VS::kBlocks + r * VS::kBlocks / 16) * 4, &vs[u]);
        }
    }
};

// One side's codes of two units to shared memory, 16 bytes a lane.  STREAM: for codes
// that nobody reads again.
template <int UNIT, int STREAM>
__device__ __forceinline__ void send_units(const uint8_t *codes, int64_t unit0, int64_t unit1, uint8_t *to) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int n = 0; n < 2 * UNIT; n += kLanes * 16) {
        const int u = UNIT >= kLanes * 16 ? n / UNIT : lane * 16 / UNIT;
        const int at = UNIT >= kLanes * 16 ? n % UNIT + lane * 16 : lane * 16 % UNIT;
        const uint8_t *from = codes + (u == 0 ? unit0 : unit1) * UNIT + at;
        __builtin_amdgcn_global_load_lds((GlobalBytes *)from, (LdsBytes *)(to + n), 16, 0, STREAM);
    }
}

template <int D, int KB, int VB>
__global__ void __launch_bounds__(kNarrowThreads, (NarrowShape<D, KB, VB>::kPerSimd))
    attn_narrow_kernel(AttnArgs a) {
    typedef NarrowShape<D, KB, VB> W;
    typedef KvSide<D, KB> KS;
    typedef KvSide<D, VB> VS;
    constexpr int kSlices = D / 32;            // MFMAs of one unit's scores
    constexpr int kRowDims = W::kRowDims;      // elements of a value row
    constexpr int kStep = kNarrowWaves * kTileKeys;
    extern __shared__ __align__(16) uint8_t lds[];
    const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int head = blockIdx.y, z = blockIdx.z;
    const RowTile tile = row_tile(a, 0, blockIdx.x);
    if (!tile.some) return;
    const KeyRange keys = key_range(a, 0, tile, blockIdx.x, head, z);
    if (!keys.some) return;

    // The tile at `key` on its way to the wave's shared memory, and which of its units
    // have pages (a bit each).  The table's entries come a tile earlier.
    const KvView &kv = a.kv;
    uint8_t *const mine = lds + wave * W::kTileBytes;
    int has = 0, entry[2];
    // the lane's four bytes of scales: of a side's unit `second` (of two), in as many loads as it takes
    const uint8_t *scale_of[W::kScaleLoads];
    bool second[W::kScaleLoads];
#pragma unroll
    for (int n = 0; n < W::kScaleLoads; ++n) {
        const int at = n * kLanes * 4 + lane * 4, region = at / W::kScaleBytes & 3;
        scale_of[n] = kv.scales[region >> 1] + at % W::kScaleBytes;
        second[n] = region & 1;
    }
    const auto look_up = [&](int key) {
#pragma unroll
        for (int u = 0; u < 2; ++u) entry[u] = kv.entry_at_scalar(tile.s, key + u * kKvUnit);
    };
    const auto send = [&](int key) {
        int64_t unit[2];
        has = 0;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int pos = key + u * kKvUnit;
            const int page = pos < keys.hi ? kv.page_in(entry[u], pos) : -1;
            has |= (page >= 0) << u;
            unit[u] = kv.unit_of(max(page, 0), head, pos);
        }
        // Codes that one tile reads go past the caches (64 sequences of 8192 keys 146 us,
        // through them 168); those that the tiles of a chunk share do not (64 tokens
        // over 4064 keys, heads of 256: 42 us, past them 52).
        if (a.reused) {
            send_units<KS::kUnitCodes, 0>(kv.codes[0], unit[0], unit[1], mine);
            send_units<VS::kUnitCodes, 0>(kv.codes[1], unit[0], unit[1], mine + W::kValuesAt);
        } else {
            send_units<KS::kUnitCodes, kStream>(kv.codes[0], unit[0], unit[1], mine);
            send_units<VS::kUnitCodes, kStream>(kv.codes[1], unit[0], unit[1], mine + W::kValuesAt);
        }
#pragma unroll
        for (int n = 0; n < W::kScaleLoads; ++n)
            __builtin_amdgcn_global_load_lds((GlobalBytes *)(scale_of[n] + (second[n] ? unit[1] : unit[0]) * W::kScaleBytes),
                                             (LdsBytes *)(mine + W::kScalesAt + n * kLanes * 4), 4, 0, 0);
    };
    int key = keys.lo + wave * kTileKeys;
    look_up(key);
    if (key < keys.hi) {
        send(key);
        look_up(key + kStep);
    }

    // The row of this lane's column, and its query operands.
    bf16x8 q[kSlices];
    const int row = tile.row0 + c;
    const bool in = row < tile.rows;
    const int i = in ? row / a.group : 0;
    const int token = in ? tile.begin + i : -1, qhead = head * a.group + (in ? row - i * a.group : 0);
    const int pos = tile.past + i;
    const int klo = a.window > 0 ? max(0, pos + 1 - a.window) : 0;
    const int khi = in ? (a.tree ? tile.past : pos + 1) : 0;
    const unsigned long long tree = in && a.tree ? a.tree[token] : 0ull;
    const uint16_t *src = a.q + max(token, 0) * a.q_stride + qhead * D;
#pragma unroll
    for (int m = 0; m < kSlices; ++m) {
        // slice m takes the lane's m-th group of eight elements of its pieces
        constexpr int per = KS::kPieceDims / 8;
        const int d = (4 * (m / per) + g) * KS::kPieceDims + 8 * (m % per);
        u32x4 w = {0, 0, 0, 0};
        if (in) w = *reinterpret_cast<const u32x4 *>(src + d);
        q[m] = __builtin_bit_cast(bf16x8, w);
    }
    if (a.info && z == 0 && threadIdx.x < kNarrowRows && in)
        a.info[int64_t(token) * a.q_heads + qhead] = RowInfo{keys.part + c, kNarrowRows, keys.splits, 0};

    // Weights are 2^(score - sub); l is their sum, lr the sum of the weights as
    // rounded to bf16, which normalises the output and comes from the smallest
    // matrix instruction (each lane's own four weights by ones).
    floatx4 o[kRowDims], lr = {0, 0, 0, 0};
    float sub = in ? kNegInf : 0.0f, l = 0.0f;       // rows that see nothing need no maximum
    const s16x4 ones = {0x3F80, 0x3F80, 0x3F80, 0x3F80};
#pragma unroll
    for (int j = 0; j < kRowDims; ++j) o[j] = floatx4{0, 0, 0, 0};

    for (; key < keys.hi; key += kStep) {
        __builtin_amdgcn_s_waitcnt(kWaitLoads);
        NarrowTile<D, KB, VB> x;
        x.load(mine, mine + W::kValuesAt, mine + W::kScalesAt);
        const bool some0 = has & 1, some1 = has & 2;
        // the tile is in registers: the next one may overwrite it
        __builtin_amdgcn_s_waitcnt(kWaitLds);
        __builtin_amdgcn_sched_barrier(0);
        if (key + kStep < keys.hi) {
            send(key + kStep);
            look_up(key + 2 * kStep);
        }
        const bool edge = (key < tile.inner_lo) | (key + kTileKeys > min(tile.inner_hi, keys.hi)) | !some0 | !some1;

        // scores of two units: lane (g, c) has keys 4 g + i of each, row c
        floatx4 s[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            s[u] = floatx4{0, 0, 0, 0};
#pragma unroll
            for (int m = 0; m < kSlices; ++m) {
                constexpr int per = KS::kPieceDims / 8;
                const int j = m / per, e = m % per;
                // the block of piece 4 j + g; the four lanes' blocks of a piece never cross a word
                const int block = ((4 * j + g) * KS::kPieceDims) / kMxBlock;
                const float unit = unit_of_byte(x.ks[u][4 * j * KS::kPieceDims / kMxBlock / 4], block & 3);
                bf16x8 k;
                if constexpr (KB == 8) k = codes8(x.k[u][j][2 * e], x.k[u][j][2 * e + 1], unit);
                else k = codes4(x.k[u][j][e], unit);
                s[u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, q[m], s[u], 0, 0, 0);
            }
        }
        unsigned seen = 0xFFu;                  // bit i: score i is of an allowed key
        if (edge) {
            const int first = key + 4 * g, last = min(khi, tile.hi);
            seen = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int at = first + (e >> 2) * kKvUnit + (e & 3);
                seen |= unsigned((at >= klo) & (at < last)) << e;
            }
            if (a.tree) {
                const int drafted = min(min(tile.n, 64), tile.hi - tile.past);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int t = first + (e >> 2) * kKvUnit + (e & 3) - tile.past;
                    seen |= (unsigned((t >= 0) & (t < drafted)) & unsigned(tree >> (t & 63))) << e;
                }
            }
            seen &= (some0 ? 0x0Fu : 0u) | (some1 ? 0xF0u : 0u);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e >> 2][e & 3] = (seen >> e) & 1u ? s[e >> 2][e & 3] : kNegInf;
        }
        // The weights, against the reference that earlier tiles left.  It moves up
        // only where their sum shows a weight too large (or none was set).
        uint32_t p[4];
        const auto weigh = [&](float ref) {
            float w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = exp2_fast(__builtin_fmaf(s[e >> 2][e & 3], a.scale_log2, -ref));
#pragma unroll
            for (int e = 0; e < 4; ++e) p[e] = pack_bf16(w[2 * e], w[2 * e + 1]);
            return ((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7]));
        };
        float total = weigh(sub == kNegInf ? 0.0f : sub);
        if (__any(sub == kNegInf || total > kMaxSum)) {
            float top = kNegInf;
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf(top, s[e >> 2][e & 3]);
            top *= a.scale_log2;
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            const float m = fmaxf(sub, top);
            const float by = m == sub ? 1.0f : exp2_fast(sub - m);
            sub = m;
            l = l * by + no_maximum(m, seen != 0);
            lr *= by;
#pragma unroll
            for (int j = 0; j < kRowDims; ++j) o[j] *= by;
            total = weigh(sub == kNegInf ? 0.0f : sub);
        }
        l += total;
#pragma unroll
        for (int e = 0; e < 4; e += 2)
            lr = __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(ones, __builtin_bit_cast(s16x4, u32x2{p[e], p[e + 1]}), lr, 0, 0, 0);

        // In an edge tile, values of keys that no row of the tile sees, or without a
        // page, become zeros, and NaN blocks too: zero weights times NaN would reach
        // every row.  The product of the NaN marks with the allowed keys says which rows
        // and elements are NaN.
        uint32_t vs[2] = {x.vs[0], x.vs[1]};
        if (edge) {
            uint32_t bad = 0;                   // bit i where key slot i's block is NaN
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int u = e >> 2, at = key + u * kKvUnit + 4 * g + (e & 3);
                const bool held = (u ? some1 : some0) && at >= tile.lo && at < tile.hi;
                const bool nan = ((vs[u] >> (8 * (e & 3))) & 0xFFu) == 0xFFu;
                bad |= unsigned(held && nan) << e;
                if (held && !nan) continue;
                vs[u] &= ~(0xFFu << (8 * (e & 3)));
                clear_token<D, VB>(x.v[u], e & 3);
            }
            if (__any(bad != 0)) {
                u32x4 mark, on;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    mark[e] = ((bad >> (2 * e)) & 1 ? 0x3F80u : 0u) | ((bad >> (2 * e + 1)) & 1 ? 0x3F800000u : 0u);
                    on[e] = ((seen >> (2 * e)) & 1 ? 0x3F80u : 0u) | ((seen >> (2 * e + 1)) & 1 ? 0x3F800000u : 0u);
                }
                const floatx4 n = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, mark), __builtin_bit_cast(bf16x8, on), floatx4{0, 0, 0, 0}, 0, 0, 0);
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                    for (int j = 0; j < kRowDims; ++j) o[j][e] = n[e] > 0.0f ? __builtin_nanf("") : o[j][e];
            }
        }
        // values: the lane's row holds D / 16 elements of eight keys; two
        // elements of a key come at a time and are paired over keys
        const bf16x8 pb = __builtin_bit_cast(bf16x8, u32x4{p[0], p[1], p[2], p[3]});
#pragma unroll
        for (int jp = 0; jp < kRowDims / 2; ++jp) {
            uint32_t w[2][4];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e) w[u][e] = value_pair<D, VB>(x.v[u], e, jp, unit_of_byte(vs[u], e));
            const u32x4 even = {low_halves(w[0][0], w[0][1]), low_halves(w[0][2], w[0][3]),
                                low_halves(w[1][0], w[1][1]), low_halves(w[1][2], w[1][3])};
            const u32x4 odd = {high_halves(w[0][0], w[0][1]), high_halves(w[0][2], w[0][3]),
                               high_halves(w[1][0], w[1][1]), high_halves(w[1][2], w[1][3])};
            o[2 * jp] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, even), pb, o[2 * jp], 0, 0, 0);
            o[2 * jp + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, odd), pb, o[2 * jp + 1], 0, 0, 0);
        }
    }

    // The waves meet: their references and sums, then their outputs, in parts.
    float *const states = reinterpret_cast<float *>(lds + W::kStatesAt);      // [sub, l, lr][wave][row]
    float *const outs = reinterpret_cast<float *>(lds);                       // [wave][row][kCols]
    const auto state = [&](int what, int w, int r) -> float & { return states[(what * kNarrowWaves + w) * kNarrowRows + r]; };
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    float norm = lr[0] + __shfl_xor(lr[0], 16);
    norm += __shfl_xor(norm, 32);
    if (g == 0) {
        state(0, wave, c) = sub;
        state(1, wave, c) = l;
        state(2, wave, c) = norm;
    }
    __syncthreads();
    float m = kNegInf;
#pragma unroll
    for (int w = 0; w < kNarrowWaves; ++w) m = fmaxf(m, state(0, w, c));
    const float by = piece_weight(sub, m);
    const int row16 = threadIdx.x >> 4, piece = threadIdx.x & 15;
    const int mine_row = tile.row0 + row16;
#pragma unroll
    for (int part = 0; part < kRowDims / W::kPart; ++part) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int j = 0; j < W::kPart; ++j)
                outs[(wave * kNarrowRows + c) * W::kCols + (4 * g + e) * W::kPart + j] = o[part * W::kPart + j][e] * by;
        __syncthreads();
        if (mine_row < tile.rows) {
            float mm = kNegInf, ll = 0.0f, rr = 0.0f;
#pragma unroll
            for (int w = 0; w < kNarrowWaves; ++w) mm = fmaxf(mm, state(0, w, row16));
#pragma unroll
            for (int w = 0; w < kNarrowWaves; ++w) {
                const float b = piece_weight(state(0, w, row16), mm);
                ll += state(1, w, row16) * b;
                rr += state(2, w, row16) * b;
            }
            float y[W::kPart];
#pragma unroll
            for (int j = 0; j < W::kPart; ++j) {
                y[j] = 0.0f;
#pragma unroll
                for (int w = 0; w < kNarrowWaves; ++w) y[j] += outs[(w * kNarrowRows + row16) * W::kCols + piece * W::kPart + j];
            }
            const int t = mine_row / a.group, at_head = head * a.group + (mine_row - t * a.group);
            const int d = piece * kRowDims + part * W::kPart;
            const bool facts = piece == 0 && part == 0;
            if (keys.splits > 1) {
                const int64_t to = keys.part + row16;
                float *dst = a.part_o + to * D + d;
#pragma unroll
                for (int j = 0; j < W::kPart; ++j) dst[j] = y[j];
                if (facts) *reinterpret_cast<float4 *>(a.part_ml + to * 4) = float4{mm, ll, rr, 0.0f};
            } else {
                const float inv = mm == kNegInf && ll == 0.0f ? 0.0f : 1.0f / rr;
                uint16_t *dst = a.out + int64_t(tile.begin + t) * a.out_stride + at_head * D + d;
#pragma unroll
                for (int j = 0; j < W::kPart; j += 2)
                    *reinterpret_cast<uint32_t *>(dst + j) = pack_bf16(y[j] * inv, y[j + 1] * inv);
                if (a.lse && facts) a.lse[int64_t(tile.begin + t) * a.q_heads + at_head] = lse_of(mm, ll);
            }
        }
        __syncthreads();
    }
}

// --------------------------------------------------------------------- join

constexpr int kMaxPieces = kMaxSplits;

// Where row u = token * q_heads + head has its parts; no pieces, or one that wrote the
// output itself, is nothing to join.  Rows of no sequence have no facts; and facts that
// point outside the workspace, as arrays that change under the call may leave them,
// are none.
__device__ __forceinline__ RowInfo row_info(const AttnArgs &a, int64_t u) {
    RowInfo r = a.info[u];
    const int token = int(u / a.q_heads);
    if (token < a.kv.offsets[0] || token >= a.kv.offsets[a.kv.seqs] || r.pieces > kMaxPieces || r.first < 0 ||
        (r.stride != kNarrowRows && r.stride != a.cut[1].rows) ||
        r.first + int64_t(r.pieces - 1) * r.stride >= a.part_rows)
        r.pieces = 0;
    return r;
}

__device__ __forceinline__ void store_row4(const AttnArgs &a, int D, int64_t u, int d, float m, float l, float lr,
                                           const float4 &y) {
    const int token = int(u / a.q_heads), qhead = int(u - int64_t(token) * a.q_heads);
    const float inv = m == kNegInf && l == 0.0f ? 0.0f : 1.0f / lr;
    uint16_t *dst = a.out + token * a.out_stride + qhead * D + d;
    *reinterpret_cast<u32x2 *>(dst) = u32x2{pack_bf16(y.x * inv, y.y * inv), pack_bf16(y.z * inv, y.w * inv)};
    if (a.lse && d == 0) a.lse[u] = lse_of(m, l);
}

// For few pieces: a thread takes four elements of a row and eight pieces at a time,
// whose loads go out together.
template <int D>
__global__ void __launch_bounds__(256) attn_join_few_kernel(AttnArgs a) {
    constexpr int kThreads = D / 4, kAtOnce = 8;
    const int64_t u = int64_t(blockIdx.x) * 256 + threadIdx.x;
    const int64_t row = u / kThreads;
    if (row >= int64_t(a.kv.tokens) * a.q_heads) return;
    const int d = int(u % kThreads) * 4;
    const RowInfo r = row_info(a, row);
    if (r.pieces <= 1) return;
    float m = kNegInf, l = 0.0f, lr = 0.0f;
    float4 y = {0, 0, 0, 0};
    for (int first = 0; first < r.pieces; first += kAtOnce) {
        float4 part[kAtOnce], o[kAtOnce];
#pragma unroll
        for (int z = 0; z < kAtOnce; ++z) {
            const int64_t from = r.first + int64_t(min(first + z, r.pieces - 1)) * r.stride;
            part[z] = *reinterpret_cast<const float4 *>(a.part_ml + from * 4);
            o[z] = *reinterpret_cast<const float4 *>(a.part_o + from * D + d);
        }
        float top = m;
#pragma unroll
        for (int z = 0; z < kAtOnce; ++z) top = fmaxf(top, part[z].x);
        const float old = piece_weight(m, top);
        m = top;
        l *= old;
        lr *= old;
        y.x *= old; y.y *= old; y.z *= old; y.w *= old;
#pragma unroll
        for (int z = 0; z < kAtOnce; ++z) {
            if (first + z >= r.pieces) break;
            const float by = piece_weight(part[z].x, m);
            l += part[z].y * by;
            lr += part[z].z * by;
            y.x += o[z].x * by; y.y += o[z].y * by; y.z += o[z].z * by; y.w += o[z].w * by;
        }
    }
    store_row4(a, D, row, d, m, l, lr, y);
}

// For many: a workgroup of 256 threads takes one row.  The threads weigh the
// pieces, then groups of D / 4 sum every kGroups-th and meet in shared memory.
template <int D>
__global__ void __launch_bounds__(256) attn_join_many_kernel(AttnArgs a) {
    constexpr int kThreads = D / 4, kGroups = 256 / kThreads;
    __shared__ float4 red[4];
    __shared__ float weight[kMaxPieces];
    __shared__ float4 sum[kGroups][kThreads];
    const RowInfo r = row_info(a, blockIdx.x);
    if (r.pieces <= 1) return;
    const int tid = threadIdx.x, wave = tid >> 6;
    constexpr int kEach = kMaxPieces / 256;
    float4 part[kEach];
    float m = kNegInf;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        const int z = tid + 256 * k;
        part[k] = float4{kNegInf, 0, 0, 0};
        if (z < r.pieces) part[k] = *reinterpret_cast<const float4 *>(a.part_ml + (r.first + int64_t(z) * r.stride) * 4);
        m = fmaxf(m, part[k].x);
    }
#pragma unroll
    for (int k = 1; k < 64; k *= 2) m = fmaxf(m, __shfl_xor(m, k));
    if ((tid & 63) == 0) red[wave].x = m;
    __syncthreads();
    m = fmaxf(fmaxf(red[0].x, red[1].x), fmaxf(red[2].x, red[3].x));
    float l = 0.0f, lr = 0.0f;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
        const int z = tid + 256 * k;
        const float by = z < r.pieces ? piece_weight(part[k].x, m) : 0.0f;
        weight[z] = by;
        l += part[k].y * by;
        lr += part[k].z * by;
    }
#pragma unroll
    for (int k = 1; k < 64; k *= 2) {
        l += __shfl_xor(l, k);
        lr += __shfl_xor(lr, k);
    }
    if ((tid & 63) == 0) {
        red[wave].y = l;
        red[wave].z = lr;
    }
    __syncthreads();
    l = red[0].y + red[1].y + red[2].y + red[3].y;
    lr = red[0].z + red[1].z + red[2].z + red[3].z;
    const int grp = tid / kThreads, d = tid % kThreads * 4;
    float4 y = {0, 0, 0, 0};
#pragma unroll 8
    for (int z = grp; z < r.pieces; z += kGroups) {
        const float4 o = *reinterpret_cast<const float4 *>(a.part_o + (r.first + int64_t(z) * r.stride) * D + d);
        const float w = weight[z];
        y.x += o.x * w; y.y += o.y * w; y.z += o.z * w; y.w += o.w * w;
    }
    sum[grp][tid % kThreads] = y;
    __syncthreads();
    if (grp != 0) return;
#pragma unroll
    for (int k = 1; k < kGroups; ++k) {
        const float4 o = sum[k][tid];
        y.x += o.x; y.y += o.y; y.z += o.z; y.w += o.w;
    }
    store_row4(a, D, blockIdx.x, d, m, l, lr, y);
}

int launch_attn_join(const AttnArgs &a, bool many, int dim, hipStream_t stream) {
    return kv_dim(dim, [&](auto tag) {
        constexpr int D = decltype(tag)::value;
        const int64_t rows = int64_t(a.kv.tokens) * a.q_heads, grid = many ? rows : ceil_div(rows * (D / 4), 256);
        if (grid >= kMaxGrid / 256) return NVFP4_ESHAPE;
        if (many) attn_join_many_kernel<D><<<unsigned(grid), 256, 0, stream>>>(a);
        else attn_join_few_kernel<D><<<unsigned(grid), 256, 0, stream>>>(a);
        return launch_status();
    });
}

template <int D, int K, int V>
static int launch_narrow(const AttnArgs &a, int64_t tiles, hipStream_t stream) {
    typedef NarrowShape<D, K, V> W;
    if (tiles >= kMaxGrid / kNarrowThreads) return NVFP4_ESHAPE;
    if (!raise_lds<attn_narrow_kernel<D, K, V>>(W::kLds)) return NVFP4_EHIP;
    attn_narrow_kernel<D, K, V><<<dim3(unsigned(tiles), unsigned(a.kv.heads), unsigned(a.cut[0].splits)),
                                         kNarrowThreads, W::kLds, stream>>>(a);
    return launch_status();
}

int launch_attn_narrow(const AttnArgs &a, int64_t tiles, int dim, int k_format, int v_format, hipStream_t stream) {
    return kv_dim(dim, [&](auto d) {
        return kv_bits(k_format, [&](auto k) {
            return kv_bits(v_format, [&](auto v) {
                return launch_narrow<decltype(d)::value, decltype(k)::value, decltype(v)::value>(a, tiles, stream);
            });
        });
    });
}

}  // namespace nvfp4
