// nvfp4_attn_narrow.hip -- attention of few query rows over the paged cache
// (decode, speculative verify) on gfx950.
#include "nvfp4_attn.h"

namespace nvfp4 {

constexpr int kNarrowWaves = 4;
constexpr int kTileKeys = 32;      // keys of a wave's tile: two units

// The table's entries of a tile's two units, wave-uniform; made pages when the tile
// is loaded, so that nothing waits for them before.
struct TileEntries {
    int entry[2];
    __device__ __forceinline__ void load(const KvView &kv, int s, int key) {
#pragma unroll
        for (int u = 0; u < 2; ++u) entry[u] = kv.entry_at(s, key + u * kKvUnit);
    }
};

// The operands of one 32-key tile as loaded.
template <int D, int KB, int VB>
struct NarrowTile {
    typedef KvSide<D, KB> KS;
    typedef KvSide<D, VB> VS;
    static constexpr int kLoads = KS::kPieces / 4;
    uint32_t k[2][kLoads][KS::kPiece / 4];
    uint32_t ks[2][(KS::kBlocks + 3) / 4];
    uint32_t v[2][VS::kSlots * VS::kSlot / 4];
    uint32_t vs[2];
    bool some[2];                  // the unit has a page (wave-uniform)

    __device__ __forceinline__ void load(const KvView &kv, const TileEntries &entries, int head, int key, int end) {
        const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int pos = key + u * kKvUnit;
            const int page = pos < end ? kv.page_in(__builtin_amdgcn_readfirstlane(entries.entry[u]), pos) : -1;
            some[u] = page >= 0;
            const int64_t unit = kv.unit_of(max(page, 0), head, pos);
            const uint8_t *kc = kv.codes[0] + unit * KS::kUnitCodes + lane * KS::kPiece;
#pragma unroll
            for (int j = 0; j < kLoads; ++j) load_words<KS::kPiece, true>(kc + j * kLanes * KS::kPiece, k[u][j]);
            load_words<KS::kBlocks>(kv.scales[0] + unit * KS::kUnitScales + r * KS::kBlocks, ks[u]);
            const uint8_t *vc = kv.codes[1] + unit * VS::kUnitCodes + lane * VS::kSlot;
#pragma unroll
            for (int j = 0; j < VS::kSlots; ++j) load_words<VS::kSlot, true>(vc + j * kLanes * VS::kSlot, &v[u][j * (VS::kSlot / 4)]);
            load_words<4>(kv.scales[1] + unit * VS::kUnitScales + (g * VS::kBlocks + r * VS::kBlocks / 16) * 4, &vs[u]);
        }
    }
};

template <int D, int KB, int VB>
__global__ void __launch_bounds__(kNarrowWaves * kLanes, D <= 128 ? 3 : 1) attn_narrow_kernel(AttnArgs a) {
    typedef KvSide<D, KB> KS;
    constexpr int kSlices = D / 32;            // MFMAs of one unit's scores
    constexpr int kRowDims = D / 16;           // elements of a value row
    const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int head = blockIdx.y, z = blockIdx.z;
    const RowTile tile = row_tile(a, 0, blockIdx.x);
    if (!tile.some) return;
    const KeyRange keys = key_range(a, 0, tile, blockIdx.x, head, z);
    if (!keys.some) return;

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

    floatx4 o[kRowDims];
    // lr: the sum of the weights as rounded, which normalises the outputs
    float mx = kNegInf, sub = 0.0f, l = 0.0f, lr = 0.0f;
#pragma unroll
    for (int j = 0; j < kRowDims; ++j) o[j] = floatx4{0, 0, 0, 0};

    const auto step = [&](const NarrowTile<D, KB, VB> &x, int key, auto edge_tag) {
        constexpr bool EDGE = decltype(edge_tag)::value != 0;
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
        uint32_t ones[4];                  // EDGE: the allowed keys as a bf16 operand of ones
        uint32_t p[4];
        float f[8];
        float top = kNegInf;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            f[i] = s[i >> 2][i & 3] * a.scale_log2;
            if constexpr (EDGE) {
                const int pos = key + (i >> 2) * kKvUnit + 4 * g + (i & 3);
                bool ok = pos >= klo && pos < khi;
                if (a.tree) {
                    const int b = pos - tile.past;
                    ok = ok || (b >= 0 && b < tile.n && b < 64 && ((tree >> (b & 63)) & 1));
                }
                ok = ok && x.some[i >> 2] && pos < tile.hi;
                if (!ok) f[i] = kNegInf;
                const uint32_t one = ok ? 0x3F80u : 0u;
                if (i & 1) ones[i >> 1] |= one << 16;
                else ones[i >> 1] = one;
            }
            top = fmaxf(top, f[i]);
        }
        if (__any(top > mx + kMaxSlack)) {
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            const float m = fmaxf(mx, top);
            const float by = m == mx ? 1.0f : exp2_fast(mx - m);
            mx = m;
            sub = m == kNegInf ? 0.0f : m;
            l *= by;
            lr *= by;
#pragma unroll
            for (int j = 0; j < kRowDims; ++j) o[j] *= by;
        }
        float e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            e[i] = exp2_fast(f[i] - sub);
            l += e[i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            p[i] = pack_bf16(e[2 * i], e[2 * i + 1]);
            lr = add_pair(p[i], lr);
        }
        // values: the lane's row holds D / 16 elements of eight keys; two
        // elements of a key come at a time and are paired over keys
        uint32_t keep[2] = {~0u, ~0u};         // EDGE: per token a byte of ones where its values count
        uint32_t bad = 0;                      // EDGE: bit i where key slot i's block is NaN
        if constexpr (EDGE) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int pos = key + u * kKvUnit + 4 * g + i;
                    const bool held = x.some[u] && pos >= tile.lo && pos < tile.hi;
                    const bool nan = ((x.vs[u] >> (8 * i)) & 0xFFu) == 0xFFu;
                    if (!held || nan) keep[u] &= ~(0xFFu << (8 * i));
                    if (held && nan) bad |= 1u << (4 * u + i);
                }
        }
#pragma unroll
        for (int jp = 0; jp < kRowDims / 2; ++jp) {
            uint32_t w[2][4];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    w[u][i] = value_pair<D, VB>(x.v[u], i, jp, unit_of_byte(x.vs[u], i));
                    if constexpr (EDGE) w[u][i] = (keep[u] >> (8 * i)) & 1u ? w[u][i] : 0u;
                }
            const u32x4 even = {low_halves(w[0][0], w[0][1]), low_halves(w[0][2], w[0][3]),
                                low_halves(w[1][0], w[1][1]), low_halves(w[1][2], w[1][3])};
            const u32x4 odd = {high_halves(w[0][0], w[0][1]), high_halves(w[0][2], w[0][3]),
                               high_halves(w[1][0], w[1][1]), high_halves(w[1][2], w[1][3])};
            const bf16x8 pb = __builtin_bit_cast(bf16x8, u32x4{p[0], p[1], p[2], p[3]});
            o[2 * jp] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, even), pb, o[2 * jp], 0, 0, 0);
            o[2 * jp + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, odd), pb, o[2 * jp + 1], 0, 0, 0);
        }
        if constexpr (EDGE) {
            // A NaN block counts only for the rows that see its key: its values
            // were left out above (zero weights times NaN would reach every
            // row), and a product of the NaN marks with the allowed keys says
            // which rows and elements are NaN.
            if (__any(bad != 0)) {
                u32x4 mark;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    mark[i] = ((bad >> (2 * i)) & 1 ? 0x3F80u : 0u) | ((bad >> (2 * i + 1)) & 1 ? 0x3F800000u : 0u);
                const bf16x8 on = __builtin_bit_cast(bf16x8, u32x4{ones[0], ones[1], ones[2], ones[3]});
                const floatx4 n = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, mark), on, floatx4{0, 0, 0, 0}, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (n[i] > 0.0f)
#pragma unroll
                        for (int j = 0; j < kRowDims; ++j) o[j][i] = __builtin_nanf("");
            }
        }
    };

    // A wave takes every fourth tile; the page numbers of its next one are
    // fetched while one is worked on.  Codes are not: three waves of a SIMD cover
    // each other's loads, and a ring of two or three tiles in registers (two
    // waves of a SIMD) measured 82 -> 92 us on 64 sequences of 4096 keys.
    constexpr int kStep = kNarrowWaves * kTileKeys;
    int key = keys.lo + wave * kTileKeys;
    TileEntries entries;
    entries.load(a.kv, tile.s, key);
    for (; key < keys.hi; key += kStep) {
        NarrowTile<D, KB, VB> x;
        x.load(a.kv, entries, head, key, keys.hi);
        entries.load(a.kv, tile.s, key + kStep);
        const bool inner = key >= tile.inner_lo && key + kTileKeys <= min(tile.inner_hi, keys.hi) && x.some[0] && x.some[1];
        if (inner) step(x, key, IntC<0>());
        else step(x, key, IntC<1>());
    }

    // Join the four waves: their maxima and sums, then their outputs, kRowDims in
    // parts of at most 8 to bound the shared memory.
    constexpr int kPart = kRowDims < 8 ? kRowDims : 8;
    constexpr int kCols = 16 * kPart + 4;              // floats of one row's part, padded against bank conflicts
    __shared__ float sm[kNarrowWaves][kNarrowRows], sl[kNarrowWaves][kNarrowRows], sr[kNarrowWaves][kNarrowRows];
    __shared__ float so[kNarrowWaves][16][kCols];
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    lr += __shfl_xor(lr, 16);
    lr += __shfl_xor(lr, 32);
    if (g == 0) {
        sr[wave][c] = lr;
        sm[wave][c] = mx;
        sl[wave][c] = l;
    }
    __syncthreads();
    float m = kNegInf;
#pragma unroll
    for (int w = 0; w < kNarrowWaves; ++w) m = fmaxf(m, sm[w][c]);
    const float by = mx == kNegInf ? (m == kNegInf ? 1.0f : 0.0f) : exp2_fast(mx - m);
#pragma unroll
    for (int part = 0; part < kRowDims / kPart; ++part) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < kPart; ++j) so[wave][c][(4 * g + i) * kPart + j] = o[part * kPart + j][i] * by;
        __syncthreads();
        // thread (row, piece): kPart / ... elements of one row
        constexpr int kEach = 16 * kPart / 16;
        const int row16 = threadIdx.x >> 4, piece = threadIdx.x & 15;
        const int row = tile.row0 + row16;
        if (row < tile.rows) {
            float mm = kNegInf, ll = 0.0f, rr = 0.0f;
#pragma unroll
            for (int w = 0; w < kNarrowWaves; ++w) mm = fmaxf(mm, sm[w][row16]);
#pragma unroll
            for (int w = 0; w < kNarrowWaves; ++w) {
                const float mw = sm[w][row16];
                const float by = mw == kNegInf ? (mm == kNegInf ? 1.0f : 0.0f) : exp2_fast(mw - mm);
                ll += sl[w][row16] * by;
                rr += sr[w][row16] * by;
            }
            float y[kEach];
#pragma unroll
            for (int j = 0; j < kEach; ++j) {
                y[j] = 0.0f;
#pragma unroll
                for (int w = 0; w < kNarrowWaves; ++w) y[j] += so[w][row16][piece * kEach + j];
            }
            const int i = row / a.group;
            const int64_t at = int64_t(tile.begin + i) * a.q_heads + head * a.group + (row - i * a.group);
            const int d = piece * kRowDims + part * kPart;
            if (keys.splits > 1) {
                const int64_t to = keys.part + row16;
                float *dst = a.part_o + to * D + d;
#pragma unroll
                for (int j = 0; j < kEach; ++j) dst[j] = y[j];
                if (piece == 0 && part == 0) {
                    float *ml = a.part_ml + to * 4;
                    *reinterpret_cast<float4 *>(ml) = float4{mm, ll, rr, 0.0f};
                }
            } else {
                const float inv = mm == kNegInf && ll == 0.0f ? 0.0f : 1.0f / rr;
                uint16_t *dst = a.out + int64_t(tile.begin + i) * a.out_stride + (head * a.group + (row - i * a.group)) * D + d;
#pragma unroll
                for (int j = 0; j < kEach; j += 2)
                    *reinterpret_cast<uint32_t *>(dst + j) = pack_bf16(y[j] * inv, y[j + 1] * inv);
                if (a.lse && piece == 0 && part == 0) a.lse[at] = lse_of(mm, ll);
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

__device__ __forceinline__ float piece_weight(float mz, float m) {
    return mz == kNegInf ? (m == kNegInf ? 1.0f : 0.0f) : exp2_fast(mz - m);
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

int launch_attn_narrow(const AttnArgs &a, int64_t tiles, int dim, int k_format, int v_format, hipStream_t stream) {
    return kv_dim(dim, [&](auto d) {
        return kv_bits(k_format, [&](auto k) {
            return kv_bits(v_format, [&](auto v) {
                constexpr int D = decltype(d)::value, K = decltype(k)::value, V = decltype(v)::value;
                constexpr int kThreads = kNarrowWaves * kLanes;
                if (tiles >= kMaxGrid / kThreads) return NVFP4_ESHAPE;
                attn_narrow_kernel<D, K, V><<<dim3(unsigned(tiles), unsigned(a.kv.heads), unsigned(a.cut[0].splits)),
                                              kThreads, 0, stream>>>(a);
                return launch_status();
            });
        });
    });
}

}  // namespace nvfp4
