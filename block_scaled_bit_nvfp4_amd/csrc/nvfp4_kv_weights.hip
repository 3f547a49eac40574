// nvfp4_kv_weights.hip -- the attention that each cached key receives, gathered over
// steps (gfx950).  Two kernels: one streams keys past a few query rows (decode steps,
// verifies), one streams the query rows of a chunk past keys that stay in registers.
//
// A weight is 2^(s * c - r) with c = scale * log2(e) and r = lse * log2(e), each rounded
// to fp32; what that loses of the weights that count, those whose score is near lse, is
// the same for a whole row, and the factor that puts it right is one operand of the sum's
// multiply-add.  Rows that count for nothing have a factor of 0.
#include "nvfp4_attn.h"

namespace nvfp4 {

constexpr int kWeighWaves = 4, kWeighThreads = kWeighWaves * kLanes;
// The most rows (new tokens x group) of a sequence for the first kernel.  40 rows of 8 heads
// take it 7.1 us over 2048 keys (the second kernel 9.5), 12.7 over 16384 (10.5) and 35 over
// 131000 (44); 80 rows, two passes, 11 (9.5), 21 (12) and 64 (52).
constexpr int kFewRows = 64;

typedef float floatx16 __attribute__((ext_vector_type(16)));

struct WeighArgs {
    KvView kv;
    const uint16_t *q;
    const float *lse;
    const unsigned long long *tree;
    float *weights;
    int64_t q_stride, width;
    int q_heads, group, window;
    uint32_t group_magic;  // (2^32 - 1) / group
    int few_rows;          // sequences of at most so many rows are the first kernel's
    float scale_log2;      // c as rounded
    float lost;            // (scale * log2(e) - c) / scale, less what kLog2e is short of log2(e)
    float decay;
};

// A row of a sequence's (new token, head of the group).
struct WeighRow {
    int i, g;
    __device__ __forceinline__ WeighRow(const WeighArgs &a, int row) {
        i = int(__umulhi(uint32_t(row), a.group_magic));     // the quotient, or one less
        g = row - i * a.group;
        const bool less = g >= a.group;
        i += less;
        g -= less ? a.group : 0;
    }
};

// KvView::sequence by scalar loads, for `s` that is the same in the whole wave.
__device__ __forceinline__ void sequence(const KvView &v, int s, int &begin, int &end, int &before) {
    typedef __attribute__((address_space(4))) const int32_t Constant;
    s = __builtin_amdgcn_readfirstlane(s);
    begin = min(max(((Constant *)v.offsets)[s], 0), v.tokens);
    end = min(max(((Constant *)v.offsets)[s + 1], begin), v.tokens);
    before = min(max(((Constant *)v.past)[s], 0), v.capacity);
}

// What turns a row's scores into weights.
struct RowFacts {
    float r, factor;
};
__device__ __forceinline__ bool counts(float lse) { return fabsf(lse) < __builtin_inff(); }
__device__ __forceinline__ RowFacts row_facts(const WeighArgs &a, float lse, bool in) {
    lse = in ? lse : 0.0f;
    const float r = lse * kLog2e;
    const float factor = exp2_fast(__builtin_fmaf(lse, a.lost, -__builtin_fmaf(lse, kLog2e, -r)));
    return RowFacts{r, in ? factor : 0.0f};
}

// The new weight of a key from what its rows add and what it had (0 for none); a key with
// a NaN or an infinity, or without a page, adds nothing.
__device__ __forceinline__ float gathered(float total, bool page, float old, float keep) {
    if (!(total < __builtin_inff()) || !page) total = 0.0f;
    return keep != 0.0f ? __builtin_fmaf(old, keep, total) : total;
}

// -------------------------------------------------------- keys past a few rows
//
// Q as the A operand of v_mfma_f32_16x16x32_bf16, RT tiles of 16 rows that stay in
// registers, and keys, 32 of a wave's step, as B: a lane of the accumulator has four
// rows' scores of one key, whose sum it takes with two exchanges between lanes for the
// other rows.  Workgroups take equal shares of all sequences' steps (64 ragged sequences
// 33.6 us, in pieces of 2048 keys 46.8).  Codes of the two steps to come are loaded ahead,
// past the caches, the table's entries a step before that.  Bound by reading the keys' codes
// (131008 keys of 8 heads of 128 dims: 28 us, 4.9 TB/s).

// A load of BYTES that nobody repeats.
template <int BYTES>
__device__ __forceinline__ void load_once(const uint8_t *p, uint32_t *w) {
    if constexpr (BYTES == 16) {
        const u32x4 t = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p));
        w[0] = t[0]; w[1] = t[1]; w[2] = t[2]; w[3] = t[3];
    } else {
        const u32x2 t = __builtin_nontemporal_load(reinterpret_cast<const u32x2 *>(p));
        w[0] = t[0]; w[1] = t[1];
    }
}

template <int D, int BITS>
struct KeyTile {
    typedef KvSide<D, BITS> S;
    static constexpr int kLoads = S::kPieces / 4, kSlices = D / 32, kPer = S::kPieceDims / 8;
    uint32_t w[2][kLoads][S::kPiece / 4], scale[2][(S::kBlocks + 3) / 4];
    float old;
    int has;               // which units have a page

    // The tile at `key` of keys before `last`; past them any tile.  `weights`: any of the
    // sequence's where the tile is past `last`.
    __device__ __forceinline__ void load(const WeighArgs &a, int head, int key, int last, const int (&entry)[2],
                                         const float *weights) {
        const int lane = threadIdx.x & 63, r = lane & 15;
        has = 0;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int pos = key + u * kKvUnit;
            const bool some = pos < last && uint32_t(entry[u]) < uint32_t(a.kv.pages);
            has |= int(some) << u;
            const int64_t unit = a.kv.unit_of(some ? entry[u] : 0, head, some ? pos : 0);
            const uint8_t *codes = a.kv.codes[0] + unit * S::kUnitCodes + lane * S::kPiece;
#pragma unroll
            for (int j = 0; j < kLoads; ++j) load_once<S::kPiece>(codes + j * kLanes * S::kPiece, w[u][j]);
            load_words<S::kBlocks>(a.kv.scales[0] + unit * S::kUnitScales + r * S::kBlocks, scale[u]);
        }
        old = weights[min(key + (lane & 31), last - 1)];
    }
    __device__ __forceinline__ bf16x8 operand(int u, int m) const {
        const int g = (threadIdx.x & 63) >> 4, j = m / kPer, e = m % kPer;
        // the block of piece 4 j + g; the four lanes' blocks of a piece never cross a word
        const int block = (4 * j + g) * S::kPieceDims / kMxBlock;
        const float unit = unit_of_byte(scale[u][4 * j * S::kPieceDims / kMxBlock / 4], block & 3);
        if constexpr (BITS == 8) return codes8(w[u][j][2 * e], w[u][j][2 * e + 1], unit);
        else return codes4(w[u][j][e], unit);
    }
};

// Sum over the lanes of the same column (lane % 16).
__device__ __forceinline__ float column_sum(float v) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

template <int D, int BITS, int RT>
__global__ void __launch_bounds__(kWeighThreads, RT * D <= 128 ? 4 : RT * D <= 256 ? 2 : 1) weigh_few_kernel(WeighArgs a) {
    typedef KeyTile<D, BITS> K;
    constexpr int kStep = kWeighWaves * 32;
    __shared__ unsigned long long words[kWeighWaves][16 * RT];       // each wave's rows' trees
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int head = blockIdx.y;
    // The workgroup's share of the head's steps, those of one sequence after another: the
    // lanes hold 64 sequences' facts at a time.
    int begins, stops, pasts, steps, upto;
    const auto sequences = [&](int base) {
        const int s = min(base + lane, a.kv.seqs - 1);
        a.kv.sequence(s, begins, stops, pasts);
        const int rows = (stops - begins) * a.group;
        const bool mine = base + lane < a.kv.seqs && rows > 0 && rows <= a.few_rows;
        steps = mine ? int((min(unsigned(pasts) + unsigned(stops - begins), unsigned(a.kv.capacity)) + kStep - 1) / kStep) : 0;
        upto = steps;
#pragma unroll
        for (int d = 1; d < kLanes; d <<= 1) {
            const int v = __shfl_up(upto, d);
            upto += lane >= d ? v : 0;
        }
        return __builtin_amdgcn_readlane(upto, 63);
    };
    uint64_t all = 0;
    int here = 0;
    for (int base = 0; base < a.kv.seqs; base += kLanes) all += uint64_t(here = sequences(base));
    uint64_t at = all * blockIdx.x / gridDim.x;
    const uint64_t to = all * (blockIdx.x + 1) / gridDim.x;
    uint64_t before = 0;
    for (int base = 0; at < to; base += kLanes) {
        if (a.kv.seqs > kLanes) here = sequences(base);
        while (at < to && at < before + uint64_t(here)) {
            const int rel = int(at - before), l = __popcll(__ballot(upto <= rel));
            const int s = base + l;
            const int begin = __builtin_amdgcn_readlane(begins, l), past = __builtin_amdgcn_readlane(pasts, l);
            const int n = __builtin_amdgcn_readlane(stops, l) - begin, rows = n * a.group;
            const int end = int(min(unsigned(past) + unsigned(n), unsigned(a.kv.capacity)));
            const int own = __builtin_amdgcn_readlane(steps, l), done = rel - (__builtin_amdgcn_readlane(upto, l) - own);
            const int take = int(min(uint64_t(own - done), to - at));
            const int last = min((done + take) * kStep, end);
            at += take;
            float *const weights = a.weights + (int64_t(s) * a.kv.heads + head) * a.width;
            const auto look_up = [&](int key, int (&entry)[2]) {
#pragma unroll
                for (int u = 0; u < 2; ++u) entry[u] = a.kv.entry_at_scalar(s, key + u * kKvUnit);
            };
            const int start = done * kStep + wave * 32;
            if (start >= last) continue;
            // more rows than the bounds said take more passes
            for (int base = 0; base < rows; base += 16 * RT) {
                const float keep = base == 0 ? a.decay : 1.0f;
                const int held = base == 0 ? (a.decay != 0.0f ? past : 0) : end;
                int key = start, entry[2];
                K tile[2];
                look_up(key, entry);
                tile[0].load(a, head, key, last, entry, weights);
                look_up(key + kStep, entry);
                tile[1].load(a, head, key + kStep, last, entry, weights);
                look_up(key + 2 * kStep, entry);
                // the rows' operands and facts
                bf16x8 q[RT][K::kSlices];
                RowFacts fact[RT][4];
                float lse[RT][5];          // of the lane's four rows of the accumulator, and of its row of the operand
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    const WeighRow w(a, min(base + 16 * t + c, rows - 1));
                    const int64_t token = begin + w.i, qhead = head * a.group + w.g;
                    const uint16_t *src = a.q + token * a.q_stride + qhead * D;
#pragma unroll
                    for (int m = 0; m < K::kSlices; ++m) {
                        const int d = (4 * (m / K::kPer) + g) * K::S::kPieceDims + 8 * (m % K::kPer);
                        q[t][m] = *reinterpret_cast<const bf16x8 *>(src + d);
                    }
                    lse[t][4] = a.lse[token * a.q_heads + qhead];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const WeighRow v(a, min(base + 16 * t + 4 * g + e, rows - 1));
                        lse[t][e] = a.lse[int64_t(begin + v.i) * a.q_heads + head * a.group + v.g];
                    }
                    if (a.tree) words[wave][16 * t + c] = a.tree[token];
                }
#pragma unroll
                for (int t = 0; t < RT; ++t) {
                    const bool in = base + 16 * t + c < rows && counts(lse[t][4]);
#pragma unroll
                    for (int m = 0; m < K::kSlices; ++m) q[t][m] = in ? q[t][m] : bf16x8{};
#pragma unroll
                    for (int e = 0; e < 4; ++e) fact[t][e] = row_facts(a, lse[t][e], base + 16 * t + 4 * g + e < rows && counts(lse[t][e]));
                }
                // the keys that every row sees
                const int inner_lo = a.window > 0 ? past + n - a.window : 0, inner_hi = a.tree ? past : past + 1;
                const auto work = [&](const K &k, int key) {
                    const bool edge = key < inner_lo || min(key + 32, end) > inner_hi;
                    float total[2];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        float sum = 0.0f;
                        bf16x8 operand[K::kSlices];
#pragma unroll
                        for (int m = 0; m < K::kSlices; ++m) operand[m] = k.operand(u, m);
#pragma unroll
                        for (int t = 0; t < RT; ++t) {
                            floatx4 x = {0, 0, 0, 0};
#pragma unroll
                            for (int m = 0; m < K::kSlices; ++m)
                                x = __builtin_amdgcn_mfma_f32_16x16x32_bf16(q[t][m], operand[m], x, 0, 0, 0);
                            float w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) w[e] = exp2_fast(__builtin_fmaf(x[e], a.scale_log2, -fact[t][e].r));
                            if (edge) {
                                const int j = key + 16 * u + c, bit = j - past;
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const int i = WeighRow(a, min(base + 16 * t + 4 * g + e, rows - 1)).i, pos = past + i;
                                    bool seen = j <= pos && (a.window == 0 || j > pos - a.window);
                                    if (a.tree && bit >= 0) seen = bit < min(n, 64) && words[wave][16 * t + 4 * g + e] >> (bit & 63) & 1;
                                    w[e] = seen ? w[e] : 0.0f;
                                }
                            }
#pragma unroll
                            for (int e = 0; e < 4; ++e) sum = __builtin_fmaf(w[e], fact[t][e].factor, sum);
                        }
                        total[u] = column_sum(sum);
                    }
                    const int at = key + lane;
                    if (lane < 32 && at < last)
                        weights[at] = gathered(lane < 16 ? total[0] : total[1], k.has >> (lane >> 4) & 1, at < held ? k.old : 0.0f, keep);
                };
                for (; key < last; key += 2 * kStep) {
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        work(tile[t], key + t * kStep);
                        if (key + (t + 1) * kStep >= last) break;
                        tile[t].load(a, head, key + (2 + t) * kStep, last, entry, weights);
                        look_up(key + (3 + t) * kStep, entry);
                    }
                }
            }
        }
        before += uint64_t(here);
    }
}

// -------------------------------------------------------- rows past many keys
//
// A wave holds 64 keys as A operands of v_mfma_f32_32x32x16_bf16 and the workgroup walks
// the query rows, 32 at a time, as B through shared memory: a lane of the accumulator has
// 16 keys' scores of one row, whose log-sum-exp it holds too, and adds its weights to
// running sums.  Only at the end are the sums of the 32 rows' lanes added.  RW
// waves of the four share keys, each with its own rows; their sums meet in shared memory.
//
// A step's rows go straight to shared memory two steps ahead, into a ring of three, so
// that one barrier a step is enough.  16-byte chunks of a row stand exchanged by the
// row's number, without which the lanes of a read would meet in the same banks.
// 2048 tokens of 40 heads over 32768 keys: 705 us, 950 TFLOP/s.  Matrix instructions take
// 43% of the cycles, the exponentials' multiply-adds and the steps' other vector work most
// of the rest: two waves a SIMD overlap them only in part, four kept in one wave's
// registers (1154 us) or both woven into one stream of instructions (798 us) do no better.

constexpr int kWideKeys = 64;              // of a wave
constexpr int kWideRows = 32;              // of a wave's step

typedef __attribute__((address_space(1))) const void GlobalMem;
typedef __attribute__((address_space(3))) void SharedMem;

// A 32-key operand of head `head` from position `key` on.
template <int D, int BITS>
struct KeyOperand {
    typedef KvSide<D, BITS> S;
    static constexpr int kSteps = D / 16, kHalf = S::kPieces / 2, kPer = S::kPieceDims / 8;
    bf16x8 k[kSteps];
    unsigned has;          // whether the first and the second 16 keys have a page

    // The element at which a lane's eight of step m start.
    static __device__ __forceinline__ int element(int m, int half) {
        return (2 * (m / kPer) + half) * S::kPieceDims + 8 * (m % kPer);
    }
    __device__ __forceinline__ void load(const KvView &v, int s, int head, int key, int end) {
        const int lane = threadIdx.x & 63, r = lane & 15, half = lane >> 5;
        const int pos = key + (lane & 16);
        const int page = pos < end ? v.page_in(v.entry_at(s, pos), pos) : -1;
        const unsigned long long lanes = __ballot(page >= 0);
        has = unsigned(lanes & 1) | unsigned(lanes >> 15 & 2);
        const int64_t unit = v.unit_of(max(page, 0), head, pos);
        uint32_t w[kHalf][S::kPiece / 4], scale[(S::kBlocks + 3) / 4];
        const uint8_t *codes = v.codes[0] + unit * S::kUnitCodes + (half * kKvUnit + r) * S::kPiece;
#pragma unroll
        for (int j = 0; j < kHalf; ++j) load_words<S::kPiece>(codes + 2 * j * kKvUnit * S::kPiece, w[j]);
        load_words<S::kBlocks>(v.scales[0] + unit * S::kUnitScales + r * S::kBlocks, scale);
#pragma unroll
        for (int m = 0; m < kSteps; ++m) {
            const int j = m / kPer, e = m % kPer;
            // the two halves' blocks of a step never cross a word
            const int block = (2 * j + half) * S::kPieceDims / kMxBlock;
            const float unit_scale = unit_of_byte(scale[2 * j * S::kPieceDims / kMxBlock / 4], block & 3);
            if constexpr (BITS == 8) k[m] = codes8(w[j][2 * e], w[j][2 * e + 1], unit_scale);
            else k[m] = codes4(w[j][e], unit_scale);
        }
    }
};

// Which of the 64 keys from position `key` on new token i (row `token` of the batch) sees.
__device__ __forceinline__ unsigned long long seen_keys(const WeighArgs &a, int past, int n, int i, int token, int key) {
    const auto below = [](int k) { return k <= 0 ? 0ull : k >= 64 ? ~0ull : (1ull << k) - 1; };
    const int pos = past + i;
    if (a.tree) {
        const unsigned long long word = a.tree[token] & below(n);
        const int d = past - key;
        return below(d) | (d >= 64 || d <= -64 ? 0ull : d >= 0 ? word << d : word >> -d);
    }
    const unsigned long long old = a.window > 0 ? below(pos - a.window + 1 - key) : 0ull;
    return below(pos + 1 - key) & ~old;
}

// The sum over the 32 lanes of each half of the wave of x[r], for the r that the lane's
// low four bits are.
__device__ __forceinline__ float column_sums(const float (&x)[16]) {
    const int lane = threadIdx.x & 63;
    float y[8], z[4], u[2];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = (lane & 8 ? x[i + 8] : x[i]) + __shfl_xor(lane & 8 ? x[i] : x[i + 8], 8);
#pragma unroll
    for (int i = 0; i < 4; ++i) z[i] = (lane & 4 ? y[i + 4] : y[i]) + __shfl_xor(lane & 4 ? y[i] : y[i + 4], 4);
#pragma unroll
    for (int i = 0; i < 2; ++i) u[i] = (lane & 2 ? z[i + 2] : z[i]) + __shfl_xor(lane & 2 ? z[i] : z[i + 2], 2);
    const float v = (lane & 1 ? u[1] : u[0]) + __shfl_xor(lane & 1 ? u[0] : u[1], 1);
    return v + __shfl_xor(v, 16);
}

// s_waitcnt operand: until at most n loads from memory are on their way.
constexpr int loads_left(int n) { return kWaitLoads | (n & 15) | n >> 4 << 14; }

template <int D, int RW>
struct WideShape {
    static constexpr int kChunks = D / 8;                            // 16-byte chunks of a row
    static constexpr int kLoadRows = kWeighThreads / kChunks;        // rows that the workgroup loads at a time
    static constexpr int kTileLoads = kWideRows / kLoadRows;         // a thread's loads of a tile
    static constexpr int kTileBytes = kWideRows * D * 2;
    static constexpr int kStepRows = RW * kWideRows;
    static constexpr int kRowBytes = RW * kTileBytes;                // of a step's tiles; each wave's log-sum-exps stand behind
    static constexpr int kStepBytes = kRowBytes + kWeighWaves * kLanes * 4;
    static constexpr int kLoads = RW * kTileLoads;
    static constexpr int kLds = 3 * kStepBytes;
    // Which chunk stands in place c of row r, and the other way round: the same for all rows
    // that a thread loads, and other ones for rows whose chunks would share banks.
    static __device__ __forceinline__ int exchanged(int r, int c) {
        return c ^ (D == 64 ? r >> 1 & 7 : D == 128 ? r & 15 : r & 7);
    }
};

// FLAT: tiles of 32 rows one after another, token by token, of sequences of few tokens;
// else tiles of 32 tokens of one head of the group, whose addresses take no arithmetic of
// the lanes.  RW: waves that share keys.
template <int D, int BITS, int RW, bool FLAT>
__global__ void __launch_bounds__(kWeighThreads, 2) weigh_many_kernel(WeighArgs a) {
    typedef KeyOperand<D, BITS> K;
    typedef WideShape<D, RW> W;
    constexpr int kKeyWaves = kWeighWaves / RW;
    constexpr unsigned kKeys = kKeyWaves * kWideKeys;
    extern __shared__ __align__(16) uint8_t lds[];
    const int lane = threadIdx.x & 63, c = lane & 31, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int key_wave = wave % kKeyWaves, row_wave = wave / kKeyWaves;
    const int head = blockIdx.y;
    // where the lane's operands stand in a step's rows
    int from[K::kSteps];
#pragma unroll
    for (int m = 0; m < K::kSteps; ++m)
        from[m] = ((row_wave * kWideRows + c) * W::kChunks + W::exchanged(c, K::element(m, half) / 8)) * 16;
    const int load_row = threadIdx.x / W::kChunks, load_chunk = W::exchanged(load_row, threadIdx.x % W::kChunks);
    // what a lane adds to a tile's address (32 tokens span less than 2^32 bytes, which the host checks)
    uint32_t offset[W::kTileLoads];
#pragma unroll
    for (int l = 0; l < W::kTileLoads; ++l)
        offset[l] = (uint32_t(load_row + l * W::kLoadRows) * uint32_t(a.q_stride) + load_chunk * 8) * 2;
    const uint32_t offset_lse = uint32_t(c) * a.q_heads * 4;
    for (int s = blockIdx.z; s < a.kv.seqs; s += gridDim.z) {
        int begin, stop, past;
        sequence(a.kv, s, begin, stop, past);
        const int n = stop - begin, rows = n * a.group, end = int(min(unsigned(past) + unsigned(n), unsigned(a.kv.capacity)));
        if (n == 0 || rows <= a.few_rows) continue;
        const uint16_t *const q = a.q + int64_t(begin) * a.q_stride + head * a.group * D;
        const float *const lses = a.lse + int64_t(begin) * a.q_heads + head * a.group;
        for (unsigned first = blockIdx.x * kKeys; first < unsigned(end); first += gridDim.x * kKeys) {
            const int key = int(first) + key_wave * kWideKeys;
            K k[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) k[u].load(a.kv, s, head, key + 32 * u, end);
            // The tokens that may see some of the workgroup's keys, the tiles of their rows, and the
            // tokens that see all of the wave's keys.
            const int i_lo = (a.tree ? 0 : max(0, int(first) - past)) & (FLAT ? -1 : -kWideRows);
            const int i_hi = a.window > 0 ? max(i_lo, int(min(int64_t(n), int64_t(first) + kKeys - 1 + a.window - past))) : n;
            const int row_lo = i_lo * a.group & -kWideRows;
            const int tiles = FLAT ? max(0, i_hi * a.group - row_lo + kWideRows - 1) / kWideRows
                                   : (i_hi - i_lo + kWideRows - 1) / kWideRows * a.group;
            const int full_lo = a.tree ? (key + kWideKeys <= past ? 0 : n) : key + kWideKeys - 1 - past;
            const int full_hi = a.window > 0 ? int(min(int64_t(n), int64_t(key) + a.window - past)) : n;

            // A tile's first token and head of the group.
            const auto advance = [&](int &i, int &g) __attribute__((always_inline)) {
                if (++g == a.group) {
                    g = 0;
                    i += kWideRows;
                }
            };
            // The rows and log-sum-exps of the step of tiles `tile`, .. on their way to shared memory
            // (where there is no such tile, or no such row, those of any); i, g: the first one's.
            const auto send = [&](int tile, int &i, int &g, int slot) __attribute__((always_inline)) {
                uint8_t *const to = lds + slot * W::kStepBytes;
                int mine_i = i, mine_g = g;
#pragma unroll
                for (int j = 0; j < RW; ++j) {
                    if (j == row_wave) {
                        mine_i = i;
                        mine_g = g;
                    }
                    const bool whole = !FLAT && i + kWideRows <= n;
                    const uint8_t *const at = reinterpret_cast<const uint8_t *>(q + i * a.q_stride + g * D);
#pragma unroll
                    for (int l = 0; l < W::kTileLoads; ++l) {
                        const uint8_t *from = at + offset[l];
                        if (!whole) {
                            const int r = load_row + l * W::kLoadRows;
                            const WeighRow w(a, min(row_lo + (tile + j) * kWideRows + r, rows - 1));
                            const int token = FLAT ? w.i : min(i + r, n - 1), of_group = FLAT ? w.g : g;
                            from = reinterpret_cast<const uint8_t *>(q + token * a.q_stride + of_group * D + load_chunk * 8);
                        }
                        __builtin_amdgcn_global_load_lds(
                            (GlobalMem *)from, (SharedMem *)(to + ((j * W::kTileLoads + l) * kWeighThreads + wave * kLanes) * 16), 16, 0, 0);
                    }
                    if (!FLAT) advance(i, g);
                }
                // each wave's own
                const uint8_t *from = reinterpret_cast<const uint8_t *>(lses + int64_t(mine_i) * a.q_heads + mine_g) + offset_lse;
                if (FLAT || mine_i + kWideRows > n) {
                    const WeighRow w(a, min(row_lo + (tile + row_wave) * kWideRows + c, rows - 1));
                    const int token = FLAT ? w.i : min(mine_i + c, n - 1), of_group = FLAT ? w.g : mine_g;
                    from = reinterpret_cast<const uint8_t *>(lses + int64_t(token) * a.q_heads + of_group);
                }
                __builtin_amdgcn_global_load_lds((GlobalMem *)from, (SharedMem *)(to + W::kRowBytes + wave * kLanes * 4), 4, 0, 0);
            };
            constexpr int kSent = W::kLoads + 1;       // a wave's loads of a step

            float sum[2][16] = {};
            int next_i = i_lo, next_g = 0, mine_i = i_lo, mine_g = 0;      // of the step to be sent, of the wave's tile
            if (!FLAT)
                for (int j = 0; j < row_wave; ++j) advance(mine_i, mine_g);
            __syncthreads();                           // the ring's last readers
            if (tiles > 0) send(0, next_i, next_g, 0);
            if (tiles > RW) send(RW, next_i, next_g, 1);
            for (int tile = 0; tile < tiles;) {
#pragma unroll
                for (int slot = 0; slot < 3; ++slot) {
                    // This step's loads have come, the next one's may be on their way: a bare
                    // barrier, since a fence would wait for them too.
                    if (tile + RW < tiles) __builtin_amdgcn_s_waitcnt(loads_left(kSent));
                    else __builtin_amdgcn_s_waitcnt(loads_left(0));
                    asm volatile("s_barrier" ::: "memory");
                    const uint8_t *const step = lds + slot * W::kStepBytes;
                    const float lse = *reinterpret_cast<const float *>(step + W::kRowBytes + wave * kLanes * 4 + c * 4);
                    if (tile + 2 * RW < tiles) send(tile + 2 * RW, next_i, next_g, slot == 0 ? 2 : slot - 1);
                    floatx16 x[2] = {};
#pragma unroll
                    for (int m0 = 0; m0 < K::kSteps; m0 += 4) {
                        bf16x8 b[4];
#pragma unroll
                        for (int m = 0; m < 4; ++m) b[m] = *reinterpret_cast<const bf16x8 *>(step + from[m0 + m]);
#pragma unroll
                        for (int m = 0; m < 4; ++m)
#pragma unroll
                            for (int u = 0; u < 2; ++u)
                                x[u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k[u].k[m0 + m], b[m], x[u], 0, 0, 0);
                    }
                    // Where not every row sees every key, or some row does not count: what is not seen
                    // is minus infinity, a weight of 0.
                    bool in = counts(lse);
                    int i = mine_i, last = mine_i + kWideRows - 1;
                    if (FLAT) {
                        const int row = row_lo + (tile + row_wave) * kWideRows;
                        i = WeighRow(a, min(row, rows - 1)).i;
                        last = row + kWideRows <= rows ? WeighRow(a, row + kWideRows - 1).i : n;
                    }
                    if (i < full_lo || last >= full_hi || tile + row_wave >= tiles || !__all(in)) {
                        int token = mine_i + c;
                        in = in && token < n && tile + row_wave < tiles;
                        if (FLAT) {
                            const int row = row_lo + (tile + row_wave) * kWideRows + c;
                            in = counts(lse) && row < rows;
                            token = WeighRow(a, min(row, rows - 1)).i;
                        }
                        unsigned long long sees = in ? seen_keys(a, past, n, min(token, n - 1), begin + min(token, n - 1), key) : 0ull;
                        sees >>= 4 * half;
#pragma unroll
                        for (int u = 0; u < 2; ++u)
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                x[u][e] = unsigned(sees >> 32 * u) >> (8 * (e / 4) + e % 4) & 1 ? x[u][e] : kNegInf;
                    }
                    const RowFacts f = row_facts(a, lse, in);
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            sum[u][e] = __builtin_fmaf(exp2_fast(__builtin_fmaf(x[u][e], a.scale_log2, -f.r)), f.factor, sum[u][e]);
                    if (!FLAT)
#pragma unroll
                        for (int j = 0; j < RW; ++j) advance(mine_i, mine_g);
                    tile += RW;
                    if (tile >= tiles) break;
                }
            }
            // lanes with bit 4 clear take the sums of the first 32 keys, the others those of the second
            const float both[2] = {column_sums(sum[0]), column_sums(sum[1])};
            const int u = lane >> 4 & 1, of_tile = 8 * (lane >> 2 & 3) + 4 * half + (lane & 3);
            float total = u ? both[1] : both[0];
            const unsigned has = (u ? k[1].has : k[0].has) >> (of_tile >> 4);
            const int of_wave = 32 * u + of_tile;
            if constexpr (RW > 1) {
                float *const meet = reinterpret_cast<float *>(lds);
                __syncthreads();                       // the last step's readers
                meet[wave * kWideKeys + of_wave] = total;
                __syncthreads();
                total = 0.0f;
#pragma unroll
                for (int w = 0; w < RW; ++w) total += meet[(w * kKeyWaves + key_wave) * kWideKeys + of_wave];
            }
            const int at = key + of_wave;
            if (row_wave == 0 && at < end) {
                float *const to = a.weights + (int64_t(s) * a.kv.heads + head) * a.width + at;
                const float old = a.decay != 0.0f && at < past ? *to : 0.0f;
                *to = gathered(total, has & 1, old, a.decay);
            }
        }
    }
}

constexpr int kFewFill = 4096;

// Workgroups along a launch's x for `tiles`; what is past them, and past the bounds, the
// workgroups walk.
static dim3 weigh_grid(const WeighArgs &a, int64_t tiles) {
    const int64_t most = 1 << 20;
    return dim3(unsigned(tiles < 1 ? 1 : tiles < most ? tiles : most), a.kv.heads, a.kv.seqs < 65535 ? a.kv.seqs : 65535);
}

template <int D, int BITS>
static int launch_few(const WeighArgs &a, int64_t context, int64_t most_rows, hipStream_t stream) {
    const int64_t steps = ceil_div(context, kWeighWaves * 32) * a.kv.seqs, all = steps * a.kv.heads;
    // Two workgroups a CU, or as many as fit where there are steps for them (32000 keys of 8
    // heads 9.5 us, with four 10.2; 64 sequences of 4095 keys 32.6, with two 37.1): with
    // more than one tile of rows two fit (8 tokens of 40 heads over 16385 keys 12.7 us, with four 19.4).
    const int64_t groups = all < kFewFill || most_rows > 16 ? 512 : 1024, each = ceil_div(groups, a.kv.heads);
    const dim3 grid(unsigned(steps < 1 ? 1 : steps < each ? steps : each), a.kv.heads);
    if (most_rows <= 16) weigh_few_kernel<D, BITS, 1><<<grid, kWeighThreads, 0, stream>>>(a);
    else if (most_rows <= 32) weigh_few_kernel<D, BITS, 2><<<grid, kWeighThreads, 0, stream>>>(a);
    else weigh_few_kernel<D, BITS, 4><<<grid, kWeighThreads, 0, stream>>>(a);
    return launch_status();
}

template <int D, int BITS, int RW>
static int launch_many_as(const WeighArgs &a, int64_t context, bool flat, hipStream_t stream) {
    typedef WideShape<D, RW> W;
    const dim3 grid = weigh_grid(a, ceil_div(context, kWeighWaves / RW * kWideKeys));
    const auto launch = [&](auto is_flat) {
        constexpr bool FLAT = decltype(is_flat)::value;
        if constexpr (W::kLds > 64 * 1024)
            if (!raise_lds<weigh_many_kernel<D, BITS, RW, FLAT>>(W::kLds)) return int(NVFP4_EHIP);
        weigh_many_kernel<D, BITS, RW, FLAT><<<grid, kWeighThreads, W::kLds, stream>>>(a);
        return launch_status();
    };
    return flat ? launch(IntC<1>()) : launch(IntC<0>());
}

template <int D, int BITS>
static int launch_many(const WeighArgs &a, int64_t context, bool even, hipStream_t stream) {
    // Tiles of a head's tokens leave places of the last one empty, half of them where the
    // lengths differ: taken where that is less than an eighth (of 40 heads, 2048 tokens over
    // 32768 keys 700 us, of rows one after another 778; 64 over 8192 12.1 against 12.9; but 4 x
    // 40 tokens over 16384 keys 71 against 48, 1 to 301 tokens of 7 sequences 126 against 98).
    const int64_t mean = a.kv.tokens / a.kv.seqs, places = ceil_div(mean, 32) * 32 + (even ? 0 : 16);
    const bool flat = 8 * places > 9 * mean || a.q_stride >= int64_t(1) << 25 || a.q_heads >= 1 << 24;
    // Waves share keys where there are not enough of them to give every CU two workgroups.
    const int64_t groups = ceil_div(context, kWeighWaves * kWideKeys) * a.kv.heads * a.kv.seqs;
    if (groups >= 512) return launch_many_as<D, BITS, 1>(a, context, flat, stream);
    if (groups >= 256 || D == 256) return launch_many_as<D, BITS, 2>(a, context, flat, stream);
    return launch_many_as<D, BITS, D == 256 ? 2 : 4>(a, context, flat, stream);
}

}  // namespace nvfp4

using namespace nvfp4;

NVFP4_API int nvfp4_kv_weights(const nvfp4_kv_cache *cache, const nvfp4_kv_batch *batch, const uint16_t *q,
                               int64_t q_stride, int q_heads, float scale, int window, const uint64_t *tree,
                               const float *lse, float decay, float *weights, int64_t width, hipStream_t stream) {
    WeighArgs a;
    if (int st = kv_check(cache, batch, a.kv)) return st;
    if (q_heads < 1 || q_heads % cache->heads != 0 || batch->tokens > (int64_t(1) << 30) / q_heads) return NVFP4_ESHAPE;
    if ((batch->tokens > 0 && (!q || !lse || !weights)) || !tscale_ok(scale) || window < 0) return NVFP4_EINVAL;
    if (!(decay >= 0.0f && decay <= 1.0f) || (tree && (window > 0 || batch->max_new > 64))) return NVFP4_EINVAL;
    if (q_stride < int64_t(q_heads) * cache->head_dim || q_stride > (int64_t(1) << 40)) return NVFP4_ESHAPE;
    if (width < a.kv.capacity || width > (int64_t(1) << 40)) return NVFP4_ESHAPE;
    if (!aligned(q, 16) || q_stride % 8 || !aligned(lse, 4) || !aligned(weights, 4) || !aligned(tree, 8)) return NVFP4_EALIGN;
    if (batch->tokens == 0) return NVFP4_OK;
    a.q = q;
    a.lse = lse;
    a.tree = reinterpret_cast<const unsigned long long *>(tree);
    a.weights = weights;
    a.q_stride = q_stride;
    a.width = width;
    a.q_heads = q_heads;
    a.group = q_heads / cache->heads;
    a.group_magic = 0xFFFFFFFFu / uint32_t(a.group);
    a.window = window;
    const double c = double(scale) * 1.4426950408889634074;
    a.scale_log2 = float(c);
    a.lost = float((c - a.scale_log2) / scale - (1.4426950408889634074 - double(kLog2e)));
    a.decay = decay;
    // Which kernels, by the bounds: that for few rows alone, that for many alone where all
    // sequences are as long, or each for its own sequences.
    const int64_t most_rows = int64_t(batch->max_new > 1 ? batch->max_new : 1) * a.group;
    const bool even = batch->tokens == int64_t(batch->seqs) * batch->max_new;      // all of the same length
    a.few_rows = most_rows <= kFewRows ? 0x7FFFFFFF : even ? -1 : kFewRows;
    const int64_t context = batch->max_context < a.kv.capacity ? batch->max_context : a.kv.capacity;
    return kv_dim(cache->head_dim, [&](auto dim) {
        return kv_bits(cache->k_format, [&](auto bits) {
            constexpr int D = decltype(dim)::value, BITS = decltype(bits)::value;
            if (most_rows <= kFewRows || !even)
                if (int st = launch_few<D, BITS>(a, context, most_rows, stream)) return st;
            return most_rows > kFewRows ? launch_many<D, BITS>(a, context, even, stream) : NVFP4_OK;
        });
    });
}
