// nvfp4_kv_weights.hip -- the attention that each cached key receives, gathered over
// steps (gfx950).
//
// A wave holds 32 keys of a head as the A operand of v_mfma_f32_32x32x16_bf16 and walks
// the query rows, 32 at a time, as B: a lane of the accumulator then has 16 keys' scores
// of one row, whose log-sum-exp it holds too, and adds its weights to 16 running sums.
// Only at the end are the sums of the 32 rows' lanes added.  Waves of a workgroup share
// keys (each takes its part of the rows; their sums meet in shared memory) or rows.
//
// A weight is 2^(s * c - r) with c = scale * log2(e) and r = lse * log2(e), each rounded
// to fp32; what that loses of the weights that count, those whose score is near lse, is
// the same for a whole row, and the factor that puts it right is one operand of the sum's
// multiply-add.  Rows that count for nothing have a factor of 0.
#include "nvfp4_attn.h"

namespace nvfp4 {

constexpr int kWeighWaves = 4, kWeighThreads = kWeighWaves * kLanes;
constexpr int kWeighTile = 32;             // keys of a wave's operand, rows of a step

typedef float floatx16 __attribute__((ext_vector_type(16)));

struct WeighArgs {
    KvView kv;
    const uint16_t *q;
    const float *lse;
    const unsigned long long *tree;
    float *weights;
    int64_t q_stride, width;
    int q_heads, group, window;
    int row_waves;         // waves of a workgroup that share keys
    float scale_log2;      // c as rounded
    float lost;            // (scale * log2(e) - c) / scale
    float decay;
};

// One 32-key operand of head `head` from position `key` on.
template <int D, int BITS>
struct KeyOperand {
    typedef KvSide<D, BITS> S;
    static constexpr int kSteps = D / 16, kHalf = S::kPieces / 2, kPer = S::kPieceDims / 8;
    bf16x8 k[kSteps];
    bool some[2];          // whether the first and the second 16 keys have a page

    // The element at which a lane's eight of step m start.
    static __device__ __forceinline__ int element(int m, int half) {
        return (2 * (m / kPer) + half) * S::kPieceDims + 8 * (m % kPer);
    }
    __device__ __forceinline__ void load(const KvView &v, int s, int head, int key, int end) {
        const int lane = threadIdx.x & 63, r = lane & 15, half = lane >> 5;
        const int pos = key + (lane & 16);
        const int page = pos < end ? v.page_in(v.entry_at(s, pos), pos) : -1;
        const unsigned long long has = __ballot(page >= 0);
        some[0] = has & 1;
        some[1] = has >> 16 & 1;
        const int64_t unit = v.unit_of(max(page, 0), head, pos);
        uint32_t w[kHalf][S::kPiece / 4] = {}, scale[(S::kBlocks + 3) / 4] = {};
        if (page >= 0) {
            const uint8_t *codes = v.codes[0] + unit * S::kUnitCodes + (half * kKvUnit + r) * S::kPiece;
#pragma unroll
            for (int j = 0; j < kHalf; ++j) load_words<S::kPiece>(codes + 2 * j * kKvUnit * S::kPiece, w[j]);
            load_words<S::kBlocks>(v.scales[0] + unit * S::kUnitScales + r * S::kBlocks, scale);
        }
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

template <int D, int BITS>
__global__ void __launch_bounds__(kWeighThreads) kv_weights_kernel(WeighArgs a) {
    typedef KeyOperand<D, BITS> K;
    __shared__ float meet[kWeighThreads];
    const int lane = threadIdx.x & 63, c = lane & 31, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int key_waves = kWeighWaves / a.row_waves;
    const int key_wave = wave % key_waves, row_wave = wave / key_waves;
    const int head = blockIdx.y;
    const unsigned group_keys = key_waves * kWeighTile;
    for (int s = blockIdx.z; s < a.kv.seqs; s += gridDim.z) {
        int begin, stop, past;
        a.kv.sequence(s, begin, stop, past);
        const int n = stop - begin, rows = n * a.group, end = int(min(unsigned(past) + unsigned(n), unsigned(a.kv.capacity)));
        if (n == 0) continue;
        for (unsigned first = blockIdx.x * group_keys; first < unsigned(end); first += gridDim.x * group_keys) {
            const int key = int(first) + key_wave * kWeighTile;
            K k;
            k.load(a.kv, s, head, key, end);
            // the rows that may see some of the keys
            const int i_lo = a.tree ? 0 : max(0, min(key, end) - past);
            const int i_hi = a.window > 0 ? max(0, int(min(int64_t(n), int64_t(key) + kWeighTile - 1 + a.window - past))) : n;
            const int row_lo = i_lo * a.group & ~(kWeighTile - 1), row_hi = key < end ? i_hi * a.group : 0;
            float sum[16] = {};
            for (int row0 = row_lo + row_wave * kWeighTile; row0 < row_hi; row0 += a.row_waves * kWeighTile) {
                const int row = row0 + c;
                const bool in = row < rows;
                const int i = in ? row / a.group : 0, token = begin + i, qhead = head * a.group + (in ? row - i * a.group : 0);
                const float lse = in ? a.lse[int64_t(token) * a.q_heads + qhead] : kNegInf;
                const bool counts = fabsf(lse) < __builtin_inff();
                const uint16_t *src = a.q + token * a.q_stride + qhead * D;
                bf16x8 q[K::kSteps];
#pragma unroll
                for (int m = 0; m < K::kSteps; ++m) {
                    u32x4 w = {0, 0, 0, 0};
                    if (counts) w = *reinterpret_cast<const u32x4 *>(src + K::element(m, half));
                    q[m] = __builtin_bit_cast(bf16x8, w);
                }
                floatx16 x = {};
#pragma unroll
                for (int m = 0; m < K::kSteps; ++m) x = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k.k[m], q[m], x, 0, 0, 0);
                constexpr float kLog2eRest = 1.92596299e-8f;       // log2(e) - kLog2e
                const float r = counts ? lse * kLog2e : 0.0f;
                const float rest = __builtin_fmaf(lse, kLog2e, -r) + lse * kLog2eRest;
                const float factor = counts ? exp2_fast(__builtin_fmaf(lse, a.lost, -rest)) : 0.0f;
                float w[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) w[e] = exp2_fast(__builtin_fmaf(x[e], a.scale_log2, -r));
                // where not every row sees every key
                const int pos = past + i;
                const int i0 = __builtin_amdgcn_readfirstlane(i), i1 = min(row0 + kWeighTile, rows) - 1;
                const bool whole = a.tree ? key + kWeighTile <= past
                                          : key + kWeighTile - 1 <= past + i0 && (a.window == 0 || key > past + i1 / a.group - a.window);
                if (!whole) {
                    const int at = key + 4 * half;
                    if (a.tree) {
                        const unsigned long long tree = in ? a.tree[token] : 0ull;
                        const int drafted = min(n, 64);
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const int j = at + 8 * (e / 4) + e % 4 - past;
                            w[e] = j < 0 || (j < drafted && tree >> (j & 63) & 1) ? w[e] : 0.0f;
                        }
                    } else {
                        const int lo = a.window > 0 ? pos - a.window : -1;
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const int j = at + 8 * (e / 4) + e % 4;
                            w[e] = j <= pos && j > lo ? w[e] : 0.0f;
                        }
                    }
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) sum[e] = __builtin_fmaf(w[e], factor, sum[e]);
            }
            float total = column_sums(sum);
            // the lane's key of the wave's 32
            const int mine = 8 * (lane >> 2 & 3) + 4 * half + (lane & 3);
            if (a.row_waves > 1) {
                __syncthreads();                       // of the tile before
                if ((lane & 16) == 0) meet[wave * kWeighTile + mine] = total;
                __syncthreads();
                total = 0.0f;
                for (int w = 0; w < a.row_waves; ++w) total += meet[(w * key_waves + key_wave) * kWeighTile + mine];
            }
            const int at = key + mine;
            if (row_wave == 0 && (lane & 16) == 0 && at < end) {
                // a key with a NaN or an infinity, or without a page, adds nothing
                if (!(total < __builtin_inff()) || !k.some[mine >> 4]) total = 0.0f;
                float *to = a.weights + (int64_t(s) * a.kv.heads + head) * a.width + at;
                if (a.decay != 0.0f && at < past) total = __builtin_fmaf(*to, a.decay, total);
                *to = total;
            }
        }
    }
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
    a.window = window;
    const double c = double(scale) * 1.4426950408889634074;
    a.scale_log2 = float(c);
    a.lost = float((c - a.scale_log2) / scale);
    a.decay = decay;
    const int64_t most_rows = int64_t(batch->max_new > 1 ? batch->max_new : 1) * a.group;
    a.row_waves = most_rows > 64 ? kWeighWaves : 1;
    const int keys = kWeighWaves / a.row_waves * kWeighTile;
    const int context = batch->max_context < a.kv.capacity ? batch->max_context : a.kv.capacity;
    // workgroups walk what is past the grid, and past the bounds
    const int64_t tiles = ceil_div(context > 1 ? context : 1, keys), most = 1 << 20;
    const dim3 grid(unsigned(tiles < most ? tiles : most), cache->heads, batch->seqs < 65535 ? batch->seqs : 65535);
    return kv_dim(cache->head_dim, [&](auto dim) {
        return kv_bits(cache->k_format, [&](auto bits) {
            kv_weights_kernel<decltype(dim)::value, decltype(bits)::value><<<grid, kWeighThreads, 0, stream>>>(a);
            return launch_status();
        });
    });
}
