// nvfp4_logprobs.hip -- log probabilities of given tokens, entropy and the likeliest
// tokens of rows of logits (gfx950).
//
// One pass over the logits: a workgroup holds kChunk of a row in registers and leaves,
// of z = scale * x, the maximum m, l = sum e^(z - m), t = sum e^(z - m) (z - m), and the
// `top` largest logits as keys.  A second launch joins a row's chunks,
//   l = sum l_c e^(m_c - m),  t = sum e^(m_c - m) (t_c + l_c (m_c - m)),
//   lse = m + log l,  entropy = log l - t / l,
// and looks the given tokens up.
//
// The largest logits of a chunk are found without sorting it: the top-th largest of a
// wave's 64 lane maxima is no larger than the chunk's top-th largest, since that many
// elements reach it.  What reaches the largest such bound of the waves, a few more than
// `top` of them, goes to shared memory, where an element's rank is the number of larger
// ones.  Where too many reach it (long runs of equal logits) the maximum is taken `top`
// times.
#include "nvfp4_host.h"

namespace nvfp4 {

typedef unsigned long long Key;           // order of the value, then of falling index; 0: none

constexpr int kLogpThreads = 256, kLogpWaves = kLogpThreads / kLanes;
constexpr int kChunk = 32 * kLogpThreads;            // logits of a workgroup
constexpr int kCandidates = 512;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNegInf = -__builtin_inff();

struct LogpArgs {
    const void *logits;
    int64_t stride;
    int n, vocab, chunks, given, top;
    float scale;
    const int *tokens;
    float *logp, *lse, *entropy, *top_logp;
    int *top_index;
    float *parts;          // [n][chunks][4]: m, l, t, unused
    Key *keys;             // [n][chunks][top]
};

// Whole numbers in the order of the values: NaN 0, then -infinity to infinity, -0 as 0.
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    const uint32_t o = b & 0x80000000u ? ~b : b | 0x80000000u;
    return x != x ? 0u : o;
}
__device__ __forceinline__ float value_of(uint32_t o) {
    return o == 0 ? __builtin_nanf("") : __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}
__device__ __forceinline__ Key key_of(uint32_t order, int index) { return Key(order) << 32 | (0xFFFFFFFFu - uint32_t(index)); }
__device__ __forceinline__ int index_of(Key k) { return int(0xFFFFFFFFu - uint32_t(k)); }

// A number that `k` lanes of the wave at least reach, the k-th largest but for the bits
// below the top 20.
__device__ __forceinline__ uint32_t reached_by(uint32_t v, int k) {
    uint32_t bound = 0;
#pragma unroll
    for (int bit = 31; bit >= 12; --bit) {
        const uint32_t t = bound | 1u << bit;
        if (__popcll(__ballot(v >= t)) >= k) bound = t;
    }
    return bound;
}

__device__ __forceinline__ Key wave_max(Key v) { return lanes_max_u64<64>(v); }

// The `top` largest of a workgroup's keys (absent ones 0) to out[0 .. top - 1], in order.
// Each thread's keys are 0 .. count - 1 of `key`, their orders' largest is `most`.
// Threads need not hold `top` keys together: what is missing is 0.
struct TopShared {
    Key list[kCandidates];
    Key wave[kLogpWaves];
    uint32_t bound[kLogpWaves];
    int found;
};
template <int UNROLL, class KeyAt>
__device__ __forceinline__ void largest(TopShared &sh, int top, int count, uint32_t most, KeyAt key, Key *out) {
    const int tid = threadIdx.x, wave = tid / kLanes;
    const uint32_t mine = reached_by(most, top);
    if ((tid & 63) == 0) sh.bound[wave] = mine;
    if (tid == 0) sh.found = 0;
    __syncthreads();
    uint32_t bound = sh.bound[0];
#pragma unroll
    for (int w = 1; w < kLogpWaves; ++w) bound = max(bound, sh.bound[w]);
    const Key least = max(Key(bound) << 32, Key(1));
    if (Key(most) << 32 >= (least & 0xFFFFFFFF00000000ull))
#pragma unroll UNROLL
        for (int i = 0; i < count; ++i) {
            const Key k = key(i);
            if (k >= least) {
                const int at = atomicAdd(&sh.found, 1);
                if (at < kCandidates) sh.list[at] = k;
            }
        }
    __syncthreads();
    const int found = sh.found;
    if (found <= kCandidates) {
        for (int i = tid; i < max(found, top); i += kLogpThreads) {
            if (i >= found) {
                out[i] = 0;
                continue;
            }
            const Key k = sh.list[i];
            int rank = 0;
            for (int j = 0; j < found; ++j) rank += sh.list[j] > k;
            if (rank < top) out[rank] = k;
        }
    } else {
        Key last = ~Key(0);
        for (int r = 0; r < top; ++r) {
            Key best = 0;
#pragma unroll UNROLL
            for (int i = 0; i < count; ++i) {
                const Key k = key(i);
                if (k < last && k > best) best = k;
            }
            best = wave_max(best);
            if ((tid & 63) == 0) sh.wave[wave] = best;
            __syncthreads();
            last = sh.wave[0];
#pragma unroll
            for (int w = 1; w < kLogpWaves; ++w) last = max(last, sh.wave[w]);
            if (tid == 0) out[r] = last;
            __syncthreads();
        }
    }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
    return v;
}
__device__ __forceinline__ float wave_largest(float v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
    return v;
}

// Sums of one part relative to its maximum.
struct Sums {
    float m, l, t;
};
// A part's sums relative to m >= s.m; parts of nothing (m = -infinity, l = 0) stay
// nothing, and a difference past fp32's range has no infinity to multiply a weight of 0.
__device__ __forceinline__ Sums moved(Sums s, float m) {
    const float d = s.m == kNegInf ? 0.0f : fmaxf(s.m - m, -1e30f);
    const float w = __builtin_amdgcn_exp2f(d * kLog2e);
    return Sums{m, s.l * w, w * __builtin_fmaf(s.l, d, s.t)};
}

template <class T>
__device__ __forceinline__ void load_logits(const T *row, int first, int vocab, float (&x)[32]);
template <>
__device__ __forceinline__ void load_logits<float>(const float *row, int first, int vocab, float (&x)[32]) {
    typedef float F4 __attribute__((ext_vector_type(4), aligned(4)));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int at = first + (i * kLogpThreads + int(threadIdx.x)) * 4;
        if (at + 4 <= vocab) {
            const F4 v = *reinterpret_cast<const F4 *>(row + at);
#pragma unroll
            for (int j = 0; j < 4; ++j) x[4 * i + j] = v[j];
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) x[4 * i + j] = at + j < vocab ? row[at + j] : kNegInf;
        }
    }
}
template <>
__device__ __forceinline__ void load_logits<uint16_t>(const uint16_t *row, int first, int vocab, float (&x)[32]) {
    typedef unsigned int U2 __attribute__((ext_vector_type(2), aligned(2)));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int at = first + (i * kLogpThreads + int(threadIdx.x)) * 4;
        if (at + 4 <= vocab) {
            const U2 v = *reinterpret_cast<const U2 *>(row + at);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                x[4 * i + j] = __uint_as_float(j & 1 ? v[j / 2] & 0xFFFF0000u : v[j / 2] << 16);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                x[4 * i + j] = at + j < vocab ? __uint_as_float(uint32_t(row[at + j]) << 16) : kNegInf;
        }
    }
}

template <class T>
__global__ void __launch_bounds__(kLogpThreads) logprobs_chunk_kernel(LogpArgs a) {
    __shared__ TopShared sh;
    __shared__ Sums sums[kLogpWaves];
    const int tid = threadIdx.x, wave = tid / kLanes;
    const int chunk = int(blockIdx.x % unsigned(a.chunks)), r = int(blockIdx.x / unsigned(a.chunks));
    const int first = chunk * kChunk;
    float x[32];
    load_logits<T>(static_cast<const T *>(a.logits) + r * a.stride, first, a.vocab, x);
    float most = x[0];
#pragma unroll
    for (int i = 1; i < 32; ++i) most = fmaxf(most, x[i]);
    const float top = wave_largest(most);
    Sums s = {top * a.scale, 0.0f, 0.0f};
    const float base = s.m == kNegInf ? 0.0f : s.m;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
        const float d = __builtin_fmaf(x[i], a.scale, -base);
        const float e = __builtin_amdgcn_exp2f(d * kLog2e);
        s.l += e;
        s.t = __builtin_fmaf(e, fmaxf(d, -1e30f), s.t);
    }
    s.l = wave_sum(s.l);
    s.t = wave_sum(s.t);
    if ((tid & 63) == 0) sums[wave] = s;
    const int64_t part = int64_t(r) * a.chunks + chunk;
    if (a.top > 0) {
        const auto key = [&](int i) {
            const int at = first + (i / 4 * kLogpThreads + tid) * 4 + i % 4;
            return at < a.vocab ? key_of(order_of(x[i]), at) : Key(0);
        };
        uint32_t reach = order_of(most);
        if (first + kChunk > a.vocab) {                  // places past the row reach nothing
            reach = 0;
#pragma unroll
            for (int i = 0; i < 32; ++i) reach = max(reach, uint32_t(key(i) >> 32));
        }
        largest<32>(sh, a.top, 32, reach, key, a.keys + part * a.top);
    } else {
        __syncthreads();
    }
    if (tid == 0) {
        float m = sums[0].m;
#pragma unroll
        for (int w = 1; w < kLogpWaves; ++w) m = fmaxf(m, sums[w].m);
        Sums all = {m, 0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < kLogpWaves; ++w) {
            const Sums o = moved(sums[w], m);
            all.l += o.l;
            all.t += o.t;
        }
        float *p = a.parts + part * 4;
        p[0] = all.m;
        p[1] = all.l;
        p[2] = all.t;
    }
}

__global__ void __launch_bounds__(kLogpThreads) logprobs_join_kernel(LogpArgs a, int dtype) {
    __shared__ TopShared sh;
    __shared__ Sums sums[kLogpWaves];
    __shared__ Key best[NVFP4_MAX_TOP];
    const int tid = threadIdx.x, wave = tid / kLanes, r = blockIdx.x;
    const float *parts = a.parts + int64_t(r) * a.chunks * 4;
    float m = kNegInf;
    for (int c = tid; c < a.chunks; c += kLogpThreads) m = fmaxf(m, parts[4 * c]);
    m = wave_largest(m);
    Sums s = {m, 0.0f, 0.0f};
    for (int c = tid; c < a.chunks; c += kLogpThreads) {
        const Sums o = moved(Sums{parts[4 * c], parts[4 * c + 1], parts[4 * c + 2]}, m);
        s.l += o.l;
        s.t += o.t;
    }
    s.l = wave_sum(s.l);
    s.t = wave_sum(s.t);
    if ((tid & 63) == 0) sums[wave] = s;
    __syncthreads();
    m = sums[0].m;
#pragma unroll
    for (int w = 1; w < kLogpWaves; ++w) m = fmaxf(m, sums[w].m);
    Sums all = {m, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < kLogpWaves; ++w) {
        const Sums o = moved(sums[w], m);
        all.l += o.l;
        all.t += o.t;
    }
    const bool nothing = m == kNegInf && all.l == 0.0f;
    const float log_l = __builtin_logf(all.l);
    const float lse = nothing ? kNegInf : m + log_l;
    const float entropy = nothing ? 0.0f : log_l - all.t / all.l;
    // z - lse without the rounding of a large lse
    const auto logp = [&](float x) { return nothing ? kNegInf : __builtin_fmaf(x, a.scale, -m) - log_l; };
    if (tid == 0) {
        if (a.lse) a.lse[r] = lse;
        if (a.entropy) a.entropy[r] = entropy;
    }
    const int64_t row = r * a.stride;
    for (int i = tid; i < a.given; i += kLogpThreads) {
        const int64_t at = int64_t(r) * a.given + i;
        const int token = a.tokens[at];
        float y = __builtin_nanf("");
        if (token >= 0 && token < a.vocab)
            y = logp(dtype == NVFP4_KV_F32 ? static_cast<const float *>(a.logits)[row + token]
                                           : __uint_as_float(uint32_t(static_cast<const uint16_t *>(a.logits)[row + token]) << 16));
        a.logp[at] = y;
    }
    if (a.top == 0) return;
    const int64_t all_keys = int64_t(a.chunks) * a.top;
    const Key *keys = a.keys + r * all_keys;
    const int count = int((all_keys - tid + kLogpThreads - 1) / kLogpThreads);
    uint32_t most = 0;
    for (int i = 0; i < count; ++i) most = max(most, uint32_t(keys[tid + int64_t(i) * kLogpThreads] >> 32));
    __syncthreads();
    largest<1>(sh, a.top, count, most, [&](int i) { return keys[tid + int64_t(i) * kLogpThreads]; }, best);
    __syncthreads();
    for (int i = tid; i < a.top; i += kLogpThreads) {
        a.top_index[int64_t(r) * a.top + i] = index_of(best[i]);
        a.top_logp[int64_t(r) * a.top + i] = logp(value_of(uint32_t(best[i] >> 32)));
    }
}

static bool logprobs_shape_ok(int64_t n, int64_t vocab, int top) {
    if (n < 0 || n > (int64_t(1) << 30) || vocab < 1 || vocab > (int64_t(1) << 30)) return false;
    if (top < 0 || top > NVFP4_MAX_TOP || top > vocab) return false;
    return n * ceil_div(vocab, kChunk) <= 0x7FFFFFFF;
}

}  // namespace nvfp4

using namespace nvfp4;

NVFP4_API size_t nvfp4_logprobs_workspace_bytes(int64_t n, int64_t vocab, int top) {
    if (!logprobs_shape_ok(n, vocab, top)) return 0;
    return size_t(n) * size_t(ceil_div(vocab, kChunk)) * (4 * sizeof(float) + size_t(top) * sizeof(Key));
}

NVFP4_API int nvfp4_logprobs(int dtype, const void *logits, int64_t n, int64_t vocab, int64_t stride, float scale,
                             const int32_t *tokens, int given, float *logp, float *lse, float *entropy, int top,
                             float *top_logp, int32_t *top_index, void *workspace, size_t workspace_bytes,
                             hipStream_t stream) {
    if (dtype != NVFP4_KV_BF16 && dtype != NVFP4_KV_F32) return NVFP4_EINVAL;
    if (!tscale_ok(scale) || given < 0 || given > 1 << 20) return NVFP4_EINVAL;
    if (!logprobs_shape_ok(n, vocab, top) || stride < vocab || stride > (int64_t(1) << 40)) return NVFP4_ESHAPE;
    if (n > 0) {
        if (!logits || (given > 0 && (!tokens || !logp)) || (top > 0 && (!top_logp || !top_index))) return NVFP4_EINVAL;
        if (given == 0 && top == 0 && !lse && !entropy) return NVFP4_EINVAL;
    }
    if (!aligned(logits, dtype == NVFP4_KV_F32 ? 4 : 2) || !aligned(tokens, 4) || !aligned(logp, 4) || !aligned(lse, 4) ||
        !aligned(entropy, 4) || !aligned(top_logp, 4) || !aligned(top_index, 4))
        return NVFP4_EALIGN;
    if (n == 0) return NVFP4_OK;
    const size_t need = nvfp4_logprobs_workspace_bytes(n, vocab, top);
    if (!workspace || workspace_bytes < need) return NVFP4_EWORKSPACE;
    if (!aligned(workspace, 16)) return NVFP4_EALIGN;
    LogpArgs a = {};
    a.logits = logits;
    a.stride = stride;
    a.n = int(n);
    a.vocab = int(vocab);
    a.chunks = int(ceil_div(vocab, kChunk));
    a.given = given;
    a.top = top;
    a.scale = scale;
    a.tokens = tokens;
    a.logp = logp;
    a.lse = lse;
    a.entropy = entropy;
    a.top_logp = top_logp;
    a.top_index = top_index;
    a.parts = static_cast<float *>(workspace);
    a.keys = reinterpret_cast<Key *>(a.parts + size_t(n) * a.chunks * 4);
    const unsigned groups = unsigned(n * a.chunks);
    if (dtype == NVFP4_KV_F32) logprobs_chunk_kernel<float><<<groups, kLogpThreads, 0, stream>>>(a);
    else logprobs_chunk_kernel<uint16_t><<<groups, kLogpThreads, 0, stream>>>(a);
    if (int st = launch_status()) return st;
    logprobs_join_kernel<<<unsigned(n), kLogpThreads, 0, stream>>>(a, dtype);
    return launch_status();
}
