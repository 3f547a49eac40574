// nvfp4_logprobs.hip -- log probabilities of given tokens, entropy and the likeliest
// tokens of rows of logits (gfx950).
//
// One pass over the logits: a workgroup holds a chunk of a row in registers and leaves,
// with d = scale * (x - m), the largest logit m, l = sum e^d, t = sum e^d d, and the `top`
// largest logits as keys.  A second launch joins a row's chunks,
//   l = sum l_c e^D,  t = sum e^D (t_c + l_c D)  with D = scale * (m_c - m),
//   lse = scale * m + log l,  entropy = log l - t / l,
// and looks the given tokens up.  Bound by reading the logits once: 512 rows of 151936 in
// fp32 take 58 us and the join 6.9 (5.4 TB/s, a large copy's rate); one row 6.0 and 5.0, two
// launches.
//
// The largest logits of a chunk are found without sorting it.  The top-th largest of a
// wave's 64 lane maxima is no larger than the chunk's top-th largest, since that many
// elements reach it, and neither is the least, over the four waves, of their
// (top / 4)-th largest; the larger of the two is close.  What reaches it, a few more than
// `top`, goes to shared memory, where an element's rank is the number of larger ones.
// Where too many reach it (equal logits, such as masked ones) the bound is taken again,
// among all threads' maxima with their places, which no two share.
#include <math.h>

#include "nvfp4_host.h"

namespace nvfp4 {

typedef unsigned long long Key;           // order of the value, then of falling index; 0: none

constexpr int kLogpThreads = 256, kLogpWaves = kLogpThreads / kLanes;
constexpr int kLong = 32, kShort = 8;      // logits of a thread
constexpr int kCandidates = 512;
constexpr int64_t kMaxGroups = (int64_t(1) << 32) / kLogpThreads - 1;     // of a launch: its threads stay below 2^32
constexpr int64_t kLogpFill = 512;                // workgroups with long chunks from which on they are taken
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNegInf = -__builtin_inff();

// Sums of one part relative to its largest logit, m.  l is in 64 bits: where one token is all
// but certain, l is 1 and a little, and that little is all of its log probability.  The
// reference is m and not scale * m, whose rounding would put the largest term off 1.
struct Sums {
    float m, t;
    double l;
};

struct LogpArgs {
    const void *logits;
    int64_t stride;
    int vocab, chunks, given, top;
    float scale;
    float pre, post;       // d = (pre * x - pre * m) * post, pre a power of two
    float to_log2;         // post * log2(e)
    const int *tokens;
    float *logp, *lse, *entropy, *top_logp;
    int *top_index;
    Sums *parts;           // [n][chunks]
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

// Values over the whole wave, in every lane: exchanges within rows of 16 lanes, then of rows.
template <int CTRL>
__device__ __forceinline__ float lane_of(float v) {
    return __uint_as_float(uint32_t(__builtin_amdgcn_update_dpp(0, int(__float_as_uint(v)), CTRL, 0xF, 0xF, false)));
}
template <class F>
__device__ __forceinline__ float over_wave(float v, F f) {
    v = f(v, lane_of<0xB1>(v));      // quad_perm [1,0,3,2]
    v = f(v, lane_of<0x4E>(v));      // quad_perm [2,3,0,1]
    v = f(v, lane_of<0x141>(v));     // row_half_mirror
    v = f(v, lane_of<0x140>(v));     // row_mirror
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = f(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return f(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
// The same sum of a 64-bit number, both of whose halves go between the lanes.
template <int CTRL>
__device__ __forceinline__ double lane_of(double v) {
    const u32x2 w = __builtin_bit_cast(u32x2, v);
    const u32x2 y = {uint32_t(__builtin_amdgcn_update_dpp(0, int(w[0]), CTRL, 0xF, 0xF, false)),
                     uint32_t(__builtin_amdgcn_update_dpp(0, int(w[1]), CTRL, 0xF, 0xF, false))};
    return __builtin_bit_cast(double, y);
}
__device__ __forceinline__ double wave_sum(double v) {
    v += lane_of<0xB1>(v);
    v += lane_of<0x4E>(v);
    v += lane_of<0x141>(v);
    v += lane_of<0x140>(v);
    u32x2 w = __builtin_bit_cast(u32x2, v);
    const auto a0 = __builtin_amdgcn_permlane16_swap(w[0], w[0], false, false);
    const auto a1 = __builtin_amdgcn_permlane16_swap(w[1], w[1], false, false);
    v = __builtin_bit_cast(double, u32x2{a0[0], a1[0]}) + __builtin_bit_cast(double, u32x2{a0[1], a1[1]});
    w = __builtin_bit_cast(u32x2, v);
    const auto b0 = __builtin_amdgcn_permlane32_swap(w[0], w[0], false, false);
    const auto b1 = __builtin_amdgcn_permlane32_swap(w[1], w[1], false, false);
    return __builtin_bit_cast(double, u32x2{b0[0], b1[0]}) + __builtin_bit_cast(double, u32x2{b0[1], b1[1]});
}
__device__ __forceinline__ float wave_sum(float v) { return over_wave(v, [](float x, float y) { return x + y; }); }
__device__ __forceinline__ float wave_largest(float v) { return over_wave(v, [](float x, float y) { return fmaxf(x, y); }); }

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

struct TopShared {
    Key list[kCandidates], most[kLogpThreads];
    Key wave[kLogpWaves], least;
    uint32_t every[kLogpWaves], quarter[kLogpWaves];
    int found;
};

// The `top` largest of a workgroup's keys to out[0 .. top - 1], in order; 0 where it has
// fewer.  A thread's largest order is `most` (0 if it has none); offer(bound, take) calls
// take for each of its keys whose order is at least `bound`, each(f) calls f for all of them.
template <class Offer, class Each>
__device__ __forceinline__ void largest(TopShared &sh, int top, uint32_t most, Offer offer, Each each, Key *out) {
    const int tid = threadIdx.x, wave = tid / kLanes;
    const uint32_t every = reached_by(most, top), quarter = reached_by(most, (top + kLogpWaves - 1) / kLogpWaves);
    if ((tid & 63) == 0) {
        sh.every[wave] = every;
        sh.quarter[wave] = quarter;
    }
    if (tid == 0) {
        sh.found = 0;
        sh.least = ~Key(0);
    }
    __syncthreads();
    uint32_t bound = sh.every[0], all = sh.quarter[0];
#pragma unroll
    for (int w = 1; w < kLogpWaves; ++w) {
        bound = max(bound, sh.every[w]);
        all = min(all, sh.quarter[w]);
    }
    bound = max(bound, all);
    const auto take = [&](Key k) {
        const int at = atomicAdd(&sh.found, 1);
        if (at < kCandidates) sh.list[at] = k;
    };
    if (most >= bound) offer(bound, take);
    __syncthreads();
    int found = sh.found;
    if (found > kCandidates) {
        Key mine = 0;
        each([&](Key k) { mine = max(mine, k); });
        sh.most[tid] = mine;
        __syncthreads();
        int larger = 0;
        for (int i = 0; i < kLogpThreads; ++i) larger += sh.most[i] > mine;
        if (tid == 0) sh.found = 0;
        if (larger < top) atomicMin(&sh.least, mine);
        __syncthreads();
        const Key least = max(sh.least, Key(1));
        if (mine >= least)
            each([&](Key k) {
                if (k >= least) take(k);
            });
        __syncthreads();
        found = sh.found;
    }
    if (found <= kCandidates) {
        for (int i = tid; i < max(found, top); i += kLogpThreads) {
            if (i >= found) {
                out[i] = 0;
                continue;
            }
            const Key k = sh.list[i];
            int rank = 0;
#pragma unroll 8
            for (int j = 0; j < found; ++j) rank += sh.list[j] > k;
            if (rank < top) out[rank] = k;
        }
    } else {
        // a few threads hold most of the largest: one after another
        Key last = ~Key(0);
        for (int r = 0; r < top; ++r) {
            Key best = 0;
            each([&](Key k) { best = k < last ? max(best, k) : best; });
            best = lanes_max_u64<64>(best);
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

// A part's sums relative to m >= s.m; parts of nothing (m = -infinity, l = 0) stay
// nothing, and a difference past fp32's range has no infinity to multiply a weight of 0.
__device__ __forceinline__ Sums moved(const LogpArgs &a, Sums s, float m) {
    // the powers of two below 1 alone: no product passes fp32's range
    const float pre = fminf(a.pre, 1.0f), post = a.pre > 1.0f ? a.scale : a.post;
    const float d = s.m == kNegInf ? 0.0f : fmaxf(__builtin_fmaf(s.m, pre, -(m * pre)) * post, -1e30f);
    const float w = __builtin_amdgcn_exp2f(d * kLog2e);
    return Sums{m, w * __builtin_fmaf(float(s.l), d, s.t), s.l * w};
}

__device__ __forceinline__ float logit(const float *row, int at) { return row[at]; }
__device__ __forceinline__ float logit(const uint16_t *row, int at) { return __uint_as_float(uint32_t(row[at]) << 16); }

// A thread's N logits, four in a row at place(0), place(4), ...: all in flight together.
// A chunk that the row's end cuts is read one by one, minus infinity past it.
template <int N, class Place>
__device__ __forceinline__ void load_logits(const float *row, bool full, int vocab, Place place, float (&x)[N]) {
    typedef float F4 __attribute__((ext_vector_type(4), aligned(4)));
    if (full) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const F4 v = *reinterpret_cast<const F4 *>(row + place(i));
#pragma unroll
            for (int j = 0; j < 4; ++j) x[i + j] = v[j];
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = place(i) < vocab ? row[place(i)] : kNegInf;
    }
}
template <int N, class Place>
__device__ __forceinline__ void load_logits(const uint16_t *row, bool full, int vocab, Place place, float (&x)[N]) {
    typedef unsigned int U2 __attribute__((ext_vector_type(2), aligned(2)));
    uint32_t w[N / 2];
    if (full) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const U2 v = *reinterpret_cast<const U2 *>(row + place(i));
            w[i / 2] = v[0];
            w[i / 2 + 1] = v[1];
        }
    } else {
        constexpr uint32_t kMasked = 0xFF80;             // minus infinity
#pragma unroll
        for (int i = 0; i < N; i += 2)
            w[i / 2] = (place(i) < vocab ? uint32_t(row[place(i)]) : kMasked) |
                       (place(i + 1) < vocab ? uint32_t(row[place(i + 1)]) : kMasked) << 16;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
}

// log x for x > 0 (NaN stays NaN): of the power of two in 64 bits, of what is left, which
// is within 0.7 .. 1.4, by its distance from 1, so that the result is good to 2^-22 of
// itself also next to x = 1.
__device__ __forceinline__ double log_of(double x) {
    double part = __builtin_amdgcn_frexp_mant(x);
    int power = __builtin_amdgcn_frexp_exp(x);
    const bool low = part < 0.70710678118654752440;
    part = low ? part + part : part;
    power -= low;
    return power * 0.69314718055994530942 + log1pf(float(part - 1.0));
}

template <class T, int N>
__global__ void __launch_bounds__(kLogpThreads, 8) logprobs_chunk_kernel(LogpArgs a) {
    __shared__ TopShared sh;
    __shared__ Sums sums[kLogpWaves];
    const int tid = threadIdx.x, wave = tid / kLanes;
    const int chunk = int(blockIdx.x % unsigned(a.chunks)), r = int(blockIdx.x / unsigned(a.chunks));
    const int first = chunk * (N * kLogpThreads);
    const T *const row = static_cast<const T *>(a.logits) + r * a.stride;
    const auto place = [&](int i) { return first + (i / 4 * kLogpThreads + tid) * 4 + i % 4; };
    float x[N];
    const bool full = first + N * kLogpThreads <= a.vocab;
    load_logits<N>(row, full, a.vocab, place, x);
    float most = x[0];
#pragma unroll
    for (int i = 1; i < N; ++i) most = fmaxf(most, x[i]);
    const float top = wave_largest(most);
    Sums s = {top, 0.0f, 0.0};
    // A `pre` of 2 is for scales whose product with log2(e) may pass fp32's range.  It is left
    // out where 2 * top may: logits that far out differ by nothing or by so much that e is 0.
    const float pre = fabsf(top) < 0x1p126f ? a.pre : fminf(a.pre, 1.0f);
    const float base = top == kNegInf ? 0.0f : top * pre;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float y = __builtin_fmaf(x[i], pre, -base);            // d / post
        const float e = __builtin_amdgcn_exp2f(y * a.to_log2);
        s.l += double(e);
        s.t = __builtin_fmaf(e, fmaxf(y, -1e30f), s.t);
    }
    s.t *= a.post;
    s.l = wave_sum(s.l);
    s.t = wave_sum(s.t);
    if ((tid & 63) == 0) sums[wave] = s;
    const int64_t part = int64_t(r) * a.chunks + chunk;
    if (a.top > 0) {
        uint32_t reach = order_of(most);
        if (!full) {                                     // places past the row reach nothing
            reach = 0;
#pragma unroll
            for (int i = 0; i < N; ++i) reach = place(i) < a.vocab ? max(reach, order_of(x[i])) : reach;
        }
        const auto offer = [&](uint32_t bound, auto take) {
            // by value; NaN only where anything is taken, and below -infinity's order there is no value
            const float limit = bound < 0x007FFFFFu ? kNegInf : value_of(bound);
#pragma unroll
            for (int i = 0; i < N; ++i)
                if ((x[i] >= limit || bound == 0) && (full || place(i) < a.vocab)) take(key_of(order_of(x[i]), place(i)));
        };
        // Rarely needed, so read again: what the rare path keeps through the kernel costs the
        // common one its occupancy.
        const auto each = [&](auto f) {
#pragma unroll 2
            for (int j = 0; j < N; j += 4) {
                float y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = place(j) + e < a.vocab ? logit(row, place(j) + e) : 0.0f;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (place(j) + e < a.vocab) f(key_of(order_of(y[e]), place(j) + e));
            }
        };
        largest(sh, a.top, reach, offer, each, a.keys + part * a.top);
    } else {
        __syncthreads();
    }
    if (tid == 0) {
        float m = sums[0].m;
#pragma unroll
        for (int w = 1; w < kLogpWaves; ++w) m = fmaxf(m, sums[w].m);
        Sums all = {m, 0.0f, 0.0};
#pragma unroll
        for (int w = 0; w < kLogpWaves; ++w) {
            const Sums o = moved(a, sums[w], m);
            all.l += o.l;
            all.t += o.t;
        }
        a.parts[part] = all;
    }
}

__global__ void __launch_bounds__(kLogpThreads) logprobs_join_kernel(LogpArgs a, int dtype) {
    __shared__ TopShared sh;
    __shared__ Sums sums[kLogpWaves];
    __shared__ Key best[NVFP4_MAX_TOP];
    const int tid = threadIdx.x, wave = tid / kLanes, r = blockIdx.x;
    const Sums *const parts = a.parts + int64_t(r) * a.chunks;
    // the chunks' keys, the first of them in registers
    constexpr int kKept = 8;
    const int64_t all_keys = int64_t(a.chunks) * a.top;
    const Key *const keys = a.keys + r * all_keys;
    Key mine[kKept];
    uint32_t reach = 0;
#pragma unroll
    for (int i = 0; i < kKept; ++i) mine[i] = tid + i * kLogpThreads < all_keys ? keys[tid + i * kLogpThreads] : Key(0);
    float m = kNegInf;
    for (int c = tid; c < a.chunks; c += kLogpThreads) m = fmaxf(m, parts[c].m);
    m = wave_largest(m);
    Sums s = {m, 0.0f, 0.0};
    for (int c = tid; c < a.chunks; c += kLogpThreads) {
        const Sums o = moved(a, parts[c], m);
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
    Sums all = {m, 0.0f, 0.0};
#pragma unroll
    for (int w = 0; w < kLogpWaves; ++w) {
        const Sums o = moved(a, sums[w], m);
        all.l += o.l;
        all.t += o.t;
    }
    const bool nothing = m == kNegInf && all.l == 0.0;
    const double log_l = log_of(all.l);
    const float lse = nothing ? kNegInf : float(__builtin_fma(double(m), double(a.scale), log_l));
    const float entropy = nothing ? 0.0f : float(log_l - all.t / all.l);
    // z - lse without the rounding of a large lse
    const auto logp = [&](float x) { return nothing ? kNegInf : float((double(x) - double(m)) * double(a.scale) - log_l); };
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
            y = logp(dtype == NVFP4_KV_F32 ? logit(static_cast<const float *>(a.logits) + row, token)
                                           : logit(static_cast<const uint16_t *>(a.logits) + row, token));
        a.logp[at] = y;
    }
    if (a.top == 0) return;
#pragma unroll
    for (int i = 0; i < kKept; ++i) reach = max(reach, uint32_t(mine[i] >> 32));
    for (int64_t i = tid + kKept * kLogpThreads; i < all_keys; i += kLogpThreads) reach = max(reach, uint32_t(keys[i] >> 32));
    const auto each = [&](auto f) {                    // 0 where there is none
#pragma unroll
        for (int i = 0; i < kKept; ++i) f(mine[i]);
        for (int64_t i = tid + kKept * kLogpThreads; i < all_keys; i += kLogpThreads) f(keys[i]);
    };
    const auto offer = [&](uint32_t bound, auto take) {
        each([&](Key k) {
            if (k && uint32_t(k >> 32) >= bound) take(k);
        });
    };
    largest(sh, a.top, reach, offer, each, best);
    __syncthreads();
    for (int i = tid; i < a.top; i += kLogpThreads) {
        a.top_index[int64_t(r) * a.top + i] = index_of(best[i]);
        a.top_logp[int64_t(r) * a.top + i] = logp(value_of(uint32_t(best[i] >> 32)));
    }
}

// Logits of a workgroup: chunks of 2048 where longer ones would leave CUs idle (one row of
// 151936: 11.0 us, of 8192 13.7; 16 rows 13.9 and 15.0; from 24 to 27 rows either takes 16),
// else of 8192 (48 rows 18.7 us, of 2048 20.6; 128 rows 26.5 and 35; 512 rows 66 and 108; in
// bf16 17.7 and 20.1, 26 and 35, 56 and 107).
static int64_t logprobs_chunk(int64_t n, int64_t vocab) {
    return (n * ceil_div(vocab, kLong * kLogpThreads) < kLogpFill ? kShort : kLong) * kLogpThreads;
}

static bool logprobs_shape_ok(int64_t n, int64_t vocab, int top) {
    if (n < 0 || n > (int64_t(1) << 30) || vocab < 1 || vocab > (int64_t(1) << 30)) return false;
    if (top < 0 || top > NVFP4_MAX_TOP || top > vocab) return false;
    return n * ceil_div(vocab, logprobs_chunk(n, vocab)) <= kMaxGroups;
}

// What a call of n rows writes to its workspace.
static size_t logprobs_need(int64_t n, int64_t vocab, int top) {
    return size_t(n) * size_t(ceil_div(vocab, logprobs_chunk(n, vocab))) * (sizeof(Sums) + size_t(top) * sizeof(Key));
}

}  // namespace nvfp4

using namespace nvfp4;

NVFP4_API size_t nvfp4_logprobs_workspace_bytes(int64_t n, int64_t vocab, int top) {
    if (!logprobs_shape_ok(n, vocab, top)) return 0;
    // that of the most rows in short chunks may be larger
    const int64_t most_short = (kLogpFill - 1) / ceil_div(vocab, kLong * kLogpThreads);
    const size_t need = logprobs_need(n, vocab, top), fewer = logprobs_need(n < most_short ? n : most_short, vocab, top);
    return need > fewer ? need : fewer;
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
    if (!workspace || workspace_bytes < logprobs_need(n, vocab, top)) return NVFP4_EWORKSPACE;
    if (!aligned(workspace, 16)) return NVFP4_EALIGN;
    LogpArgs a = {};
    a.logits = logits;
    a.stride = stride;
    a.vocab = int(vocab);
    const bool short_chunks = logprobs_chunk(n, vocab) == kShort * kLogpThreads;
    a.chunks = int(ceil_div(vocab, logprobs_chunk(n, vocab)));
    a.given = given;
    a.top = top;
    a.scale = scale;
    // Of a scale below 1 the power of two goes to the logits, whose difference might pass
    // fp32's range where its product does not; of the largest a 2.
    int power;
    const float part = frexpf(scale, &power);            // scale = part * 2^power, part in 1/2 .. 1
    a.pre = scale < 1.0f ? ldexpf(1.0f, power - 1) : scale < 0x1p126f ? 1.0f : 2.0f;
    a.post = scale < 1.0f ? 2.0f * part : scale / a.pre;
    a.to_log2 = float(double(a.post) * 1.4426950408889634074);
    a.tokens = tokens;
    a.logp = logp;
    a.lse = lse;
    a.entropy = entropy;
    a.top_logp = top_logp;
    a.top_index = top_index;
    a.parts = static_cast<Sums *>(workspace);
    a.keys = reinterpret_cast<Key *>(a.parts + size_t(n) * a.chunks);
    const unsigned groups = unsigned(n * a.chunks);
    const auto launch = [&](auto kernel) { kernel<<<groups, kLogpThreads, 0, stream>>>(a); };
    if (dtype == NVFP4_KV_F32) launch(short_chunks ? logprobs_chunk_kernel<float, kShort> : logprobs_chunk_kernel<float, kLong>);
    else launch(short_chunks ? logprobs_chunk_kernel<uint16_t, kShort> : logprobs_chunk_kernel<uint16_t, kLong>);
    if (int st = launch_status()) return st;
    logprobs_join_kernel<<<unsigned(n), kLogpThreads, 0, stream>>>(a, dtype);
    return launch_status();
}
