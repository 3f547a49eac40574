// nvfp4_rope.hip -- rotary positions of one or several axes (gfx950).
//
// A thread owns four pairs of one token (or eight elements of the part that does not
// turn) and takes them through several heads: the angle, its sine and cosine are
// worked out once for all of them.  Angles are taken in quarter turns in 64 bits,
// t = position * frequency * 2 / pi: t less its nearest whole number is exact to
// 2^-53 of t, at a position of 2^20 better than 2^-31 of a turn, and what is left, at
// most an eighth of a turn, is rounded to fp32.  Sine and cosine of that are their
// power series to x^9 and x^10 (the next terms are below 2^-29 at pi / 4).
#include "nvfp4_host.h"

namespace nvfp4 {

constexpr int kRopeThreads = 256;
constexpr int64_t kRopeMost = int64_t(1) << 32;   // threads are counted in 32 bits
constexpr int64_t kRopeFill = 1 << 19;             // units of eight elements
constexpr double kTwoOverPi = 0.63661977236758134308;
constexpr float kHalfPi = 1.57079632679489661923f;

struct RopeSet {
    const void *in;
    void *out;
    int64_t in_stride, out_stride;
    int first;             // heads of the sets before it
    bool f32;              // type of `out`
};

struct RopeArgs {
    RopeSet set[NVFP4_MAX_ROPE];
    int count, heads;      // sets, heads of all of them
    int dim, rotary, adjacent;
    int units, turning;    // units of eight elements of a head, and those that turn
    int slots;             // threads that share a token's unit: thread s takes heads s, s + slots, ...
    uint32_t threads;      // in all
    int tokens, axes;
    const int *positions;
    const double *freqs;
    const uint8_t *axis;
    float factor;
};

__device__ __forceinline__ floatx4 load4(const float *p) { return *reinterpret_cast<const floatx4 *>(p); }
__device__ __forceinline__ floatx4 load4(const uint16_t *p) {
    const u32x2 w = *reinterpret_cast<const u32x2 *>(p);
    return floatx4{__uint_as_float(w[0] << 16), __uint_as_float(w[0] & 0xFFFF0000u), __uint_as_float(w[1] << 16),
                   __uint_as_float(w[1] & 0xFFFF0000u)};
}
// STREAM: past the caches.
template <bool STREAM, class V>
__device__ __forceinline__ void put(V *p, V v) {
    if constexpr (STREAM) __builtin_nontemporal_store(v, p);
    else *p = v;
}
template <bool STREAM>
__device__ __forceinline__ void store4(float *p, floatx4 x) { put<STREAM>(reinterpret_cast<floatx4 *>(p), x); }
template <bool STREAM>
__device__ __forceinline__ void store4(uint16_t *p, floatx4 x) {
    u32x2 w;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        bf16x2 v;
        v[0] = static_cast<__bf16>(x[2 * i]);
        v[1] = static_cast<__bf16>(x[2 * i + 1]);
        w[i] = as_u32(v);
    }
    put<STREAM>(reinterpret_cast<u32x2 *>(p), w);
}

// Cosine and sine of `turns` quarter turns.
__device__ __forceinline__ void turn(double turns, float &c, float &s) {
    const double whole = __builtin_rint(turns);
    const float x = float(turns - whole) * kHalfPi;
    const int quarter = int(whole - 4.0 * __builtin_floor(whole * 0.25));
    const float y = x * x;
    float p = __builtin_fmaf(y, 1.0f / 362880, -1.0f / 5040);
    p = __builtin_fmaf(y, p, 1.0f / 120);
    p = __builtin_fmaf(y, p, -1.0f / 6);
    const float sine = __builtin_fmaf(x * y, p, x);
    float q = __builtin_fmaf(y, -1.0f / 3628800, 1.0f / 40320);
    q = __builtin_fmaf(y, q, -1.0f / 720);
    q = __builtin_fmaf(y, q, 1.0f / 24);
    q = __builtin_fmaf(y, q, -0.5f);
    const float cosine = __builtin_fmaf(y, q, 1.0f);
    const float a = quarter & 1 ? sine : cosine, b = quarter & 1 ? cosine : sine;
    c = (quarter + 1) & 2 ? -a : a;
    s = quarter & 2 ? -b : b;
}

template <class T, int HEADS>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(RopeArgs a) {
    constexpr bool STREAM = HEADS > 1;                 // outputs that no cache would hold
    const uint32_t at = blockIdx.x * uint32_t(kRopeThreads) + threadIdx.x;
    if (at >= a.threads) return;
    const uint32_t per_token = uint32_t(a.units * a.slots);
    const int token = int(at / per_token), rest = int(at % per_token);
    const int slot = rest / a.units, unit = rest % a.units;
    const bool turns = unit < a.turning;
    const bool half = turns && !a.adjacent;            // pairs half the rotary part apart
    const int lo = half ? 4 * unit : 8 * unit, hi = half ? a.rotary / 2 + lo : lo + 4;

    floatx4 x[HEADS], y[HEADS];
    int of[HEADS];                                     // the head's set
#pragma unroll
    for (int i = 0; i < HEADS; ++i) {
        const int h = min(slot + i * a.slots, a.heads - 1);
        of[i] = 0;
        for (int k = 1; k < a.count; ++k) of[i] += h >= a.set[k].first;
        const RopeSet &r = a.set[of[i]];
        const T *p = static_cast<const T *>(r.in) + token * r.in_stride + (h - r.first) * a.dim;
        x[i] = load4(p + lo);
        y[i] = load4(p + hi);
    }
    float c[4], s[4];
    if (turns) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int pair = 4 * unit + i;
            const int axis = a.axis ? a.axis[pair] : 0;
            const int position = axis < a.axes ? a.positions[int64_t(axis) * a.tokens + token] : 0;
            turn(position * (a.freqs[pair] * kTwoOverPi), c[i], s[i]);
            c[i] *= a.factor;
            s[i] *= a.factor;
        }
    }
#pragma unroll
    for (int i = 0; i < HEADS; ++i) {
        const int h = slot + i * a.slots;
        if (h >= a.heads) break;
        if (half) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float u = x[i][j], v = y[i][j];
                x[i][j] = __builtin_fmaf(u, c[j], -(v * s[j]));
                y[i][j] = __builtin_fmaf(v, c[j], u * s[j]);
            }
        } else if (turns) {
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
                float u = x[i][j], v = x[i][j + 1];
                x[i][j] = __builtin_fmaf(u, c[j / 2], -(v * s[j / 2]));
                x[i][j + 1] = __builtin_fmaf(v, c[j / 2], u * s[j / 2]);
                u = y[i][j], v = y[i][j + 1];
                y[i][j] = __builtin_fmaf(u, c[2 + j / 2], -(v * s[2 + j / 2]));
                y[i][j + 1] = __builtin_fmaf(v, c[2 + j / 2], u * s[2 + j / 2]);
            }
        }
        const RopeSet &r = a.set[of[i]];
        const int64_t to = token * r.out_stride + (h - r.first) * a.dim;
        if (r.f32) {
            store4<STREAM>(static_cast<float *>(r.out) + to + lo, x[i]);
            store4<STREAM>(static_cast<float *>(r.out) + to + hi, y[i]);
        } else {
            store4<STREAM>(static_cast<uint16_t *>(r.out) + to + lo, x[i]);
            store4<STREAM>(static_cast<uint16_t *>(r.out) + to + hi, y[i]);
        }
    }
}

template <class T, int HEADS>
static int rope_launch(RopeArgs &a, hipStream_t stream) {
    a.slots = int(ceil_div(a.heads, HEADS));
    const int64_t threads = int64_t(a.tokens) * a.units * a.slots;
    if (threads >= kRopeMost) return NVFP4_ESHAPE;
    a.threads = uint32_t(threads);
    rope_kernel<T, HEADS><<<grid_1d(threads, kRopeThreads), kRopeThreads, 0, stream>>>(a);
    return launch_status();
}

template <class T>
static int rope_typed(RopeArgs &a, hipStream_t stream) {
    // Four heads a thread where the card is full all the same (2048 tokens of 48 heads of 128
    // 16.7 us, a head a thread 28), their outputs past the caches (18.2 through them).
    if (int64_t(a.tokens) * a.units * a.heads >= kRopeFill) return rope_launch<T, 4>(a, stream);
    return rope_launch<T, 1>(a, stream);
}

}  // namespace nvfp4

using namespace nvfp4;

NVFP4_API int nvfp4_rope(const nvfp4_rope_rows *rows, int count, int dtype, int64_t tokens, int head_dim,
                         int rotary_dim, int adjacent, const int32_t *positions, int axes, const double *freqs,
                         const uint8_t *axis, float factor, hipStream_t stream) {
    if (!rows || count < 1 || count > NVFP4_MAX_ROPE || tokens < 0 || axes < 1 || !freqs || !tscale_ok(factor))
        return NVFP4_EINVAL;
    if (dtype != NVFP4_KV_BF16 && dtype != NVFP4_KV_F32) return NVFP4_EINVAL;
    if (tokens > 0 && !positions) return NVFP4_EINVAL;
    if (head_dim < 8 || head_dim > 1024 || head_dim % 8 || rotary_dim < 8 || rotary_dim > head_dim || rotary_dim % 8)
        return NVFP4_ESHAPE;
    if (tokens > (int64_t(1) << 30) || axes > 256) return NVFP4_ESHAPE;
    RopeArgs a = {};
    for (int i = 0; i < count; ++i) {
        const nvfp4_rope_rows &r = rows[i];
        if (tokens > 0 && (!r.in || !r.out)) return NVFP4_EINVAL;
        if (r.out_type != NVFP4_KV_BF16 && r.out_type != NVFP4_KV_F32) return NVFP4_EINVAL;
        if (r.heads < 1 || r.heads > 65535) return NVFP4_ESHAPE;
        const int64_t wide = int64_t(r.heads) * head_dim, most = int64_t(1) << 40;
        if (r.in_stride < wide || r.out_stride < wide || r.in_stride > most || r.out_stride > most) return NVFP4_ESHAPE;
        if (!aligned(r.in, 16) || !aligned(r.out, 16)) return NVFP4_EALIGN;
        if (r.in_stride % (dtype == NVFP4_KV_F32 ? 4 : 8) || r.out_stride % (r.out_type == NVFP4_KV_F32 ? 4 : 8))
            return NVFP4_EALIGN;
        // in place a thread reads what it writes, and nothing else, only where both are laid out the same
        if (r.in && r.in == r.out && (r.out_type != dtype || r.in_stride != r.out_stride)) return NVFP4_EINVAL;
        a.set[i] = RopeSet{r.in, r.out, r.in_stride, r.out_stride, a.heads, r.out_type == NVFP4_KV_F32};
        a.heads += r.heads;
    }
    if (!aligned(freqs, 8) || !aligned(positions, 4)) return NVFP4_EALIGN;
    if (tokens == 0) return NVFP4_OK;
    a.count = count;
    a.dim = head_dim;
    a.rotary = rotary_dim;
    a.adjacent = adjacent != 0;
    a.units = head_dim / 8;
    a.turning = rotary_dim / 8;
    a.tokens = int(tokens);
    a.axes = axes;
    a.positions = positions;
    a.freqs = freqs;
    a.axis = axis;
    a.factor = factor;
    return dtype == NVFP4_KV_F32 ? rope_typed<float>(a, stream) : rope_typed<uint16_t>(a, stream);
}
