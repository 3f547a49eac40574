// nvfp4_rope.hip -- rotary positions of one or several axes (gfx950).
//
// A unit of four pairs, or eight of bf16 rows where their halves stand on 16 bytes, is a
// thread's; of many tokens a workgroup works out each pair's sine and cosine once and
// keeps them in shared memory for all heads.  Bound by its bytes: 16384 tokens of 48 heads
// of 128 in bf16 take 69.6 us, 5.8 TB/s, the outputs stored past the caches (76 us
// through them); 64 tokens of 40 heads 3.5 us, a launch.  Angles are taken in quarter turns
// in 64 bits, t = position * frequency * 2 / pi: t less its nearest whole number is exact
// to 2^-53 of t, at a position of 2^20 better than 2^-31 of a turn, and what is left, at
// most an eighth of a turn, is rounded to fp32.  Sine and cosine of that are their power
// series to x^9 and x^10 (the next terms are below 2^-29 at pi / 4).
#include "nvfp4_host.h"

namespace nvfp4 {

constexpr int kRopeThreads = 256;
constexpr int64_t kRopeMost = int64_t(1) << 34;   // units of eight elements
constexpr int64_t kRopeMostGroups = (int64_t(1) << 32) / kRopeThreads - 1;     // of a launch: its threads stay below 2^32
// Workgroups from which rope_many_kernel is the faster one (256 tokens of 48 heads of 128,
// 256 of them, 4.3 us against 5.3; 300 of 32 heads of 72, 57 of them, 5.3 against 3.9).
constexpr int64_t kRopeFill = 128;
constexpr int kRopeTurns = 512;                    // of a workgroup
constexpr double kTwoOverPi = 0.63661977236758134308;
constexpr float kHalfPi = 1.57079632679489661923f;

struct RopeSet {
    const void *in;
    void *out;
    int64_t in_stride, out_stride;
    int first;             // heads of the sets before it
    bool f32;              // type of `out`
};

// How rope_many_kernel's workgroups, from `first` on, share a set: `span` tokens of `per`
// of its heads each, `ranges` of which are all of them.
struct RopeShare {
    unsigned first;
    int heads, per, ranges, span;
    uint32_t token_magic, last_magic;
};

struct RopeArgs {
    RopeSet set[NVFP4_MAX_ROPE];
    int count, heads;      // sets, heads of all of them
    int dim, rotary, adjacent;
    int units, turning;    // units of eight elements of a head, and those that turn
    uint32_t threads;      // rope_few_kernel's
    RopeShare share[NVFP4_MAX_ROPE];
    uint32_t unit_magic, pair_magic;
    int tokens, axes;
    const int *positions;
    const double *freqs;
    const uint8_t *axis;
    float factor;
};

// Where a unit of 8 * WIDE elements of a head stands: in two halves, which hold the two
// elements of pairs that stand apart, or pair after pair.
struct RopeUnit {
    bool turns, apart;
    int lo, hi;
    __device__ __forceinline__ RopeUnit(const RopeArgs &a, int unit, int wide) {
        turns = unit * wide < a.turning;
        apart = turns && !a.adjacent;
        lo = (apart ? 4 : 8) * wide * unit;
        hi = lo + (apart ? a.rotary / 2 : 4 * wide);
    }
};

// The set of head h of all, by choice among scalars: lanes' own loads of it would be
// waited for before each row's.
__device__ __forceinline__ RopeSet set_of(const RopeArgs &a, int h) {
    RopeSet r = a.set[0];
#pragma unroll
    for (int k = 1; k < NVFP4_MAX_ROPE; ++k) {
        const bool here = k < a.count && h >= a.set[k].first;
        r.in = here ? a.set[k].in : r.in;
        r.out = here ? a.set[k].out : r.out;
        r.in_stride = here ? a.set[k].in_stride : r.in_stride;
        r.out_stride = here ? a.set[k].out_stride : r.out_stride;
        r.first = here ? a.set[k].first : r.first;
        r.f32 = here ? a.set[k].f32 : r.f32;
    }
    return r;
}

// 4 * WIDE elements as they are in memory, and as numbers.
template <class T, int WIDE>
struct Raw {
    typedef uint32_t Words __attribute__((ext_vector_type(WIDE * sizeof(T))));
    Words w;
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (sizeof(Words) <= 16) {
            w = *reinterpret_cast<const Words *>(p);
        } else {
#pragma unroll
            for (int i = 0; i < int(sizeof(Words)) / 16; ++i) {
                const u32x4 t = reinterpret_cast<const u32x4 *>(p)[i];
                w[4 * i] = t[0]; w[4 * i + 1] = t[1]; w[4 * i + 2] = t[2]; w[4 * i + 3] = t[3];
            }
        }
    }
    __device__ __forceinline__ void numbers(floatx4 (&x)[WIDE]) const {
#pragma unroll
        for (int i = 0; i < 4 * WIDE; ++i)
            x[i / 4][i % 4] = __uint_as_float(sizeof(T) == 4 ? w[i] : i % 2 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    }
};
// STREAM: past the caches.
template <bool STREAM, class V>
__device__ __forceinline__ void put(V *p, V v) {
    if constexpr (STREAM) __builtin_nontemporal_store(v, p);
    else *p = v;
}
template <bool STREAM, int WIDE>
__device__ __forceinline__ void store(const RopeSet &r, int64_t at, const floatx4 (&x)[WIDE]) {
    if (r.f32) {
#pragma unroll
        for (int w = 0; w < WIDE; ++w) put<STREAM>(reinterpret_cast<floatx4 *>(static_cast<float *>(r.out) + at) + w, x[w]);
    } else {
        typedef uint32_t Words __attribute__((ext_vector_type(2 * WIDE)));
        Words t;
#pragma unroll
        for (int i = 0; i < 2 * WIDE; ++i) {
            bf16x2 v;
            v[0] = static_cast<__bf16>(x[i / 2][2 * (i % 2)]);
            v[1] = static_cast<__bf16>(x[i / 2][2 * (i % 2) + 1]);
            t[i] = as_u32(v);
        }
        put<STREAM>(reinterpret_cast<Words *>(static_cast<uint16_t *>(r.out) + at), t);
    }
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

// A pair of a token: its (cosine, sine), times the factor.
struct RopeTurn {
    int axis, position;
    double freq;
    __device__ __forceinline__ void load_pair(const RopeArgs &a, int pair) {
        axis = a.axis ? a.axis[pair] : 0;
        freq = a.freqs[pair];
    }
    __device__ __forceinline__ void load_position(const RopeArgs &a, int token) {
        const bool some = axis < a.axes;
        position = a.positions[int64_t(some ? axis : 0) * a.tokens + token];
        position = some ? position : 0;
    }
    __device__ __forceinline__ float2 operator()(float factor) const {
        float c, s;
        turn(position * (freq * kTwoOverPi), c, s);
        return make_float2(c * factor, s * factor);
    }
};

// u, v: the elements of a pair.
__device__ __forceinline__ void turn_pair(float2 t, float u, float v, float &to_u, float &to_v) {
    to_u = __builtin_fmaf(u, t.x, -(v * t.y));
    to_v = __builtin_fmaf(v, t.x, u * t.y);
}

// A unit turned; t: of its pairs.
template <int WIDE>
__device__ __forceinline__ void turn_unit(bool apart, const float2 *t, floatx4 (&x)[WIDE], floatx4 (&y)[WIDE]) {
    if (apart) {
#pragma unroll
        for (int w = 0; w < WIDE; ++w)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float u = x[w][j], v = y[w][j];
                float to_u, to_v;
                turn_pair(t[4 * w + j], u, v, to_u, to_v);
                x[w][j] = to_u;
                y[w][j] = to_v;
            }
    } else {
#pragma unroll
        for (int w = 0; w < 2 * WIDE; ++w)
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
                floatx4 &z = w < WIDE ? x[w] : y[w - WIDE];
                const float u = z[j], v = z[j + 1];
                float to_u, to_v;
                turn_pair(t[2 * w + j / 2], u, v, to_u, to_v);
                z[j] = to_u;
                z[j + 1] = to_v;
            }
    }
}

// A thread to a unit of one head of one token.
template <class T>
__global__ void __launch_bounds__(kRopeThreads) rope_few_kernel(RopeArgs a) {
    const uint32_t at = blockIdx.x * uint32_t(kRopeThreads) + threadIdx.x;
    if (at >= a.threads) return;
    const uint32_t per_token = uint32_t(a.units * a.heads);
    const int token = int(at / per_token), rest = int(at % per_token);
    const int h = rest / a.units, unit = rest % a.units;
    const RopeUnit u(a, unit, 1);
    const RopeSet r = set_of(a, h);
    const T *p = static_cast<const T *>(r.in) + token * r.in_stride + (h - r.first) * a.dim;
    Raw<T, 1> lo, hi;
    lo.load(p + u.lo);
    hi.load(p + u.hi);
    floatx4 x[1], y[1];
    lo.numbers(x);
    hi.numbers(y);
    if (u.turns) {
        RopeTurn w[4];
        float2 t[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i].load_pair(a, 4 * unit + i);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i].load_position(a, token);
#pragma unroll
        for (int i = 0; i < 4; ++i) t[i] = w[i](a.factor);
        turn_unit<1>(u.apart, t, x, y);
    }
    const int64_t to = token * r.out_stride + (h - r.first) * a.dim;
    store<false, 1>(r, to + u.lo, x);
    store<false, 1>(r, to + u.hi, y);
}

// The quotient of e >= 0 by what `magic` is of, exact while 4 * e times that is below 2^32.
static uint32_t magic_of(int d) { return uint32_t(((1ull << 32) + 2 * d - 1) / (2 * d)); }
__device__ __forceinline__ int quotient(int e, uint32_t magic) { return int(__umulhi(2 * uint32_t(e) + 1, magic)); }

// A workgroup to `span` tokens of `per` heads, whose sines and cosines, each worked out
// once, stand in shared memory; ITEMS units of 8 * WIDE elements a thread, whose loads
// are on their way meanwhile.
template <class T, int WIDE, int ITEMS>
__global__ void __launch_bounds__(kRopeThreads) rope_many_kernel(RopeArgs a) {
    __shared__ __align__(16) float2 turns[kRopeTurns];
    int set = 0;
    for (int k = 1; k < a.count; ++k) set += blockIdx.x >= a.share[k].first;
    const RopeSet &r = a.set[set];
    const RopeShare &f = a.share[set];
    const int block = int(blockIdx.x - f.first), token0 = block / f.ranges * f.span, head0 = block % f.ranges * f.per;
    const int span = min(f.span, a.tokens - token0), per = min(f.per, f.heads - head0);
    const int pairs = a.rotary / 2, units = a.units / WIDE, items = span * per * units;
    int thread = threadIdx.x;
    const auto place = [&](int i, int &token, int &h, int &unit) __attribute__((always_inline)) {
        const int item = i * kRopeThreads + thread, at = min(item, items - 1);
        // of the last heads there may be fewer
        token = quotient(at, per == f.per ? f.token_magic : f.last_magic);
        const int rest = at - token * per * units;
        h = quotient(rest, a.unit_magic);
        unit = rest - h * units;
        token += token0;
        h += head0;
        return item < items;
    };
    // What the angles are of first: the rows' loads are on their way while the angles'
    // sines and cosines are worked out.
    constexpr int kMine = kRopeTurns / kRopeThreads;
    RopeTurn mine[kMine];
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
        const int i = min(k * kRopeThreads + thread, span * pairs - 1);
        mine[k].load_pair(a, i - quotient(i, a.pair_magic) * pairs);
    }
#pragma unroll
    for (int k = 0; k < kMine; ++k)
        mine[k].load_position(a, token0 + quotient(min(k * kRopeThreads + thread, span * pairs - 1), a.pair_magic));
    asm volatile("" ::: "memory");
    Raw<T, WIDE> lo[ITEMS], hi[ITEMS];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        int token, h, unit;
        place(i, token, h, unit);
        const RopeUnit u(a, unit, WIDE);
        const T *p = static_cast<const T *>(r.in) + token * r.in_stride + h * a.dim;
        lo[i].load(p + u.lo);
        hi[i].load(p + u.hi);
    }
#pragma unroll
    for (int k = 0; k < kMine; ++k)
        if (k * kRopeThreads + thread < span * pairs) turns[k * kRopeThreads + thread] = mine[k](a.factor);
    __syncthreads();
    asm volatile("" : "+v"(thread));                   // places are worked out again rather than kept
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        int token, h, unit;
        if (!place(i, token, h, unit)) break;
        const RopeUnit u(a, unit, WIDE);
        floatx4 x[WIDE], y[WIDE];
        lo[i].numbers(x);
        hi[i].numbers(y);
        if (u.turns) {
            float2 t[4 * WIDE];
            const floatx4 *const from = reinterpret_cast<const floatx4 *>(turns + (token - token0) * pairs + 4 * WIDE * unit);
#pragma unroll
            for (int j = 0; j < 2 * WIDE; ++j) {
                const floatx4 two = from[j];
                t[2 * j] = make_float2(two[0], two[1]);
                t[2 * j + 1] = make_float2(two[2], two[3]);
            }
            turn_unit<WIDE>(u.apart, t, x, y);
        }
        const int64_t to = token * r.out_stride + h * a.dim;
        store<true, WIDE>(r, to + u.lo, x);
        store<true, WIDE>(r, to + u.hi, y);
    }
}

template <class T, int WIDE, int ITEMS>
static int launch_rope_many(RopeArgs &a, hipStream_t stream) {
    const int units = a.units / WIDE, most = kRopeThreads * ITEMS, pairs = a.rotary / 2;
    int64_t blocks = 0;
    for (int k = 0; k < a.count; ++k) {
        RopeShare &f = a.share[k];
        f.first = unsigned(blocks);
        f.heads = (k + 1 < a.count ? a.set[k + 1].first : a.heads) - a.set[k].first;
        f.per = int(ceil_div(f.heads, ceil_div(int64_t(f.heads) * units, most)));
        if (f.per * units > most) f.per = most / units;
        f.ranges = int(ceil_div(f.heads, f.per));
        f.span = min(most / (f.per * units), kRopeTurns / pairs);
        f.token_magic = magic_of(f.per * units);
        f.last_magic = magic_of((f.heads - (f.ranges - 1) * f.per) * units);
        blocks += ceil_div(a.tokens, f.span) * f.ranges;
    }
    if (blocks > kRopeMostGroups) return NVFP4_ESHAPE;
    a.unit_magic = magic_of(units);
    a.pair_magic = magic_of(pairs);
    rope_many_kernel<T, WIDE, ITEMS><<<unsigned(blocks), kRopeThreads, 0, stream>>>(a);
    return launch_status();
}

template <class T>
static int rope_typed(RopeArgs &a, hipStream_t stream) {
    // ITEMS: with more of them fewer workgroups stay on a CU, with fewer their sines and
    // cosines weigh more (16384 tokens of 48 heads of 128 in bf16 69.6 us with 3, 72.0 with 4;
    // 16383 of 32 heads of 72 35.5 us with 6, 37.6 with 8).
    const bool wide = sizeof(T) == 2 && a.units % 2 == 0 && a.turning % 2 == 0;
    const int64_t units = int64_t(a.tokens) * a.heads * a.units, block = kRopeThreads * (sizeof(T) == 2 ? 6 : 3);
    if (units >= kRopeFill * block) {
        if constexpr (sizeof(T) == 2) return wide ? launch_rope_many<T, 2, 3>(a, stream) : launch_rope_many<T, 1, 6>(a, stream);
        else return launch_rope_many<T, 1, 3>(a, stream);
    }
    a.threads = uint32_t(units);
    rope_few_kernel<T><<<grid_1d(units, kRopeThreads), kRopeThreads, 0, stream>>>(a);
    return launch_status();
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
        for (int k = 0; k < i; ++k)
            if (r.out && (r.out == rows[k].out || r.out == rows[k].in || r.in == rows[k].out)) return NVFP4_EINVAL;
        a.set[i] = RopeSet{r.in, r.out, r.in_stride, r.out_stride, a.heads, r.out_type == NVFP4_KV_F32};
        a.heads += r.heads;
    }
    if (!aligned(freqs, 8) || !aligned(positions, 4)) return NVFP4_EALIGN;
    if (tokens == 0) return NVFP4_OK;
    if (tokens * (head_dim / 8) * a.heads >= kRopeMost) return NVFP4_ESHAPE;
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
