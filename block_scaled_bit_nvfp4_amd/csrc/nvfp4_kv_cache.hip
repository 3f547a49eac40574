// nvfp4_kv_cache.hip -- the paged key/value cache: the host checks that its
// entry points share, and the kernels that quantise new tokens into it and read
// them back (gfx950).
#include "nvfp4_kv.h"

namespace nvfp4 {

static bool kv_shape_ok(int format, int32_t pages, int32_t page_tokens, int32_t heads, int32_t dim) {
    if (format != NVFP4_KV_MXFP8 && format != NVFP4_KV_MXFP4) return false;
    if (pages < 1 || pages > kKvMaxPages || heads < 1 || heads > 65535) return false;
    if (page_tokens < 16 || page_tokens > 1024 || (page_tokens & (page_tokens - 1))) return false;
    return dim == 64 || dim == 128 || dim == 256;
}

int kv_check(const nvfp4_kv_cache *c, const nvfp4_kv_batch *b, KvView &v) {
    if (!c || !b) return NVFP4_EINVAL;
    if (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales) return NVFP4_EINVAL;
    if (!kv_shape_ok(c->k_format, c->pages, c->page_tokens, c->heads, c->head_dim) ||
        !kv_shape_ok(c->v_format, c->pages, c->page_tokens, c->heads, c->head_dim))
        return NVFP4_ESHAPE;
    if (!b->page_table || !b->offsets || !b->past || b->seqs < 1 || b->table_width < 1) return NVFP4_EINVAL;
    if (b->tokens < 0 || b->max_new < 0 || b->max_context < 0) return NVFP4_EINVAL;
    // positions, and rows of heads, are 32-bit in the kernels
    if (int64_t(b->table_width) * c->page_tokens > kKvMaxPositions) return NVFP4_ESHAPE;
    if (b->tokens > (int64_t(1) << 30) / c->heads) return NVFP4_ESHAPE;
    if (!aligned(c->k_codes, 16) || !aligned(c->k_scales, 16) || !aligned(c->v_codes, 16) ||
        !aligned(c->v_scales, 16) || !aligned(b->page_table, 4) || !aligned(b->offsets, 4) || !aligned(b->past, 4))
        return NVFP4_EALIGN;
    v.codes[0] = c->k_codes;
    v.codes[1] = c->v_codes;
    v.scales[0] = c->k_scales;
    v.scales[1] = c->v_scales;
    v.pages = c->pages;
    v.page_shift = __builtin_ctz(unsigned(c->page_tokens));
    v.heads = c->heads;
    v.table = b->page_table;
    v.offsets = b->offsets;
    v.past = b->past;
    v.width = b->table_width;
    v.seqs = b->seqs;
    v.tokens = int(b->tokens);
    v.capacity = b->table_width << v.page_shift;
    return NVFP4_OK;
}

// ------------------------------------------------------------------- append

// The 16 elements of one thread, as floats.
__device__ __forceinline__ void load16(const float *p, float (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 f = reinterpret_cast<const float4 *>(p)[i];
        x[4 * i] = f.x; x[4 * i + 1] = f.y; x[4 * i + 2] = f.z; x[4 * i + 3] = f.w;
    }
}
__device__ __forceinline__ void load16(const uint16_t *p, float (&x)[16]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const u32x4 w = reinterpret_cast<const u32x4 *>(p)[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
            x[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
        }
    }
}
// Stores of 16 elements a lane, four lanes in a row.  The lanes of a four exchange
// their words, so that each store instruction writes whole 64-byte runs.
template <int CTRL>
__device__ __forceinline__ uint32_t of_four(uint32_t w) {
    return uint32_t(__builtin_amdgcn_update_dpp(0, int(w), CTRL, 0xF, 0xF, false));
}
template <int FROM>
__device__ __forceinline__ void store_run(float *p, const float (&x)[16], int q) {
    u32x4 w;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t a = of_four<FROM * 0x55>(__float_as_uint(x[j])), b = of_four<FROM * 0x55>(__float_as_uint(x[4 + j]));
        const uint32_t c = of_four<FROM * 0x55>(__float_as_uint(x[8 + j])), d = of_four<FROM * 0x55>(__float_as_uint(x[12 + j]));
        w[j] = q & 2 ? (q & 1 ? d : c) : (q & 1 ? b : a);
    }
    reinterpret_cast<u32x4 *>(p)[4 * FROM] = w;
}
__device__ __forceinline__ void store16(float *p, const float (&x)[16], int q) {
    p += 4 * q - 16 * q;
    store_run<0>(p, x, q);
    store_run<1>(p, x, q);
    store_run<2>(p, x, q);
    store_run<3>(p, x, q);
}
// The values are bf16 values (or lose bits below bf16's smallest subnormal
// only), so the conversion does not round.
__device__ __forceinline__ void store16(uint16_t *p, const float (&x)[16], int q) {
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        bf16x2 v;
        v[0] = static_cast<__bf16>(x[2 * j]);
        v[1] = static_cast<__bf16>(x[2 * j + 1]);
        w[j] = as_u32(v);
    }
    u32x4 lo, hi;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t a = of_four<0x50>(w[j]), b = of_four<0x50>(w[4 + j]);     // lanes 0 0 1 1
        const uint32_t c = of_four<0xFA>(w[j]), d = of_four<0xFA>(w[4 + j]);     // lanes 2 2 3 3
        lo[j] = q & 1 ? b : a;
        hi[j] = q & 1 ? d : c;
    }
    p += 8 * q - 16 * q;
    reinterpret_cast<u32x4 *>(p)[0] = lo;
    reinterpret_cast<u32x4 *>(p)[4] = hi;
}

// Exponent E of a block's scale from the bits of its largest magnitude.
template <int BITS>
__device__ __forceinline__ int block_exponent(uint32_t amax_bits) {
    const float a = __uint_as_float(amax_bits);
    if (amax_bits == 0u) return -127;
    const int e = __builtin_amdgcn_frexp_expf(a);       // a in [2^(e-1), 2^e)
    const int E = BITS == 4 ? e - 3 : e - (__builtin_amdgcn_frexp_mantf(a) <= 0.875f ? 9 : 8);
    return max(E, -127);                                // at most 125
}

// Quantise 16 elements with unit 2^E (bad: store zeros): 16 bytes for BITS = 8,
// 8 for BITS = 4, in element order.  x * 2^-E is exact wherever it matters (it
// underflows only far below half the smallest code) and the conversions round
// to nearest even.
template <int BITS>
__device__ __forceinline__ void quantise16(const float (&x)[16], int E, bool bad, uint32_t (&w)[BITS / 2]) {
#pragma unroll
    for (int i = 0; i < BITS / 2; ++i) {
        uint32_t c = 0;
        if constexpr (BITS == 8) {
            float y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = __builtin_amdgcn_ldexpf(x[4 * i + j], -E);
            c = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], int(c), false);
            c = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], int(c), true);
        } else {
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = __builtin_amdgcn_ldexpf(x[8 * i + j], -E);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[0], y[1], 1.0f, 0);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[2], y[3], 1.0f, 1);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[4], y[5], 1.0f, 2);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[6], y[7], 1.0f, 3);
        }
        w[i] = bad ? 0u : c;
    }
}

template <int BYTES>
struct BytesT;
template <> struct BytesT<2> { typedef uint16_t type; };
template <> struct BytesT<4> { typedef uint32_t type; };
template <> struct BytesT<8> { typedef u32x2 type; };
template <> struct BytesT<16> { typedef u32x4 type; };

// Copy the NW words of 16 elements between registers and the places of a unit
// that hold them: runs of RUN bytes, `at(byte)` giving a run's offset.
template <int RUN, bool LOAD, int NW, class At>
__device__ __forceinline__ void move16(uint8_t *unit, uint32_t (&w)[NW], At at) {
    typedef typename BytesT<RUN>::type T;
#pragma unroll
    for (int k = 0; k < NW * 4 / RUN; ++k) {
        T *p = reinterpret_cast<T *>(unit + at(k * RUN));
        if constexpr (RUN == 2) {
            if (LOAD) w[k / 2] |= uint32_t(*p) << (16 * (k & 1));
            else *p = T(w[k / 2] >> (16 * (k & 1)));
        } else {
            constexpr int N = RUN / 4;
            if constexpr (LOAD) {
                const T t = *p;
                if constexpr (N == 1) w[k] = t;
                else
#pragma unroll
                    for (int i = 0; i < N; ++i) w[N * k + i] = t[i];
            } else {
                if constexpr (N == 1) *p = w[k];
                else {
                    T t;
#pragma unroll
                    for (int i = 0; i < N; ++i) t[i] = w[N * k + i];
                    *p = t;
                }
            }
        }
    }
}

// Moves the codes of elements 16 part .. of token r of a unit.
template <int D, int BITS, int SIDE, bool LOAD>
__device__ __forceinline__ void move_codes(uint8_t *unit, int r, int part, uint32_t (&w)[BITS / 2]) {
    typedef KvSide<D, BITS> S;
    const int first = part * 2 * BITS;
    if constexpr (SIDE == 0) {
        constexpr int run = S::kPiece < 2 * BITS ? S::kPiece : 2 * BITS;
        move16<run, LOAD>(unit, w, [&](int b) { return S::key_code(r, first + b); });
    } else {
        move16<S::kPart, LOAD>(unit, w, [&](int b) { return S::value_code(r, first + b); });
    }
}

// The places in the cache of a thread's N token rows t0, t0 + 1, ...
template <int N>
struct KvPlaces {
    int64_t unit[N];
    int r[N];              // the token of the unit
    bool in[N], ok[N];     // whether the row is one of the batch's, and has a page
};
template <int N>
__device__ __forceinline__ KvPlaces<N> kv_places(const KvView &v, int t0, int head) {
    // the wave's first token finds its sequence together; a later lane's is a
    // few sequences on at most
    int s = wave_count_le(v.seqs, __builtin_amdgcn_readfirstlane(t0), [&](int i) { return v.offsets[i]; }) - 1;
    s = max(s, 0);
    int begin = 0, end = 0, before = 0, seq[N], pos[N], entry[N];
    KvPlaces<N> p;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int t = t0 + i;
        if (i == 0 || t >= end) {
            while (s + 1 < v.seqs && v.offsets[s + 1] <= t) ++s;
            v.sequence(s, begin, end, before);
        }
        seq[i] = s;
        pos[i] = before + (t - begin);
        p.in[i] = t >= begin && t < end;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) entry[i] = v.entry_at(seq[i], pos[i]);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int page = p.in[i] ? v.page_in(entry[i], pos[i]) : -1;
        p.ok[i] = page >= 0;
        p.unit[i] = v.unit_of(max(page, 0), head, max(pos[i], 0));
        p.r[i] = pos[i] & (kKvUnit - 1);
    }
    return p;
}

// What a thread of append and read takes: 16 elements of a head of N tokens in a row.
template <int N, int D>
struct KvThread {
    int t0, head, part;
    bool in;
    __device__ __forceinline__ KvThread(const KvView &v) {
        constexpr int kParts = D / 16;
        const int64_t u = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
        const int64_t rows = int64_t((v.tokens + N - 1) / N) * v.heads;
        in = u < rows * kParts;
        const int row = int(in ? u / kParts : rows - 1);
        part = int(u % kParts);
        const int group = row / v.heads;
        head = row - group * v.heads;
        t0 = group * N;
    }
};

// One thread takes 16 elements of a head of a token; two neighbours share a block.
// Bound by bytes (2 or 4 read and 1 or 1/2 written per element) for a chunk of tokens,
// and by the launch for a few.  Measured: 2048 tokens of 8 heads of 128 from float32 to
// 4 bits 7 us, 64 tokens 3.4 us.
template <int D, int BITS, int SIDE, class T>
__device__ __forceinline__ void append16(const KvView &v, const KvPlaces<1> &p, const T *src, int part) {
    typedef KvSide<D, BITS> S;
    float x[16];
    if (p.in[0]) load16(src, x);
    uint32_t amax = 0;
#pragma unroll
    for (int e = 0; e < 16; ++e) amax = max(amax, __float_as_uint(x[e]) & 0x7FFFFFFFu);
    amax = max(amax, uint32_t(__builtin_amdgcn_update_dpp(0, int(amax), 0xB1, 0xF, 0xF, false)));   // the neighbour's
    if (!p.ok[0]) return;
    const bool bad = amax >= 0x7F800000u;
    const int E = block_exponent<BITS>(bad ? 0u : amax);
    uint32_t w[BITS / 2];
    quantise16<BITS>(x, E, bad, w);
    const int64_t unit = p.unit[0];
    move_codes<D, BITS, SIDE, false>(v.codes[SIDE] + unit * S::kUnitCodes, p.r[0], part, w);
    if ((part & 1) == 0) {
        const int at = SIDE == 0 ? S::key_scale(p.r[0], part / 2) : S::value_scale(p.r[0], part / 2);
        v.scales[SIDE][unit * S::kUnitScales + at] = uint8_t(bad ? 0xFF : E + 127);
    }
}

template <int D, class T>
__global__ void __launch_bounds__(256) kv_append_kernel(KvView v, int k_bits, int v_bits, const T *__restrict__ k,
                                                        int64_t k_stride, const T *__restrict__ x, int64_t v_stride) {
    const KvThread<1, D> a(v);
    const KvPlaces<1> p = kv_places<1>(v, a.t0, a.head);
    if (!a.in) return;                                   // neighbours return together
    const int side = blockIdx.y;
    const T *src = (side == 0 ? k + a.t0 * k_stride : x + a.t0 * v_stride) + a.head * D + a.part * 16;
    if (side == 0) {
        if (k_bits == 8) append16<D, 8, 0>(v, p, src, a.part);
        else append16<D, 4, 0>(v, p, src, a.part);
    } else {
        if (v_bits == 8) append16<D, 8, 1>(v, p, src, a.part);
        else append16<D, 4, 1>(v, p, src, a.part);
    }
}

// --------------------------------------------------------------------- read

// The same way back, of N tokens that share the search for their places and have their
// loads in flight together: one pass, bound by bytes (65521 tokens of 8 heads of 128 from
// 8 bits 92 us, 4.5 TB/s read and written; a large copy reaches 4.8).  The values are
// exact products of a code and a power of two.
template <int N, int D, int BITS, int SIDE, class T>
__device__ __forceinline__ void read16(const KvView &v, const KvPlaces<N> &p, T *dst, int64_t stride, int part) {
    typedef KvSide<D, BITS> S;
    uint32_t w[N][BITS / 2] = {};
    uint8_t scale[N] = {};
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (!p.ok[i]) continue;
        const int b = part / 2;
        move_codes<D, BITS, SIDE, true>(v.codes[SIDE] + p.unit[i] * S::kUnitCodes, p.r[i], part, w[i]);
        scale[i] = v.scales[SIDE][p.unit[i] * S::kUnitScales + (SIDE == 0 ? S::key_scale(p.r[i], b) : S::value_scale(p.r[i], b))];
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (!p.in[i]) continue;
        float x[16];
        const float unit = e8m0_f32(scale[i]);           // tokens without a page: zeros by their codes
#pragma unroll
        for (int k = 0; k < BITS / 2; ++k) {
            if constexpr (BITS == 8) {
                const float2 lo = e4m3x2_f32(w[i][k], 0), hi = e4m3x2_f32(w[i][k], 1);
                x[4 * k] = lo.x * unit; x[4 * k + 1] = lo.y * unit;
                x[4 * k + 2] = hi.x * unit; x[4 * k + 3] = hi.y * unit;
            } else {
                const bf16x8 c = e2m1x8_bf16(w[i][k]);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[8 * k + j] = float(c[j]) * unit;
            }
        }
        store16(dst + i * stride, x, part & 3);
    }
}

template <int N, int D, class T>
__global__ void __launch_bounds__(256) kv_read_kernel(KvView v, int k_bits, int v_bits, T *__restrict__ k,
                                                      int64_t k_stride, T *__restrict__ x, int64_t v_stride) {
    const int side = blockIdx.y;
    if ((side == 0 ? k : x) == nullptr) return;
    const KvThread<N, D> a(v);
    KvPlaces<N> p = kv_places<N>(v, a.t0, a.head);
    if (!a.in) return;
    const int64_t stride = side == 0 ? k_stride : v_stride;
    T *dst = (side == 0 ? k : x) + a.t0 * stride + a.head * D + a.part * 16;
    if (side == 0) {
        if (k_bits == 8) read16<N, D, 8, 0>(v, p, dst, stride, a.part);
        else read16<N, D, 4, 0>(v, p, dst, stride, a.part);
    } else {
        if (v_bits == 8) read16<N, D, 8, 1>(v, p, dst, stride, a.part);
        else read16<N, D, 4, 1>(v, p, dst, stride, a.part);
    }
}

// Checks of the float side of append and read, and their grid.
static int kv_rows_check(const nvfp4_kv_cache *c, int dtype, const void *p, int64_t stride) {
    if (!p) return NVFP4_OK;
    const int size = dtype == NVFP4_KV_F32 ? 4 : 2;
    const int64_t wide = int64_t(c->heads) * c->head_dim;
    if (stride < wide || stride > (int64_t(1) << 40)) return NVFP4_ESHAPE;
    return aligned(p, 16) && stride * size % 16 == 0 ? NVFP4_OK : NVFP4_EALIGN;
}

// Workgroups along the rows of a launch of N token rows a thread; 0 past the grid's limit.
static unsigned kv_groups(const KvView &v, int n, int dim) {
    const int64_t groups = ceil_div(ceil_div(v.tokens, n) * v.heads * (dim / 16), 256);
    return groups < kMaxGrid / 256 ? unsigned(groups) : 0u;
}

template <int D, class T>
static int kv_launch_append(const KvView &v, int k_bits, int v_bits, const T *k, int64_t k_stride, const T *x,
                            int64_t v_stride, hipStream_t stream) {
    // One token row a thread: two are as good (16384 tokens 64.6 us, two 62.8; 2048
    // tokens 12.6, 13.2).
    const unsigned g = kv_groups(v, 1, D);
    if (g == 0) return NVFP4_ESHAPE;
    kv_append_kernel<D, T><<<dim3(g, 2), 256, 0, stream>>>(v, k_bits, v_bits, k, k_stride, x, v_stride);
    return launch_status();
}

template <int N, int D, class T>
static int kv_launch_read_rows(const KvView &v, int k_bits, int v_bits, T *k, int64_t k_stride, T *x, int64_t v_stride,
                               hipStream_t stream) {
    const unsigned g = kv_groups(v, N, D);
    if (g == 0) return NVFP4_ESHAPE;
    kv_read_kernel<N, D, T><<<dim3(g, 2), 256, 0, stream>>>(v, k_bits, v_bits, k, k_stride, x, v_stride);
    return launch_status();
}

template <int D, class T>
static int kv_launch_read(const KvView &v, int k_bits, int v_bits, T *k, int64_t k_stride, T *x, int64_t v_stride,
                          hipStream_t stream) {
    // Two token rows a thread where the card is full all the same (65521 tokens: 91.7
    // us, one row 95.2, four 91.5; 1500 tokens of 4 heads of 256: 9.3, 9.9, 10.0).
    constexpr int64_t kFill = 1 << 17;
    if (int64_t(v.tokens) * v.heads * (D / 16) >= kFill)
        return kv_launch_read_rows<2, D, T>(v, k_bits, v_bits, k, k_stride, x, v_stride, stream);
    return kv_launch_read_rows<1, D, T>(v, k_bits, v_bits, k, k_stride, x, v_stride, stream);
}

template <bool APPEND, int D, class T>
static int kv_launch(const nvfp4_kv_cache *c, const KvView &v, void *k, int64_t k_stride, void *x, int64_t v_stride,
                     hipStream_t stream) {
    const int kb = c->k_format == NVFP4_KV_MXFP8 ? 8 : 4, vb = c->v_format == NVFP4_KV_MXFP8 ? 8 : 4;
    T *const ks = static_cast<T *>(k), *const xs = static_cast<T *>(x);
    if constexpr (APPEND) return kv_launch_append<D, T>(v, kb, vb, ks, k_stride, xs, v_stride, stream);
    else return kv_launch_read<D, T>(v, kb, vb, ks, k_stride, xs, v_stride, stream);
}

template <bool APPEND>
static int kv_move(const nvfp4_kv_cache *cache, const nvfp4_kv_batch *batch, int dtype, void *k, int64_t k_stride,
                   void *x, int64_t v_stride, hipStream_t stream) {
    KvView v;
    if (int st = kv_check(cache, batch, v)) return st;
    if (dtype != NVFP4_KV_BF16 && dtype != NVFP4_KV_F32) return NVFP4_EINVAL;
    if (batch->tokens > 0 && (APPEND ? !k || !x : !k && !x)) return NVFP4_EINVAL;
    if (int st = kv_rows_check(cache, dtype, k, k_stride)) return st;
    if (int st = kv_rows_check(cache, dtype, x, v_stride)) return st;
    if (batch->tokens == 0) return NVFP4_OK;
    return kv_dim(cache->head_dim, [&](auto dim) {
        constexpr int D = decltype(dim)::value;
        return dtype == NVFP4_KV_F32 ? kv_launch<APPEND, D, float>(cache, v, k, k_stride, x, v_stride, stream)
                                     : kv_launch<APPEND, D, uint16_t>(cache, v, k, k_stride, x, v_stride, stream);
    });
}

}  // namespace nvfp4

using namespace nvfp4;

NVFP4_API size_t nvfp4_kv_code_bytes(int format, int32_t pages, int32_t page_tokens, int32_t heads,
                                     int32_t head_dim) {
    if (!kv_shape_ok(format, pages, page_tokens, heads, head_dim)) return 0;
    return size_t(pages) * heads * page_tokens * (head_dim * (format == NVFP4_KV_MXFP8 ? 8 : 4) / 8);
}

NVFP4_API size_t nvfp4_kv_scale_bytes(int format, int32_t pages, int32_t page_tokens, int32_t heads,
                                      int32_t head_dim) {
    if (!kv_shape_ok(format, pages, page_tokens, heads, head_dim)) return 0;
    return size_t(pages) * heads * page_tokens * (head_dim / kMxBlock);
}

NVFP4_API int nvfp4_kv_append(const nvfp4_kv_cache *cache, const nvfp4_kv_batch *batch, int dtype, const void *k,
                              int64_t k_stride, const void *v, int64_t v_stride, hipStream_t stream) {
    return kv_move<true>(cache, batch, dtype, const_cast<void *>(k), k_stride, const_cast<void *>(v), v_stride,
                         stream);
}

NVFP4_API int nvfp4_kv_read(const nvfp4_kv_cache *cache, const nvfp4_kv_batch *batch, int dtype, void *k,
                            int64_t k_stride, void *v, int64_t v_stride, hipStream_t stream) {
    return kv_move<false>(cache, batch, dtype, k, k_stride, v, v_stride, stream);
}
