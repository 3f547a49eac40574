// nvfp4_attn_wide.hip -- attention of many query rows over the paged cache
// (prefill chunks, wide verifies) on gfx950.
//
// A workgroup owns 32 rows per wave and walks the keys in tiles of kKeys = 8192 / D.
// Keys and values are decoded to bf16 once per workgroup, into shared memory and
// as whole operands of v_mfma_f32_32x32x16_bf16: the waves read them with
// conflict-free 16-byte loads, and the cache's byte order makes each thread's share
// of the decode one load and a few stores.  Two buffers: while the waves work on one
// tile, the next one's codes, loaded a tile earlier, are decoded into the other,
// so a tile costs one barrier.
#include <mutex>

#include "nvfp4_attn.h"

namespace nvfp4 {

typedef float floatx16 __attribute__((ext_vector_type(16)));

// The shape at head dimension D: 256 rows in 8 waves, two to a SIMD, whose matrix
// and vector instructions overlap; at D = 256 a row's accumulators and query
// operands take 192 registers of a lane, so 4 waves, one to a SIMD, and 128 rows.
template <int D>
struct WideShape {
    static constexpr int kWaves = D == 256 ? 4 : 8;
    static constexpr int kThreads = kWaves * kLanes;
    static constexpr int kRows = 32 * kWaves;
    static constexpr int kKeys = 8192 / D;             // of a tile
    static constexpr int kUnits = kKeys / kKvUnit;
    static constexpr int kBlocks32 = kKeys / 32;
    static constexpr int kDimSteps = D / 16;           // MFMAs of a 32-key block's scores
    static constexpr int kDimBlocks = D / 32;          // accumulators of the output
    static constexpr int kSide = kKeys * D * 2;        // bytes of a tile's keys (and of its values): 16 KiB
    static constexpr int kMarks = kKeys * (D / kMxBlock);
    static constexpr int kBuffer = 2 * kSide + kMarks;
    static constexpr int kLds = 2 * kBuffer;
};

// One thread's share of a tile between its load and its store to shared memory.
template <int D, int KB, int VB>
struct WideStage {
    typedef WideShape<D> W;
    typedef KvSide<D, KB> KS;
    typedef KvSide<D, VB> VS;
    // keys: 16 elements of one key; values: two keys' (D = 64: four keys')
    // elements of a row, 16 or (D = 256) 32
    static constexpr int kKeyItems = kKvUnit * D / 16;               // of a unit
    static constexpr int kKeyEach = W::kUnits * kKeyItems / W::kThreads;
    static constexpr int kTokens = D == 64 ? 4 : 2;
    static constexpr int kValueItems = kKvUnit / kTokens * 16;
    static constexpr int kValueEach = W::kUnits * kValueItems / W::kThreads;
    static constexpr int kRowDims = D / 16;
    static constexpr int kValueWords = kTokens * kRowDims * VB / 32;
    static_assert(kValueEach == 1, "one value item per thread");

    uint32_t k[kKeyEach][KB / 2], ks[kKeyEach];
    uint32_t v[kValueWords], vs;

    // The place of a key item: unit, token, and which 16 elements.
    static __device__ __forceinline__ void key_item(int e, int &unit, int &r, int &part) {
        unit = e / kKeyItems;
        const int i = e % kKeyItems;
        if (KB == 4 && KS::kPiece == 16) {          // two items of a piece side by side
            r = (i >> 1) & 15;
            part = (i >> 5) * 2 + (i & 1);
        } else {
            r = i & 15;
            part = i >> 4;
        }
    }
    // The place of a value item: unit, quad (half + 2 * upper), which tokens, row.
    static __device__ __forceinline__ void value_item(int e, int &unit, int &quad, int &pair, int &r) {
        unit = e / kValueItems;
        const int i = e % kValueItems;
        r = i & 15;
        if (D == 64) {
            quad = i >> 4;
            pair = 0;
        } else {
            quad = ((i >> 4) & 1) * 2 + (i >> 6);
            pair = (i >> 5) & 1;
        }
    }

    // `pages`: lane u holds the page of the tile's unit u (or -1).
    __device__ __forceinline__ void load(const KvView &kv, int pages, int head, int key) {
        const int tid = threadIdx.x;
#pragma unroll
        for (int n = 0; n < kKeyEach; ++n) {
            int unit, r, part;
            key_item(n * W::kThreads + tid, unit, r, part);
            unit = __builtin_amdgcn_readfirstlane(unit);
            const int page = max(__builtin_amdgcn_readlane(pages, unit), 0);
            const int64_t u = kv.unit_of(page, head, key + unit * kKvUnit);
            load_words<2 * KB>(kv.codes[0] + u * KS::kUnitCodes + KS::key_code(r, part * 2 * KB), k[n]);
            ks[n] = kv.scales[0][u * KS::kUnitScales + KS::key_scale(r, part / 2)];
        }
        int unit, quad, pair, r;
        value_item(tid, unit, quad, pair, r);
        unit = __builtin_amdgcn_readfirstlane(unit);
        const int page = max(__builtin_amdgcn_readlane(pages, unit), 0);
        const int64_t u = kv.unit_of(page, head, key + unit * kKvUnit);
        const uint8_t *base = kv.codes[1] + u * VS::kUnitCodes;
        const int t0 = quad * 4 + pair * 2;
        constexpr int kRun = VS::kSlotTokens < kTokens ? VS::kPart : kValueWords * 4;   // contiguous bytes
#pragma unroll
        for (int n = 0; n < kValueWords * 4 / kRun; ++n)
            load_words<kRun>(base + VS::value_code(t0 + n * VS::kSlotTokens, r * VS::kPart), v + n * kRun / 4);
        load_words<kTokens>(kv.scales[1] + u * VS::kUnitScales + VS::value_scale(t0, r * VS::kBlocks / 16), &vs);
    }

    // Decode to the operands in `lds`.  EDGE: values of keys outside lo..hi - 1 or
    // without a page, and NaN blocks, become zeros, the latter marked.
    template <bool EDGE>
    __device__ __forceinline__ void store(uint8_t *lds, int key, int lo, int hi, unsigned some) const {
        const int tid = threadIdx.x;
#pragma unroll
        for (int n = 0; n < kKeyEach; ++n) {
            int unit, r, part;
            key_item(n * W::kThreads + tid, unit, r, part);
            const float scale = __uint_as_float(ks[n] << 23);
            const int row = (unit & 1) * 16 + r;
            bf16x8 *dst = reinterpret_cast<bf16x8 *>(lds) + ((unit >> 1) * W::kDimSteps + part) * kLanes + row;
            if constexpr (KB == 8) {
                dst[0] = codes8(k[n][0], k[n][1], scale);
                dst[32] = codes8(k[n][2], k[n][3], scale);
            } else {
                dst[0] = codes4(k[n][0], scale);
                dst[32] = codes4(k[n][1], scale);
            }
        }
        int unit, quad, pair, r;
        value_item(tid, unit, quad, pair, r);
        uint32_t keep[kTokens];
        if constexpr (EDGE) {
            uint8_t *marks = lds + 2 * W::kSide;
#pragma unroll
            for (int i = 0; i < kTokens; ++i) {
                const int token = quad * 4 + pair * 2 + i, pos = key + unit * kKvUnit + token;
                const bool held = ((some >> unit) & 1) && pos >= lo && pos < hi;
                const bool nan = ((vs >> (8 * i)) & 0xFFu) == 0xFFu;
                keep[i] = held && !nan ? ~0u : 0u;
                marks[(unit * kKvUnit + token) * VS::kBlocks + r * VS::kBlocks / 16] = held && nan ? 1 : 0;
            }
        }
        // operand (unit, dim block, half, row): eight keys, the quad's four at
        // 8 * (quad / 2) bytes
        uint8_t *dst = lds + W::kSide + (unit * W::kDimBlocks * kLanes + (quad & 1) * 32 + r) * 16 + (quad >> 1) * 8 + pair * 4;
#pragma unroll
        for (int jp = 0; jp < kRowDims / 2; ++jp) {
            uint32_t w[kTokens];
#pragma unroll
            for (int i = 0; i < kTokens; ++i) {
                w[i] = value_pair<D, VB>(v, i, jp, unit_of_byte(vs, i));
                if constexpr (EDGE) w[i] &= keep[i];
            }
            uint8_t *at = dst + jp * kLanes * 16;
            if constexpr (kTokens == 4) {
                *reinterpret_cast<u32x2 *>(at) = u32x2{low_halves(w[0], w[1]), low_halves(w[2], w[3])};
                *reinterpret_cast<u32x2 *>(at + 16 * 16) = u32x2{high_halves(w[0], w[1]), high_halves(w[2], w[3])};
            } else {
                *reinterpret_cast<uint32_t *>(at) = low_halves(w[0], w[1]);
                *reinterpret_cast<uint32_t *>(at + 16 * 16) = high_halves(w[0], w[1]);
            }
        }
    }
};

// The pages of the tile at `key`: lane u (u < units) that of its unit u.
template <int D>
__device__ __forceinline__ int wide_pages(const KvView &kv, int s, int key, int end) {
    const int u = threadIdx.x & 63, pos = key + u * kKvUnit;
    return u < WideShape<D>::kUnits && pos < end ? kv.page_of(s, pos) : -1;
}

template <int D, int KB, int VB>
__global__ void __launch_bounds__(WideShape<D>::kThreads) attn_wide_kernel(AttnArgs a) {
    typedef WideShape<D> W;
    extern __shared__ __align__(16) uint8_t lds[];
    const int lane = threadIdx.x & 63, h = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // heads first: the tiles of a head, which read the same keys, meet in few
    // XCDs' caches; a sequence's last tiles, which have the most keys, go first
    const int item = int(gridDim.x / a.kv.heads) - 1 - int(blockIdx.x / a.kv.heads);
    const RowTile tile = row_tile(a, item, W::kRows);
    if (!tile.some || a.narrow_rows >= tile.rows) return;
    const int head = blockIdx.x % a.kv.heads, z = blockIdx.y;
    const KeyRange keys = key_range(a.split[1], tile, z);
    if (z > 0 && z >= keys.splits) return;

    const int row = tile.row0 + wave * 32 + (lane & 31);
    const bool in = row < tile.rows;
    const int i = in ? row / a.group : 0;
    const int token = tile.begin + i, qhead = head * a.group + (in ? row - i * a.group : 0);
    const int pos = tile.past + i;
    const int klo = a.window > 0 ? max(0, pos + 1 - a.window) : 0;
    const int khi = in ? (a.tree ? tile.past : pos + 1) : 0;
    const unsigned long long tree = in && a.tree ? a.tree[token] : 0ull;
    bf16x8 q[W::kDimSteps];
    {
        const uint16_t *src = a.q + token * a.q_stride + qhead * D + 8 * h;
#pragma unroll
        for (int m = 0; m < W::kDimSteps; ++m) {
            u32x4 w = {0, 0, 0, 0};
            if (in) w = *reinterpret_cast<const u32x4 *>(src + 16 * m);
            q[m] = __builtin_bit_cast(bf16x8, w);
        }
    }
    floatx16 o[W::kDimBlocks];
#pragma unroll
    for (int d = 0; d < W::kDimBlocks; ++d) o[d] = floatx16{};
    float mx = kNegInf, sub = 0.0f, l = 0.0f, lr = 0.0f;
    const float scale = a.scale_log2;

    const auto work = [&](const uint8_t *buf, int key, unsigned some, auto edge_tag) {
        constexpr bool EDGE = decltype(edge_tag)::value != 0;
        const bf16x8 *kop = reinterpret_cast<const bf16x8 *>(buf) + lane;
        const bf16x8 *vop = reinterpret_cast<const bf16x8 *>(buf + W::kSide) + lane;
        floatx16 s[W::kBlocks32];
        float top = kNegInf;
#pragma unroll
        for (int b = 0; b < W::kBlocks32; ++b) {
            s[b] = floatx16{};
#pragma unroll
            for (int m = 0; m < W::kDimSteps; ++m)
                s[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kop[(b * W::kDimSteps + m) * kLanes], q[m], s[b], 0, 0, 0);
        }
        unsigned ones[W::kBlocks32];          // EDGE: bit e where score e of the block is allowed
#pragma unroll
        for (int b = 0; b < W::kBlocks32; ++b) {
            if constexpr (EDGE) {
                ones[b] = 0;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int at = key + b * 32 + 8 * (e >> 2) + 4 * h + (e & 3);
                    bool ok = at >= klo && at < khi;
                    if (a.tree) {
                        const int t = at - tile.past;
                        ok = ok || (t >= 0 && t < tile.n && t < 64 && ((tree >> (t & 63)) & 1));
                    }
                    ok = ok && ((some >> (2 * b + (e >> 3))) & 1) && at < tile.hi;
                    if (!ok) s[b][e] = kNegInf;
                    ones[b] |= ok ? 1u << e : 0u;
                }
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) top = fmaxf(top, s[b][e]);
        }
        top *= scale;
        if (__any(top > mx + kMaxSlack)) {
            top = fmaxf(top, __shfl_xor(top, 32));
            const float m = fmaxf(mx, top);
            const float by = m == mx ? 1.0f : exp2_fast(mx - m);
            mx = m;
            sub = m == kNegInf ? 0.0f : m;
            l *= by;
            lr *= by;
#pragma unroll
            for (int d = 0; d < W::kDimBlocks; ++d) o[d] *= by;
        }
#pragma unroll
        for (int b = 0; b < W::kBlocks32; ++b) {
            uint32_t p[8];
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
                const float x = exp2_fast(__builtin_fmaf(s[b][e], scale, -sub));
                const float y = exp2_fast(__builtin_fmaf(s[b][e + 1], scale, -sub));
                l += x;
                l += y;
                p[e / 2] = pack_bf16(x, y);
                lr = add_pair(p[e / 2], lr);
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const bf16x8 pb = __builtin_bit_cast(bf16x8, u32x4{p[4 * u], p[4 * u + 1], p[4 * u + 2], p[4 * u + 3]});
#pragma unroll
                for (int d = 0; d < W::kDimBlocks; ++d)
                    o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vop[((2 * b + u) * W::kDimBlocks + d) * kLanes], pb, o[d], 0, 0, 0);
            }
        }
        if constexpr (EDGE) {
            // NaN blocks, left out of the product above, reach the rows that see
            // their keys: the product of the marks with the allowed keys tells
            const uint8_t *marks = buf + 2 * W::kSide;
            const uint32_t word = *reinterpret_cast<const uint32_t *>(marks + 4 * lane);      // kMarks is 256
            if (__any(word != 0)) {
                const int block = (lane & 15) * (D / kMxBlock) / 16;
#pragma unroll
                for (int u = 0; u < W::kUnits; ++u) {
                    u32x4 mark, on;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t two = 0, two1 = 0;
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int slot = 2 * e + k, t = 8 * (slot >> 2) + 4 * h + (slot & 3);
                            two |= (marks[(u * kKvUnit + t) * (D / kMxBlock) + block] ? 0x3F80u : 0u) << (16 * k);
                            two1 |= ((ones[u >> 1] >> (8 * (u & 1) + slot)) & 1 ? 0x3F80u : 0u) << (16 * k);
                        }
                        mark[e] = two;
                        on[e] = two1;
                    }
                    const floatx16 n = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, mark), __builtin_bit_cast(bf16x8, on), floatx16{}, 0, 0, 0);
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (n[e] > 0.0f)
#pragma unroll
                            for (int d = 0; d < W::kDimBlocks; ++d) o[d][e] = __builtin_nanf("");
                }
            }
        }
    };

    // The walk.  Of tile t: its page numbers are loaded at t - 3, its codes at
    // t - 2, decoded at t - 1.
    static_assert(W::kMarks == 256, "a word of marks per lane");
    const unsigned all = (1u << W::kUnits) - 1;
    const auto valid = [&](int pages) { return unsigned(__ballot(pages >= 0)) & all; };
    const auto is_edge = [&](int key, unsigned some) {
        return key < tile.inner_lo || key + W::kKeys > min(tile.inner_hi, keys.hi) || some != all;
    };
    WideStage<D, KB, VB> stage;
    if (keys.lo < keys.hi) {
        int key = keys.lo;
        int pages = wide_pages<D>(a.kv, tile.s, key, keys.hi);
        stage.load(a.kv, pages, head, key);
        unsigned some = valid(pages), some1;
        pages = wide_pages<D>(a.kv, tile.s, key + W::kKeys, keys.hi);
        if (is_edge(key, some)) stage.template store<true>(lds, key, tile.lo, tile.hi, some);
        else stage.template store<false>(lds, key, tile.lo, tile.hi, some);
        stage.load(a.kv, pages, head, key + W::kKeys);
        some1 = valid(pages);
        pages = wide_pages<D>(a.kv, tile.s, key + 2 * W::kKeys, keys.hi);
        __syncthreads();
        for (int buf = 0;; buf ^= 1) {
            const int next = key + W::kKeys;
            uint8_t *const other = lds + (buf ^ 1) * W::kBuffer;
            if (next < keys.hi) {
                if (is_edge(next, some1)) stage.template store<true>(other, next, tile.lo, tile.hi, some1);
                else stage.template store<false>(other, next, tile.lo, tile.hi, some1);
                stage.load(a.kv, pages, head, next + W::kKeys);
            }
            const unsigned some2 = valid(pages);
            pages = wide_pages<D>(a.kv, tile.s, next + 2 * W::kKeys, keys.hi);
            if (is_edge(key, some)) work(lds + buf * W::kBuffer, key, some, IntC<1>());
            else work(lds + buf * W::kBuffer, key, some, IntC<0>());
            key = next;
            if (key >= keys.hi) break;
            some = some1;
            some1 = some2;
            __syncthreads();
        }
    }

    l += __shfl_xor(l, 32);
    lr += __shfl_xor(lr, 32);
    if (!in) return;
    const int64_t at = int64_t(token) * a.q_heads + qhead;
    // lane (h, row) holds value rows r = 8 x + 4 h + y, each D / 16 elements in
    // a row: element 2 d + jj of it in o[d][8 jj + 4 x + y]
    constexpr int kRowDims = D / 16;
    if (keys.splits > 1) {
        float *dst = a.part_o + (int64_t(z) * a.kv.tokens * a.q_heads + at) * D;
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y)
#pragma unroll
                for (int j = 0; j < kRowDims; j += 4) {
                    const int e = 4 * x + y;
                    *reinterpret_cast<float4 *>(dst + (8 * x + 4 * h + y) * kRowDims + j) =
                        float4{o[j / 2][e], o[j / 2][8 + e], o[j / 2 + 1][e], o[j / 2 + 1][8 + e]};
                }
        if (h == 0) *reinterpret_cast<float4 *>(a.part_ml + (int64_t(z) * a.kv.tokens * a.q_heads + at) * 4) = float4{mx, l, lr, 0.0f};
        return;
    }
    const float inv = mx == kNegInf && l == 0.0f ? 0.0f : 1.0f / lr;
    uint16_t *dst = a.out + token * a.out_stride + qhead * D;
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y)
#pragma unroll
            for (int j = 0; j < kRowDims; j += 4) {
                const int e = 4 * x + y;
                *reinterpret_cast<u32x2 *>(dst + (8 * x + 4 * h + y) * kRowDims + j) =
                    u32x2{pack_bf16(o[j / 2][e] * inv, o[j / 2][8 + e] * inv), pack_bf16(o[j / 2 + 1][e] * inv, o[j / 2 + 1][8 + e] * inv)};
            }
    if (a.lse && h == 0) a.lse[at] = lse_of(mx, l);
}

// The kernels' shared memory passes the default limit; it is raised once per
// device and kernel.
template <int D, int K, int V>
static bool wide_lds_ok() {
    constexpr int kDevices = 64;
    static std::once_flag once[kDevices];
    static bool ok[kDevices];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kDevices) return false;
    std::call_once(once[dev], [&] {
        ok[dev] = hipFuncSetAttribute(reinterpret_cast<const void *>(attn_wide_kernel<D, K, V>),
                                      hipFuncAttributeMaxDynamicSharedMemorySize, WideShape<D>::kLds) == hipSuccess;
    });
    return ok[dev];
}

int wide_rows(int dim) { return kv_dim(dim, [](auto d) { return WideShape<decltype(d)::value>::kRows; }); }

int launch_attn_wide(const AttnArgs &a, int dim, int k_format, int v_format, hipStream_t stream) {
    return kv_dim(dim, [&](auto d) {
        return kv_bits(k_format, [&](auto k) {
            return kv_bits(v_format, [&](auto v) {
                constexpr int D = decltype(d)::value, K = decltype(k)::value, V = decltype(v)::value;
                typedef WideShape<D> W;
                const int64_t groups = tile_items(a.kv.tokens, a.group, a.kv.seqs, W::kRows) * a.kv.heads;
                if (groups >= kMaxGrid / W::kThreads) return NVFP4_ESHAPE;
                if (!wide_lds_ok<D, K, V>()) return NVFP4_EHIP;
                attn_wide_kernel<D, K, V><<<dim3(unsigned(groups), unsigned(a.split[1].splits)), W::kThreads, W::kLds,
                                            stream>>>(a);
                return launch_status();
            });
        });
    });
}

}  // namespace nvfp4
