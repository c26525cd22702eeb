// The AdamW step over many tensors at once.
//
// m <- b1 m + (1 - b1) g, v <- b2 v + (1 - b2) g^2, w <- (1 - lr wd) w - lr c1 m /
// (sqrt(c2) sqrt(v) + eps), c1 and c2 the bias corrections; all in fp32.  Bound by HBM:
// each element's weight and states are read and written once, its gradient read once.
// The tensors' addresses travel in the launch's arguments, as many as 4 KB hold, so that
// there is no table to keep on the device and a captured step holds them; a workgroup
// takes 4096 consecutive elements of one tensor, a lane four neighbouring ones at a time
// (whole lines of fp32 per instruction; eight with 8-bit states, a tile of which is then
// one row of 16 lanes), all of them in flight together.  A workgroup whose elements all
// lie inside its tensor runs without their checks.
//
// States in 8 bits are e4m3 codes in tiles of 128 with a power of two each; v is kept as
// its root, whose range is the root of v's: a tile's roots reach from its largest down to
// 2^-18 of it, v's values to 2^-36.  Codes are rounded stochastically: a step moves v by
// about 1 - b2 of itself, far below half a step of the codes, and rounding to nearest
// would leave it where it is for good.  (The roundings spread the roots: a step's adds (1 - b2) / 32
// to / 16 of a root's square to its variance, codes being 1/16 to 1/8 apart, and of the sum about
// 1 / 2 (1 - b2) steps' last: a deviation of 11 to 18 %.)  The random numbers, the codes and the update are
// arithmetic enough to bound this form (12 bytes and 56 vector instructions an element):
// hence one root for the update and the code, square root and reciprocal from the
// hardware's instructions (1 ulp each, against 20 instructions of the exact division),
// and the conversion that rounds by given random bits.  Measured, of 1.46 x 10^9 bf16
// weights without a master, fp32 gradients: 3.2 ms, 5.4 TB/s (4.9 ms with two exact roots,
// an exact division and rounding in integers); 0.81 x 10^9 with masters and fp32 states, 30
// bytes each: 4.3 to 4.5 ms, 5.4 to 5.7 TB/s.
#include "mx.h"

#include <math.h>
#include <type_traits>

namespace moe {

namespace {

constexpr int per_lane(bool s8) { return s8 ? 8 : 4; }  // neighbouring elements
// Elements of a workgroup; one piece a lane in a launch of fewer such chunks than two to a CU,
// so that more CUs have some (93 tensors, 175 chunks: 5.7 us against 7.7; many chunks keep
// four pieces of a lane under way, 5.4 TB/s).
constexpr int kChunk = 4096;
constexpr int64_t kFewChunks = 512;
constexpr int kTile = 128;

// A launch's tensors, F addresses each: w, g, m, v, then the scales of 8-bit states, then
// the master.
constexpr int addresses(bool s8, bool master) { return 4 + 2 * s8 + master; }
constexpr int capacity(int f) { return 3936 / (8 * f + 10); }
template <int F>
struct Table {
    static constexpr int kMax = capacity(F);
    uint64_t p[F][kMax];
    uint32_t first[kMax];  // its first workgroup
    uint32_t index[kMax];  // its place in the call
    uint16_t last[kMax];   // elements of its last workgroup, less one
    int count;
    uint32_t groups;
};
struct Step {
    float lr, b1, b1c, b2, b2c, eps, wd, c1, c2;  // c1, c2: 1 / (1 - b1^step), the root of 1 / (1 - b2^step)
    uint32_t key_seed_lo, key_seed_hi;
    double log2_b1, log2_b2;  // of the betas, for a step on the device
    int64_t step;
    const float *grad_scale;
    const int64_t *step_ptr;
    const float *lr_ptr;
};

// A published 32-bit integer hash (C. Wellons, "Prospecting for hash functions").
__host__ __device__ __forceinline__ uint32_t mix(uint32_t x) {
    x ^= x >> 16;
    x *= 0x7feb352du;
    x ^= x >> 15;
    x *= 0x846ca68bu;
    return x ^ (x >> 16);
}

// E elements of a piece from i on, n of them there (n >= E: all).
template <bool BF16, int E>
__device__ __forceinline__ void load(const void *p, uint32_t i, int n, float (&v)[E]) {
    if (n >= E) {
#pragma unroll
        for (int q = 0; q < E; q += 4) {
            if (BF16) {
                uint2 w;
                __builtin_memcpy(&w, static_cast<const uint16_t *>(p) + i + q, 8);
                v[q] = bf16_to_f32(w.x & 0xffffu);
                v[q + 1] = __uint_as_float(w.x & 0xffff0000u);
                v[q + 2] = bf16_to_f32(w.y & 0xffffu);
                v[q + 3] = __uint_as_float(w.y & 0xffff0000u);
            } else {
                __builtin_memcpy(&v[q], static_cast<const float *>(p) + i + q, 16);
            }
        }
    } else {
#pragma unroll
        for (int k = 0; k < E; ++k)
            v[k] = k >= n ? 0.f : BF16 ? bf16_to_f32(static_cast<const uint16_t *>(p)[i + k]) : static_cast<const float *>(p)[i + k];
    }
}
// E elements as T (a bf16's bits, an fp32).
template <class T, int E>
__device__ __forceinline__ void store(void *p, uint32_t i, int n, const T (&v)[E]) {
    T *const d = static_cast<T *>(p) + i;
    if (n >= E) {
        __builtin_memcpy(d, v, sizeof(v));
    } else {
#pragma unroll
        for (int k = 0; k < E; ++k)
            if (k < n) d[k] = v[k];
    }
}
__device__ __forceinline__ uint2 load_codes8(const void *p, uint32_t i, int n) {
    const uint8_t *const c = static_cast<const uint8_t *>(p) + i;
    uint2 w = {0u, 0u};
    if (n >= 8) {
        __builtin_memcpy(&w, c, 8);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < n) (k < 4 ? w.x : w.y) |= (uint32_t)c[k] << (8 * (k & 3));
    }
    return w;
}
__device__ __forceinline__ void store_codes8(void *p, uint32_t i, int n, uint2 w) {
    uint8_t *const c = static_cast<uint8_t *>(p) + i;
    if (n >= 8) {
        __builtin_memcpy(c, &w, 8);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < n) c[k] = (uint8_t)((k < 4 ? w.x : w.y) >> (8 * (k & 3)));
    }
}

// The root, 1 ulp (the instruction takes a subnormal for 0).
__device__ __forceinline__ float root(float v) {
    const bool tiny = v < 0x1p-96f;
    const float r = __builtin_amdgcn_sqrtf(tiny ? v * 0x1p64f : v);
    return tiny ? r * 0x1p-32f : r;
}

__device__ __forceinline__ void decode8(uint2 w, uint32_t byte, float (&v)[8]) {
    const float s = e8m0_value(byte);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int x = (int)(h ? w.y : w.x);
        const f32x2_hw lo = __builtin_amdgcn_cvt_pk_f32_fp8(x, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(x, true);
        v[4 * h] = lo[0] * s;
        v[4 * h + 1] = lo[1] * s;
        v[4 * h + 2] = hi[0] * s;
        v[4 * h + 3] = hi[1] * s;
    }
}

// Scale byte of the tile that a row of 16 lanes holds, eight values each: the smallest
// power of two at or above the largest magnitude / 448, at least 2^-126; 127 for zeros,
// 255 where a value is not finite.
__device__ __forceinline__ uint32_t tile_byte16(const float (&v)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = max(m, __float_as_uint(v[k]) & 0x7fffffffu);
    m = row_max(m);
    const uint32_t b = (uint32_t)max((int)(m >> 23) - 8 + ((m & 0x7fffffu) > 0x600000u ? 1 : 0), 1);
    return m == 0 ? 127u : m >= 0x7f800000u ? 255u : b;
}

// e4m3 codes, up with the probability of what lies above the code below: sixteen random
// bits (the low ones for m, the high ones for the root) against the dropped bits of the
// mantissa, or, below 2^-6, against the fraction of the multiples of 2^-9 (cut to its
// first sixteen bits): what the conversion does with bits in its operand's upper half.
template <bool ROOT>
__device__ __forceinline__ uint2 encode8(const float (&v)[8], uint32_t byte, const uint32_t (&h)[8]) {
    const float inv = __uint_as_float((254u - byte) << 23);  // (a byte is 247 at most, or 255)
    float a[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        a[k] = v[k] * inv;
        // above 0, but not below the least code
        if (ROOT) a[k] = fmaxf(a[k], fminf(v[k] * 0x1p126f, 0x1p-9f));
    }
    uint2 w = {0u, 0u};
#define CODE(K) __builtin_amdgcn_cvt_sr_fp8_f32(a[K], ROOT ? h[K] & 0xffff0000u : h[K] << 16, (K) < 4 ? w.x : w.y, (K) & 3)
    w.x = CODE(0); w.x = CODE(1); w.x = CODE(2); w.x = CODE(3);
    w.y = CODE(4); w.y = CODE(5); w.y = CODE(6); w.y = CODE(7);
#undef CODE
    return byte == 255u ? uint2{0u, 0u} : w;
}

// bf16 of a weight, up in magnitude with the probability of the dropped bits (an
// infinity stays one, a NaN quiet).
__device__ __forceinline__ uint16_t stochastic_bf16(float w, uint32_t h) {
    const uint32_t more = (h * 0x9E3779B1u) >> 16;
    return (uint16_t)((__float_as_uint(w) + (w == w ? more : 0u)) >> 16);
}

template <bool WBF, bool GBF, bool S8, bool MASTER, int CHUNK>
__global__ __launch_bounds__(256) void k_adamw(Table<addresses(S8, MASTER)> tab, Step st) {
    constexpr int E = per_lane(S8), kPieces = CHUNK / 256 / E;
    constexpr bool SR = WBF && !MASTER;
    float gs = 1.0f;
    if (st.grad_scale) {
        gs = *st.grad_scale;
        if (!(gs - gs == 0.0f)) return;
    }
    // the tensor that this workgroup's elements lie in: the last that begins at or before it
    const int lane = threadIdx.x & 63;
    const int a = lane < tab.count ? lane : 0, b = lane + 64 < tab.count ? lane + 64 : 0;
    const uint32_t fa = tab.first[a], fb = tab.first[b];
    const int t = __popcll(__ballot(lane < tab.count && fa <= blockIdx.x)) + __popcll(__ballot(lane + 64 < tab.count && fb <= blockIdx.x)) - 1;
    const uint32_t chunk = blockIdx.x - tab.first[t], behind = t + 1 < tab.count ? tab.first[t + 1] : tab.groups;
    const int left = blockIdx.x + 1 == behind ? tab.last[t] + 1 : CHUNK;  // elements of this workgroup
    const int64_t base = (int64_t)chunk * CHUNK;

    const float lr = st.lr_ptr ? *st.lr_ptr : st.lr;
    float c1 = st.c1, c2 = st.c2;
    int64_t step = st.step;
    if (st.step_ptr) {
        step = *st.step_ptr;
        c1 = (float)(1.0 / (1.0 - exp2((double)step * st.log2_b1)));
        c2 = (float)sqrt(1.0 / (1.0 - exp2((double)step * st.log2_b2)));
    }
    const float keep = 1.0f - lr * st.wd;
    uint32_t inner = 0;
    if (S8 || SR) {
        const uint32_t key = mix(st.key_seed_lo ^ mix(st.key_seed_hi ^ mix((uint32_t)step ^ mix(tab.index[t]))));
        inner = mix((uint32_t)((uint64_t)base >> 32) + key);
    }
    auto of = [&](int which, int bytes) { return reinterpret_cast<uint8_t *>(tab.p[which][t]) + base * bytes; };
    uint8_t *const pw = of(0, WBF ? 2 : 4), *const pg = of(1, GBF ? 2 : 4), *const pm = of(2, S8 ? 1 : 4), *const pv = of(3, S8 ? 1 : 4);
    uint8_t *const pms = S8 ? reinterpret_cast<uint8_t *>(tab.p[S8 ? 4 : 0][t]) + base / kTile : nullptr;
    uint8_t *const pvs = S8 ? reinterpret_cast<uint8_t *>(tab.p[S8 ? 5 : 0][t]) + base / kTile : nullptr;
    uint8_t *const pf = MASTER ? of(MASTER ? addresses(S8, MASTER) - 1 : 0, 4) : nullptr;

    auto body = [&](auto whole) {
        constexpr bool WHOLE = decltype(whole)::value;
        float w[kPieces][E], g[kPieces][E], m[kPieces][E], v[kPieces][E];
        uint2 mc[kPieces], vc[kPieces];
        uint32_t mb[kPieces], vb[kPieces];
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            const uint32_t i = (uint32_t)E * (256 * p + threadIdx.x);
            const int n = WHOLE ? E : left - (int)i;
            if (MASTER) load<false>(pf, i, n, w[p]);
            else load<WBF>(pw, i, n, w[p]);
            load<GBF>(pg, i, n, g[p]);
            if constexpr (S8) {
                mc[p] = load_codes8(pm, i, n);
                vc[p] = load_codes8(pv, i, n);
                mb[p] = n > 0 ? pms[i / kTile] : 127u;
                vb[p] = n > 0 ? pvs[i / kTile] : 127u;
            } else {
                load<false>(pm, i, n, m[p]);
                load<false>(pv, i, n, v[p]);
            }
        }
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
            const uint32_t i = (uint32_t)E * (256 * p + threadIdx.x);
            const int n = WHOLE ? E : left - (int)i;
            if constexpr (S8) {
                decode8(mc[p], mb[p], m[p]);
                decode8(vc[p], vb[p], v[p]);
            }
#pragma unroll
            for (int k = 0; k < E; ++k) {
                const float gk = g[p][k] * gs;
                const float mk = m[p][k] * st.b1 + gk * st.b1c;
                const float vk = (S8 ? v[p][k] * v[p][k] : v[p][k]) * st.b2 + gk * gk * st.b2c;
                const float r = root(vk);
                w[p][k] = w[p][k] * keep - lr * (mk * c1 * __builtin_amdgcn_rcpf(r * c2 + st.eps));
                m[p][k] = mk;
                v[p][k] = S8 ? r : vk;
            }
            uint32_t h[E];
            if (S8 || SR) {
                const uint32_t at = ((uint32_t)base + i) ^ inner;  // (of a multiple of E)
#pragma unroll
                for (int k = 0; k < E; ++k) h[k] = mix(at ^ (uint32_t)k);
            }
            if constexpr (S8) {
                if (!WHOLE) {  // what lies past the tensor does not count towards its last tile
#pragma unroll
                    for (int k = 0; k < E; ++k)
                        if (k >= n) m[p][k] = v[p][k] = 0.f;
                }
                const uint32_t bm = tile_byte16(m[p]), bv = tile_byte16(v[p]);
                if ((WHOLE || n > 0) && (threadIdx.x & 15) == 0) {
                    pms[i / kTile] = (uint8_t)bm;
                    pvs[i / kTile] = (uint8_t)bv;
                }
                store_codes8(pm, i, n, encode8<false>(m[p], bm, h));
                store_codes8(pv, i, n, encode8<true>(v[p], bv, h));
            } else {
                store<float>(pm, i, n, m[p]);
                store<float>(pv, i, n, v[p]);
            }
            if (MASTER) store<float>(pf, i, n, w[p]);
            if constexpr (WBF) {
                uint16_t o[E];
#pragma unroll
                for (int k = 0; k < E; k += 2) {
                    const uint32_t two = SR ? 0u : pack_bf16x2(w[p][k], w[p][k + 1]);
                    o[k] = SR ? stochastic_bf16(w[p][k], h[k]) : (uint16_t)two;
                    o[k + 1] = SR ? stochastic_bf16(w[p][k + 1], h[k + 1]) : (uint16_t)(two >> 16);
                }
                store<uint16_t>(pw, i, n, o);
            } else {
                store<float>(pw, i, n, w[p]);
            }
        }
    };
    if (left == CHUNK) body(std::true_type{});
    else body(std::false_type{});
}

template <bool WBF, bool GBF, bool S8, bool MASTER>
hipError_t go(const Step &st, const AdamWTensor *tensors, int count, hipStream_t s) {
    constexpr int F = addresses(S8, MASTER);
    static_assert(sizeof(Table<F>) + sizeof(Step) <= 4096, "the launch's arguments");
    static_assert(Table<F>::kMax <= 128, "two to a lane");
    constexpr int kSmall = 256 * per_lane(S8);
    for (int at = 0; at < count;) {
        int64_t chunks = 0;  // of all the tensors that are left: those of one launch, or more
        for (int i = at; i < count && chunks < kFewChunks; ++i) chunks += (tensors[i].n + kChunk - 1) / kChunk;
        const int chunk = chunks < kFewChunks ? kSmall : kChunk;
        Table<F> tab{};
        int64_t groups = 0;
        while (at < count && tab.count < Table<F>::kMax) {
            const AdamWTensor &t = tensors[at];
            const int64_t more = (t.n + chunk - 1) / chunk;
            if (groups + more >= (1LL << 24)) break;
            auto put = [&](int f, const void *p) { tab.p[f][tab.count] = reinterpret_cast<uint64_t>(p); };
            put(0, t.w);
            put(1, t.g);
            put(2, t.m);
            put(3, t.v);
            if (S8) {
                put(S8 ? 4 : 0, t.m_scales);
                put(S8 ? 5 : 0, t.v_scales);
            }
            if (MASTER) put(F - 1, t.master);
            tab.first[tab.count] = (uint32_t)groups;
            tab.index[tab.count] = t.index;
            tab.last[tab.count++] = (uint16_t)(t.n - (more - 1) * chunk - 1);
            groups += more;
            ++at;
        }
        tab.groups = (uint32_t)groups;
        if (chunk == kSmall) hipLaunchKernelGGL((k_adamw<WBF, GBF, S8, MASTER, kSmall>), dim3((uint32_t)groups), dim3(256), 0, s, tab, st);
        else hipLaunchKernelGGL((k_adamw<WBF, GBF, S8, MASTER, kChunk>), dim3((uint32_t)groups), dim3(256), 0, s, tab, st);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}
template <bool WBF, bool GBF>
hipError_t go(const AdamWTypes &ty, const Step &st, const AdamWTensor *tensors, int count, hipStream_t s) {
    if constexpr (WBF) {
        if (ty.master) return ty.states8 ? go<WBF, GBF, true, true>(st, tensors, count, s) : go<WBF, GBF, false, true>(st, tensors, count, s);
    }
    return ty.states8 ? go<WBF, GBF, true, false>(st, tensors, count, s) : go<WBF, GBF, false, false>(st, tensors, count, s);
}

}  // namespace

hipError_t launch_adamw(const AdamWRule &r, const AdamWTypes &ty, const AdamWTensor *tensors, int count, hipStream_t s) {
    // a launch takes fewer than 2^32 threads: 2^24 workgroups; one tensor has at most 2^23
    static_assert(kAdamWMaxN / kChunk <= (1LL << 23), "one tensor fits a launch");
    Step st{};
    st.lr = (float)r.lr;
    st.b1 = (float)r.beta1;
    st.b1c = (float)(1.0 - r.beta1);
    st.b2 = (float)r.beta2;
    st.b2c = (float)(1.0 - r.beta2);
    st.eps = (float)r.eps;
    st.wd = (float)r.weight_decay;
    st.c1 = (float)(1.0 / (1.0 - pow(r.beta1, (double)r.step)));
    st.c2 = (float)sqrt(1.0 / (1.0 - pow(r.beta2, (double)r.step)));
    st.log2_b1 = log2(r.beta1);
    st.log2_b2 = log2(r.beta2);
    st.key_seed_lo = (uint32_t)r.seed;
    st.key_seed_hi = (uint32_t)(r.seed >> 32);
    st.step = r.step;
    st.grad_scale = r.grad_scale;
    st.step_ptr = r.step_ptr;
    st.lr_ptr = r.lr_ptr;
    if (ty.w_bf16) return ty.g_bf16 ? go<true, true>(ty, st, tensors, count, s) : go<true, false>(ty, st, tensors, count, s);
    return ty.g_bf16 ? go<false, true>(ty, st, tensors, count, s) : go<false, false>(ty, st, tensors, count, s);
}

int adamw_tensors(const AdamWTypes &ty) { return capacity(addresses(ty.states8, ty.master)); }

}  // namespace moe
