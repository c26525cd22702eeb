// Expert choice from router logits, its gradient, and the sequence-wise balance
// loss.
//
//   scores   s = sigmoid(l) or softmax(l) over the row
//   choice   a = s + bias (the bias steers the choice only); the experts are
//            cut into groups, the best groups by max or top-two sum of a stay
//            open, the k largest a inside them are chosen; ties to the lower id
//   weights  scale * s_j, over the chosen scores' sum when renormalised
// The choice is that of 64-bit scores: it decides whole numbers, and an fp32
// score's rounding would decide them differently from one exp to the next.
// Without a bias the order of the scores is the order of the logits, so the
// logits themselves are compared and nothing is rounded.
//
// k_select (one wave per token, lane l holds the experts l, l + 64, ...) computes
// every score in 64 bits.  k_select_fast (16 lanes per token) chooses by fp32
// scores, whose error it knows, and hands a token to the 64-bit code where the
// border between chosen and not, of experts or of groups, is nearer than that.
#include "device.h"
#include "kernels.h"

namespace moe {

namespace {

// Totally ordered key of a double (larger value -> larger key); 1 for a NaN,
// which ranks below every number, and never 0, which marks an expert that
// cannot be chosen.  -0 and +0 get the same key.
__device__ __forceinline__ uint64_t f64_order_key(double v) {
    if (v != v) return 1;
    const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);
    return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
__device__ __forceinline__ double f64_from_order_key(uint64_t k) {
    return __longlong_as_double((long long)((k >> 63) ? (k & 0x7fffffffffffffffull) : ~k));
}

__device__ __forceinline__ float wave_sum_f32(float v) {
#pragma unroll
    for (int s = 32; s >= 1; s >>= 1) v += __shfl_xor(v, s, kWave);
    return v;
}
__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
    for (int s = 32; s >= 1; s >>= 1) v += __shfl_xor(v, s, kWave);
    return v;
}

// Orders a wave's own LDS stores before its lanes' loads of each other's values.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

template <bool BF16>
__device__ __forceinline__ float load_logit(const void *row, int e) {
    return BF16 ? bf16_to_f32(static_cast<const uint16_t *>(row)[e]) : static_cast<const float *>(row)[e];
}

__device__ __forceinline__ float sigmoid_f32(float l) { return 1.0f / (1.0f + expf(-l)); }

// e^(l - m) of a softmax whose maximum is m; a row of -inf has no mass at all.
__device__ __forceinline__ float softmax_term(float l, float m) { return m == -INFINITY ? 0.f : expf(l - m); }

// The n largest of the keys of a wave (key[q] of lane l: item l + 64 q; 0 = no
// item), as a bit mask over q in each lane; equal keys go to the lower item.
template <int Q>
__device__ __forceinline__ uint32_t wave_top(uint64_t (&key)[Q], int n) {
    const int lane = threadIdx.x & 63;
    uint32_t chosen = 0;
    for (int r = 0; r < n; ++r) {
        uint64_t m = key[0];
#pragma unroll
        for (int q = 1; q < Q; ++q) m = key[q] > m ? key[q] : m;
        m = wave_max_u64(m);
        bool open = m != 0;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const uint64_t at = __ballot(key[q] == m);
            if (open && at != 0) {
                open = false;
                if (lane == __ffsll((unsigned long long)at) - 1) {
                    chosen |= 1u << q;
                    key[q] = 0;
                }
            }
        }
    }
    return chosen;
}

// The choice for one token in 64 bits: the chosen experts as a bit mask over q
// in each lane (expert lane + 64 q).  score64: this wave's E doubles in LDS,
// open: its group flags.
template <int Q>
__device__ __forceinline__ uint32_t choose64(const SelectRule &r, const float (&l)[Q], const float *__restrict__ bias,
                                             double *score64, uint8_t *open) {
    const int lane = threadIdx.x & 63;
    double s[Q];
    if (r.softmax) {
        float m = -INFINITY;
#pragma unroll
        for (int q = 0; q < Q; ++q) m = fmaxf(m, l[q]);
        m = wave_max_f32(m, kWave);
        double sum = 0.0;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            s[q] = lane + 64 * q < r.E && m != -INFINITY ? exp((double)l[q] - (double)m) : 0.0;
            sum += s[q];
        }
        sum = wave_sum_f64(sum);
#pragma unroll
        for (int q = 0; q < Q; ++q) s[q] = m == -INFINITY ? 0.0 : s[q] / sum;
    } else {
#pragma unroll
        for (int q = 0; q < Q; ++q) s[q] = 1.0 / (1.0 + exp(-(double)l[q]));
    }
    uint64_t key[Q];
    double a[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int e = lane + 64 * q;
        a[q] = bias && e < r.E ? s[q] + (double)bias[e] : s[q];
        key[q] = e < r.E ? f64_order_key(bias ? a[q] : (double)l[q]) : 0;
    }
    if (r.topk_group < r.n_group) {
        const int per = r.E / r.n_group;
        // without a bias, the best of a group is that of its logits
        const bool by_logit = !bias && !r.top_two;
#pragma unroll
        for (int q = 0; q < Q; ++q)
            if (lane + 64 * q < r.E) score64[lane + 64 * q] = by_logit ? (double)l[q] : a[q];
        wave_sync();
        uint64_t gkey[Q];
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int g = lane + 64 * q;
            gkey[q] = 0;
            if (g >= r.n_group) continue;
            uint64_t k1 = 0, k2 = 0;
            for (int i = 0; i < per; ++i) {
                const uint64_t k = f64_order_key(score64[g * per + i]);
                k2 = k > k1 ? k1 : (k > k2 ? k : k2);
                k1 = k > k1 ? k : k1;
            }
            if (r.top_two && k1 > 1 && k2 > 1)
                k1 = f64_order_key(f64_from_order_key(k1) + f64_from_order_key(k2));
            else if (r.top_two && per > 1)
                k1 = 1;  // fewer than two numbers: behind every group that has two
            gkey[q] = k1;
        }
        const uint32_t go = wave_top<Q>(gkey, r.topk_group);
#pragma unroll
        for (int q = 0; q < Q; ++q)
            if (lane + 64 * q < r.n_group) open[lane + 64 * q] = (go >> q) & 1;
        wave_sync();
#pragma unroll
        for (int q = 0; q < Q; ++q)
            if (key[q] != 0 && !open[(lane + 64 * q) / per]) key[q] = 0;
    }
    return wave_top<Q>(key, r.k);
}

// The chosen ids in ascending order and their weights.
template <int Q>
__device__ __forceinline__ void store_choice(const SelectRule &r, int64_t t, uint32_t chosen, const float (&l)[Q],
                                             int32_t *__restrict__ idx, float *__restrict__ wts) {
    const int lane = threadIdx.x & 63;
    float s[Q], total;
    if (r.softmax) {
        // relative to the largest logit that the denominator has
        float m = -INFINITY, sum = 0.f;
#pragma unroll
        for (int q = 0; q < Q; ++q)
            if (!r.renorm || ((chosen >> q) & 1)) m = fmaxf(m, l[q]);
        m = wave_max_f32(m, kWave);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            s[q] = softmax_term(l[q], m);
            if (lane + 64 * q < r.E && (!r.renorm || ((chosen >> q) & 1))) sum += s[q];
        }
        total = wave_sum_f32(sum);
    } else {
        float sum = 0.f;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            s[q] = sigmoid_f32(l[q]);
            if ((chosen >> q) & 1) sum += s[q];
        }
        total = r.renorm ? wave_sum_f32(sum) : 1.f;
    }
    int base = 0;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const bool mine = (chosen >> q) & 1;
        const uint64_t at = __ballot(mine);
        if (mine) {
            const int64_t o = t * r.k + base + __popcll(at & ((1ull << lane) - 1));
            idx[o] = lane + 64 * q;
            wts[o] = total == 0.f ? 0.f : r.scale * (s[q] / total);
        }
        base += __popcll(at);
    }
}

template <int Q, bool BF16>
__global__ __launch_bounds__(256) void k_select(SelectRule r, int T, const void *__restrict__ logits, int64_t ld,
                                                const float *__restrict__ bias, int32_t *__restrict__ idx,
                                                float *__restrict__ wts) {
    __shared__ double score64[4][64 * Q];
    __shared__ uint8_t open[4][64 * Q];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * 4 + wave;
    if (t >= T) return;
    const void *row = static_cast<const char *>(logits) + t * ld * (BF16 ? 2 : 4);
    float l[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) l[q] = lane + 64 * q < r.E ? load_logit<BF16>(row, lane + 64 * q) : -INFINITY;
    const uint32_t chosen = choose64<Q>(r, l, bias, score64[wave], open[wave]);
    store_choice<Q>(r, t, chosen, l, idx, wts);
}

// -------------------------------------------------------- sixteen lanes per token

template <int CTRL>
__device__ __forceinline__ float dpp_f32(float v) { return __uint_as_float(dpp_u32<CTRL>(__float_as_uint(v))); }
// v of the lane N below in its row of 16, 0 for the first N.
template <int N>
__device__ __forceinline__ uint32_t row_shr(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x110 + N, 0xf, 0xf, true);
}

__device__ __forceinline__ uint32_t row_min(uint32_t v) {
#define STEP(C) v = min(v, dpp_u32<C>(v));
    MOE_ROW_STEPS(STEP)
#undef STEP
    return v;
}
__device__ __forceinline__ uint32_t row_add(uint32_t v) {
#define STEP(C) v += dpp_u32<C>(v);
    MOE_ROW_STEPS(STEP)
#undef STEP
    return v;
}
__device__ __forceinline__ float row_sum(float v) {
#define STEP(C) v += dpp_f32<C>(v);
    MOE_ROW_STEPS(STEP)
#undef STEP
    return v;
}
__device__ __forceinline__ float row_maxf(float v) {
#define STEP(C) v = fmaxf(v, dpp_f32<C>(v));
    MOE_ROW_STEPS(STEP)
#undef STEP
    return v;
}

// Lanes of the row whose v is larger than this lane's.
__device__ __forceinline__ int row_rank(uint32_t v) {
    int n = 0;
#define ROR(N) n += dpp_u32<0x120 + N>(v) > v;
    ROR(1) ROR(2) ROR(3) ROR(4) ROR(5) ROR(6) ROR(7) ROR(8) ROR(9) ROR(10) ROR(11) ROR(12) ROR(13) ROR(14) ROR(15)
#undef ROR
    return n;
}

// 31-bit ordered key of a number (its last mantissa bit goes), never 0.
__device__ __forceinline__ uint32_t key31(float v) { return f32_order_key(v + 0.f) >> 1; }
__device__ __forceinline__ float from_key31(uint32_t k) { return f32_from_order_key(k << 1); }

// e^v to choose by: the product's rounding and log2(e)'s, each a half step of the exponent, are left in.
__device__ __forceinline__ float fast_exp(float v) { return __builtin_amdgcn_exp2f(1.4426950408889634f * v); }

// e^v to two steps of fp32: what the exponent's rounding left out goes back to first order, e^c = 1 + c.  At most a
// half step of an exponent that exp2 does not take to 0 or infinity, 2^-18; past those c can be anything, and only
// its sign and finiteness are kept.
__device__ __forceinline__ float exp_f32(float v) {
    const float t = 1.44269502162933349609375f * v;  // log2(e) = this + 1.92596299e-8
    const float c = __builtin_fmaf(v, 1.92596299e-8f, __builtin_fmaf(v, 1.44269502162933349609375f, -t));
    return __builtin_amdgcn_exp2f(t) * __builtin_fmaf(fminf(fmaxf(c, -1.f), 1.f), 0.693147182464599609375f, 1.f);
}

// The n <= Q experts from e0 on of a row that begins `at` elements into p, -inf
// behind them (what is loaded there is another expert of the row).  vec: lanes
// begin at 16 bytes (or all of a lane's), and n is Q or 0.
template <int Q, bool BF16>
__device__ __forceinline__ void load_row(const void *p, int64_t at, int e0, int n, bool vec, float (&l)[Q]) {
    const int first = n > 0 ? e0 : 0, last = n > 0 ? n - 1 : 0;
    const char *row = static_cast<const char *>(p) + (at + first) * (BF16 ? 2 : 4);
    if (vec && BF16) {
        constexpr int W = Q >= 8 ? 4 : 2;  // words per load
#pragma unroll
        for (int c = 0; c < Q / 2; c += W) {
            uint32_t w[4];
            if (W == 4) {
                const i32x4 v = *reinterpret_cast<const i32x4 *>(row + 4 * c);
                w[0] = (uint32_t)v[0]; w[1] = (uint32_t)v[1]; w[2] = (uint32_t)v[2]; w[3] = (uint32_t)v[3];
            } else {
                const uint2 v = *reinterpret_cast<const uint2 *>(row + 4 * c);
                w[0] = v.x; w[1] = v.y;
            }
#pragma unroll
            for (int i = 0; i < W; ++i) {
                l[2 * (c + i)] = bf16_to_f32(w[i] & 0xffffu);
                l[2 * (c + i) + 1] = bf16_to_f32(w[i] >> 16);
            }
        }
    } else if (vec) {
#pragma unroll
        for (int c = 0; c < Q; c += 4) {
            const f32x4 v = *reinterpret_cast<const f32x4 *>(row + 4 * c);
#pragma unroll
            for (int i = 0; i < 4; ++i) l[c + i] = v[i];
        }
    } else {
#pragma unroll
        for (int q = 0; q < Q; ++q) l[q] = load_logit<BF16>(row, min(q, last));
    }
#pragma unroll
    for (int q = 0; q < Q; ++q) l[q] = q < n ? l[q] : -INFINITY;
}

// Four experts per lane and load, 64 experts on for the next: the expert of a
// lane's value q.  Sixteen lanes then read and write a row in order.
__device__ __forceinline__ int spread(int sub, int q) { return (q >> 2) * 64 + 4 * sub + (q & 3); }

// A row's experts spread over its sixteen lanes, `behind` behind the last one.
// vec: rows begin at four values, E is a multiple of four.
template <int Q, bool BF16>
__device__ __forceinline__ void load_spread(const void *p, int64_t at, int sub, int E, bool vec, float behind,
                                            float (&l)[Q]) {
    const char *row = static_cast<const char *>(p) + at * (BF16 ? 2 : 4);
#pragma unroll
    for (int c = 0; c < Q; c += 4) {
        const int e = spread(sub, c);
        if (vec) {
            const int from = e < E ? e : 0;
            if (BF16) {
                const uint2 v = *reinterpret_cast<const uint2 *>(row + 2 * from);
                l[c] = bf16_to_f32(v.x & 0xffffu);
                l[c + 1] = bf16_to_f32(v.x >> 16);
                l[c + 2] = bf16_to_f32(v.y & 0xffffu);
                l[c + 3] = bf16_to_f32(v.y >> 16);
            } else {
                const f32x4 v = *reinterpret_cast<const f32x4 *>(row + 4 * from);
                l[c] = v[0]; l[c + 1] = v[1]; l[c + 2] = v[2]; l[c + 3] = v[3];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) l[c + i] = load_logit<BF16>(row, min(e + i, E - 1));
        }
    }
#pragma unroll
    for (int q = 0; q < Q; ++q) l[q] = spread(sub, q) < E ? l[q] : behind;
}
// Whether load_spread can load whole vectors of rows ld apart, and of dense fp32
// rows beside them.
bool spread_vec(int E, bool bf16, const void *logits, int64_t ld, const void *a, const void *b) {
    const int64_t bytes = bf16 ? 8 : 16;
    return E % 4 == 0 && reinterpret_cast<uintptr_t>(logits) % bytes == 0 && ld % 4 == 0 &&
           reinterpret_cast<uintptr_t>(a) % 16 == 0 && reinterpret_cast<uintptr_t>(b) % 16 == 0;
}

// How a row's groups lie over sixteen lanes.
struct LaneMap {
    int groups, per;          // groups of so many experts
    int lanes, shift;         // lanes per group, a power of two, and its logarithm
    int run;                  // experts per lane, the group's last lane with what is left
};
LaneMap lane_map(const SelectRule &r) {
    LaneMap m{r.topk_group < r.n_group ? r.n_group : 1, 0, 16, 4, 0};
    m.per = r.E / m.groups;
    while (m.lanes > 1 && m.lanes * m.groups > 16) m.lanes /= 2, --m.shift;
    m.run = (m.per + m.lanes - 1) / m.lanes;
    return m;
}

// What the keys are made of: bf16 logits with the id in the low bits (no two
// alike, nothing rounded), fp32 logits, or the biased fp32 scores.
enum { KEY_BF16 = 0, KEY_F32 = 1, KEY_SCORE = 2 };

template <int CTRL>
__device__ __forceinline__ double dpp_f64(double v) {
    return __longlong_as_double((long long)dpp_u64<CTRL>((uint64_t)__double_as_longlong(v)));
}

// Lanes of the row with a larger v, or the same and a lower id.
__device__ __forceinline__ int row_rank64(double v, int id) {
    int n = 0;
#define ROR(N)                                                       \
    {                                                                \
        const double o = dpp_f64<0x120 + N>(v);                      \
        const int oid = (int)dpp_u32<0x120 + N>((uint32_t)id);       \
        n += o > v || (o == v && oid < id);                          \
    }
    ROR(1) ROR(2) ROR(3) ROR(4) ROR(5) ROR(6) ROR(7) ROR(8) ROR(9) ROR(10) ROR(11) ROR(12) ROR(13) ROR(14) ROR(15)
#undef ROR
    return n;
}

__device__ __forceinline__ double sigmoid64(float l) { return 1.0 / (1.0 + exp(-(double)l)); }

// Whether this lane's group is among the best ones, by 64-bit scores.  cand: the
// lane's experts that can be one of its group's two best; lq: its logits in LDS.
__device__ __forceinline__ bool settle_groups(uint32_t cand, const float *lq, const float *__restrict__ bias, int e0,
                                              const LaneMap &map, int group, bool top_two, int want) {
    double d1 = -INFINITY, d2 = -INFINITY;
    for (; cand; cand &= cand - 1) {
        const int q = __ffs(cand) - 1;
        double v = bias || top_two ? sigmoid64(lq[q]) : (double)lq[q];
        if (bias) v += (double)bias[e0 + q];
        d2 = fmax(d2, fmin(d1, v));
        d1 = fmax(d1, v);
    }
#define STEP(C, LANES)                                           \
    if (map.lanes >= LANES) {                                    \
        const double o1 = dpp_f64<C>(d1), o2 = dpp_f64<C>(d2);   \
        d2 = fmax(fmin(d1, o1), fmax(d2, o2));                   \
        d1 = fmax(d1, o1);                                       \
    }
    STEP(0xB1, 2) STEP(0x4E, 4) STEP(0x141, 8) STEP(0x140, 16)
#undef STEP
    return row_rank64(top_two && map.per > 1 ? d1 + d2 : d1, group) < want;
}

// Which of the experts of a row that are near its border are chosen, by 64-bit
// scores: `need` of them.  near: the lane's, bit q; list: 16 values and ids of the
// row in LDS.  Returns them by bit q; of more than 16 none is settled (false).
struct BorderList {
    double v[16];
    int32_t id[16];
};
__device__ __forceinline__ bool settle_border(uint32_t &near, int need, const float *lq, const float *__restrict__ bias,
                                              int e0, BorderList *list) {
    const int sub = threadIdx.x & 15, mine = __popc(near), all = (int)row_add((uint32_t)mine);
    uint32_t pos = (uint32_t)mine;
    pos += row_shr<1>(pos);
    pos += row_shr<2>(pos);
    pos += row_shr<4>(pos);
    pos += row_shr<8>(pos);
    pos -= (uint32_t)mine;
    if (all <= 16) {
        uint32_t at = pos;
        for (uint32_t c = near; c; c &= c - 1, ++at) {
            const int q = __ffs(c) - 1;
            list->v[at] = bias ? sigmoid64(lq[q]) + (double)bias[e0 + q] : (double)lq[q];
            list->id[at] = e0 + q;
        }
    }
    wave_sync();
    const bool on = all <= 16 && sub < all;
    const int rank = row_rank64(on ? list->v[on ? sub : 0] : -INFINITY, on ? list->id[on ? sub : 0] : 1 << 20);
    wave_sync();
    if (on) list->id[sub] = rank < need;
    wave_sync();
    uint32_t out = 0;
    if (all <= 16) {
        uint32_t at = pos;
        for (uint32_t c = near; c; c &= c - 1, ++at)
            if (list->id[at]) out |= c & -c;
    }
    near = out;
    return all <= 16;
}

// Sixteen lanes per token, four tokens per wave (FULL: every lane has Q experts, in
// whole vectors, and none is masked).  A lane holds up to Q neighbouring
// experts of one group, each group has 1, 2, 4, 8 or 16 neighbouring lanes (LaneMap;
// all experts are one group where none is closed).  Keys are 31-bit unsigned numbers (0: not an expert, or its group is
// closed), so that with the largest key below m wanted, k - m as an unsigned
// number is at least 2^31 for a key below m and less for the others, and the
// largest difference is the answer: one subtraction and half a three-way maximum
// per key and round, four exchanges, k + 1 rounds.
//
// A sigmoid's doubts are settled where they arise, by the 64-bit scores of the few
// experts that they are about (settle_groups, settle_border); a softmax's, whose
// 64-bit scores need the whole row, and rows with a NaN go to choose64.
//
// fp32 scores: exp2 and reciprocal are off by one unit each, the exponent's
// rounding moves a sigmoid by at most s (1 - s) |l| 2^-24 < 2^-26, a softmax by p x
// 2^-24 with p x < 0.37 besides its sum's 30 roundings, the bias's addition and
// the key's lost bit by 2^-23 of the sum.  Two neighbours are in doubt when they
// are nearer than 2^-20 (sigmoid) or 2^-17 (softmax) plus 2^-21 of their size: twice
// those errors with room.  That is also where equal keys end up.
//
// 8 of 256 experts in 8 groups, biased sigmoid: 16384 tokens 13 us (17.8 MB; the wave
// per token takes 52), 32 tokens 5.5 us: bound by the instructions and latencies of
// one round of waves, about 1000 instructions per four tokens.  Without the
// settling of borders, its few 64-bit tokens made that 17 us.
template <int Q, int KEY, bool BF16, bool FULL>
__global__ __launch_bounds__(256) void k_select_fast(SelectRule r, LaneMap map, bool vec, int T,
                                                     const void *__restrict__ logits, int64_t ld,
                                                     const float *__restrict__ bias, int32_t *__restrict__ idx,
                                                     float *__restrict__ wts) {
    constexpr int QS = Q / 4;  // experts per lane in the 64-bit code
    __shared__ __attribute__((aligned(16))) float sc[4][64 * Q];  // the scores; 64-bit ones in the 64-bit code
    __shared__ uint8_t open64[4][64 * QS];
    __shared__ BorderList lists[4][4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, sub = lane & 15;
    const int64_t t0 = ((int64_t)blockIdx.x * 4 + wave) * 4;
    if (t0 >= T) return;
    const int64_t t = min(t0 + (lane >> 4), (int64_t)T - 1);
    const bool mine = t0 + (lane >> 4) < T;
    const int group = sub >> map.shift, e1 = (sub & (map.lanes - 1)) * map.run;  // in the group
    const int e0 = FULL ? sub * Q : group * map.per + e1;
    const int n = FULL ? Q : group < map.groups ? min(map.run, map.per - e1) : 0;
    float l[Q], b[Q];
    load_row<Q, BF16>(logits, t * ld, e0, n, FULL || vec, l);
    if (KEY == KEY_SCORE) load_row<Q, false>(bias, 0, e0, n, FULL || vec, b);
    // a NaN ranks behind every number: the 64-bit code's business (a biased score's is looked for below)
    bool doubt = false;
    if (KEY != KEY_SCORE) {
#pragma unroll
        for (int q = 0; q < Q; ++q) doubt |= l[q] != l[q];
    }

    float s[Q], total = 1.f, m = 0.f;
    if (r.softmax) {
        m = l[0];
#pragma unroll
        for (int q = 1; q < Q; ++q) m = fmaxf(m, l[q]);
        m = row_maxf(m);
        doubt |= !(fabsf(m) < INFINITY);
        total = 0.f;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            s[q] = fast_exp(l[q] - m);
            total += s[q];
        }
        total = row_sum(total);
        const float inv = 1.0f / total;
#pragma unroll
        for (int q = 0; q < Q; ++q) s[q] *= inv;
    } else {
#pragma unroll
        for (int q = 0; q < Q; ++q) s[q] = __builtin_amdgcn_rcpf(1.0f + fast_exp(-l[q]));
    }
    uint32_t key[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        if (KEY == KEY_SCORE) {
            b[q] += s[q];  // (-inf behind the last expert)
            doubt |= b[q] != b[q];
            key[q] = key31(b[q]);
        } else if (KEY == KEY_F32) {
            key[q] = key31(l[q]);
        } else {
            key[q] = ((f32_order_key(l[q] + 0.f) >> 16) << 15) | (uint32_t)(0x7fff - (e0 + q));
        }
        key[q] = q < n ? key[q] : 0;
    }
    const float near = r.softmax ? 7.62939453125e-6f : 9.5367431640625e-7f;  // 2^-17, 2^-20

    if (r.topk_group < r.n_group) {
        uint32_t g;
        const bool rounded = KEY == KEY_SCORE || r.top_two;
        float a1 = -INFINITY, a2 = -INFINITY;
        if (r.top_two) {
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                const float v = KEY == KEY_SCORE ? b[q] : q < n ? s[q] : -INFINITY;
                a2 = __builtin_amdgcn_fmed3f(a1, a2, v);  // a2 <= a1: the second of the three
                a1 = fmaxf(a1, v);
            }
#define STEP(C, LANES)                                         \
    if (map.lanes >= LANES) {                            \
        const float o1 = dpp_f32<C>(a1), o2 = dpp_f32<C>(a2);  \
        a2 = fmaxf(fminf(a1, o1), fmaxf(a2, o2));              \
        a1 = fmaxf(a1, o1);                                    \
    }
            STEP(0xB1, 2) STEP(0x4E, 4) STEP(0x141, 8) STEP(0x140, 16)
#undef STEP
            const float sum = map.per == 1 ? a1 : a1 + a2;
            doubt |= group < map.groups && sum != sum;
            g = group < map.groups ? key31(sum) : 0;
        } else {
            g = key[0];
#pragma unroll
            for (int q = 1; q < Q; ++q) g = max(g, key[q]);
#define STEP(C, LANES) \
    if (map.lanes >= LANES) g = max(g, dpp_u32<C>(g));
            STEP(0xB1, 2) STEP(0x4E, 4) STEP(0x141, 8) STEP(0x140, 16)
#undef STEP
        }
        const int want = r.topk_group * map.lanes;
        bool is_open = row_rank(g) < want;
        // equal groups at the border open together
        bool unsure = row_add(is_open ? 1u : 0u) != (uint32_t)want;
        if (rounded) {
            const uint32_t lo = row_min(is_open ? g : 0x7fffffffu), hi = row_max(is_open ? 0u : g);
            const float x = from_key31(lo), y = hi ? from_key31(hi) : -INFINITY;
            unsure |= !(x - y > 2.f * (near + 4.76837158203125e-7f * fabsf(x)));
        }
        if (r.softmax) {
            doubt |= unsure;
        } else if (__ballot(unsure)) {
            // those that fp32 leaves among their group's two best, or its best
            uint32_t cand = 0;
            const float lo = r.top_two && map.per > 1 ? a2 : from_key31(g);
            const float from = lo - 2.f * (near + 4.76837158203125e-7f * fabsf(lo));
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                sc[wave][lane * Q + q] = l[q];
                const float v = KEY == KEY_SCORE ? b[q] : r.top_two ? s[q] : l[q];
                if (unsure && q < n && !(v < from)) cand |= 1u << q;
            }
            wave_sync();
            const bool settled = settle_groups(cand, &sc[wave][lane * Q], bias, e0, map, group, r.top_two, want);
            is_open = unsure ? settled : is_open;
            wave_sync();
        }
#pragma unroll
        for (int q = 0; q < Q; ++q) key[q] = is_open ? key[q] : 0;
    }

    uint32_t at = 0x80000000u, kth = 0;
    const int rounds = KEY == KEY_SCORE ? r.k + 1 : r.k;
    for (int i = 0; i < rounds; ++i) {
        uint32_t d = key[0] - at;
#pragma unroll
        for (int q = 1; q < Q; ++q) d = max(d, key[q] - at);
        d = row_max(d);
        // none below: nothing (0) from here on, and no k-th, though the largest key wraps round to it
        at = d >= 0x80000000u ? at + d : 0;
        if (i == r.k - 1) kth = at;
    }
    // bit Q - 1 - q: expert e0 + q is chosen
    uint32_t chosen = 0;
#pragma unroll
    for (int q = 0; q < Q; ++q) chosen = __builtin_amdgcn_alignbit(chosen, (kth - 1u) - key[q], 31);
    bool unsure = row_add(__popc(chosen)) != (uint32_t)r.k || kth <= 1u;
    if (KEY == KEY_SCORE) {
        const float x = from_key31(kth), y = at ? from_key31(at) : -INFINITY;
        unsure |= !(x - y > near + 4.76837158203125e-7f * fabsf(x));
    }
    if (r.softmax && KEY == KEY_SCORE) {
        doubt |= unsure;
    } else if (__ballot(unsure)) {
        // the k-th largest again, equal keys counted one by one
        uint32_t kk = 0x80000000u, seen = 0;
        for (int i = 0; i < r.k; ++i) {
            uint32_t d = key[0] - kk, same = 0;
#pragma unroll
            for (int q = 1; q < Q; ++q) d = max(d, key[q] - kk);
            d = row_max(d);
            const uint32_t below = d >= 0x80000000u ? kk + d : 0;
#pragma unroll
            for (int q = 0; q < Q; ++q) same += key[q] == below;
            same = row_add(same);
            if (seen < (uint32_t)r.k && below) {
                kk = below;
                seen += same;
            }
        }
        const bool found = seen >= (uint32_t)r.k && kk != 0x80000000u;
        // above it by more than the error: chosen; within it: settled by 64-bit scores
        uint32_t hi = kk, lo = kk;
        if (KEY == KEY_SCORE) {
            const float x = from_key31(kk), tol = near + 4.76837158203125e-7f * fabsf(x);
            hi = key31(x + tol);
            lo = key31(x - tol);
        }
        uint32_t sure = 0, border = 0;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            if (unsure) sc[wave][lane * Q + q] = l[q];
            sure |= key[q] > hi ? 1u << q : 0;
            border |= key[q] <= hi && key[q] >= lo && key[q] != 0 ? 1u << q : 0;
        }
        if (!unsure || !found) border = 0;
        wave_sync();
        const int need = r.k - (int)row_add(__popc(sure));
        const bool settled = settle_border(border, need, &sc[wave][lane * Q], KEY == KEY_SCORE ? bias : nullptr, e0,
                                           &lists[wave][lane >> 4]);
        if (unsure) {
            chosen = __brev(sure | border) >> (32 - Q);
            doubt |= !settled || !found || row_add(__popc(chosen)) != (uint32_t)r.k;
        }
        wave_sync();
    }
    const uint32_t count = __popc(chosen);

    // the chosen experts' scores as store_choice has them: fast_exp's error, enough to choose by, grows
    // with the logit (2^-19 of the score at -32).  A sum that underflows is left to the 64-bit code's way: a
    // softmax's there is relative to the largest chosen, a sigmoid's keeps fp32's subnormals
    float sum = 0.f;
#pragma unroll
    for (int q = 0; q < Q; ++q) sc[wave][lane * Q + q] = l[q];
    for (uint32_t left = chosen << (32 - Q); left != 0;) {
        const int q = __clz(left);
        left &= ~(0x80000000u >> q);
        float &v = sc[wave][lane * Q + q];
        v = r.softmax ? softmax_term(v, m) : sigmoid_f32(v);
        sum += v;
    }
    sum = row_sum(sum);
    doubt |= r.renorm && !(sum > 1e-30f);
    if (!r.renorm) sum = r.softmax ? total : 1.f;
    uint32_t pos = count;
    pos += row_shr<1>(pos);
    pos += row_shr<2>(pos);
    pos += row_shr<4>(pos);
    pos += row_shr<8>(pos);
    pos -= count;
    doubt = row_add(doubt ? 1u : 0u) != 0;
    wave_sync();
    if (mine && !doubt) {
        int32_t *io = idx + t * r.k + pos;
        float *wo = wts + t * r.k + pos;
        for (uint32_t left = chosen << (32 - Q); left != 0;) {
            const int q = __clz(left);
            left &= ~(0x80000000u >> q);
            *io++ = e0 + q;
            *wo++ = r.scale * (sc[wave][lane * Q + q] / sum);  // (scale / sum alone may be past fp32)
        }
    }
    wave_sync();
    // the tokens in doubt, one after the other, in 64 bits
    const uint64_t left = __ballot(mine && doubt);
    for (int i = 0; i < 4; ++i) {
        if (!((left >> (16 * i)) & 1)) continue;
        const void *rw = static_cast<const char *>(logits) + (t0 + i) * ld * (BF16 ? 2 : 4);
        float v[QS];
#pragma unroll
        for (int q = 0; q < QS; ++q) v[q] = lane + 64 * q < r.E ? load_logit<BF16>(rw, lane + 64 * q) : -INFINITY;
        const uint32_t c = choose64<QS>(r, v, bias, reinterpret_cast<double *>(sc[wave]), open64[wave]);
        store_choice<QS>(r, t0 + i, c, v, idx, wts);
    }
}

// ------------------------------------------------------------- the sequences

// How many i of [0, n) have holds(i), which holds for the first ones and no
// others.  The wave looks at sixty-four of them at a time.
template <typename F>
__device__ __forceinline__ int count_leading(int n, F holds) {
    const int lane = threadIdx.x & 63;
    int lo = 0;
    while (n > 64) {
        const int step = (n + 63) / 64;
        const int i = min(lane * step + step, n) - 1;
        const int full = __popcll(__ballot(holds(lo + i)));
        if (full == 64) return lo + n;
        lo += full * step;
        n = min(step, n - full * step);
        if (n <= 0) return lo;
    }
    return lo + __popcll(__ballot(lane < n && holds(lo + min(lane, n - 1))));
}

// The sequence of [0, n) that holds token t, or n behind the last one: how many
// end at or before t.
__device__ __forceinline__ int sequence_of(const int32_t *__restrict__ off, int n, int t) {
    return count_leading(n, [&](int i) { return off[1 + i] <= t; });
}

// The gradient with respect to the logits of one token:
//   weights, renormalised: r_j (c dw_j - sum_i c dw_i r_i) with r the chosen
//     shares, times (1 - s_j) for a sigmoid; as they are: sigmoid c dw_j s_j
//     (1 - s_j), softmax p_e (c dw_e - sum_j c dw_j p_j) over all experts;
//   balance: p'_e (b_e - sum_i b_i p'_i), times (1 - s_e) for a sigmoid, with p'
//     the scores over their sum and b_e = alpha dloss load_e / tokens.
// Written in the shares r and p' (never in ds / S), nothing overflows where a
// row's scores are tiny; a row with no score at all has no gradient.
//
// Sixteen lanes per token as in k_select_fast; the chosen experts' gradients, made
// by the lanes of their places in idx, reach their experts through LDS.  dense:
// every logit has a gradient; else the row is not read but for the chosen.
// 16384 tokens of 256, weights and balance loss: 13 us for 34.6 MB; a wave per
// token took 17, and with each lane's experts side by side in memory (64 bytes
// per lane, so that an instruction touched as many lines as lanes) 14.3.
template <int Q, bool BF16>
__global__ __launch_bounds__(256) void k_select_backward(SelectRule r, bool vec, int T, const void *__restrict__ logits,
                                                         int64_t ld, const int32_t *__restrict__ idx,
                                                         const float *__restrict__ dw, BalanceGrad b,
                                                         float *__restrict__ dlogits) {
    __shared__ __attribute__((aligned(16))) float acc[4][64 * Q];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, sub = lane & 15;
    const int64_t t0 = ((int64_t)blockIdx.x * 4 + wave) * 4;
    if (t0 >= T) return;
    const int64_t t = min(t0 + (lane >> 4), (int64_t)T - 1);
    const bool mine = t0 + (lane >> 4) < T;
    const bool dense = b.seq || (r.softmax && !r.renorm);
    float p[Q], x[Q], m = -INFINITY, total = 0.f;
    float *const row_acc = &acc[wave][(lane & 48) * Q];  // by expert
    // what the places of idx say, asked for ahead of all else
    const int places = dw ? (r.k + 15) / 16 : 0;
    float d[4], le[4];
    int e[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (i >= places) continue;
        const int j = 16 * i + sub;
        e[i] = j < r.k ? idx[t * r.k + j] : -1;
        d[i] = j < r.k ? dw[t * r.k + j] : 0.f;
    }
    if (dense) {
        load_spread<Q, BF16>(logits, t * ld, sub, r.E, vec, -INFINITY, p);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (i >= places) continue;
        const bool on = e[i] >= 0 && e[i] < r.E;
        if (!on) e[i] = -1;
        le[i] = load_logit<BF16>(static_cast<const char *>(logits) + t * ld * (BF16 ? 2 : 4), on ? e[i] : 0);
        le[i] = on ? le[i] : -INFINITY;
        d[i] = on ? d[i] : 0.f;
    }
    // the balance loss's coefficients of the row's sequence
    float f[Q], scale = 0.f;
    if (b.seq) {
        const int last = (int)min(t0 + 3, (int64_t)T - 1);
        int s = sequence_of(b.seq, b.n_seq, (int)t0);
        if (sequence_of(b.seq, b.n_seq, last) != s) {
#pragma unroll
            for (int i = 1; i < 4; ++i) {
                const int si = sequence_of(b.seq, b.n_seq, min((int)t0 + i, last));
                s = (lane >> 4) >= i ? si : s;
            }
        }
        const int at = min(s, b.n_seq - 1), start = b.seq[at], end = b.seq[at + 1];
        if (s < b.n_seq && t >= start && t < end) scale = b.alpha * b.dloss[at] / (float)(end - start);
        load_spread<Q, false>(b.load, (int64_t)at * r.E, sub, r.E, vec, 1.f, f);
    }
    float mean = 0.f;  // softmax weights as they are: sum_j c dw_j p_j
#pragma unroll
    for (int q = 0; q < Q; ++q) row_acc[spread(sub, q)] = 0.f;
    wave_sync();
    if (dense) {
        if (r.softmax) {
#pragma unroll
            for (int q = 0; q < Q; ++q) m = fmaxf(m, p[q]);
            m = row_maxf(m);
        }
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            // p becomes the score, x what gives a sigmoid's 1 - p = x p
            if (r.softmax) {
                p[q] = m == -INFINITY ? 0.f : exp_f32(p[q] - m);
            } else {
                x[q] = exp_f32(-p[q]);
                p[q] = __builtin_amdgcn_rcpf(1.0f + x[q]);
            }
            total += p[q];
        }
        total = row_sum(total);
    }
    if (dw) {
        float share[4], mc = -INFINITY, S = 0.f, cross = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < places) mc = fmaxf(mc, le[i]);
        if (r.softmax) mc = r.renorm ? row_maxf(mc) : m;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i >= places) continue;
            share[i] = e[i] < 0 ? 0.f : r.softmax ? softmax_term(le[i], mc) : sigmoid_f32(le[i]);
            S += share[i];
        }
        S = r.renorm ? row_sum(S) : r.softmax ? total : 1.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i >= places) continue;
            share[i] = S == 0.f ? 0.f : share[i] / S;
            cross += d[i] * share[i];
        }
        cross = row_sum(cross);
        if (r.softmax && !r.renorm) mean = r.scale * cross;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i >= places) continue;
            // the scale behind the share: their product is the gradient's size, the scale's with dw may be past fp32
            d[i] = r.scale * (share[i] * (r.renorm ? d[i] - cross : d[i]) * (r.softmax ? 1.f : sigmoid_f32(-le[i])));
            if (e[i] >= 0) row_acc[e[i]] = d[i];
        }
    }
    wave_sync();
    float g[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) g[q] = row_acc[spread(sub, q)];
    if (dense) {
        const float inv = total == 0.f ? 0.f : 1.f / total;
        float dot = 0.f;
        if (b.seq) {
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                // from the mean load, 1: the shares' sum is 1, so a constant has no gradient, and
                // what is left rounds by its own size
                f[q] = scale * (f[q] - 1.f);
                dot += f[q] * (p[q] * inv);
            }
            dot = row_sum(dot);
        }
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const float rest = r.softmax || x[q] > 1e30f ? 1.f : x[q] * p[q];
            g[q] += p[q] * inv * ((b.seq ? f[q] - dot : 0.f) * rest - mean);
        }
    }
    if (!mine) return;
    float *o = dlogits + t * r.E;
#pragma unroll
    for (int c = 0; c < Q; c += 4) {
        const int e = spread(sub, c);
        if (vec) {
            if (e < r.E) *reinterpret_cast<f32x4 *>(o + e) = f32x4{g[c], g[c + 1], g[c + 2], g[c + 3]};
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (e + i < r.E) o[e + i] = g[c + i];
        }
    }
}

// Partial sums of the balance loss.  The tokens are cut at every kBalanceTokens and
// at every sequence: the piece of sequence s that lies in the c-th kBalanceTokens
// tokens is number c + s (ascending in both, so no two share one), and workgroup
// and slot of that number leave the sum of its tokens' shares and the count of
// choices per expert.  Sixteen lanes per token, each lane sums its own experts.
// 16384 tokens of 256 in 9 sequences: 10 us, bound by the latency of its loads and
// exchanges in turn; 128 tokens per piece took 13, a workgroup for all sequences of
// its tokens 12.7 (and, with 59 sequences in 258 tokens, 30 more).
template <int Q, bool BF16>
__global__ __launch_bounds__(512) void k_balance_part(SelectRule r, bool vec, int T, const void *__restrict__ logits,
                                                      int64_t ld, const int32_t *__restrict__ idx,
                                                      const int32_t *__restrict__ seq, int n_seq,
                                                      float *__restrict__ part, int32_t *__restrict__ count) {
    __shared__ float share[8][16 * Q];
    __shared__ int32_t hist[16 * Q];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, sub = lane & 15;
    const int64_t slot = blockIdx.x;
    // the last sequence whose first piece has this number or less
    const int s = count_leading(n_seq, [&](int i) { return (int64_t)max(seq[i], 0) / kBalanceTokens + i <= slot; }) - 1;
    if (s < 0) return;
    const int64_t c0 = (slot - s) * kBalanceTokens;
    const int t = (int)min(max(c0, (int64_t)max(seq[s], 0)), (int64_t)T);
    const int end = (int)min(min(c0 + kBalanceTokens, (int64_t)max(seq[s + 1], 0)), (int64_t)T);
    if (t >= end) return;
    // this thread's first choice, asked for ahead of the scores
    const int64_t first = (int64_t)t * r.k + tid, behind = (int64_t)end * r.k;
    const int mine = first < behind ? idx[first] : -1;
    for (int e = tid; e < 16 * Q; e += 512) hist[e] = 0;
    float sum[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) sum[q] = 0.f;
    for (int u0 = t + 4 * wave; u0 < end; u0 += 32) {
        const int u = u0 + (lane >> 4);
        float p[Q], m = -INFINITY, total = 0.f;
        load_spread<Q, BF16>(logits, (int64_t)min(u, end - 1) * ld, sub, r.E, vec, -INFINITY, p);
        if (r.softmax) {
#pragma unroll
            for (int q = 0; q < Q; ++q) m = fmaxf(m, p[q]);
            m = row_maxf(m);
        }
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            p[q] = r.softmax ? (m == -INFINITY ? 0.f : exp_f32(p[q] - m)) : __builtin_amdgcn_rcpf(1.0f + exp_f32(-p[q]));
            total += p[q];
        }
        total = row_sum(total);
        const float c = u < end && total != 0.f ? 1.f / total : 0.f;
#pragma unroll
        for (int q = 0; q < Q; ++q) sum[q] += p[q] * c;
    }
    // the wave's four rows, then the waves, in a fixed order
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        sum[q] += __shfl_xor(sum[q], 16, kWave);
        sum[q] += __shfl_xor(sum[q], 32, kWave);
        if (lane < 16) share[wave][spread(sub, q)] = sum[q];
    }
    __syncthreads();
    if (mine >= 0 && mine < r.E) atomicAdd(&hist[mine], 1);
    for (int64_t i = first + 512; i < behind; i += 512) {
        const int e = idx[i];
        if (e >= 0 && e < r.E) atomicAdd(&hist[e], 1);
    }
    __syncthreads();
    for (int e = tid; e < r.E; e += 512) {
        float v = share[0][e];
#pragma unroll
        for (int w = 1; w < 8; ++w) v += share[w][e];
        part[slot * r.E + e] = v;
        count[slot * r.E + e] = hist[e];
    }
}

// One workgroup per sequence: its slots added in order (by 1024 / width slices, the
// slices in order), load_e = E count_e / (k n), loss = alpha sum_e load_e mean_e.
// A sequence without tokens has no loss and no load.
template <int WIDTH>
__global__ __launch_bounds__(1024) void k_balance_sum(int E, int k, int T, const int32_t *__restrict__ seq, float alpha,
                                                      const float *__restrict__ part, const int32_t *__restrict__ count,
                                                      float *__restrict__ loss, float *__restrict__ load) {
    constexpr int kSlices = 1024 / WIDTH;
    __shared__ double sums[kSlices][WIDTH];
    __shared__ int32_t counts[kSlices][WIDTH];
    __shared__ double wsum[16];
    const int s = blockIdx.x, tid = threadIdx.x, e = tid % WIDTH, slice = tid / WIDTH;
    const int a = min(max(seq[s], 0), T), b = min(max(seq[s + 1], 0), T), n = b - a;
    double sum = 0.0;
    int c = 0;
    if (n > 0 && e < E) {
        const int64_t first = a / kBalanceTokens + s, last = (b - 1) / kBalanceTokens + s;
#pragma unroll 8
        for (int64_t i = first + slice; i <= last; i += kSlices) {
            sum += part[i * E + e];
            c += count[i * E + e];
        }
    }
    sums[slice][e] = sum;
    counts[slice][e] = c;
    __syncthreads();
    double mine = 0.0;
    if (tid < E) {
#pragma unroll
        for (int i = 1; i < kSlices; ++i) {
            sum += sums[i][e];
            c += counts[i][e];
        }
        const double f = n > 0 ? (double)E * (double)c / ((double)k * n) : 0.0;
        load[(int64_t)s * E + e] = (float)f;
        if (n > 0) mine = f * sum / n;
    }
    mine = wave_sum_f64(mine);
    if ((tid & 63) == 0) wsum[tid >> 6] = mine;
    __syncthreads();
    if (tid == 0) {
        double v = 0.0;
        for (int w = 0; w < 16; ++w) v += wsum[w];
        loss[s] = (float)((double)alpha * v);
    }
}

int balance_blocks(int T) { return (T + kBalanceTokens - 1) / kBalanceTokens; }

}  // namespace

// LAUNCH(experts per lane): the next power of two of E over LANES.
#define MOE_BY_WIDTH(LAUNCH, LANES)                      \
    do {                                                 \
        if (a.rule.E <= 64) LAUNCH(64 / LANES);          \
        else if (a.rule.E <= 128) LAUNCH(128 / LANES);   \
        else if (a.rule.E <= 256) LAUNCH(256 / LANES);   \
        else if (a.rule.E <= 512) LAUNCH(512 / LANES);   \
        else LAUNCH(1024 / LANES);                       \
    } while (0)

hipError_t launch_select(const SelectArgs &a, hipStream_t s) {
    const SelectRule &r = a.rule;
    const dim3 block(256);
    // Sixteen lanes hold up to 32 experts each; more of them, or more than 16 groups,
    // are left to the wave per token.
    LaneMap map = lane_map(r);
    if (map.lanes * map.groups <= 16 && map.run <= 32) {
        const dim3 grid((unsigned)(((int64_t)a.T + 15) / 16));
        const int Q = map.run <= 4 ? 4 : map.run <= 8 ? 8 : map.run <= 16 ? 16 : 32;
        // whole vectors: a group's lanes all full, or empty
        const int64_t bytes = a.bf16 ? 2 : 4, step = Q * bytes < 16 ? Q * bytes : 16;
        const bool vec = map.per % Q == 0 && reinterpret_cast<uintptr_t>(a.logits) % step == 0 &&
                         a.ld * bytes % step == 0 && reinterpret_cast<uintptr_t>(a.bias) % 16 == 0;
        if (vec) map.run = Q;
        const bool full = vec && r.E == 16 * Q;
#define FAST_KEY(QQ, KEY, BF16)                                                                                     \
    do {                                                                                                            \
        if (full) hipLaunchKernelGGL((k_select_fast<QQ, KEY, BF16, true>), grid, block, 0, s, r, map, vec, a.T,     \
                                     a.logits, a.ld, a.bias, a.idx, a.weights);                                     \
        else hipLaunchKernelGGL((k_select_fast<QQ, KEY, BF16, false>), grid, block, 0, s, r, map, vec, a.T,         \
                                a.logits, a.ld, a.bias, a.idx, a.weights);                                          \
    } while (0)
#define FAST(QQ)                                                    \
    do {                                                            \
        if (a.bias && a.bf16) FAST_KEY(QQ, KEY_SCORE, true);        \
        else if (a.bias) FAST_KEY(QQ, KEY_SCORE, false);            \
        else if (a.bf16) FAST_KEY(QQ, KEY_BF16, true);              \
        else FAST_KEY(QQ, KEY_F32, false);                          \
    } while (0)
        if (Q == 4) FAST(4);
        else if (Q == 8) FAST(8);
        else if (Q == 16) FAST(16);
        else FAST(32);
#undef FAST
#undef FAST_KEY
        return hipGetLastError();
    }
    // (a wave per token: fewer than 2^32 threads to a launch)
    constexpr int kRows = 1 << 25;
    for (int t0 = 0; t0 < a.T; t0 += kRows) {
        const int n = a.T - t0 < kRows ? a.T - t0 : kRows;
        const dim3 grid((unsigned)((n + 3) / 4));
        const void *logits = static_cast<const char *>(a.logits) + t0 * a.ld * (a.bf16 ? 2 : 4);
        int32_t *idx = a.idx + (int64_t)t0 * r.k;
        float *weights = a.weights + (int64_t)t0 * r.k;
#define GO(Q)                                                                                                       \
    do {                                                                                                            \
        if (a.bf16) hipLaunchKernelGGL((k_select<Q, true>), grid, block, 0, s, r, n, logits, a.ld, a.bias, idx,     \
                                       weights);                                                                    \
        else hipLaunchKernelGGL((k_select<Q, false>), grid, block, 0, s, r, n, logits, a.ld, a.bias, idx, weights); \
    } while (0)
        MOE_BY_WIDTH(GO, 64);
#undef GO
    }
    return hipGetLastError();
}

hipError_t launch_select_backward(const SelectBackwardArgs &a, hipStream_t s) {
    const dim3 grid((unsigned)(((int64_t)a.T + 15) / 16)), block(256);
#define GO(Q)                                                                                                          \
    do {                                                                                                               \
        const bool vec = spread_vec(a.rule.E, a.bf16, a.logits, a.ld, a.dlogits, a.balance.load);                      \
        if (a.bf16) hipLaunchKernelGGL((k_select_backward<Q, true>), grid, block, 0, s, a.rule, vec, a.T, a.logits,    \
                                       a.ld, a.idx, a.dweights, a.balance, a.dlogits);                                 \
        else hipLaunchKernelGGL((k_select_backward<Q, false>), grid, block, 0, s, a.rule, vec, a.T, a.logits, a.ld,    \
                                a.idx, a.dweights, a.balance, a.dlogits);                                              \
    } while (0)
    MOE_BY_WIDTH(GO, 16);
#undef GO
    return hipGetLastError();
}

size_t balance_ws_bytes(int T, int E, int n_seq) {
    return ((size_t)balance_blocks(T) + n_seq) * E * (sizeof(float) + sizeof(int32_t));
}

hipError_t launch_balance_loss(const BalanceArgs &a, void *ws, hipStream_t s) {
    const size_t slots = (size_t)balance_blocks(a.T) + a.n_seq;
    float *part = static_cast<float *>(ws);
    int32_t *count = reinterpret_cast<int32_t *>(part + slots * a.rule.E);
    const dim3 grid((unsigned)slots), block(512);
#define GO(Q)                                                                                                         \
    do {                                                                                                              \
        const bool vec = spread_vec(a.rule.E, a.bf16, a.logits, a.ld, nullptr, nullptr);                              \
        if (a.bf16) hipLaunchKernelGGL((k_balance_part<Q, true>), grid, block, 0, s, a.rule, vec, a.T, a.logits,      \
                                       a.ld, a.idx, a.seq, a.n_seq, part, count);                                     \
        else hipLaunchKernelGGL((k_balance_part<Q, false>), grid, block, 0, s, a.rule, vec, a.T, a.logits, a.ld,      \
                                a.idx, a.seq, a.n_seq, part, count);                                                  \
    } while (0)
    MOE_BY_WIDTH(GO, 16);
#undef GO
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
#define GO(W)                                                                                                         \
    hipLaunchKernelGGL(k_balance_sum<W>, dim3(a.n_seq), dim3(1024), 0, s, a.rule.E, a.rule.k, a.T, a.seq, a.alpha,    \
                       part, count, a.loss, a.load)
    MOE_BY_WIDTH(GO, 1);
#undef GO
    return hipGetLastError();
}
#undef MOE_BY_WIDTH

}  // namespace moe
