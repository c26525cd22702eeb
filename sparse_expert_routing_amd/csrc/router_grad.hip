// The router projection's gradient from that of its logits:
//   dx[t, n] = dx_in[t, n] + sum_e dl[t, e] w[e, n],   dw[e, n] = sum_t dl[t, e] x[t, n]
// with fp32's accuracy, on the 16-bit matrix cores (16x the fp32 ones' rate).
//
// Each fp32 operand becomes a few 16-bit terms whose products are exact in fp32:
//   - dx, K = 256: a row of dl and a column of w are each scaled by a power of
//     two so that their largest magnitude lies in [2^14, 2^15), then v = hi + mid
//     in fp16 (hi = rne(v), mid = rne(v - hi): 22 bits, down to 2^-39 of the
//     row's largest).  hi hi + hi mid + mid hi leaves out mid mid, 2^-22 of a
//     product; the sum is scaled back by the two exponents together (ldexp).
//   - dw, K = T: x is bf16 as it is; dl = hi + mid + lo in bf16, each the top 8
//     bits of what is left, 24 bits and exact.  An fp32 x is split the same way,
//     and the six products of at least 2^-16 of the whole are summed.
// An infinity or NaN in dl, w or an fp32 x makes the sums it enters NaN.
#include "device.h"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kE = 256;
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i16x4 *lds_i16x4_t;
typedef __attribute__((address_space(3))) void lds_void;

__device__ __forceinline__ void dma16(const void *src, void *lds) {
    __builtin_amdgcn_global_load_lds(src, (lds_void *)lds, 16, 0, 0);
}
// This wave's loads and LDS reads are done, and every wave's.
__device__ __forceinline__ void all_landed() {
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_waitcnt((7 << 4));  // vmcnt(0), lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

// The exponent e of the scale 2^e that brings a largest magnitude (its bits)
// into [2^14, 2^15); 0 for zero, and no more than 2^126, which fp32's
// subnormals do not fill.
__device__ __forceinline__ int scale_exp(uint32_t amax_bits) {
    if (amax_bits == 0) return 0;
    return min(14 - ((int)(amax_bits >> 23) - 127), 126);
}

__device__ __forceinline__ uint32_t f16_bits(_Float16 v) { return (uint32_t)__builtin_bit_cast(uint16_t, v); }

// v = hi + mid in fp16 (bits).
__device__ __forceinline__ void split_f16(float v, uint32_t &hi, uint32_t &mid) {
    const _Float16 h = (_Float16)v;
    hi = f16_bits(h);
    mid = f16_bits((_Float16)(v - (float)h));
}

// v = t[0] + t[1] + t[2] in bf16 (bits), each the top of what is left: exact.
__device__ __forceinline__ void split_bf16(float v, uint32_t (&t)[3]) {
    t[0] = __float_as_uint(v) >> 16;
    v -= bf16_to_f32(t[0]);
    t[1] = __float_as_uint(v) >> 16;
    v -= bf16_to_f32(t[1]);
    t[2] = __float_as_uint(v) >> 16;
}

// Position of 16-byte piece c of row r in the dw product's A tiles, rows of 32
// bytes: eight rows that are read together lie in different banks.
constexpr int kStageK = 16;  // K per stage of the dw product
__device__ __forceinline__ int piece32(int r, int c) { return r * kStageK + ((c ^ ((r >> 3) & 1)) * 8); }

struct RgWs {
    uint16_t *dlh;   // [Tp/32][2][16][64][8] fp16 terms of the scaled rows of dl, as dx's fragments: 32 rows,
                     // term, 16 of K, lane, 8 values; zeros behind T
    int32_t *er;     // [T] their exponents
    uint16_t *wh;    // [2][d][256] fp16 terms of the scaled columns of w
    int32_t *ec;     // [d]
    uint16_t *dlt;   // [Tp/16][3][256][16] bf16 terms of dl, transposed by stages of 16 tokens, zeros behind T
    uint16_t *xs;    // [3][T][d] bf16 terms of an fp32 x
    float *part;     // [S][256][d] partial sums of dw
    int Tp, S;
    size_t bytes;
};

// How the two products are cut into workgroups.  Large problems: 128 columns per dx
// block and 256 per dw block, about one of each per CU.  Below, 32 and 64, two
// workgroups per CU: T = 2048, d = 4096 50 us instead of 64 (T = d = 4096, where the
// large tiles begin: 82 and 89 with bf16 x, 140 and 132 with fp32 x; T = 16384,
// d = 2048: 182 and 146).
struct Cut {
    bool small;
    int dx_cols, dw_cols, dx_split, dw_split;
};
Cut cut_of(int T, int d) {
    Cut c{};
    const int rounds = (T + 255) / 256, stages = (T + kStageK - 1) / kStageK;
    c.small = (int64_t)((d + 127) / 128) * rounds < 512;
    c.dx_cols = c.small ? 32 : 128;
    c.dw_cols = c.small ? 64 : 256;
    const int dx_tiles = (d + c.dx_cols - 1) / c.dx_cols, dw_tiles = (d + c.dw_cols - 1) / c.dw_cols;
    // dx: its 8 waves have one chunk of 32 tokens at least
    c.dx_split = 256 / dx_tiles;
    c.dx_split = c.dx_split < 1 ? 1 : c.dx_split > rounds ? rounds : c.dx_split;
    // dw: eight stages at least.  Neighbouring workgroups take different splits, so with a
    // multiple of 8 each XCD works on its own tokens and keeps their dl terms in its L2: worth
    // a sixteenth of the CUs (d = 2560, T = 12000: 24 splits 49 us, 25 52), not an eighth
    // (T = 16384: d = 7168 9 splits 148 us, 8 155; d = 5120 12 splits 109, 8 143).
    c.dw_split = 256 / dw_tiles;
    if (c.dw_split / 8 * 8 * 16 >= c.dw_split * 15) c.dw_split = c.dw_split / 8 * 8;
    const int most = (stages + 7) / 8;
    c.dw_split = c.dw_split < 1 ? 1 : c.dw_split > most ? most : c.dw_split;
    return c;
}

RgWs carve(char *base, int T, int d, bool x_bf16) {
    RgWs w{};
    size_t o = 0;
    auto take = [&](size_t n) -> char * {
        char *p = base ? base + o : nullptr;
        o += (n + 255) / 256 * 256;
        return p;
    };
    w.Tp = (T + 31) / 32 * 32;
    w.S = cut_of(T, d).dw_split;
    w.dlh = reinterpret_cast<uint16_t *>(take((size_t)2 * w.Tp * kE * 2));
    w.er = reinterpret_cast<int32_t *>(take((size_t)w.Tp * 4));
    w.wh = reinterpret_cast<uint16_t *>(take((size_t)2 * d * kE * 2));
    w.ec = reinterpret_cast<int32_t *>(take((size_t)d * 4));
    w.dlt = reinterpret_cast<uint16_t *>(take((size_t)3 * kE * w.Tp * 2));
    w.xs = x_bf16 ? nullptr : reinterpret_cast<uint16_t *>(take((size_t)3 * T * d * 2));
    w.part = w.S == 1 ? nullptr : reinterpret_cast<float *>(take((size_t)w.S * kE * d * 4));
    w.bytes = o;
    return w;
}

// The operands' terms in one launch.  Workgroups [0, nw): 16 columns of w each;
// [nw, nw + nt): 32 rows of dl each; the rest, for an fp32 x: 2048 of its values.
// A thread's loads are all asked for before the first is used: at small sizes this
// launch is one such round trip.
__global__ __launch_bounds__(512) void k_rg_split(int T, int d, int nw, int nt, const float *__restrict__ w,
                                                  const float *__restrict__ dl, const float *__restrict__ x, RgWs ws) {
    __shared__ __attribute__((aligned(16))) float tile[32][kE + 4];
    __shared__ int row_exp[32];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    if ((int)blockIdx.x < nw) {
        // thread: column n, experts 8 part .. +7
        const int col = tid & 15, part = tid >> 4, n = blockIdx.x * 16 + col;
        float v[8];
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = w[(int64_t)(part * 8 + i) * d + n];
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
        uint32_t *most = reinterpret_cast<uint32_t *>(&tile[0][0]);
        most[tid] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 32; ++i) m = max(m, most[16 * i + col]);
        const int e = scale_exp(m);
        if (part == 0) ws.ec[n] = -e;
        i32x4 hi, mid;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t h0, m0, h1, m1;
            split_f16(ldexpf(v[2 * i], e), h0, m0);
            split_f16(ldexpf(v[2 * i + 1], e), h1, m1);
            hi[i] = (int)(h0 | (h1 << 16));
            mid[i] = (int)(m0 | (m1 << 16));
        }
        uint16_t *o = ws.wh + (int64_t)n * kE + part * 8;
        *reinterpret_cast<i32x4 *>(o) = hi;
        *reinterpret_cast<i32x4 *>(o + (int64_t)d * kE) = mid;
        return;
    }
    if ((int)blockIdx.x >= nw + nt) {
        const int64_t at = ((int64_t)(blockIdx.x - nw - nt) * 512 + tid) * 4, n = (int64_t)T * d;
        if (at >= n) return;  // n is a multiple of 4
        const f32x4 v = *reinterpret_cast<const f32x4 *>(x + at);
        uint32_t t[4][3];
#pragma unroll
        for (int i = 0; i < 4; ++i) split_bf16(v[i], t[i]);
#pragma unroll
        for (int j = 0; j < 3; ++j)
            *reinterpret_cast<uint2 *>(ws.xs + j * n + at) = uint2{t[0][j] | (t[1][j] << 16), t[2][j] | (t[3][j] << 16)};
        return;
    }
    const int t0 = (blockIdx.x - nw) * 32;
    f32x4 v[4];  // wave: rows 4 wave .. +3; lane: 4 experts
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = t0 + 4 * wave + i;
        v[i] = t < T ? *reinterpret_cast<const f32x4 *>(dl + (int64_t)t * kE + 4 * lane) : f32x4{0.f, 0.f, 0.f, 0.f};
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 4 * wave + i;
        *reinterpret_cast<f32x4 *>(&tile[r][4 * lane]) = v[i];
        uint32_t m = 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) m = max(m, __float_as_uint(v[i][c]) & 0x7fffffffu);
        for (int s = 32; s >= 1; s >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, s, kWave));
        if (lane == 0) {
            row_exp[r] = scale_exp(m);
            ws.er[t0 + r] = -row_exp[r];
        }
    }
    __syncthreads();
    // thread: 8 experts of a row, the 16 bytes of one lane of a fragment
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const int at = c * 512 + tid, m = at & 31, k = 8 * (at >> 5), e = row_exp[m];
        const f32x4 v0 = *reinterpret_cast<const f32x4 *>(&tile[m][k]);
        const f32x4 v1 = *reinterpret_cast<const f32x4 *>(&tile[m][k + 4]);
        i32x4 hi, mid;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t h0, m0, h1, m1;
            split_f16(ldexpf(i < 2 ? v0[2 * i] : v1[2 * i - 4], e), h0, m0);
            split_f16(ldexpf(i < 2 ? v0[2 * i + 1] : v1[2 * i - 3], e), h1, m1);
            hi[i] = (int)(h0 | (h1 << 16));
            mid[i] = (int)(m0 | (m1 << 16));
        }
        uint16_t *o = ws.dlh + (int64_t)(t0 / 32) * 2 * 32 * kE + at * 8;
        *reinterpret_cast<i32x4 *>(o) = hi;
        *reinterpret_cast<i32x4 *>(o + 32 * kE) = mid;
    }
    // thread: expert tid % 256, 16 of the tokens in a row
    const int ex = tid & (kE - 1), half = tid >> 8;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        i32x4 o[3];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t a[3], b[3];
            split_bf16(tile[16 * half + 8 * c + 2 * i][ex], a);
            split_bf16(tile[16 * half + 8 * c + 2 * i + 1][ex], b);
#pragma unroll
            for (int j = 0; j < 3; ++j) o[j][i] = (int)(a[j] | (b[j] << 16));
        }
#pragma unroll
        for (int j = 0; j < 3; ++j)
            *reinterpret_cast<i32x4 *>(ws.dlt + ((int64_t)(t0 / kStageK + half) * 3 + j) * kE * kStageK +
                                       piece32(ex, c)) = o[j];
    }
}

// ------------------------------------------------------------------- dx

// Position of 16-byte piece c of row r in an LDS tile of 512-byte rows: rows
// that are read together lie in different banks.
__device__ __forceinline__ int piece512(int r, int c) { return r * kE + ((c ^ (r & 15)) * 8); }

// A workgroup keeps its 32 NJ columns' terms of w in LDS (32 NJ KB) and its 8 waves
// walk 32-token chunks: their dl terms come straight from memory (each wave
// has its own rows, so LDS would not save a read), laid out so that a fragment is
// 1 KB in a row; there is no barrier in the loop.  32x32x16 tiles, NJ per wave; lane: column n, so a store is 128 bytes
// of a row.  Block z of S, tile y.
template <int NJ>
__device__ __forceinline__ void dx_block(int T, int d, const RgWs &ws, const int32_t *__restrict__ er,
                                         const float *dx_in, float *dx, uint16_t *sw, int z, int S, int y) {
    constexpr int kDxN = 32 * NJ;
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n0 = y * kDxN;
    // 64 NJ rows (term, n) of 512 bytes, two per load instruction
#pragma unroll
    for (int i = 0; i < 4 * NJ; ++i) {
        const int r = 2 * (wave * 4 * NJ + i) + g, n = min(n0 + (r & (kDxN - 1)), d - 1);
        const int c = (lane & 31) ^ (r & 15);
        dma16(ws.wh + ((int64_t)(r / kDxN) * d + n) * kE + 8 * c, sw + 2 * (wave * 4 * NJ + i) * kE);
    }
    const int chunks = (T + 31) / 32;
    const int c0 = (int)((int64_t)chunks * z / S), c1 = (int)((int64_t)chunks * (z + 1) / S);
    int ec[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) ec[j] = ws.ec[min(n0 + 32 * j + (lane & 31), d - 1)];
    all_landed();
    // LDS: row 32 j + lane % 32 of a term at + 16 KB j, piece 2 ks + g by one xor
    const uint32_t row_off = (uint32_t)piece512(lane & 31, g);
    // a part of K: two steps of 16; buffer, term, step
    constexpr int kParts = 8, kSteps = 16 / kParts;
    f16x8 a[2][2][kSteps];
    auto load = [&](int ch, int p, f16x8 (&v)[2][kSteps]) {
        const uint16_t *from = ws.dlh + (int64_t)ch * 2 * 32 * kE + p * kSteps * 512 + 8 * lane;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            v[0][s] = *reinterpret_cast<const f16x8 *>(from + s * 512);
            v[1][s] = *reinterpret_cast<const f16x8 *>(from + 32 * kE + s * 512);
        }
    };
    f32x16 acc[NJ];
    // w's fragments of a step are read from LDS during the step before: step, block, term
    f16x8 w[2][NJ][2];
    auto fetch = [&](int step, f16x8 (&v)[NJ][2]) {
        const uint16_t *h = sw + (row_off ^ (uint32_t)(16 * step));
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            v[j][0] = *reinterpret_cast<const f16x8 *>(h + 32 * j * kE);
            v[j][1] = *reinterpret_cast<const f16x8 *>(h + (kDxN + 32 * j) * kE);
        }
    };
    auto part = [&](int p, const f16x8 (&v)[2][kSteps]) {
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int step = kSteps * p + s;
            fetch((step + 1) & 15, w[(step + 1) & 1]);
            const f16x8(&b)[NJ][2] = w[step & 1];
#pragma unroll
            for (int j = 0; j < NJ; ++j) acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v[1][s], b[j][0], acc[j], 0, 0, 0);
#pragma unroll
            for (int j = 0; j < NJ; ++j) acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v[0][s], b[j][1], acc[j], 0, 0, 0);
#pragma unroll
            for (int j = 0; j < NJ; ++j) acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v[0][s], b[j][0], acc[j], 0, 0, 0);
#pragma unroll
            for (int j = 0; j < NJ; ++j) {  // two LDS reads among three products
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);
            }
        }
    };
    // A part is asked for two parts ahead of its use, the next chunk's first two ahead of a
    // chunk's stores: stores count as loads in flight do, in order, so nothing waits for them
    // but what comes a part later.
    if (c0 + wave < c1) {
        load(c0 + wave, 0, a[0]);
        load(c0 + wave, 1, a[1]);
        fetch(0, w[0]);
    }
    for (int ch = c0 + wave; ch < c1; ch += 8) {
        const int next = min(ch + 8, c1 - 1);
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[j] = f32x16{};
#pragma unroll
        for (int p = 0; p < kParts / 2; ++p) {
            part(p, a[p & 1]);
            __builtin_amdgcn_sched_barrier(0);
            load(ch, p + 2, a[p & 1]);
        }
        // lane: column n0 + 32 j + lane % 32, tokens t0 + 8 q + 4 g + r; what is added to the
        // sums is asked for here, half the products ahead of its use
        const int t0 = ch * 32 + 4 * g, n = n0 + (lane & 31);
        const bool whole = ch * 32 + 32 <= T && n0 + kDxN <= d;
        const int64_t at0 = (int64_t)t0 * d + n;
        f32x16 in[NJ];
        if (dx_in == nullptr) {
#pragma unroll
            for (int j = 0; j < NJ; ++j) in[j] = f32x16{};
        } else if (whole) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
#pragma unroll
                for (int j = 0; j < NJ; ++j) in[j][i] = dx_in[at0 + (int64_t)(8 * (i >> 2) + (i & 3)) * d + 32 * j];
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    const int row = 8 * (i >> 2) + (i & 3);
                    in[j][i] = t0 + row < T && n + 32 * j < d ? dx_in[at0 + (int64_t)row * d + 32 * j] : 0.f;
                }
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int p = kParts / 2; p < kParts; ++p) {
            part(p, a[p & 1]);
            __builtin_amdgcn_sched_barrier(0);
            load(p + 2 < kParts ? ch : next, (p + 2) % kParts, a[p & 1]);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int lo = er[ch * 32 + 8 * q + r], hi = er[ch * 32 + 8 * q + 4 + r];  // wave-uniform
                const int e = g ? hi : lo;
#pragma unroll
                for (int j = 0; j < NJ; ++j) acc[j][4 * q + r] = ldexpf(acc[j][4 * q + r], e + ec[j]) + in[j][4 * q + r];
            }
        if (whole) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
#pragma unroll
                for (int j = 0; j < NJ; ++j) dx[at0 + (int64_t)(8 * (i >> 2) + (i & 3)) * d + 32 * j] = acc[j][i];
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    const int row = 8 * (i >> 2) + (i & 3);
                    if (t0 + row < T && n + 32 * j < d) dx[at0 + (int64_t)row * d + 32 * j] = acc[j][i];
                }
        }
    }
}

// ------------------------------------------------------------------- dw

// A 16-byte load per lane into LDS, written as assembly: the compiler sees no
// LDS write, so it does not wait for the loads in flight before the LDS reads
// of a stage that has landed (it cannot tell the stages apart).  The loop's own
// vmcnt waits and barriers order them.  The LDS address goes in through M0; the
// s_nop covers the M0 write before the load.
__device__ __forceinline__ void dma16_unseen(const void *src, const uint16_t *lds) {
    const uint32_t to = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_void *)lds);
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off" : : "v"(src), "{m0}"(to) : "memory");
}

// 256 experts x 64 NB columns per workgroup, 8 waves of 64 x 32 NB, stages of K = 16
// in a ring (NB = 4, bf16 x: 5 of three terms of dl^T, 24 KB, and x, 8 KB: 160 KB),
// all but one of them in flight.  x lies K-major and is read with transposing LDS reads:
// within each 16 lanes, lane 4a + c receives element c of the 8 bytes that lanes a,
// a+4, a+8, a+12 point at; its 16-byte piece c of row k sits at c ^ 4 (k % 4) (rows
// of 512 bytes) or c ^ 2 (k % 4) (128 bytes, where two rows share the banks).
template <int NX, int NB>
constexpr int dw_stage() { return 3 * kE * kStageK + NX * kStageK * 64 * NB; }  // elements
// Stages in the ring: what one workgroup per CU has room for, or two (NB = 1).
template <int NX, int NB>
constexpr int dw_ring() { return NB == 1 ? (NX == 1 ? 3 : 2) : (NX == 1 ? 5 : 3); }
template <int NX, int NB>
__device__ __forceinline__ void dw_block(int T, int d, const RgWs &ws, const uint16_t *__restrict__ x,
                                         float *__restrict__ out, uint16_t *smem, int z, int S, int y) {
    constexpr int kDwN = 64 * NB, kPieces = kDwN / 8, kTurn = NB == 4 ? 4 : 2;
    constexpr int kA = 3 * kE * kStageK, kX = kStageK * kDwN;  // elements per stage
    constexpr int kBuf = kA + NX * kX, kRing = dw_ring<NX, NB>();
    constexpr int kRowsPer = 64 / kPieces;                // rows of x per load instruction
    constexpr int kXWaves = kStageK / kRowsPer;           // waves that load x
    constexpr int kLoads = 3 + NX;                        // per wave and stage
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const int n0 = y * kDwN;
    const int stages = ws.Tp / kStageK;
    const int s0 = (int)((int64_t)stages * z / S), s1 = (int)((int64_t)stages * (z + 1) / S);
    out += (int64_t)z * kE * d;

    // A: 24 KB in a row, 3 KB per wave; x: some rows of each term (waves behind the last
    // row load the first ones' again, so that every wave counts the same loads)
    const uint16_t *asrc = ws.dlt + wave * 3 * 512 + 8 * lane;
    const int xblk = wave % kXWaves, xk = kRowsPer * xblk + lane / kPieces;
    const int xn = min(n0 + 8 * ((lane % kPieces) ^ (kTurn * (xk & 3))), d - 8);
    auto issue = [&](int st, uint16_t *to) {
        st = min(st, s1 - 1);  // behind the end the last stage again, never read: the loads stay countable
#pragma unroll
        for (int i = 0; i < 3; ++i)
            dma16_unseen(asrc + (int64_t)st * kA + i * 512, to + (wave * 3 + i) * 512);
        const int64_t t = min(st * kStageK + xk, T - 1);
#pragma unroll
        for (int u = 0; u < NX; ++u)
            dma16_unseen(x + (u * (int64_t)T + t) * d + xn, to + kA + u * kX + kRowsPer * xblk * kDwN);
    };
    f32x16 acc[2][NB];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[i][j] = f32x16{};
    const int h = lane >> 4, b = lane & 15;
    const int bk = 8 * (h >> 1) + (b >> 2);  // + 4 for the second read
    auto step = [&](const uint16_t *st) {
        bf16x8 a[3][2];
#pragma unroll
        for (int m = 0; m < 3; ++m)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                a[m][i] = *reinterpret_cast<const bf16x8 *>(st + m * kE * kStageK +
                                                            piece32(wm * 64 + 32 * i + (lane & 31), g));
#pragma unroll
        for (int j = 0; j < NB; ++j)
#pragma unroll
            for (int u = 0; u < NX; ++u) {
                const int col = wn * 32 * NB + 32 * j + 16 * (h & 1) + 4 * (b & 3);
                const uint16_t *p = st + kA + u * kX + bk * kDwN + ((((col >> 3) ^ (kTurn * (bk & 3))) << 3) | (col & 7));
                const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t)p);
                const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t)(p + 4 * kDwN));
                const bf16x8 xb = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
                for (int m = 2 - u; m >= 0; --m)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[m][i], xb, acc[i][j], 0, 0, 0);
            }
    };
#pragma unroll
    for (int i = 0; i < kRing - 1; ++i) issue(s0 + i, smem + i * kBuf);
    int at = 0, next = kRing - 1;
    for (int st = s0; st < s1; ++st) {
        // all but the youngest kRing - 2 stages of this wave's loads have landed and its LDS
        // reads are done; behind the barrier every wave's, and the stage before is no longer read
        constexpr int kLeft = kLoads * (kRing - 2);
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
        __builtin_amdgcn_s_waitcnt((kLeft & 15) | (7 << 4) | ((kLeft >> 4) << 14));
        __builtin_amdgcn_s_barrier();
        __atomic_signal_fence(__ATOMIC_SEQ_CST);
        issue(st + kRing - 1, smem + next * kBuf);
        step(smem + at * kBuf);
        at = at == kRing - 1 ? 0 : at + 1;
        next = next == kRing - 1 ? 0 : next + 1;
    }
    all_landed();  // nothing is on its way into LDS when the workgroup ends
    // lane: column n0 + 32 NB wn + 32 j + lane % 32, experts 64 wm + 32 i + 8 q + 4 g + r
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            const int n = n0 + wn * 32 * NB + 32 * j + (lane & 31);
            if (n >= d) continue;
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    out[(int64_t)(wm * 64 + 32 * i + 8 * q + 4 * g + r) * d + n] = acc[i][j][4 * q + r];
        }
}

struct RgGrid {
    int dx_split, dx_tiles, dw_split, dw_tiles;
};

// Large problems, one launch each.  T = 16384, d = 7168: dx 241 us at its fastest of ten
// launches, 4.0 TB/s of what it reads and writes (267 on average, under the profiler),
// dw 149 us (178), the matrix cores 67% busy at 2.0 GHz; 422 us in all with the terms
// and the sum (fp32 library products: 1247).  On one card each:
// both in one launch 548 against 522 us, dx with two workgroups of 64 columns on a CU
// 551 against 506; dx's columns and tokens in even shares for all 256 CUs (224 have
// work here) 475 against 479, not kept.
constexpr int kLargeNJ = 4, kLargeNB = 4;
__global__ __launch_bounds__(512, 1) void k_rg_dx(int T, int d, const RgWs ws, const RgGrid p,
                                                  const int32_t *__restrict__ er, const float *dx_in, float *dx) {
    __shared__ __attribute__((aligned(1024))) uint16_t smem[2 * 32 * kLargeNJ * kE];
    dx_block<kLargeNJ>(T, d, ws, er, dx_in, dx, smem, blockIdx.x % p.dx_split, p.dx_split, blockIdx.x / p.dx_split);
}
template <int NX>
__global__ __launch_bounds__(512, 1) void k_rg_dw(int T, int d, const RgWs ws, const RgGrid p,
                                                  const uint16_t *__restrict__ x, float *__restrict__ out) {
    __shared__ __attribute__((aligned(1024))) uint16_t smem[dw_ring<NX, kLargeNB>() * dw_stage<NX, kLargeNB>()];
    dw_block<NX, kLargeNB>(T, d, ws, x, out, smem, blockIdx.x % p.dw_split, p.dw_split, blockIdx.x / p.dw_split);
}
// Small ones, both in one launch, the dx blocks first, two workgroups per CU: T = 301,
// d = 896 6.0 us, where the large tiles in two launches took 31; T = d = 2048 22.6 us
// (one workgroup per CU 24.2), about 10 TB/s of terms read out of the L2s.
template <int NX>
__global__ __launch_bounds__(512, 4) void k_rg_small(int T, int d, const RgWs ws, const RgGrid p,
                                                     const int32_t *__restrict__ er, const float *dx_in, float *dx,
                                                     const uint16_t *__restrict__ x, float *__restrict__ out) {
    constexpr int kDwLds = dw_ring<NX, 1>() * dw_stage<NX, 1>(), kDxLds = 2 * 32 * kE;
    __shared__ __attribute__((aligned(1024))) uint16_t smem[kDwLds > kDxLds ? kDwLds : kDxLds];
    const int ndx = p.dx_split * p.dx_tiles, at = (int)blockIdx.x - ndx;
    if (at < 0) dx_block<1>(T, d, ws, er, dx_in, dx, smem, blockIdx.x % p.dx_split, p.dx_split, blockIdx.x / p.dx_split);
    else dw_block<NX, 1>(T, d, ws, x, out, smem, at % p.dw_split, p.dw_split, at / p.dw_split);
}

// dw = the S partial sums added in order, 4 values per thread.
__global__ __launch_bounds__(256) void k_rg_sum(int64_t n4, int S, const f32x4 *__restrict__ part,
                                                f32x4 *__restrict__ dw) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n4) return;
    f32x4 v = part[i];
#pragma unroll 4
    for (int z = 1; z < S; ++z) v += part[(int64_t)z * n4 + i];
    dw[i] = v;
}

}  // namespace

size_t router_grad_ws_bytes(int T, int d, bool x_bf16) { return carve(nullptr, T, d, x_bf16).bytes; }

hipError_t launch_router_grad(const RouterGradArgs &a, void *workspace, hipStream_t s) {
    const int T = a.T, d = a.d;
    const RgWs ws = carve(static_cast<char *>(workspace), T, d, a.x_bf16);
    const int nw = d / 16, nt = ws.Tp / 32;
    const int64_t nx = a.x_bf16 ? 0 : ((int64_t)T * d / 4 + 511) / 512;
    if (nw + nt + nx > INT32_MAX) return hipErrorInvalidValue;
    hipLaunchKernelGGL(k_rg_split, dim3((unsigned)(nw + nt + nx)), dim3(512), 0, s, T, d, nw, nt, a.w, a.dlogits,
                       static_cast<const float *>(a.x_bf16 ? nullptr : a.x), ws);
    const Cut c = cut_of(T, d);
    const RgGrid p{c.dx_split, (d + c.dx_cols - 1) / c.dx_cols, c.dw_split, (d + c.dw_cols - 1) / c.dw_cols};
    const int ndx = p.dx_split * p.dx_tiles, ndw = p.dw_split * p.dw_tiles;
    const dim3 block(512);
    float *out = ws.S == 1 ? a.dw : ws.part;
    const uint16_t *x = a.x_bf16 ? static_cast<const uint16_t *>(a.x) : ws.xs;
#define GO(NX)                                                                                                     \
    do {                                                                                                           \
        if (c.small) {                                                                                             \
            hipLaunchKernelGGL(k_rg_small<NX>, dim3(ndx + ndw), block, 0, s, T, d, ws, p, ws.er, a.dx_in, a.dx, x, \
                               out);                                                                               \
        } else {                                                                                                   \
            hipLaunchKernelGGL(k_rg_dx, dim3(ndx), block, 0, s, T, d, ws, p, ws.er, a.dx_in, a.dx);                \
            hipLaunchKernelGGL(k_rg_dw<NX>, dim3(ndw), block, 0, s, T, d, ws, p, x, out);                          \
        }                                                                                                          \
    } while (0)
    if (a.x_bf16) GO(1);
    else GO(3);
#undef GO
    if (ws.S > 1) {
        const int64_t n4 = (int64_t)kE * d / 4;
        hipLaunchKernelGGL(k_rg_sum, dim3((unsigned)((n4 + 255) / 256)), dim3(256), 0, s, n4, ws.S,
                           reinterpret_cast<const f32x4 *>(ws.part), reinterpret_cast<f32x4 *>(a.dw));
    }
    return hipGetLastError();
}

}  // namespace moe
