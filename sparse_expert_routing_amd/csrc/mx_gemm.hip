// Products grouped by expert on weights in four bits (OCP MX e2m1), activations in
// e4m3 or e2m1, with ragged group sizes; plain, or as the gate and up products of a
// SwiGLU whose result is packed again.
//
// out[r, n] = sum over blocks b of 32 of 2^(sx(r,b) + sw(n,b) - 254) sum_k x(r,k) w(n,k):
// the block-scaled matrix instruction v_mfma_scale_f32_32x32x64_f8f6f4 takes the codes
// and the E8M0 bytes as they are and sums in fp32, so the kernel is the movement of its
// operands.
//   - a persistent grid computes tiles of BM rows x 256 weight rows; a stage is KS of K:
//     the tile's bytes of x and w and a 32-bit word of scales per row and 128 columns;
//   - stages stream global -> LDS (buffer loads with an LDS destination) through a ring
//     of NS slots without a break from tile to tile: the loads run NS stages ahead of the
//     products, over the tile's end, and land under the epilogue;
//   - a stage is KS / 64 steps of products; a step's fragments are read from the LDS
//     during the step before.  Once a stage's last fragments are in registers and the
//     next stage has landed for every wave, the stage's one barrier frees its slot for
//     the loads of stage + NS, half of them under its last step, half under the next
//     stage's first;
//   - 16-byte pieces of a row sit at positions permuted by the row, so that the 32 rows
//     that a fragment read touches spread over the banks;
//   - the weights are the instruction's first operand: the accumulators then hold the
//     transposed block, each lane one row of the output and runs of 4 columns, which
//     the epilogues want (wide stores, a block of 32 columns in two lanes);
//   - bytes past an operand's end, of rows past the group's and of columns past K, are
//     dropped by the buffer's range check and read as zeros; scale bytes past K are
//     masked, since a byte of 255 would make them NaN.
// BM by the average rows of a group; k_mx_few where the tiles are few.
//
// Measured.  512 rows on 256 experts, 2048 x 7168, e4m3 rows: 260 to 290 us, the 1.72 GB of
// weights that have rows at 5.9 TB/s or more (a sixth of them from the Infinity Cache, from
// pass to pass): bound by HBM.  131072 rows on 32 experts, 7168 x 2048, e2m1 rows: 1.19 to
// 1.25 ms, 3.1 to 3.2 PFLOP/s; the gate and up of 131072 rows on 256 experts, 2048 x 7168, e4m3
// rows: 3.75 to 3.99 ms, 2.0 PFLOP/s.  These are bound by the cycles of a tile first, with one
// wave to a SIMD and nothing beside it.  Counted in the kernel at K = 2048, a tile of e2m1 rows
// takes 43500 (some 39600 without the counters): the epilogue 9000, the next tile's setup 4500,
// eight stages 3690 each where the matrix instructions need 2048, waits and barriers 1500 of it
// all; one of e4m3 rows 58500: 8800, 7900 and sixteen stages of 2620.  Without the loads of x the
// cycles are the same.  The card's power is the smaller part: of operands of zeros the product
// takes 1.09 ms, and the whole FFN 4.75 where it takes 5.7 to 5.8.
#include "mx.h"

namespace moe {

namespace {

constexpr int BN = 256;          // weight rows of a tile
constexpr int kPanel = 128;      // columns of a word of scales
constexpr int kTable = 264 * 4;  // row tiles before every fourth group
constexpr int kQueue = 4;        // tiles between the loads and the products, at most NS + 1
constexpr int kGroupM = 8;       // row tiles side by side
// An offset past the end of every resource (nothing may be added to it).
constexpr uint32_t kOob = 0xFFFF0000u;

enum { MX_BF16 = 0, MX_F32 = 1, MX_SWIGLU = 2 };

// Large tiles (BM = 256): four waves of 128 x 128, all 512 registers of a SIMD's lanes each
// (eight waves of 64 x 128 read each fragment once more: e2m1 activations 14 % slower, e4m3
// 1 % faster); e2m1 rows are loaded by 128 bytes, 256 of K, since the L2s serve about one
// request per clock and channel, of 64 bytes or of 128.  Small ones: two workgroups to a CU,
// so that one's loads run under the other's waits, 128 of K.
template <int AF, int BM>
struct Cfg {
    static constexpr int W = 4;                                                 // waves
    static constexpr int WGS = BM == 256 ? 1 : 2;                               // workgroups to a CU
    static constexpr int KS = BM == 256 && AF == kMxE2M1 ? 256 : 128;           // K of a stage
    static constexpr int KP = KS / kPanel;                                      // its words of scales per row
    static constexpr int S = KS / 64;                                           // its steps
    static constexpr int ARB = AF == kMxE2M1 ? KS / 2 : KS, BRB = KS / 2;       // bytes of a row in a stage
    static constexpr int KB = W * 1024;                                         // bytes of a load of all waves
    static constexpr int AI = BM * ARB / KB > 0 ? BM * ARB / KB : 1;            // loads of x, of w per wave and stage
    static constexpr int BI = BN * BRB / KB;
    static constexpr int AW = (BM > 64 ? BM : 64) * 4, BW = BN * 4;             // bytes of a panel's scales
    static constexpr int WI = 2;                                                // loads of a panel's scales
    static constexpr int SLOT = (AI + BI) * KB + KP * (AW + BW);
    static constexpr int L = AI + BI + WI * KP;                                 // loads per wave and stage
    static constexpr int LF = S == 4 ? L - 2 * (L / 3) : (L + 1) / 2;           // of them under the last step
    static constexpr bool LIST = BM == 256;                                     // tiles from a list
    static constexpr int LDS = 160 * 1024 / WGS, REST = kTable + W * kQueue * 16;
    static constexpr int FIT = (LDS - REST) / SLOT, NS = FIT < 3 ? FIT : 3;
    static constexpr int WM = BM >= 64 ? W / 2 : 1, WN = W / WM;                // waves over rows and weight rows
    static constexpr int TM = BM / 32 / WM, TN = BN / 32 / WN;                  // 32 x 32 blocks of a wave
    static_assert((NS == 3 && S == 2) || (NS == 2 && S == 4), "which steps load");
    static_assert(TM == 4 || TM == 1, "the products' loops by the row blocks with rows in them");
    static_assert(NS >= 2 && NS + 1 <= kQueue && (NS - 1) * L < 64, "the ring, and the counter of loads");
};

// t / d for t below 2^31: the high half of a product (d = 1: m = 0).
struct Div {
    uint32_t m, s;
};
template <class D>
__device__ __forceinline__ int of(const D &d, int t) {
    return d.m == 0 ? t : (int)(__umulhi((uint32_t)t, d.m) >> d.s);
}
Div div_by(uint32_t d) {
    if (d == 1) return Div{0, 0};
    uint32_t l = 1;
    while ((1ull << l) < d) ++l;
    return Div{(uint32_t)((1ull << (31 + l)) / d + 1), l - 1};
}

struct MxParams {
    int G, M, N, K;
    Div nt, gnt, by_k;  // column tiles; those of kGroupM row tiles; k
    const uint8_t *x;
    const uint32_t *xs;
    int x_rows, xs_rows;  // rows of x, of its scales (xs_rows = M: in the product's own order)
    bool xs_gathered;
    const i32x4 *tiles;  // large tiles: k_mx_tiles's list
    const int32_t *row_src, *offsets;
    const uint8_t *w0, *w1;
    const uint32_t *s0, *s1;
    void *out;
    uint8_t *h;
    uint32_t *hs;
};

typedef __attribute__((address_space(3))) void lds_void_t;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void *p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ const void *uniform(const void *p) {
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return reinterpret_cast<const void *>(((uint64_t)hi << 32) | lo);
}
// 16 (4) bytes per lane to consecutive places of the LDS.
__device__ __forceinline__ void to_lds16(__amdgpu_buffer_rsrc_t r, uint32_t off, uint8_t *lds) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_t *)(lds), 16, off, 0, 0, 0);
}
__device__ __forceinline__ void to_lds4(__amdgpu_buffer_rsrc_t r, uint32_t off, uint8_t *lds) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_t *)(lds), 4, off, 0, 0, 0);
}
// Waits until at most N vector memory operations of this wave are under way, and for
// its LDS reads.
template <int N>
__device__ __forceinline__ void wait_loads() {
    static_assert(N >= 0 && N < 64, "the counter's range");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
}

// Position of the 16-byte piece c of tile row `row`: rows of 128 bytes (8 pieces), and
// of 64 (4 pieces: any 8 neighbouring rows of the 32 meet all positions of 128 bytes,
// any 16 those of 256).
template <int BYTES>
__device__ __forceinline__ int swizzle(int row) {
    return BYTES == 128 ? (row & 7) ^ ((row >> 3) & 1) : ((row >> 2) & 1) | ((((row >> 1) ^ (row >> 3)) & 1) << 1);
}

// A fragment: 32 rows by the step's 64 of K.  Of those lane half g takes 16 g .. + 15 and
// 32 + 16 g .. + 15 of e4m3, 32 g .. + 31 of e2m1.  The pieces of a row's steps lie where
// bits 5 and 6 of the first one's address are turned over, whatever the row's swizzle.
template <int F>
struct Frag;
template <>
struct Frag<kMxE2M1> {
    i32x4 v;
    static constexpr int kStep = 32;
    // at: the first step's piece of the wave's first rows; more: bytes from those to the
    // fragment's (of a multiple of 16 rows, which share a swizzle)
    __device__ __forceinline__ void read(const uint8_t *lds, uint32_t at, int step, int more) {
        v = *reinterpret_cast<const i32x4 *>(lds + (at ^ (uint32_t)(kStep * step)) + more);
    }
    __device__ __forceinline__ i32x8 operand() const { return i32x8{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }
};
template <>
struct Frag<kMxE4M3> {
    i32x8 v;
    static constexpr int kStep = 64;
    __device__ __forceinline__ void read(const uint8_t *lds, uint32_t at, int step, int more) {
        const i32x4 lo = *reinterpret_cast<const i32x4 *>(lds + (at ^ (uint32_t)(kStep * step)) + more);
        const i32x4 hi = *reinterpret_cast<const i32x4 *>(lds + (at ^ (uint32_t)(kStep * step + 32)) + more);
        v = i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    }
    __device__ __forceinline__ i32x8 operand() const { return v; }
};

// acc += w x^T of a 32 x 32 block and 64 of K; byte 2 HALF of a lane's scale word is
// that of its row and block.
template <int AF, int HALF, class W, class X>
__device__ __forceinline__ f32x16 mma(const W &w, const X &x, f32x16 c, uint32_t sw, uint32_t sx) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w.operand(), x.operand(), c, 4, AF == kMxE2M1 ? 4 : 0, 2 * HALF,
                                                           (int)sw, 2 * HALF, (int)sx);
}
template <int I>
struct Int {
    static constexpr int value = I;
};

__device__ __forceinline__ float swiglu(float g, float u) {
    return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * g)) * u;
}

// An accumulator's value, read where it is used: left to the compiler, all 256 of a lane
// are copied out of the accumulation registers at once and spill.  The caller has waited
// for the matrix instructions (settle).
__device__ __forceinline__ float acc_read(float x) {
    float r;
    asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(r) : "a"(x));
    return r;
}
// Lanes 16 .. 31 and 48 .. 63 of a with lanes 0 .. 15 and 32 .. 47 of b: lanes of row r
// and r + 16 that held parts a and b of their rows then hold a and b of row r in a, of row
// r + 16 in b.
__device__ __forceinline__ void swap16(uint32_t (&a)[4], uint32_t (&b)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const auto x = __builtin_amdgcn_permlane16_swap(a[i], b[i], false, false);
        a[i] = x[0];
        b[i] = x[1];
    }
}
// The longest matrix instruction's result may be read 19 wait states behind it.
__device__ __forceinline__ void settle() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_nop 15\n\ts_nop 15");
    __builtin_amdgcn_sched_barrier(0);
}

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return min(max(v, lo), hi); }

// The launch's arguments, read anew from where they lie: kept in registers from a kernel's
// start to its end they crowd out the products' (a tile needs them twice).
typedef const __attribute__((address_space(4))) MxParams *Args;
__device__ __forceinline__ Args args() {
    Args q = reinterpret_cast<Args>(reinterpret_cast<uintptr_t>(__builtin_amdgcn_kernarg_segment_ptr()));
    asm volatile("" : "+s"(q));
    return q;
}

template <int AF, int BM, int EPI>
__global__ __launch_bounds__((64 * Cfg<AF, BM>::W), (Cfg<AF, BM>::WGS)) void k_mx_gemm(MxParams p) {
    using C = Cfg<AF, BM>;
    constexpr bool DUAL = EPI == MX_SWIGLU;
    constexpr int BC = DUAL ? BN / 2 : BN;  // output columns of a tile
    constexpr int TM = C::TM, TN = C::TN, NS = C::NS, L = C::L, LF = C::LF, AI = C::AI, BI = C::BI, KP = C::KP, S = C::S, KS = C::KS;
    constexpr int W = C::W, KB = C::KB, ARB = C::ARB, BRB = C::BRB, AKB = AF == kMxE2M1 ? 32 : 16;  // AKB: K of a 16-byte piece
    // stores of an epilogue, at least (every lane issues them all)
    constexpr int kStores = DUAL ? TM * TN / 2 : EPI == MX_BF16 ? 2 * TM * TN : 4 * TM * TN;
    // (one array: beside a second one the compiler has every LDS read wait for the loads
    // under way)
    __shared__ __attribute__((aligned(1024))) uint8_t ring[NS * C::SLOT + C::REST];
    int *const first = reinterpret_cast<int *>(ring + NS * C::SLOT);
    i32x4 *const queue = reinterpret_cast<i32x4 *>(ring + NS * C::SLOT + kTable) + kQueue * (threadIdx.x >> 6);  // the wave's own

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / C::WN, wn = wave % C::WN, g = lane >> 5, l31 = lane & 31;
    const int nk = (p.K + KS - 1) / KS, tail = p.K % KS;
    const int NT = (p.N + BC - 1) / BC;
    const uint32_t xrow = (uint32_t)(AF == kMxE2M1 ? p.K / 2 : p.K), wrow = (uint32_t)p.K / 2;  // bytes

    // first[i]: row tiles of the groups before 4 i
    // (constant memory: read through the scalar cache, apart from the loads under way)
    auto tiles_of = [&](auto offsets, int M, int e, int &lo, int &hi) {
        lo = clampi(offsets[e], 0, M);
        hi = clampi(offsets[e + 1], lo, M);
        return (hi - lo + BM - 1) / BM;
    };
    typedef const __attribute__((address_space(4))) i32x4 *List;
    const List list = reinterpret_cast<List>(reinterpret_cast<uintptr_t>(p.tiles));
    int total;
    if constexpr (C::LIST) {
        total = list[0][0] / kGroupM * kGroupM * NT;
    } else {
        int *const sums = reinterpret_cast<int *>(ring);
        int s = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            int lo, hi;
            if (4 * tid + i < p.G) s += tiles_of(p.offsets, p.M, 4 * tid + i, lo, hi);
        }
        const int incl = wave_incl_scan(s);
        if (lane == 63) sums[wave] = incl;
        __syncthreads();
        int at = incl - s;
        for (int w = 0; w < wave; ++w) at += sums[w];
        first[tid] = at;
        if (tid == 255) first[256] = at + s;
        __syncthreads();
        // (offsets that do not ascend may make more of them than there can be)
        total = (int)min((int64_t)__builtin_amdgcn_readfirstlane(first[256]) * NT, (int64_t)(0x7fffffff - (1 << 20)));
    }
    const int P = gridDim.x;

    // Loads of x (w): instruction i of wave w fills KB W i + w of the tile, lane l its l-th
    // piece; the piece of the row that belongs there is the same for every i.
    constexpr int ARPI = 1024 / ARB, BRPI = 1024 / BRB;  // rows of an instruction
    const int apiece = (lane & (ARB / 16 - 1)) ^ swizzle<ARB>(ARPI * (wave & 1) + lane / (ARB / 16));
    const int bpiece = (lane & (BRB / 16 - 1)) ^ swizzle<BRB>(BRPI * (wave & 1) + lane / (BRB / 16));
    // a lane whose piece lies past K in the last, partial stage
    const bool acut = tail && apiece * AKB >= tail, bcut = tail && bpiece * 32 >= tail;
    const uint64_t words_step = (uint64_t)p.G * p.N;  // of w's scales, from panel to panel
    // w: rows past the matrix lie past the resource's end
    constexpr int BH = DUAL ? BI / 2 : BI;  // instructions of one matrix
    const uint32_t boff = (uint32_t)(BRPI * wave + lane / (BRB / 16)) * wrow + (uint32_t)bpiece * 16u, bstep = W * BRPI * wrow;

    // ------------------------------------------------ the loads' side: a tile and its stage
    int lt, lkp = 0, lcount = 0;  // lcount: tiles begun
    uint32_t aoff[AI], soff = kOob, wsoff = kOob;  // soff, wsoff: of the scales that the lane loads
    // where the stage begins, and the bytes from there on (0 behind the last tile: the
    // loads fetch nothing, and the count of them stays the same)
    const uint8_t *pa, *pb0, *pb1;
    const uint32_t *pas, *pbs;
    uint32_t a_left, b_left, as_left, bs_left;
    // A list's entry of tile t, asked for a tile ahead.  Row tiles go by eights, side by side
    // over the columns, so that those that read one slice of the weights run together.
    i32x4 ahead = {0, 0, 0, 0};
    auto entry = [&](int t) {
        const int wide = kGroupM * NT;
        return list[1 + of(p.gnt, t) * kGroupM + ((t - of(p.gnt, t) * wide) & (kGroupM - 1))];
    };
    auto setup = [&](int t) {
        const Args q = args();
        int lane = threadIdx.x & 63;
        asm volatile("" : "+v"(lane));  // what follows of it is computed here, not kept
        const int asub = lane / (ARB / 16), apiece = (lane & (ARB / 16 - 1)) ^ swizzle<ARB>(ARPI * (wave & 1) + asub);
        const int M = q->M, N = q->N, x_rows = q->x_rows, wide = (N + BC - 1) / BC;
        const int32_t *const row_src = q->row_src;
        int e, m0, rows, ln0;
        if constexpr (C::LIST) {
            e = ahead[2];
            m0 = ahead[0];
            rows = ahead[1];
            ln0 = (t - of(q->gnt, t) * (kGroupM * wide)) / kGroupM * BC;
            if (t + P < total) ahead = entry(t + P);
        } else {
            const auto offsets = reinterpret_cast<const __attribute__((address_space(4))) int32_t *>(reinterpret_cast<uintptr_t>(q->offsets));
            const int rt = of(q->nt, t);
            // the group that row tile rt lies in: by sixteens, by fours, among four
            const int q16 = __popcll(__ballot(first[4 * lane] <= rt)) - 1;
            const int q4 = __popcll(__ballot(lane < 4 && first[4 * q16 + (lane & 3)] <= rt)) - 1;
            e = __builtin_amdgcn_readfirstlane(4 * (4 * q16 + q4));
            int f0 = __builtin_amdgcn_readfirstlane(first[4 * q16 + q4]), lo, hi;
            int n = tiles_of(offsets, M, e, lo, hi);
            while (rt >= f0 + n) {
                f0 += n;
                e = __builtin_amdgcn_readfirstlane(e + 1);
                n = tiles_of(offsets, M, e, lo, hi);
            }
            // a group's tiles: kGroupM row tiles side by side, so that those that read one
            // slice of the weights run together
            const int u = t - wide * f0, j = of(q->gnt, u), gm = min(kGroupM, n - kGroupM * j), within = u - j * kGroupM * wide;
            const int col = (int)(((float)within + 0.5f) * (1.0f / (float)gm));  // within / gm, exact below 2^20
            m0 = __builtin_amdgcn_readfirstlane(lo + (kGroupM * j + within - col * gm) * BM);
            rows = min(__builtin_amdgcn_readfirstlane(hi) - m0, BM);
            ln0 = __builtin_amdgcn_readfirstlane(col * BC);
        }
        const int m_end = m0 + rows;
        queue[lcount & (kQueue - 1)] = i32x4{m0, rows, ln0, 0};
        ++lcount;
        // x: from the tile's first row, or all of it where rows are gathered
        pa = static_cast<const uint8_t *>(uniform(row_src ? q->x : q->x + (uint64_t)m0 * xrow));
        a_left = (row_src ? (uint32_t)x_rows : (uint32_t)rows) * xrow;
        pas = q->xs;
        as_left = (uint32_t)q->xs_rows * 4u;
        const uint64_t w_first = (uint64_t)e * N + ln0;
        pb0 = static_cast<const uint8_t *>(uniform(q->w0 + w_first * wrow));
        if (DUAL) pb1 = static_cast<const uint8_t *>(uniform(q->w1 + w_first * wrow));
        pbs = static_cast<const uint32_t *>(uniform((DUAL && wave >= 2 ? q->s1 : q->s0) + w_first));
        b_left = (uint32_t)min(N - ln0, BC) * wrow;
        bs_left = (uint32_t)min(N - ln0, BC) * 4u;
        const int tr_words = (64 * wave + lane) & (BM - 1);
        int row[AI + 1];
#pragma unroll
        for (int i = 0; i <= AI; ++i) {
            const int tr = i < AI ? ARPI * (W * i + wave) + asub : tr_words;
            row[i] = tr < BM && m0 + tr < m_end ? m0 + tr : -1;
        }
        if (row_src) {
            int src[AI + 1];
#pragma unroll
            for (int i = 0; i <= AI; ++i) src[i] = row_src[max(row[i], m0)];
#pragma unroll
            for (int i = 0; i <= AI; ++i) {
                const int token = of(q->by_k, src[i] & 0x7fffffff);
                row[i] = row[i] >= 0 && src[i] >= 0 && token < x_rows ? token : -1;
            }
        }
        if (q->xs_gathered) row[AI] = tr_words < BM && m0 + tr_words < m_end ? m0 + tr_words : -1;
        const uint32_t base = row_src ? 0u : (uint32_t)m0;
#pragma unroll
        for (int i = 0; i < AI; ++i) aoff[i] = row[i] >= 0 ? ((uint32_t)row[i] - base) * xrow + (uint32_t)apiece * 16u : kOob;
        soff = row[AI] >= 0 ? (uint32_t)row[AI] * 4u : kOob;
        const int r = (64 * wave + lane) & (BC - 1);
        wsoff = ln0 + r < N ? (uint32_t)r * 4u : kOob;
    };

    // Load i of the stage into a slot.
    auto load_part = [&](uint32_t slot, int i) {
        const bool last = lkp == nk - 1;
        if (i < AI) {
            to_lds16(rsrc(pa, a_left), last && acut ? kOob : aoff[i], ring + (slot + W * i * 1024 + wave * 1024));
        } else if (i < AI + BI) {
            const int k = i - AI;
            to_lds16(rsrc(k >= BH ? pb1 : pb0, b_left), last && bcut ? kOob : boff + (uint32_t)(k % BH) * bstep,
                     ring + (slot + AI * KB + W * k * 1024 + wave * 1024));
        } else {
            // (the second panel of a stage that has one: none past K)
            const int h = (i - AI - BI) / C::WI;
            const bool none = h > 0 && (lkp * KP + h) * kPanel >= p.K;
            const uint32_t words = slot + (AI + BI) * KB + h * (C::AW + C::BW);
            if (((i - AI - BI) & 1) == 0) {
                to_lds4(rsrc(pas + (uint64_t)(h * p.xs_rows), none ? 0u : as_left), soff, ring + (words + (wave * 256 & (C::AW - 1))));
            } else {
                to_lds4(rsrc(pbs + (uint64_t)h * words_step, none ? 0u : bs_left), wsoff, ring + (words + C::AW + wave * 256));
            }
        }
    };
    auto next_stage = [&]() {
        if (++lkp < nk) {
            pa += ARB;
            pb0 += BRB;
            if (DUAL) pb1 += BRB;
            pas += (uint64_t)p.xs_rows * KP;
            pbs += words_step * KP;
            if (a_left) {
                a_left -= ARB;
                b_left -= BRB;
            }
        } else {
            lkp = 0;
            lt += P;
            // (the list's last eight may end in tiles of no rows)
            if constexpr (C::LIST) {
                while (lt < total && ahead[1] == 0) {
                    lt += P;
                    if (lt < total) ahead = entry(lt);
                }
            }
            if (lt < total) setup(lt);
            else a_left = b_left = as_left = bs_left = 0;
        }
    };

    // Every XCD's P / 8 workgroups take P / 8 consecutive tiles at a time, or an eighth of
    // fewer ones: one L2 shares their operands (2999 rows on 60 ragged groups, 1000 x 1376, 316
    // tiles: 19.3 us; 22.3 with neighbouring tiles on different XCDs).
    const int share = min(P, total + 7) >> 3;
    if ((int)(blockIdx.x >> 3) >= share) return;
    lt = (blockIdx.x & 7) * share + (blockIdx.x >> 3);
    if constexpr (C::LIST) {
        for (; lt < total; lt += P) {
            ahead = entry(lt);
            if (ahead[1]) break;
        }
    }
    if (lt >= total) return;
    setup(lt);
    for (int s = 0; s < NS; ++s) {
#pragma unroll
        for (int i = 0; i < L; ++i)
            if (NS == 2 || s + 1 < NS || i < LF) load_part((uint32_t)(s * C::SLOT), i);
        if (s + 1 < NS) next_stage();
    }

    // ------------------------------------------------ the products' side
    // Row blocks of 32 alternate between the waves, so that a short tile costs both half.
    Frag<AF> a0[TM];  // the next stage's first step
    Frag<kMxE2M1> b0[TN];
    uint32_t wa[KP][TM], wb[KP][TN];  // words of the next stage
    auto arow = [&](int i) { return 32 * (C::WM * i + wm) + l31; };
    // a wave's weight rows: TN blocks in a row, or half of them of the gate's columns and
    // half of the up's
    constexpr int BJ = DUAL ? TN / 2 : TN;
    const int brow0 = wn * (BC / C::WN) + l31;
    auto brows = [&](int j) { return (j / BJ) * BC + 32 * (j % BJ); };
    const uint32_t a_at = arow(0) * ARB + ((g ^ swizzle<ARB>(arow(0))) * 16), b_at = AI * KB + brow0 * BRB + ((g ^ swizzle<BRB>(brow0)) * 16);
    const uint32_t words0 = (AI + BI) * KB + l31 * 4;
    auto words_a = [&](uint32_t slot, int i) {
#pragma unroll
        for (int h = 0; h < KP; ++h)
            wa[h][i] = *reinterpret_cast<const uint32_t *>(ring + (words0 + (slot + wm * 128)) + (h * (C::AW + C::BW) + C::WM * i * 128));
    };
    auto words_b = [&](uint32_t slot, int j) {
#pragma unroll
        for (int h = 0; h < KP; ++h)
            wb[h][j] = *reinterpret_cast<const uint32_t *>(ring + (words0 + (slot + wn * (BC / C::WN) * 4)) +
                                                           (h * (C::AW + C::BW) + C::AW + brows(j) * 4));
    };
    auto read_a = [&](Frag<AF> &f, uint32_t slot, int i, int step) { f.read(ring, a_at + slot, step, C::WM * 32 * i * ARB); };
    auto read_b = [&](Frag<kMxE2M1> &f, uint32_t slot, int j, int step) { f.read(ring, b_at + slot, step, brows(j) * BRB); };
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    wait_loads<NS == 2 ? L : (NS - 2) * L + LF>();
    __builtin_amdgcn_s_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
#pragma unroll
    for (int i = 0; i < TM; ++i) { read_a(a0[i], 0, i, 0); words_a(0, i); }
#pragma unroll
    for (int j = 0; j < TN; ++j) { read_b(b0[j], 0, j, 0); words_b(0, j); }

    uint32_t at = 0;  // the stage's slot
    int count = 0;
    // The slot that the stage before left.  Its loads' second half follows in the next
    // stage, behind a tile's stores at its end, where NS - 2 stages are there meanwhile; in a
    // ring of two slots it goes ahead of the stores.
    uint32_t before = (NS - 1) * C::SLOT;
    for (; count < lcount; ++count) {  // (the loads have begun the tile that is next, if there is one)
        const i32x4 place = queue[count & (kQueue - 1)];
        const int cm0 = __builtin_amdgcn_readfirstlane(place[0]), rows = __builtin_amdgcn_readfirstlane(place[1]);
        const int cn0 = __builtin_amdgcn_readfirstlane(place[2]);
        f32x16 acc[TM][TN];
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

        // the tile's stages, NB row blocks of the wave with rows in them
        auto run = [&](auto nb) {
            constexpr int NB = decltype(nb)::value;
            constexpr int X = TM * TN;  // places of a step's products
            uint32_t sa[KP][TM], sb[KP][TN];
            Frag<AF> a1[TM];
            Frag<kMxE2M1> b1[TN];
            // Step st's products, in between: the fragments of step sn from a slot (with a
            // stage's words for its first), and loads lo .. hi - 1 of the loads' stage
            auto step = [&](auto st_, auto sn_, uint32_t from, uint32_t into, auto lo_, auto hi_) {
                constexpr int st = decltype(st_)::value, sn = decltype(sn_)::value, lo = decltype(lo_)::value, hi = decltype(hi_)::value;
                constexpr int span = hi > lo ? hi - lo : 1;
#pragma unroll
                for (int x = 0; x < X; ++x) {
#pragma unroll
                    for (int r = 0; r < TM + TN; ++r)
                        if (r * X / (TM + TN) == x) {
                            if (r < TN) {
                                if (sn == 0 || NB > 0) read_b((sn & 1 ? b1 : b0)[r], from, r, sn);
                                if (sn == 0) words_b(from, r);
                            } else {
                                if (sn == 0 || r - TN < NB) read_a((sn & 1 ? a1 : a0)[r - TN], from, r - TN, sn);
                                if (sn == 0) words_a(from, r - TN);
                            }
                        }
                    __builtin_amdgcn_sched_barrier(0);
                    if (x / TN < NB)
                        acc[x / TN][x % TN] = mma<AF, (st & 1)>((st & 1 ? b1 : b0)[x % TN], (st & 1 ? a1 : a0)[x / TN], acc[x / TN][x % TN],
                                                               sb[st / 2][x % TN], sa[st / 2][x / TN]);
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int i = lo; i < hi; ++i)
                        if ((i - lo) * X / span == x) load_part(into, i);
                    __builtin_amdgcn_sched_barrier(0);
                }
            };
            for (int kp = 0; kp < nk; ++kp) {
                const uint32_t slot = at, next = at + C::SLOT == NS * C::SLOT ? 0 : at + C::SLOT;
                at = next;
#pragma unroll
                for (int h = 0; h < KP; ++h) {
                    // the panel's blocks inside K
                    const int blocks = kp == nk - 1 && tail ? (tail - h * kPanel) / 32 : 4;
                    const uint32_t mask = blocks >= 4 ? ~0u : blocks <= 0 ? 0u : (1u << (8 * blocks)) - 1u;
#pragma unroll
                    for (int i = 0; i < TM; ++i) sa[h][i] = (wa[h][i] & mask) >> (8 * g);
#pragma unroll
                    for (int j = 0; j < TN; ++j) sb[h][j] = (wb[h][j] & mask) >> (8 * g);
                }
                if constexpr (NS == 2) {
                    if (kp > 0) {
#pragma unroll
                        for (int i = LF; i < LF + (L - LF) / 2; ++i) load_part(before, i);
                    }
                    step(Int<0>{}, Int<1>{}, slot, before, Int<0>{}, Int<0>{});
                } else {
                    step(Int<0>{}, Int<1>{}, slot, before, Int<LF>{}, Int<L>{});
                }
                if constexpr (S == 4) {
                    if (kp > 0) {
#pragma unroll
                        for (int i = LF + (L - LF) / 2; i < L; ++i) load_part(before, i);
                    }
                    step(Int<1>{}, Int<2>{}, slot, before, Int<0>{}, Int<0>{});
                    step(Int<2>{}, Int<3>{}, slot, before, Int<0>{}, Int<0>{});
                }
                // (the products stay on this side of what branches below)
#pragma unroll
                for (int i = 0; i < NB; ++i)
#pragma unroll
                    for (int j = 0; j < TN; ++j) asm volatile("" : "+a"(acc[i][j]));
                // the slot's fragments are in registers, the next stage has landed; behind a
                // tile's first stage's loads lie the epilogue's stores
                __atomic_signal_fence(__ATOMIC_SEQ_CST);
                if (kp == 0 && count > 0) wait_loads<((NS - 2) * L + kStores < 63 ? (NS - 2) * L + kStores : 63)>();
                else wait_loads<(NS - 2) * L>();
                __builtin_amdgcn_s_barrier();
                __atomic_signal_fence(__ATOMIC_SEQ_CST);
                next_stage();
                step(Int<S - 1>{}, Int<0>{}, next, slot, Int<0>{}, Int<LF>{});
                before = slot;
            }
        };
        const int nb = ((rows + 31) / 32 - wm + C::WM - 1) / C::WM;
        if constexpr (TM == 4) {
            if (nb >= 4) run(Int<4>{});
            else if (nb == 3) run(Int<3>{});
            else if (nb == 2) run(Int<2>{});
            else if (nb == 1) run(Int<1>{});
            else run(Int<0>{});
        } else {
            run(Int<TM>{});
        }
        if constexpr (NS == 2) {
#pragma unroll
            for (int i = LF; i < L; ++i) load_part(before, i);
        }
        settle();

        // A lane holds rows cm0 + arow(i), and of each 32-column block the columns
        // 8 q + 4 g .. + 3; lanes l and l + 32 hold one row.
        const Args o = args();
        const int N = o->N;
        const int odd = (lane >> 4) & 1;
        if constexpr (DUAL) {
            const uint32_t hrow = (uint32_t)(AF == kMxE2M1 ? N / 2 : N);
            const __amdgpu_buffer_rsrc_t rh = rsrc(uniform(o->h + (uint64_t)cm0 * hrow), (uint32_t)rows * hrow);
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                const uint32_t row = (uint32_t)arow(i);
#pragma unroll
                for (int j = 0; j < TN / 2; ++j) {
                    __builtin_amdgcn_sched_barrier(0);  // one block's accumulators at a time
                    const int col = cn0 + wn * (BC / C::WN) + 32 * j;
                    float h[16];
                    uint32_t m = 0;
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        h[r] = swiglu(acc_read(acc[i][j][r]), acc_read(acc[i][j + TN / 2][r]));
                        m = max(m, __float_as_uint(h[r]) & 0x7fffffffu);
                    }
                    const auto both = __builtin_amdgcn_permlane32_swap(m, m, false, false);
                    const uint32_t byte = mx_block_byte<AF>(max(both[0], both[1]));
                    const float inv = e8m0_inverse(byte == 255u ? 127u : byte);
#pragma unroll
                    for (int r = 0; r < 16; ++r) h[r] = byte == 255u ? 0.f : h[r] * inv;
                    const bool ok = row < (uint32_t)rows && col < N;
                    if constexpr (AF == kMxE4M3) {
                        uint32_t w[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q) w[q] = e4m3x4(h[4 * q], h[4 * q + 1], h[4 * q + 2], h[4 * q + 3]);
                        // lane l takes the block's first 16 columns of the row, l + 32 the others
                        const auto lo = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
                        const auto hi = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
                        __builtin_amdgcn_raw_buffer_store_b128(i32x4{(int)lo[0], (int)lo[1], (int)hi[0], (int)hi[1]}, rh,
                                                               ok ? row * hrow + (uint32_t)(col + 16 * g) : kOob, 0, 0);
                    } else {
                        uint32_t w[2] = {0u, 0u};
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            w[q] = e2m1x2<0>(w[q], h[8 * q], h[8 * q + 1]);
                            w[q] = e2m1x2<1>(w[q], h[8 * q + 2], h[8 * q + 3]);
                            w[q] = e2m1x2<2>(w[q], h[8 * q + 4], h[8 * q + 5]);
                            w[q] = e2m1x2<3>(w[q], h[8 * q + 6], h[8 * q + 7]);
                        }
                        const auto x = __builtin_amdgcn_permlane32_swap(w[0], w[1], false, false);
                        typedef int i32x2 __attribute__((ext_vector_type(2)));
                        const i32x2 v = {(int)((x[0] & 0xffffu) | (x[1] << 16)), (int)((x[0] >> 16) | (x[1] & 0xffff0000u))};
                        __builtin_amdgcn_raw_buffer_store_b64(v, rh, ok ? row * hrow + (uint32_t)(col / 2 + 8 * g) : kOob, 0, 0);
                    }
                    if (ok && g == 0)
                        reinterpret_cast<uint8_t *>(o->hs)[((uint64_t)(col / kPanel) * o->M + cm0 + row) * 4 + (col / 32) % 4] = (uint8_t)byte;
                }
            }
        } else {
            constexpr uint32_t ES = EPI == MX_BF16 ? 2 : 4;
            const uint32_t orow = (uint32_t)N * ES;
            const __amdgpu_buffer_rsrc_t ro = rsrc(uniform(static_cast<uint8_t *>(o->out) + (uint64_t)cm0 * orow), (uint32_t)rows * orow);
            const bool wide = orow % 16 == 0 && reinterpret_cast<uintptr_t>(o->out) % 16 == 0;
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                const uint32_t row = (uint32_t)arow(i);
                // (rows past the tile's begin at the resource's end: with a column's offset
                // on top, at most 2^31 + 2^23, they stay behind it, where kOob would wrap)
                const uint32_t at0 = min(row, (uint32_t)rows) * orow;
                auto at16 = [&](int h) {  // of the row that a lane holds a part of behind swap16
                    return min(row - (uint32_t)(16 * odd) + (uint32_t)(16 * h), (uint32_t)rows) * orow;
                };
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    __builtin_amdgcn_sched_barrier(0);  // one block's accumulators at a time
                    const int col = cn0 + wn * (BN / C::WN) + 32 * j;
                    if (wide) {
                        if constexpr (EPI == MX_BF16) {
                            uint32_t w[4][2];
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                w[q][0] = pack_bf16x2(acc_read(acc[i][j][4 * q]), acc_read(acc[i][j][4 * q + 1]));
                                w[q][1] = pack_bf16x2(acc_read(acc[i][j][4 * q + 2]), acc_read(acc[i][j][4 * q + 3]));
                            }
                            // columns 16 h + 8 g .. + 7 of a row in one lane, v[h]; then, with the
                            // neighbouring 16 lanes, all 32 columns of 16 rows to a store: 64 bytes
                            // of a row together
                            uint32_t v[2][4];
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const auto x = __builtin_amdgcn_permlane32_swap(w[2 * h][0], w[2 * h + 1][0], false, false);
                                const auto y = __builtin_amdgcn_permlane32_swap(w[2 * h][1], w[2 * h + 1][1], false, false);
                                v[h][0] = x[0]; v[h][1] = y[0]; v[h][2] = x[1]; v[h][3] = y[1];
                            }
                            swap16(v[0], v[1]);
                            const int c = col + 16 * odd + 8 * g;
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                __builtin_amdgcn_raw_buffer_store_b128(i32x4{(int)v[h][0], (int)v[h][1], (int)v[h][2], (int)v[h][3]}, ro,
                                                                       c < N ? at16(h) + (uint32_t)c * 2u : kOob, 0, 0);
                        } else {
                            // (two runs of 8 columns, 16 rows of both to a store)
#pragma unroll
                            for (int q = 0; q < 4; q += 2) {
                                uint32_t v[2][4];
#pragma unroll
                                for (int h = 0; h < 2; ++h)
#pragma unroll
                                    for (int r = 0; r < 4; ++r) v[h][r] = __float_as_uint(acc_read(acc[i][j][4 * (q + h) + r]));
                                swap16(v[0], v[1]);
                                const int c = col + 8 * q + 8 * odd + 4 * g;
#pragma unroll
                                for (int h = 0; h < 2; ++h)
                                    __builtin_amdgcn_raw_buffer_store_b128(i32x4{(int)v[h][0], (int)v[h][1], (int)v[h][2], (int)v[h][3]}, ro,
                                                                           c < N ? at16(h) + (uint32_t)c * 4u : kOob, 0, 0);
                            }
                        }
                    } else {
#pragma unroll
                        for (int r = 0; r < 16; ++r) {
                            const int c = col + 8 * (r >> 2) + 4 * g + (r & 3);
                            const uint32_t o = c < N ? at0 + (uint32_t)c * ES : kOob;
                            if constexpr (EPI == MX_BF16)
                                __builtin_amdgcn_raw_buffer_store_b16((uint16_t)f32_to_bf16(acc_read(acc[i][j][r])), ro, o, 0, 0);
                            else
                                __builtin_amdgcn_raw_buffer_store_b32(__float_as_int(acc_read(acc[i][j][r])), ro, o, 0, 0);
                        }
                    }
                }
            }
        }
    }
}

// Products of so few tiles that most of the card would have none: 32 rows x 32 weight rows
// to a workgroup, its eight waves taking every eighth panel of K, fragments straight from
// memory (no byte is used twice), the waves' sums joined in the LDS.  Latency: of one row x
// 7168, K = 2048, 4.7 us, 1.6 of them its 7.8 MB.
constexpr int kFewWaves = 8;
template <int AF, int EPI>
__global__ __launch_bounds__(64 * kFewWaves) void k_mx_few(MxParams p) {
    constexpr int U = 2;  // panels under way
    __shared__ float sums[kFewWaves][16][64];
    __shared__ int tiles[kFewWaves], place[3];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), g = lane >> 5, l31 = lane & 31;
    {  // the group of row tile blockIdx.y
        int lo[2], n[2];
        int hi[2], s = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int e = 2 * tid + i;
            lo[i] = hi[i] = 0;
            if (e < p.G) {
                lo[i] = clampi(p.offsets[e], 0, p.M);
                hi[i] = clampi(p.offsets[e + 1], lo[i], p.M);
            }
            n[i] = (hi[i] - lo[i] + 31) / 32;
            s += n[i];
        }
        if (tid == 0) place[1] = 0;
        const int incl = wave_incl_scan(s);
        if (lane == 63) tiles[wave] = incl;
        __syncthreads();
        int at = incl - s;
        for (int w = 0; w < wave; ++w) at += tiles[w];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int j = (int)blockIdx.y - at;
            if (j >= 0 && j < n[i]) {
                place[0] = lo[i] + 32 * j;
                place[1] = min(hi[i] - lo[i] - 32 * j, 32);
                place[2] = 2 * tid + i;
            }
            at += n[i];
        }
        __syncthreads();
    }
    const int m0 = __builtin_amdgcn_readfirstlane(place[0]), rows = __builtin_amdgcn_readfirstlane(place[1]);
    const int e = __builtin_amdgcn_readfirstlane(place[2]), n0 = blockIdx.x * 32;
    if (rows == 0) return;
    // rows past the tile's and weight rows past the matrix repeat the last: what they give is
    // not stored; a row of none of x counts as zeros
    int row = m0 + min(l31, rows - 1);
    bool none = false;
    if (p.row_src) {
        const int src = p.row_src[row], token = of(p.by_k, src & 0x7fffffff);
        none = src < 0 || token >= p.x_rows;
        row = none ? 0 : token;
    }
    const uint64_t wr = (uint64_t)e * p.N + min(n0 + l31, p.N - 1);
    const uint8_t *const x = p.x + (uint64_t)row * (AF == kMxE2M1 ? p.K / 2 : p.K);
    const uint8_t *const w = p.w0 + wr * (uint32_t)(p.K / 2);
    const int blocks = p.K / 32, panels = (blocks + 3) / 4;
    f32x16 acc;
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[r] = 0.f;
    for (int p0 = wave; p0 < panels; p0 += U * kFewWaves) {
        uint32_t sw[U], sx[U];
        Frag<kMxE2M1> fw[U][2];
        Frag<AF> fx[U][2];
        const i32x4 zero = {0, 0, 0, 0};
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int pn = p0 + u * kFewWaves;
            const bool in = pn < panels;
            sw[u] = in ? p.s0[(uint64_t)pn * p.G * p.N + wr] : 0u;
            sx[u] = in && !none ? p.xs[(uint64_t)pn * p.x_rows + row] : 0u;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int b = 4 * pn + 2 * h;  // the step's first block
                fw[u][h].v = b + g < blocks ? *reinterpret_cast<const i32x4 *>(w + (b + g) * 16) : zero;
                if constexpr (AF == kMxE2M1) {
                    fx[u][h].v = b + g < blocks && !none ? *reinterpret_cast<const i32x4 *>(x + (b + g) * 16) : zero;
                } else {
                    const i32x4 c = b < blocks && !none ? *reinterpret_cast<const i32x4 *>(x + b * 32 + 16 * g) : zero;
                    const i32x4 d = b + 1 < blocks && !none ? *reinterpret_cast<const i32x4 *>(x + b * 32 + 32 + 16 * g) : zero;
                    fx[u][h].v = i32x8{c[0], c[1], c[2], c[3], d[0], d[1], d[2], d[3]};
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int left = blocks - 4 * (p0 + u * kFewWaves);
            const uint32_t mask = left >= 4 ? ~0u : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
            const uint32_t a = (sw[u] & mask) >> (8 * g), b = (sx[u] & mask) >> (8 * g);
            acc = mma<AF, 0>(fw[u][0], fx[u][0], acc, a, b);
            acc = mma<AF, 1>(fw[u][1], fx[u][1], acc, a, b);
        }
    }
#pragma unroll
    for (int r = 0; r < 16; ++r) sums[wave][r][lane] = acc[r];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 1024 / (64 * kFewWaves); ++i) {
        const int r = wave + kFewWaves * i, col = n0 + 8 * (r >> 2) + 4 * g + (r & 3);
        if (l31 >= rows || col >= p.N) continue;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kFewWaves; ++w) v += sums[w][r][lane];
        const uint64_t at = (uint64_t)(m0 + l31) * p.N + col;
        if (EPI == MX_BF16) static_cast<uint16_t *>(p.out)[at] = (uint16_t)f32_to_bf16(v);
        else static_cast<float *>(p.out)[at] = v;
    }
}

// The large tiles' rows: list[0] = {row tiles, rounded up to eight}, list[1 + i] = {first
// row, rows, group} of row tile i (no rows: those that fill up the last eight).  A group of
// offsets that do not ascend has no rows; what there is of row tiles past the list's room,
// which then may be, is left out.
__global__ __launch_bounds__(256) void k_mx_tiles(int G, int M, const int32_t *__restrict__ offsets, i32x4 *__restrict__ list, int room) {
    constexpr int BM = 256;
    __shared__ int first[kMxMaxGroups + 1];
    __shared__ int sums[4];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int n[4], s = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int e = 4 * tid + i;
        n[i] = 0;
        if (e < G) {
            const int lo = clampi(offsets[e], 0, M), hi = clampi(offsets[e + 1], lo, M);
            n[i] = (hi - lo + BM - 1) / BM;
        }
        s += n[i];
    }
    const int incl = wave_incl_scan(s);
    if (lane == 63) sums[wave] = incl;
    __syncthreads();
    int at = incl - s;
    for (int w = 0; w < wave; ++w) at += sums[w];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        first[4 * tid + i] = at;
        at += n[i];
    }
    if (tid == 255) first[kMxMaxGroups] = at;
    __syncthreads();
    const int R = min(first[kMxMaxGroups], room), filled = (R + kGroupM - 1) / kGroupM * kGroupM, i = blockIdx.x * 256 + tid;
    if (i == 0) list[0] = i32x4{filled, 0, 0, 0};
    if (i >= filled) return;
    if (i >= R) {
        list[1 + i] = i32x4{0, 0, 0, 0};
        return;
    }
    int lo = 0, hi = kMxMaxGroups - 1;
    while (lo < hi) {  // the last group that begins at or before row tile i
        const int mid = (lo + hi + 1) / 2;
        if (first[mid] <= i) lo = mid;
        else hi = mid - 1;
    }
    const int a = clampi(offsets[lo], 0, M), b = clampi(offsets[lo + 1], a, M), m0 = a + (i - first[lo]) * BM;
    list[1 + i] = i32x4{m0, min(b - m0, BM), lo, 0};
}

// out[p, r] = words[p, row_src[r] / k]: a panel's words in the order of the product's rows
// (an entry of no row of x: 0, which no code is read with).  23 us for 131072 rows of 7168.
__global__ __launch_bounds__(256) void k_mx_words(int M, int x_rows, Div by_k, const int32_t *__restrict__ row_src,
                                                  const uint32_t *__restrict__ words, uint32_t *__restrict__ out, int panels) {
    const int r = blockIdx.x * 256 + threadIdx.x;
    if (r >= M) return;
    const int src = row_src[r], token = of(by_k, src & 0x7fffffff);
    const bool ok = src >= 0 && token < x_rows;
    for (int p = blockIdx.y; p < panels; p += gridDim.y) out[(int64_t)p * M + r] = ok ? words[(int64_t)p * x_rows + token] : 0u;
}

int cu_count() {
    static int cached[64];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
    if (cached[dev] == 0) {
        int n = 0;
        if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0) n = 256;
        cached[dev] = n;
    }
    return cached[dev];
}

// Rows of a group up to which tiles of 32 rows, of 64 rows are taken (their sizes spread:
// past half a tile many groups need two, which read the weights twice).  Measured at random
// sizes, N = 2048, e4m3, in us: tiles of 32 against 64 at 10 rows of 32 groups, K = 7168,
// 44.1 against 45.1, at 24 rows 69.8 against 48.5; of 256 groups, K = 1024, 51.4 against 53.9
// and 67.8 against 61.0.  Tiles of 64 against 256 at 40 rows of the 32 groups 51.7 against
// 59.9, at 72 rows 92.3 against 68.9; of the 256 groups at 48 rows 76.2 against 100.9, at 128
// rows 130.2 against 129.3.
constexpr int kSmallRows = 16, kLargeRows = 64;
int rows_of_group(int M, int G) { return (M + G - 1) / G; }
// Tiles of 32 rows x 256 weight rows up to which k_mx_few takes a product.  Measured, few
// against tiles in us, e4m3, K = 2048 unless given: 1 row x 7168 (28) 4.7 against 10.5; 1 x
// 2048, K = 7168 (8) 7.9 against 26.4; 8 groups' row x 4096, K = 7168 (128) 25.7 against
// 29.3; 128 x 7168 (140) 17.3 against 28.1; 8 groups' row x 7168 (224) 20.2 against 14.2.  That
// border comes early where one group has many rows: of 4096 x 4096, 319 rows (160) take 32.8 us by
// few, 320 rows 49.3 by tiles of 256 rows, of which there are 32 for 256 CUs.
constexpr int kFewTiles = 160;
int64_t row_tiles(int G, int M) { return M < M / 32 + G ? M : M / 32 + G; }  // of 32 rows, at most
bool few(int G, int M, int N) { return row_tiles(G, M) * ((N + BN - 1) / BN) <= kFewTiles; }

template <int AF, int BM>
void launch(MxParams p, int epi, hipStream_t s) {
    const int columns = epi == MX_SWIGLU ? BN / 2 : BN;
    p.nt = div_by((uint32_t)((p.N + columns - 1) / columns));
    p.gnt = div_by((uint32_t)((p.N + columns - 1) / columns * kGroupM));
    const dim3 grid((Cfg<AF, BM>::WGS * cu_count() + 7) / 8 * 8);
    if (epi == MX_BF16) hipLaunchKernelGGL((k_mx_gemm<AF, BM, MX_BF16>), grid, dim3(64 * Cfg<AF, BM>::W), 0, s, p);
    else if (epi == MX_F32) hipLaunchKernelGGL((k_mx_gemm<AF, BM, MX_F32>), grid, dim3(64 * Cfg<AF, BM>::W), 0, s, p);
    else hipLaunchKernelGGL((k_mx_gemm<AF, BM, MX_SWIGLU>), grid, dim3(64 * Cfg<AF, BM>::W), 0, s, p);
}
template <int AF>
void launch(const MxParams &p, int epi, hipStream_t s) {
    const int avg = rows_of_group(p.M, p.G);
    if (epi != MX_SWIGLU && few(p.G, p.M, p.N)) {
        const dim3 grid((p.N + 31) / 32, (uint32_t)row_tiles(p.G, p.M));
        if (epi == MX_BF16) hipLaunchKernelGGL((k_mx_few<AF, MX_BF16>), grid, dim3(64 * kFewWaves), 0, s, p);
        else hipLaunchKernelGGL((k_mx_few<AF, MX_F32>), grid, dim3(64 * kFewWaves), 0, s, p);
        return;
    }
    if (avg <= kSmallRows) launch<AF, 32>(p, epi, s);
    else if (avg <= kLargeRows) launch<AF, 64>(p, epi, s);
    else launch<AF, 256>(p, epi, s);
}

}  // namespace

bool large_tiles(const MxProductArgs &a) { return rows_of_group(a.M, a.G) > kLargeRows && (a.swiglu || !few(a.G, a.M, a.N)); }
// Row tiles of large tiles, at most; their list's entries, behind which the gathered rows'
// scales lie.
size_t large_rows(const MxProductArgs &a) { return (size_t)a.M / 256 + a.G; }
size_t list_size(const MxProductArgs &a) { return large_rows(a) + kGroupM + 1; }
size_t mx_product_ws_bytes(const MxProductArgs &a) {
    return large_tiles(a) ? list_size(a) * 16 + (size_t)a.M * ((a.K + kPanel - 1) / kPanel) * 4 : 0;
}

hipError_t launch_mx_product(const MxProductArgs &a, hipStream_t s) {
    MxParams p{};
    p.G = a.G;
    p.M = a.M;
    p.N = a.N;
    p.K = a.K;
    p.x = a.x.codes;
    p.xs = a.x.scales;
    p.x_rows = p.xs_rows = a.x_rows;
    p.by_k = div_by((uint32_t)a.k);
    p.row_src = a.row_src;
    p.offsets = a.offsets;
    p.w0 = a.w.codes;
    p.s0 = a.w.scales;
    p.w1 = a.up.codes;
    p.s1 = a.up.scales;
    p.out = a.out;
    p.h = a.h;
    p.hs = a.h_scales;
    const bool large = large_tiles(a);
    if (large) {
        i32x4 *const list = static_cast<i32x4 *>(a.ws);
        hipLaunchKernelGGL(k_mx_tiles, dim3((uint32_t)((list_size(a) + 255) / 256)), dim3(256), 0, s, a.G, a.M, a.offsets, list,
                           (int)large_rows(a));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        p.tiles = list;
    }
    if (large && a.row_src) {
        // a tile reads its rows' words as one run; gathered by every tile they were as many
        // requests as the rows' codes
        const int panels = (a.K + kPanel - 1) / kPanel;
        uint32_t *const words = reinterpret_cast<uint32_t *>(static_cast<i32x4 *>(a.ws) + list_size(a));
        hipLaunchKernelGGL(k_mx_words, dim3((a.M + 255) / 256, panels < 8 ? panels : 8), dim3(256), 0, s, a.M, a.x_rows, p.by_k, a.row_src,
                           a.x.scales, words, panels);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        p.xs = words;
        p.xs_rows = a.M;
        p.xs_gathered = true;
    }
    const int epi = a.swiglu ? MX_SWIGLU : a.out_bf16 ? MX_BF16 : MX_F32;
    if (a.x_format == kMxE4M3) launch<kMxE4M3>(p, epi, s);
    else launch<kMxE2M1>(p, epi, s);
    return hipGetLastError();
}

}  // namespace moe
