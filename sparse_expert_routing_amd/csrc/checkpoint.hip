// Activation checkpoints in 8 bits, and the combine's gradient from them.
//
// A row is cut into tiles of 128 columns (the last may be shorter).  A tile has
// one E8M0 scale 2^x, the smallest power of two at or above its largest
// magnitude over the format's largest value (448 for e4m3, 127 for integers),
// and a code per value: v / 2^x rounded to nearest even.  The quotient is exact, or
// below fp32's normal numbers, where the code is 0 either way; so a code is off by
// half a step of its format and by nothing else: at most 2^-4 of the value (e4m3,
// above its subnormals), 1/127 of the tile's largest (integers: half of a scale that
// is less than twice the largest over 127).  A tile that holds an infinity or a NaN
// gets scale byte 255, the format's NaN, and reads back as NaN throughout: a lost
// activation shows.
#include "device.h"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kTile = 128;

// The E8M0 byte of a tile: from the exponent of its largest magnitude, one more
// where the mantissa is past the format's (448 = 1.75 * 2^8, 127 = 1.984375 *
// 2^6).  At least 1 (2^-126), so the scale and its reciprocal are normal
// numbers; 127 (scale 1) for an all-zero tile; 255 where a value is not finite.
template <int FMT>
__device__ __forceinline__ uint32_t tile_byte(uint32_t amax_bits) {
    constexpr uint32_t kMant = FMT == kCkptE4M3 ? 0x600000u : 0x7e0000u;
    constexpr int kShift = FMT == kCkptE4M3 ? 8 : 6;
    if (amax_bits == 0) return 127u;
    if (amax_bits >= 0x7f800000u) return 255u;
    const int e = (int)(amax_bits >> 23) - kShift + ((amax_bits & 0x7fffffu) > kMant ? 1 : 0);
    return (uint32_t)max(e, 1);
}

__device__ __forceinline__ float pow2_of_byte(uint32_t b) {
    return b == 255u ? __uint_as_float(0x7fc00000u) : b == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(b << 23);
}
// 2^-x of a scale byte 1 .. 254.
__device__ __forceinline__ float inverse_pow2(uint32_t b) {
    return b == 254u ? __uint_as_float(0x00400000u) : __uint_as_float((254u - b) << 23);
}

// Four codes in one word.
template <int FMT>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
    if (FMT == kCkptE4M3) return e4m3x4(a, b, c, d);
    const uint32_t x = (uint32_t)(int)__builtin_rintf(a) & 0xffu, y = (uint32_t)(int)__builtin_rintf(b) & 0xffu,
                   z = (uint32_t)(int)__builtin_rintf(c) & 0xffu, w = (uint32_t)(int)__builtin_rintf(d) & 0xffu;
    return x | (y << 8) | (z << 16) | (w << 24);
}

template <int FMT>
__device__ __forceinline__ void decode4(uint32_t w, float (&v)[4]) {
    if (FMT == kCkptE4M3) {
        const f32x2_hw lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
        const f32x2_hw hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
        v[0] = lo[0]; v[1] = lo[1]; v[2] = hi[0]; v[3] = hi[1];
    } else {
        v[0] = (float)(int8_t)(w & 0xffu); v[1] = (float)(int8_t)((w >> 8) & 0xffu);
        v[2] = (float)(int8_t)((w >> 16) & 0xffu); v[3] = (float)(int8_t)(w >> 24);
    }
}

// Eight values of a row: consecutive (VEC), or 16 columns apart, so that sixteen
// lanes read and write neighbouring ones; n: columns of the row from the first
// on (VEC: 8 or more).
template <bool BF16, bool VEC>
__device__ __forceinline__ void load8(const void *src, int64_t at, int n, float (&v)[8]) {
    if (VEC && BF16) {
        const i32x4 w = *reinterpret_cast<const i32x4 *>(static_cast<const uint16_t *>(src) + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16_to_f32((uint32_t)w[i] & 0xffffu);
            v[2 * i + 1] = bf16_to_f32((uint32_t)w[i] >> 16);
        }
    } else if (VEC) {
        const f32x4 a = *reinterpret_cast<const f32x4 *>(static_cast<const float *>(src) + at);
        const f32x4 b = *reinterpret_cast<const f32x4 *>(static_cast<const float *>(src) + at + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) { v[i] = a[i]; v[4 + i] = b[i]; }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = 16 * i >= n ? 0.f : BF16 ? bf16_to_f32(static_cast<const uint16_t *>(src)[at + 16 * i])
                                            : static_cast<const float *>(src)[at + 16 * i];
    }
}

template <bool BF16, bool VEC>
__device__ __forceinline__ void store8(void *dst, int64_t at, int n, const float (&v)[8]) {
    if (VEC && BF16) {
        i32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = (int)pack_bf16x2(v[2 * i], v[2 * i + 1]);
        __builtin_nontemporal_store(w, reinterpret_cast<i32x4 *>(static_cast<uint16_t *>(dst) + at));
    } else if (VEC) {
        __builtin_nontemporal_store(f32x4{v[0], v[1], v[2], v[3]}, reinterpret_cast<f32x4 *>(static_cast<float *>(dst) + at));
        __builtin_nontemporal_store(f32x4{v[4], v[5], v[6], v[7]}, reinterpret_cast<f32x4 *>(static_cast<float *>(dst) + at + 4));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (16 * i < n) {
                if (BF16) static_cast<uint16_t *>(dst)[at + 16 * i] = (uint16_t)f32_to_bf16(v[i]);
                else static_cast<float *>(dst)[at + 16 * i] = v[i];
            }
    }
}

// A tile's place: row and column of its first value.  FLAT: rows are dense and
// hold whole tiles, so a tile is 128 values in a row of the whole array; else one
// division per tile by the tiles of a row, from the row of the workgroup's first.
struct TilePlace {
    int64_t row;
    int first;  // tile of the row that the workgroup begins with
};
template <bool FLAT>
__device__ __forceinline__ TilePlace place_of(int64_t base, int ntile) {
    if (FLAT) return TilePlace{0, 0};
    const int64_t row = base / ntile;
    return TilePlace{row, (int)(base - row * ntile)};
}

// Tiles of a lane in flight: four of a large dense array, so that a wave has enough
// loads under way, one otherwise, where there are too few tiles to fill the card so
// (2408 tiles: 4 us a pass with one, 8 with four) or places cost registers.  Four
// against one, us, e4m3:
//   bf16 there and back: 65536 tiles 12.3, 12.2 (the calls'), 131072 19.2, 19.8,
//     524288 69.6, 71.3, 131072 x 7168 979, 993
//   fp32 pack, whose loads are twice as long, always with one: 262144 tiles 25.5, 24.7,
//     131072 x 7168 886, 809
//   fp32 unpack, whose stores skip every other 16 bytes: 262144 tiles 53, 47, 1.8 million
//     387, 364, 2.1 419, 420, 2.8 389, 551, 131072 x 7168 1091, 1477
constexpr int kManyTiles = 65536;
constexpr int unroll_of(bool flat) { return flat ? 4 : 1; }

// Sixteen lanes per tile, eight values each.
template <bool BF16, int FMT, bool VEC, bool FLAT>
__global__ __launch_bounds__(256) void k_pack(int64_t rows, int cols, int ntile, const void *__restrict__ src, int64_t ld,
                                              uint8_t *__restrict__ codes, uint8_t *__restrict__ scales) {
    constexpr int kUnroll = unroll_of(FLAT);
    const int sub = threadIdx.x & 15, group = threadIdx.x >> 4;
    const int64_t tiles = rows * ntile, step = (int64_t)gridDim.x * (16 * kUnroll);
    for (int64_t base = (int64_t)blockIdx.x * (16 * kUnroll); base < tiles; base += step) {
        const TilePlace at = place_of<FLAT>(base, ntile);
        float v[kUnroll][8];
        int64_t from[kUnroll];  // where the lane's values lie in codes
        int n[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t tile = base + 16 * u + group;
            int64_t row = 0;
            int c = VEC ? sub * 8 : sub;
            if (!FLAT) {
                const uint32_t k = (uint32_t)(at.first + 16 * u + group), q = k / (uint32_t)ntile;
                row = at.row + q;
                c += (int)(k - q * ntile) * kTile;
            }
            n[u] = tile < tiles ? (FLAT ? 8 : min(kTile - (VEC ? 0 : sub), cols - c)) : 0;
            from[u] = FLAT ? tile * kTile + c : row * cols + c;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[u][i] = 0.f;
            if (n[u] > 0) load8<BF16, VEC>(src, FLAT ? from[u] : row * ld + c, n[u], v[u]);
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[u][i]) & 0x7fffffffu);
            const uint32_t byte = tile_byte<FMT>(row_max(m));
            if (base + 16 * u + group >= tiles) continue;
            if (sub == 0) scales[base + 16 * u + group] = (uint8_t)byte;
            if (n[u] <= 0) continue;
            const float inv = inverse_pow2(byte);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[u][i] = byte == 255u ? 0.f : v[u][i] * inv;
            const uint2 w = uint2{encode4<FMT>(v[u][0], v[u][1], v[u][2], v[u][3]),
                                  encode4<FMT>(v[u][4], v[u][5], v[u][6], v[u][7])};
            if (VEC) {
                *reinterpret_cast<uint2 *>(codes + from[u]) = w;
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (16 * i < n[u]) codes[from[u] + 16 * i] = (uint8_t)((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
            }
        }
    }
}

template <bool BF16, int FMT, bool VEC, bool FLAT>
__global__ __launch_bounds__(256) void k_unpack(int64_t rows, int cols, int ntile, const uint8_t *__restrict__ codes,
                                                const uint8_t *__restrict__ scales, void *__restrict__ dst, int64_t ld) {
    constexpr int kUnroll = unroll_of(FLAT);
    const int sub = threadIdx.x & 15, group = threadIdx.x >> 4;
    const int64_t tiles = rows * ntile, step = (int64_t)gridDim.x * (16 * kUnroll);
    for (int64_t base = (int64_t)blockIdx.x * (16 * kUnroll); base < tiles; base += step) {
        const TilePlace at = place_of<FLAT>(base, ntile);
        uint2 w[kUnroll];
        uint32_t byte[kUnroll];
        int64_t to[kUnroll];
        int n[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int64_t tile = base + 16 * u + group;
            int64_t row = 0;
            int c = VEC ? sub * 8 : sub;
            if (!FLAT) {
                const uint32_t k = (uint32_t)(at.first + 16 * u + group), q = k / (uint32_t)ntile;
                row = at.row + q;
                c += (int)(k - q * ntile) * kTile;
            }
            n[u] = tile < tiles ? (FLAT ? 8 : min(kTile - (VEC ? 0 : sub), cols - c)) : 0;
            const int64_t from = FLAT ? tile * kTile + c : row * cols + c;
            to[u] = FLAT ? from : row * ld + c;
            w[u] = uint2{0u, 0u};
            byte[u] = 127u;
            if (n[u] <= 0) continue;
            byte[u] = scales[tile];
            if (VEC) {
                w[u] = *reinterpret_cast<const uint2 *>(codes + from);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (16 * i < n[u]) (i < 4 ? w[u].x : w[u].y) |= (uint32_t)codes[from + 16 * i] << (8 * (i & 3));
            }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            if (n[u] <= 0) continue;
            const float scale = pow2_of_byte(byte[u]);
            float lo[4], hi[4], v[8];
            decode4<FMT>(w[u].x, lo);
            decode4<FMT>(w[u].y, hi);
#pragma unroll
            for (int i = 0; i < 4; ++i) { v[i] = lo[i] * scale; v[4 + i] = hi[i] * scale; }
            store8<BF16, VEC>(dst, to[u], n[u], v);
        }
    }
}

// ------------------------------------------------------- the combine's gradient

template <bool F32>
__device__ __forceinline__ void put8(void *base, int64_t at, const float (&v)[8]) {
    store8<!F32, true>(base, at, 8, v);
}

// Eight consecutive saved values of row r at column c: as they lie in memory, so
// that several rows' loads are in flight, and then their values.
template <int FMT>
struct Saved8 {
    i32x4 w;  // bf16: all four words; 8-bit: the first two
    uint32_t byte;
    __device__ __forceinline__ void load(const Saved &y, int64_t r, int d, int ntile, int c) {
        if (FMT == kCkptBF16) {
            w = *reinterpret_cast<const i32x4 *>(static_cast<const uint16_t *>(y.data) + r * d + c);
        } else {
            const uint2 v = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(y.data) + r * d + c);
            w = i32x4{(int)v.x, (int)v.y, 0, 0};
            byte = y.scales[r * ntile + c / kTile];
        }
    }
    __device__ __forceinline__ void values(float (&v)[8]) const {
        if (FMT == kCkptBF16) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = bf16_to_f32((uint32_t)w[i] & 0xffffu);
                v[2 * i + 1] = bf16_to_f32((uint32_t)w[i] >> 16);
            }
        } else {
            const float scale = pow2_of_byte(byte);
            float lo[4], hi[4];
            decode4<FMT>((uint32_t)w[0], lo);
            decode4<FMT>((uint32_t)w[1], hi);
#pragma unroll
            for (int i = 0; i < 4; ++i) { v[i] = lo[i] * scale; v[4 + i] = hi[i] * scale; }
        }
    }
};

// Bound by memory: T = 16384, d = 7168 from e4m3 674 us, 4.9 TB/s (one wave per token
// 702); T = 2048, d = 2048 from int8 21 us (one wave and a row's load at a time 37,
// stores through the caches 26).
//
// W waves per token, each on every W-th run of 512 columns.  A row_of entry outside
// [0, T*8) is a choice that was not dispatched: it has no row to write and its
// gradient is 0.
template <int FMT, bool F32, int W>
__global__ __launch_bounds__(256) void k_combine_backward(int T, int d, int ntile, const float *__restrict__ dy, Saved y,
                                                          const int32_t *__restrict__ row_of, const float *__restrict__ w,
                                                          void *__restrict__ dyp, void *__restrict__ dys,
                                                          float *__restrict__ dg) {
    __shared__ float part[4][8];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t = (int64_t)blockIdx.x * (4 / W) + wave / W;
    float mine = 0.f;
    if (t < T) {
        int r[8];
        float g[8], dot[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            r[j] = row_of[t * 8 + j];
            if (r[j] < 0 || (int64_t)r[j] >= (int64_t)T * 8) r[j] = -1;
            g[j] = w[t * 8 + j];
            dot[j] = 0.f;
        }
        for (int c = 8 * lane + 512 * (wave % W); c < d; c += 512 * W) {
            float v[8];
            Saved8<FMT> in[8];
            load8<false, true>(dy, t * d + c, 8, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) in[j].load(y, max(r[j], 0), d, ntile, c);
            if (dys) put8<F32>(dys, t * d + c, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float s[8], o[8];
                in[j].values(s);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    dot[j] += v[i] * s[i];
                    o[i] = g[j] * v[i];
                }
                if (r[j] >= 0) put8<F32>(dyp, (int64_t)r[j] * d + c, o);
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float v = dot[j];
#pragma unroll
            for (int s = 32; s >= 1; s >>= 1) v += __shfl_xor(v, s, kWave);
            if (lane == j) mine = r[j] >= 0 ? v : 0.f;
        }
    }
    if (W == 1) {
        if (t < T && lane < 8) dg[t * 8 + lane] = mine;
        return;
    }
    if (lane < 8) part[wave][lane] = mine;
    __syncthreads();
    if (t < T && wave % W == 0 && lane < 8) {
#pragma unroll
        for (int i = 1; i < W; ++i) mine += part[wave + i][lane];
        dg[t * 8 + lane] = mine;
    }
}

bool aligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// Whether every eight columns can be read and written as whole vectors.
bool vec_ok(const CkptArgs &a, const void *plain) {
    return a.cols % 8 == 0 && a.ld % (a.bf16 ? 8 : 4) == 0 && aligned(plain, 16) && aligned(a.codes, 8);
}

// Whether it is one run of many whole tiles.
bool flat_ok(const CkptArgs &a) {
    return a.cols % kTile == 0 && a.ld == a.cols && a.rows * (a.cols / kTile) >= kManyTiles;
}

// Tiles of a row of any number of columns.
int tiles_of(int cols) { return cols / kTile + (cols % kTile != 0); }

unsigned tile_grid(int64_t tiles, bool flat) {
    const int64_t per = 16 * unroll_of(flat), n = (tiles + per - 1) / per;
    return (unsigned)(n < (1 << 22) ? n : (1 << 22));
}

}  // namespace

// F32_FLAT: whether KERNEL has a form for many fp32 tiles.
#define MOE_CKPT_TYPES(KERNEL, F32_FLAT, FMT, ...)                                                        \
    do {                                                                                                  \
        if (a.bf16 && flat) hipLaunchKernelGGL((KERNEL<true, FMT, true, true>), __VA_ARGS__);             \
        else if (a.bf16 && vec) hipLaunchKernelGGL((KERNEL<true, FMT, true, false>), __VA_ARGS__);        \
        else if (a.bf16) hipLaunchKernelGGL((KERNEL<true, FMT, false, false>), __VA_ARGS__);              \
        else if (flat) hipLaunchKernelGGL((KERNEL<false, FMT, true, F32_FLAT>), __VA_ARGS__);             \
        else if (vec) hipLaunchKernelGGL((KERNEL<false, FMT, true, false>), __VA_ARGS__);                 \
        else hipLaunchKernelGGL((KERNEL<false, FMT, false, false>), __VA_ARGS__);                         \
    } while (0)
#define MOE_CKPT_VARIANTS(KERNEL, F32_FLAT, ...)                                                          \
    do {                                                                                                  \
        if (a.format == kCkptE4M3) MOE_CKPT_TYPES(KERNEL, F32_FLAT, kCkptE4M3, __VA_ARGS__);              \
        else MOE_CKPT_TYPES(KERNEL, F32_FLAT, kCkptI8, __VA_ARGS__);                                      \
    } while (0)

hipError_t launch_checkpoint_pack(const CkptArgs &a, hipStream_t s) {
    const int ntile = tiles_of(a.cols);
    const bool vec = vec_ok(a, a.src), flat = vec && a.bf16 && flat_ok(a);
    const dim3 grid(tile_grid(a.rows * ntile, flat)), block(256);
    MOE_CKPT_VARIANTS(k_pack, false, grid, block, 0, s, a.rows, a.cols, ntile, a.src, a.ld, a.codes, a.scales);
    return hipGetLastError();
}

hipError_t launch_checkpoint_unpack(const CkptArgs &a, hipStream_t s) {
    const int ntile = tiles_of(a.cols);
    const bool vec = vec_ok(a, a.dst), flat = vec && flat_ok(a);
    const dim3 grid(tile_grid(a.rows * ntile, flat)), block(256);
    MOE_CKPT_VARIANTS(k_unpack, true, grid, block, 0, s, a.rows, a.cols, ntile, a.codes, a.scales, a.dst, a.ld);
    return hipGetLastError();
}
#undef MOE_CKPT_VARIANTS
#undef MOE_CKPT_TYPES

// Waves per token: four share a wide row, whose one wave would have too few loads in
// flight; they cost an exchange, and idle where 512 columns are all.  Four against one,
// us, int8: T = 16384, d = 512 59, 47; 1024 95, 96; 1536 142, 146; 2048 190, 202; 4096
// 379, 387; T = 2048, d = 1024 12.6, 12.1; 1536 16.9, 16.4; 2048 20.8, 20.9; 4096 46, 52.
static int combine_waves(int d) { return d >= 2048 ? 4 : 1; }

bool combine_backward_ok(int T, int d) { return (int64_t)T * combine_waves(d) < (1LL << 26); }

hipError_t launch_combine_backward(int T, int d, const float *dy, const Saved &y, const int32_t *row_of,
                                   const float *weights, void *dyp, void *dys, float *dg, bool f32_out, hipStream_t s) {
    const int ntile = tiles_of(d);
    const dim3 block(256);
#define GO_W(FMT, W)                                                                                               \
    do {                                                                                                           \
        const dim3 grid((unsigned)(((int64_t)T * W + 3) / 4));                                                     \
        if (f32_out) hipLaunchKernelGGL((k_combine_backward<FMT, true, W>), grid, block, 0, s, T, d, ntile, dy, y, \
                                        row_of, weights, dyp, dys, dg);                                            \
        else hipLaunchKernelGGL((k_combine_backward<FMT, false, W>), grid, block, 0, s, T, d, ntile, dy, y,        \
                                row_of, weights, dyp, dys, dg);                                                    \
    } while (0)
#define GO(FMT)                                  \
    do {                                         \
        if (combine_waves(d) == 4) GO_W(FMT, 4); \
        else GO_W(FMT, 1);                       \
    } while (0)
    if (y.format == kCkptE4M3) GO(kCkptE4M3);
    else if (y.format == kCkptI8) GO(kCkptI8);
    else GO(kCkptBF16);
#undef GO
#undef GO_W
    return hipGetLastError();
}

}  // namespace moe
