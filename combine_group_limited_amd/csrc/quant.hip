// quant.hip -- MXFP4 quantisation and its inverse.
//
// Format (OCP Microscaling Formats specification v1.0): 32 consecutive
// columns share one E8M0 scale 2^(b - 127); the elements are E2M1 (0, 0.5, 1,
// 1.5, 2, 3, 4, 6 and their negatives), two to a byte, the even column in the
// low half.  Rule (section 6.3 of that specification): with amax the block's
// largest magnitude, b - 127 = floor(log2 amax) - 2, clamped to [-127, 127];
// an element is x / 2^(b - 127) rounded to nearest, ties to the even code,
// saturated to +-6.  floor(log2 amax) is the exponent field, so b is that
// field minus 2 (0 at least; all-zero and tiny blocks get 0).  A block that
// holds a NaN or an infinity has no scale: it gets b = 255 (NaN) and codes 0.
//
// A row is a whole number of blocks, so the rows are one run of blocks: a
// wavefront takes 64 blocks in four loads, in each of which 4 lanes hold a
// block, 8 columns each.  The scales of the four loads' blocks are stored as
// one byte per lane.
//
// Bound by memory: 131072 rows of 7168 bf16 columns take 384 us one way (6.2
// TB/s read and written) and 406 us back (5.9), where a plain copy reaches 5.7
// and a read alone 7.0; 128 rows take 2.8 us, a launch.
#include "device.h"
#include "launch.h"

namespace ep {

namespace {

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr int kBlock = 32;      // columns per scale
constexpr int kBlocksPerWave = 64;
constexpr int kWaves = 4;       // wavefronts per workgroup
constexpr uint32_t kNaNScale = 255u;

__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
    v = max(v, dpp_u32<kDppXor1>(v));
    return max(v, dpp_u32<kDppXor2>(v));
}

// a dword as two bf16 values (by value: a bit cast of a vector's element reads
// its first)
__device__ __forceinline__ bf16x2 bf16_pair(int w) { return __builtin_bit_cast(bf16x2, w); }

__device__ __forceinline__ uint32_t umax16x2(uint32_t a, uint32_t b) {
    const u16x2 m = __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b));
    return __builtin_bit_cast(uint32_t, m);
}

// The block's E8M0 scale from the largest exponent field among its values.
__device__ __forceinline__ uint32_t block_scale(uint32_t field) {
    return field == 255u ? kNaNScale : (field > 2u ? field - 2u : 0u);
}

// Eight columns of a block, 16-bit or 32-bit, and their largest magnitude's
// exponent field over the block.
struct Bf16Eight {
    static constexpr int kBytes = 16;
    i32x4 v;
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, int at) {
        v = __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, kStream);
    }
    __device__ __forceinline__ uint32_t field() const {
        constexpr uint32_t kMag = 0x7FFF7FFFu;
        uint32_t m = umax16x2((uint32_t)v.x & kMag, (uint32_t)v.y & kMag);
        m = umax16x2(m, umax16x2((uint32_t)v.z & kMag, (uint32_t)v.w & kMag));
        return quad_max(max(m & 0xFFFFu, m >> 16)) >> 7;
    }
    __device__ __forceinline__ uint32_t codes(float scale) const {
        uint32_t q = 0u;
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, bf16_pair(v.x), scale, 0);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, bf16_pair(v.y), scale, 1);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, bf16_pair(v.z), scale, 2);
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, bf16_pair(v.w), scale, 3);
    }
};

struct F32Eight {
    static constexpr int kBytes = 32;
    i32x4 a, b;
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, int at) {
        a = __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, kStream);
        b = __builtin_amdgcn_raw_buffer_load_b128(r, at + 16, 0, kStream);
    }
    __device__ __forceinline__ uint32_t field() const {
        constexpr uint32_t kMag = 0x7FFFFFFFu;
        uint32_t m = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max(m, max((uint32_t)a[i] & kMag, (uint32_t)b[i] & kMag));
        return quad_max(m) >> 23;
    }
    __device__ __forceinline__ uint32_t codes(float scale) const {
        uint32_t q = 0u;
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, __int_as_float(a.x), __int_as_float(a.y), scale, 0);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, __int_as_float(a.z), __int_as_float(a.w), scale, 1);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, __int_as_float(b.x), __int_as_float(b.y), scale, 2);
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, __int_as_float(b.z), __int_as_float(b.w), scale, 3);
    }
};

// Buffer bytes of a wavefront's run of 64 blocks of `block_bytes`, `left`
// blocks before the end: accesses beyond read zero and store nothing.
__device__ __forceinline__ uint32_t run_bytes(long left, int block_bytes) {
    return (uint32_t)((left < kBlocksPerWave ? left : kBlocksPerWave) * block_bytes);
}

template <class Eight>
__global__ __launch_bounds__(kWaves * 64) void quantize_kernel(const uint8_t* __restrict__ x,
                                                               uint8_t* __restrict__ codes,
                                                               uint8_t* __restrict__ scales, long blocks) {
    const int lane = threadIdx.x & 63;
    const long stride = (long)gridDim.x * kWaves * kBlocksPerWave;
    for (long b0 = ((long)blockIdx.x * kWaves + (threadIdx.x >> 6)) * kBlocksPerWave; b0 < blocks; b0 += stride) {
        constexpr int kIn = 4 * Eight::kBytes;  // bytes of a block
        const auto xr = buffer_rsrc(x + b0 * kIn, run_bytes(blocks - b0, kIn));
        const auto cr = buffer_rsrc(codes + b0 * (kBlock / 2), run_bytes(blocks - b0, kBlock / 2));
        const auto sr = buffer_rsrc(scales + b0, run_bytes(blocks - b0, 1));
        Eight v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i].load(xr, (i * 64 + lane) * Eight::kBytes);
        uint32_t mine = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t s = block_scale(v[i].field());
            uint32_t q = v[i].codes(__uint_as_float(s << 23));
            q = s == kNaNScale ? 0u : q;
            __builtin_amdgcn_raw_buffer_store_b32((int)q, cr, (i * 64 + lane) * 4, 0, kStream);
            mine = (lane & 3) == i ? s : mine;
        }
        // lane 4 j + i stores the scale of block 16 i + j
        __builtin_amdgcn_raw_buffer_store_b8((char)mine, sr, (lane & 3) * 16 + (lane >> 2), 0, kStream);
    }
}

template <bool WIDE>
__global__ __launch_bounds__(kWaves * 64) void dequantize_kernel(const uint8_t* __restrict__ codes,
                                                                 const uint8_t* __restrict__ scales,
                                                                 uint8_t* __restrict__ out, long blocks) {
    const int lane = threadIdx.x & 63;
    const long stride = (long)gridDim.x * kWaves * kBlocksPerWave;
    for (long b0 = ((long)blockIdx.x * kWaves + (threadIdx.x >> 6)) * kBlocksPerWave; b0 < blocks; b0 += stride) {
        constexpr int kOut = kBlock * (WIDE ? 4 : 2);  // bytes of a block
        const auto cr = buffer_rsrc(codes + b0 * (kBlock / 2), run_bytes(blocks - b0, kBlock / 2));
        const auto sr = buffer_rsrc(scales + b0, run_bytes(blocks - b0, 1));
        const auto orr = buffer_rsrc(out + b0 * kOut, run_bytes(blocks - b0, kOut));
        uint32_t q[4], s[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            q[i] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(cr, (i * 64 + lane) * 4, 0, kStream);
            s[i] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(sr, i * 16 + (lane >> 2), 0, kCached);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool nan = s[i] == kNaNScale;
            const float scale = __uint_as_float(s[i] << 23);
            if constexpr (WIDE) {
                f32x2 f[4];
                f[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], scale, 0);
                f[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], scale, 1);
                f[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], scale, 2);
                f[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], scale, 3);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    i32x4 o;
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        o[c] = nan ? 0x7FC00000 : __float_as_int(f[2 * h + (c >> 1)][c & 1]);
                    __builtin_amdgcn_raw_buffer_store_b128(o, orr, (i * 64 + lane) * 32 + h * 16, 0, kStream);
                }
            } else {
                i32x4 o;
                o.x = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[i], scale, 0));
                o.y = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[i], scale, 1));
                o.z = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[i], scale, 2));
                o.w = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[i], scale, 3));
                if (nan) o = i32x4{0x7FC07FC0, 0x7FC07FC0, 0x7FC07FC0, 0x7FC07FC0};
                __builtin_amdgcn_raw_buffer_store_b128(o, orr, (i * 64 + lane) * 16, 0, kStream);
            }
        }
    }
}

// One wavefront per run of 64 blocks, up to a grid that fills the chip many
// times over; beyond, the wavefronts stride.
int grid_of(long blocks) {
    constexpr long kMaxGrid = 1 << 20;
    const long g = (blocks + kWaves * kBlocksPerWave - 1) / (kWaves * kBlocksPerWave);
    return (int)(g < kMaxGrid ? g : kMaxGrid);
}

}  // namespace

hipError_t launch_mxfp4_quantize(long blocks, bool wide, const void* x, uint8_t* codes, uint8_t* scales,
                                 hipStream_t stream) {
    if (blocks == 0) return hipSuccess;
    const uint8_t* p = static_cast<const uint8_t*>(x);
    if (wide)
        hipLaunchKernelGGL(quantize_kernel<F32Eight>, dim3(grid_of(blocks)), dim3(kWaves * 64), 0, stream, p, codes,
                           scales, blocks);
    else
        hipLaunchKernelGGL(quantize_kernel<Bf16Eight>, dim3(grid_of(blocks)), dim3(kWaves * 64), 0, stream, p, codes,
                           scales, blocks);
    return hipGetLastError();
}

hipError_t launch_mxfp4_dequantize(long blocks, bool wide, const uint8_t* codes, const uint8_t* scales, void* out,
                                   hipStream_t stream) {
    if (blocks == 0) return hipSuccess;
    uint8_t* p = static_cast<uint8_t*>(out);
    if (wide)
        hipLaunchKernelGGL(dequantize_kernel<true>, dim3(grid_of(blocks)), dim3(kWaves * 64), 0, stream, codes, scales,
                           p, blocks);
    else
        hipLaunchKernelGGL(dequantize_kernel<false>, dim3(grid_of(blocks)), dim3(kWaves * 64), 0, stream, codes,
                           scales, p, blocks);
    return hipGetLastError();
}

}  // namespace ep
