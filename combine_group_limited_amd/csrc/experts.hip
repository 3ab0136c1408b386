// experts.hip -- the experts' products between dispatch and combine.
//
// Row r of the receive buffer belongs to expert e(r) and becomes
//   y[r, n] = sum_k x[r, k] W[e(r)][n, k]
// with W in MXFP4 (quant.hip's format) and x either dispatch's FP8 rows (E4M3
// and a 32-bit scale for every 128 columns) or MXFP4 rows.  The gated form
// has 2 N weight rows, N gate rows and then N up rows, and gives
//   h[r, n] = gate * sigmoid(gate) * up
// in bf16 or, for the next product, in MXFP4.
//
// The matrix instruction multiplies 16 x 128 weights by 128 x 16 activations;
// lane (g, m) (g = lane / 16, m = lane % 16) holds 32 columns of weight row m
// and 32 of activation row m: columns 32 g .. 32 g + 31 in MXFP4, 16 g .. 16 g
// + 15 and 64 + 16 g .. 64 + 16 g + 15 in FP8.  It also holds one E8M0 scale
// for columns 32 g .. 32 g + 31 of each row, which the instruction applies
// itself.  FP8 rows pass a scale of 1; their 32-bit scale of the 128 columns
// multiplies the instruction's result into the sums.  All sums are 32-bit.
//
// The instruction adds the 32 products of a block as fixed-point numbers below
// the largest of them.  MXFP4 products fit and add up exactly, but E4M3's 17
// binades do not: measured on random codes, a result is off by up to 2^-11 of
// the largest product.  Eight binades of E4M3 fit, so FP8 rows go through the
// instruction in two halves, codes of 2 and above and codes below 2, the
// second result starting from the first; that is exact up to one rounding to
// 32 bits, at half the rate.
//
// The result has weight rows along its registers: lane (g, m) holds rows
// 4 g .. 4 g + 3 of a 16-row weight tile for activation row m.  The 16 weight rows of a wavefront's NT tiles are chosen
// so that a lane's NT x 4 results are consecutive columns of y: tile i, row
// 4 g + r is column 4 (NT g + i) + r (in the gated form, the gate tiles and
// the up tiles each).
//
// How many rows an expert has is known on the device only.  Every workgroup
// finds its tile from the counts, so nothing waits for the host; the grid is
// an upper bound, and workgroups past the last tile end at once.
#include "device.h"
#include "launch.h"

namespace ep {

namespace {

typedef int32_t i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kFp8 = 0, kFp4 = 4;  // matrix instruction operand formats
constexpr int kStep = 128;         // columns of a matrix instruction
constexpr int kNT = 4;             // 16-row weight tiles per wavefront
constexpr int kUnit = 127;         // E8M0 scale of 1

enum Epilogue { kPlain, kGated, kGatedMx };

// a constant as a function argument
template <int I>
struct Int {
    static constexpr int value = I;
    __device__ constexpr operator int() const { return I; }
};

// Output columns of a wavefront's kNT weight tiles.
template <int EPI>
constexpr int kCols = EPI == kPlain ? 16 * kNT : 8 * kNT;

// One lane's 32 columns of an activation row (16-byte pieces).
template <bool FP8>
struct XPiece {
    i32x4 v[FP8 ? 2 : 1];
};

// The E4M3 codes of magnitude 2 and above (bit 6 set), zero in the others'
// places.
__device__ __forceinline__ i32x4 upper_codes(i32x4 v) {
    i32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t one = ((uint32_t)v[i] >> 6) & 0x01010101u;
        r[i] = v[i] & (int)((one << 8) - one);
    }
    return r;
}

template <bool FP8>
__device__ __forceinline__ i32x8 operand(const XPiece<FP8>& p) {
    if constexpr (FP8) return __builtin_shufflevector(p.v[0], p.v[1], 0, 1, 2, 3, 4, 5, 6, 7);
    else return i32x8{p.v[0].x, p.v[0].y, p.v[0].z, p.v[0].w, 0, 0, 0, 0};
}

// c + w x, 16 weight rows by 16 activation rows over 128 columns; WB and XB are
// the bytes of `ws` and `xs` that hold the scales.
template <bool FP8, int WB, int XB>
__device__ __forceinline__ f32x4 multiply(i32x4 w, int ws, const XPiece<FP8>& x, int xs, f32x4 c) {
    const i32x8 a = {w.x, w.y, w.z, w.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, operand<FP8>(x), c, kFp4, FP8 ? kFp8 : kFp4, WB, ws,
                                                            XB, xs);
}

// Row of the weights that lane row `a` (0 .. 15) of tile 0 loads, for output
// columns from n0 on, and how many rows further tile i's row lies.
template <int EPI>
__device__ __forceinline__ int weight_row(int n0, int a) {
    return n0 + (EPI == kPlain ? kNT : kNT / 2) * 4 * (a >> 2) + (a & 3);
}
template <int EPI>
__device__ __forceinline__ int tile_rows(int i, int N) {
    return EPI == kPlain ? 4 * i : (i >= kNT / 2 ? N : 0) + 4 * (i % (kNT / 2));
}

// Byte offset that lies outside every buffer resource here (all are below
// 2^31 bytes).
constexpr int kOutside = (int)0x80000000;

// `at` where i < n, else outside every resource, without a branch (one would
// split the loops below, and matrix instructions would move past it).
__device__ __forceinline__ int offset_if(int at, int i, int n) { return at | (((n - 1 - i) >> 31) & kOutside); }

// gate * sigmoid(gate) * up.  The hardware exponential and reciprocal are good
// to about a unit in the 22nd bit here; the result is rounded to 8 bits or
// fewer.
__device__ __forceinline__ float gated(float gate, float up) {
    const float e = __builtin_amdgcn_exp2f(gate * -0x1.715476p+0f);
    return gate * __builtin_amdgcn_rcpf(1.0f + e) * up;
}

// ---------------------------------------------------------------- the tiles

// Rows of expert e, from expert_offset (packed rows) or counts (`cap` rows
// each), clamped so that no list leads outside the receive buffer.  Beyond the
// experts the list reads zero, which is no rows.
struct Rows {
    const int32_t* list;
    int cap;    // rows per expert, or 0: packed
    int E, nrows;
    __device__ __forceinline__ int at(int i) const {
        const auto r = buffer_rsrc(list, (uint32_t)(E + (cap ? 0 : 1)) * 4u);
        const int v = __builtin_amdgcn_raw_buffer_load_b32(r, i * 4, 0, kCached), hi = cap ? cap : nrows;
        return min(max(v, 0), hi);
    }
    __device__ __forceinline__ int first(int e) const { return cap ? e * cap : at(e); }
    __device__ __forceinline__ int count(int e) const {
        const int lo = at(e), hi = at(e + 1);
        return cap ? lo : max(hi - lo, 0);
    }
};

struct Tile {
    int e;       // expert
    int row0;    // first receive row
    int rows;    // rows of the tile
    int n;       // column tile
};

// Tile number v of the launch, in XCD-contiguous order; false when there is
// none.  Inside an expert, groups of kGroup row tiles take the column tiles in
// turn, so that tiles running at once share weights and rows.  A lane first
// sums the tiles of a run of experts, then the wavefront looks into the run
// that holds the tile.  Every wavefront of a workgroup finds the same tile.
template <int BM>
__device__ __forceinline__ bool find_tile(const Rows& rows, uint32_t ntiles, uint32_t v, Tile& t) {
    constexpr uint32_t kGroup = 4;
    constexpr int kMost = 1024 / kWave;
    const int lane = threadIdx.x & 63, run = (rows.E + kWave - 1) / kWave;
    const auto tiles_of = [&](int e) { return (rows.count(e) + BM - 1) / BM; };
    int mine = 0;
    const auto add = [&](auto first, auto last) {
        int n[decltype(last)::value];
#pragma unroll
        for (int i = first; i < last; ++i) n[i] = tiles_of(lane * run + i);
#pragma unroll
        for (int i = first; i < last; ++i) mine += i < run ? n[i] : 0;
    };
    add(Int<0>(), Int<4>());
    if (run > 4) add(Int<4>(), Int<kMost>());
    int upto = wave_inclusive_sum(mine);
    const uint32_t n = (uint32_t)__builtin_amdgcn_readlane(upto, 63) * ntiles;
    if (v >= n) return false;
    const uint32_t q = n >> 3, r = n & 7, x = v & 7;
    const uint32_t at = x * q + (x < r ? x : r) + (v >> 3);
    const int row_tile = (int)(at / ntiles);  // counting the column tiles within a row tile
    const int owner = __builtin_ctzll(__ballot(upto > row_tile));
    const int before = __builtin_amdgcn_readlane(upto - mine, owner);
    const int e0 = owner * run;
    mine = lane < run ? tiles_of(e0 + lane) : 0;
    upto = wave_inclusive_sum(mine) + before;
    const int l = __builtin_ctzll(__ballot(upto > row_tile));
    const uint32_t have = (uint32_t)__builtin_amdgcn_readlane(mine, l);
    const uint32_t local = at - (uint32_t)__builtin_amdgcn_readlane(upto - mine, l) * ntiles;
    const uint32_t group = local / (kGroup * ntiles), in = local - group * kGroup * ntiles;
    const uint32_t wide = min(kGroup, have - group * kGroup);
    const int m = (int)(group * kGroup + in % wide);
    t.e = e0 + l;
    t.n = (int)(in / wide);
    t.row0 = rows.first(t.e) + m * BM;
    t.rows = min(BM, rows.count(t.e) - m * BM);
    return true;
}

struct Product {
    const uint8_t* x;
    const void* xs;
    const uint8_t* w;
    const uint8_t* ws;
    void* y;
    uint8_t* ys;  // scales of MXFP4 output
    Rows rows;
    int K, N;     // columns of x, columns of y
};

// Buffer resources of a tile's rows and of its expert's weights.
template <bool FP8, int EPI>
struct Sources {
    __amdgpu_buffer_rsrc_t x, xs, w, ws;
    __device__ __forceinline__ Sources(const Product& p, const Tile& t) {
        const uint32_t xrow = FP8 ? p.K : p.K / 2, srow = FP8 ? p.K / 128 * 4 : p.K / 32;
        const uint32_t wrows = EPI == kPlain ? p.N : 2 * p.N;
        x = buffer_rsrc(p.x + (size_t)t.row0 * xrow, t.rows * xrow);
        xs = buffer_rsrc(static_cast<const uint8_t*>(p.xs) + (size_t)t.row0 * srow, t.rows * srow);
        w = buffer_rsrc(p.w + (size_t)t.e * wrows * (p.K / 2), wrows * (uint32_t)(p.K / 2));
        ws = buffer_rsrc(p.ws + (size_t)t.e * wrows * (p.K / 32), wrows * (uint32_t)(p.K / 32));
    }
};

// E8M0 scale of a block of 32 whose largest magnitude has the bits `amax`
// (quant.hip's rule) and the codes of four values under it.
__device__ __forceinline__ uint32_t mx_scale(uint32_t amax) {
    const uint32_t f = amax >> 23;
    return f == 255u ? 255u : (f > 2u ? f - 2u : 0u);
}

__device__ __forceinline__ uint32_t mx_codes4(float a, float b, float c, float d, uint32_t s) {
    const float scale = __uint_as_float(s << 23);
    uint32_t q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, a, b, scale, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, c, d, scale, 1);
    return s == 255u ? 0u : q & 0xFFFFu;
}

// Largest magnitude as bits, so that a NaN among the values stays the largest.
__device__ __forceinline__ uint32_t mag(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// -------------------------------------------------- few rows per expert

// A workgroup takes MT x 16 rows by kCols columns; its KS wavefronts share the
// columns of x among them, STEPS x 128 at a time in turn, and their sums are
// added through LDS in order.  Weights and rows go straight to registers, the
// next piece while the present one is multiplied.
template <bool FP8, int EPI, int MT, int KS, int STEPS>
__global__ __launch_bounds__(64 * KS) void thin_kernel(Product p, int ntiles) {
    constexpr int BM = 16 * MT;
    __shared__ f32x4 part[KS][MT * kNT][kWave];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = lane >> 4, m = lane & 15;
    const int K = p.K, N = p.N, steps = (K + kStep - 1) / kStep, blocks = K / 32;

    struct Piece {
        i32x4 w[STEPS][kNT];
        int ws[STEPS][kNT];
        XPiece<FP8> x[STEPS][MT];
        int xs[STEPS][MT];
    };

    Tile t;
    if (!find_tile<BM>(p.rows, ntiles, blockIdx.x, t)) return;
    {
        const Sources<FP8, EPI> src(p, t);
        const int n0 = t.n * kCols<EPI>;
        // a lane's weight rows are all inside or all outside (N is a multiple
        // of 32); scalar offsets take no part in the bounds check
        const int wrow = weight_row<EPI>(n0, m);
        const int wat = wrow < N ? wrow * (K / 2) + g * 16 : kOutside;
        const int wsat = wrow < N ? wrow * (K / 32) + g : kOutside;
        int xat[MT], xsat[MT];
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            const int row = j * 16 + m;
            xat[j] = row * (FP8 ? K : K / 2) + g * 16;
            xsat[j] = FP8 ? row * (K / 32) : row * (K / 32) + g;
        }
        // past the last step (and the last block of MXFP4 rows) these read zeros
        const auto load = [&](Piece& q, int step0) {
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                const int step = step0 + s, b = step * 4 + g;
                const int wto = offset_if(wat, b, blocks), wsto = offset_if(wsat, b, blocks);
#pragma unroll
                for (int i = 0; i < kNT; ++i) {
                    const int row = tile_rows<EPI>(i, N);
                    q.w[s][i] = __builtin_amdgcn_raw_buffer_load_b128(src.w, wto, row * (K / 2) + step * 64, kCached);
                    q.ws[s][i] =
                        (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(src.ws, wsto, row * blocks + step * 4, kCached);
                }
#pragma unroll
                for (int j = 0; j < MT; ++j) {
                    const int xto = offset_if(xat[j], b, blocks), xsto = offset_if(xsat[j], b, blocks);
                    q.x[s][j].v[0] =
                        __builtin_amdgcn_raw_buffer_load_b128(src.x, xto, step * (FP8 ? 128 : 64), kCached);
                    if constexpr (FP8) {
                        q.x[s][j].v[1] =
                            __builtin_amdgcn_raw_buffer_load_b128(src.x, xto + 64, step * 128, kCached);
                        q.xs[s][j] = __builtin_amdgcn_raw_buffer_load_b32(src.xs, xsto, step * 4, kCached);
                    } else {
                        q.xs[s][j] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(src.xs, xsto, step * 4, kCached);
                    }
                }
            }
        };

        f32x4 acc[MT][kNT];
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
            for (int i = 0; i < kNT; ++i) acc[j][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        const auto use = [&](const Piece& q) {
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
#pragma unroll
                for (int j = 0; j < MT; ++j) {
                    XPiece<FP8> high, low;
                    if constexpr (FP8) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            high.v[h] = upper_codes(q.x[s][j].v[h]);
                            low.v[h] = q.x[s][j].v[h] ^ high.v[h];
                        }
                    }
#pragma unroll
                    for (int i = 0; i < kNT; ++i) {
                        if constexpr (FP8) {
                            f32x4 r = {0.0f, 0.0f, 0.0f, 0.0f};
                            r = multiply<true, 0, 0>(q.w[s][i], q.ws[s][i], low, kUnit, r);
                            r = multiply<true, 0, 0>(q.w[s][i], q.ws[s][i], high, kUnit, r);
                            const float sc = __int_as_float(q.xs[s][j]);
#pragma unroll
                            for (int c = 0; c < 4; ++c) acc[j][i][c] = __builtin_fmaf(sc, r[c], acc[j][i][c]);
                        } else {
                            acc[j][i] = multiply<false, 0, 0>(q.w[s][i], q.ws[s][i], q.x[s][j], q.xs[s][j], acc[j][i]);
                        }
                    }
                }
            }
        };
        constexpr int kRun = KS * STEPS;
        Piece a, b;
        load(a, wave * STEPS);
        for (int at = wave * STEPS; at < steps; at += 2 * kRun) {
            load(b, at + kRun);
            use(a);
            load(a, at + 2 * kRun);
            use(b);
        }

#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
            for (int i = 0; i < kNT; ++i) part[wave][j * kNT + i][lane] = acc[j][i];
        __syncthreads();
        const auto sum = [&](int tile, int from) {
            f32x4 s = part[0][tile][from];
#pragma unroll
            for (int w = 1; w < KS; ++w) {
                const f32x4 o = part[w][tile][from];
#pragma unroll
                for (int c = 0; c < 4; ++c) s[c] += o[c];
            }
            return s;
        };
        // four columns of a row to a thread, the threads of a row side by side
        constexpr int kPer = kCols<EPI> / 4;
        for (int q = threadIdx.x; q < BM * kPer; q += 64 * KS) {
            const int row = q / kPer, c = q % kPer;      // c = (kNT or kNT / 2) g + i
            constexpr int kI = EPI == kPlain ? kNT : kNT / 2;
            const int from = (c / kI) * 16 + (row & 15), tile = (row >> 4) * kNT + c % kI;
            f32x4 o = sum(tile, from);
            const int n = n0 + 4 * c;
            const size_t yrow = (size_t)t.row0 + row;
            const bool on = row < t.rows && n < N;
            if constexpr (EPI != kPlain) {
                const f32x4 up = sum(tile + kI, from);
#pragma unroll
                for (int i = 0; i < 4; ++i) o[i] = gated(o[i], up[i]);
            }
            if constexpr (EPI != kGatedMx) {
                if (on) {
                    uint2 d;
                    d.x = pack_bf16x2(o[0], o[1]);
                    d.y = pack_bf16x2(o[2], o[3]);
                    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.y) + yrow * N + n) = d;
                }
            } else {
                // eight adjacent threads hold a block of 32
                uint32_t a = max(max(mag(o[0]), mag(o[1])), max(mag(o[2]), mag(o[3])));
                a = max(a, dpp_u32<kDppXor1>(a));
                a = max(a, dpp_u32<kDppXor2>(a));
                a = max(a, dpp_u32<kDppHalfMirror>(a));
                const uint32_t s = mx_scale(a);
                if (on) {
                    *reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(p.y) + (yrow * N + n) / 2) =
                        (uint16_t)mx_codes4(o[0], o[1], o[2], o[3], s);
                    if (c == 0) p.ys[yrow * (N / 32) + n / 32] = (uint8_t)s;
                }
            }
        }
    }
}

// ------------------------------------------------- many rows per expert

// A workgroup takes 128 rows by 8 x kCols columns with 8 wavefronts side by
// side, each all 128 rows by kCols columns.  The rows of a 128-column step go
// through LDS (two buffers), as do the weights' scales of four steps at a
// time, turned so that a lane reads its four tiles' bytes at once; a
// wavefront's weights are its own and go straight to registers, several steps
// ahead.  Every step has one barrier.  Tiles of up to 64 rows multiply only half.
constexpr int kTileWaves = 8, kTileMT = 8, kTileRows = 16 * kTileMT, kTileThreads = 64 * kTileWaves;

template <bool FP8, int EPI>
__global__ __launch_bounds__(kTileThreads, 1) void tile_kernel(Product p, int ntiles) {
    constexpr int kMT = kTileMT;
    constexpr int kChunks = FP8 ? 8 : 4;                         // 16-byte chunks of a row's step
    constexpr int kPer = kTileRows * kChunks / kTileThreads;     // chunks staged by a thread
    constexpr int kParts = FP8 ? 2 : 1;                          // FP8: low codes, then high codes
    constexpr int kWSets = 2, kXSets = FP8 ? 1 : 2;    // steps of weights and rows in registers
    __shared__ i32x4 rows_lds[2][kParts][kTileRows * kChunks];
    __shared__ __align__(16) uint8_t xs_lds[2][kTileRows * 4];
    __shared__ __align__(16) uint8_t ws_lds[2][4][kTileThreads * 4];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g = lane >> 4, m = lane & 15;
    const int K = p.K, N = p.N, steps = (K + kStep - 1) / kStep, blocks = K / 32;

    // 16-byte chunk c of row r lies at a place of its own in the row, so that
    // the eight rows read together fall into different banks
    const auto place = [](int r, int c) {
        if constexpr (FP8) return r * kChunks + (c ^ (r & 7));
        else return r * kChunks + (c ^ ((r >> 1) & 3));
    };

    Tile t;
    if (!find_tile<kTileRows>(p.rows, ntiles, blockIdx.x, t)) return;
    const Sources<FP8, EPI> src(p, t);
    const int n0 = (t.n * kTileWaves + wave) * kCols<EPI>;

    // this lane's weights
    const int wrow = weight_row<EPI>(n0, m);
    const int wat = wrow < N ? wrow * (K / 2) + g * 16 : kOutside;
    // this thread's chunks of the rows: chunk tid and those kStride rows apart
    constexpr int kStride = kTileThreads / kChunks;
    const int xrow = tid / kChunks, xbytes = FP8 ? K : K / 2;
    const int xat = xrow * xbytes + tid % kChunks * 16;
    const int xto = place(xrow, tid % kChunks);
    // its row scale: FP8 one of a row (four threads the same), MXFP4 one byte;
    // row 16 i + c lies at 8 c + i, where the lanes c read their eight rows
    const int srow = tid >> 2, sto = (srow & 15) * 8 + (srow >> 4);
    // its weight row's scales: tile i, lane row a of this wavefront's tiles
    const int vtile = lane >> 4, vrow = weight_row<EPI>(n0, m) + tile_rows<EPI>(vtile, N);
    const int vat = wrow < N ? vrow * blocks : kOutside;
    const int vshift = vat & 3;  // rows of scales need not be a multiple of 4 bytes

    struct Staged {
        i32x4 x[kPer];
        int xs;
    };
    struct Scales {
        i32x4 v;
        int more;
    };
    const auto load_rows = [&](Staged& q, int step) {
        const int i = FP8 ? step : step * 4 + (tid & 3), n = FP8 ? steps : blocks;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int at = offset_if(xat + j * kStride * xbytes, i, n);
            q.x[j] = __builtin_amdgcn_raw_buffer_load_b128(src.x, at, step * (FP8 ? 128 : 64), kCached);
        }
        if constexpr (FP8) {
            q.xs = __builtin_amdgcn_raw_buffer_load_b32(src.xs, offset_if(srow * blocks, i, n), step * 4, kCached);
        } else {
            const int at = offset_if(srow * blocks + (tid & 3), i, n);
            q.xs = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(src.xs, at, step * 4, kCached);
        }
    };
    const auto store_rows = [&](const Staged& q, int buf) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int to = xto + j * kStride * kChunks;
            if constexpr (FP8) {
                const i32x4 high = upper_codes(q.x[j]);
                rows_lds[buf][0][to] = q.x[j] ^ high;
                rows_lds[buf][kParts - 1][to] = high;
            } else {
                rows_lds[buf][0][to] = q.x[j];
            }
        }
        if constexpr (FP8) *reinterpret_cast<int*>(&xs_lds[buf][sto * 4]) = q.xs;
        else xs_lds[buf][(tid & 3) * kTileRows + sto] = (uint8_t)q.xs;
    };
    const auto load_weights = [&](i32x4 (&w)[kNT], int step) {
        const int at = offset_if(wat, step * 4 + g, blocks);
#pragma unroll
        for (int i = 0; i < kNT; ++i)
            w[i] = __builtin_amdgcn_raw_buffer_load_b128(src.w, at, tile_rows<EPI>(i, N) * (K / 2) + step * 64,
                                                         kCached);
    };
    // the scales of steps 4 four .. 4 four + 3: 16 bytes of a row, from the
    // aligned words that hold them
    const auto load_scales = [&](Scales& q, int four) {
        const int at = offset_if(vat - vshift, four * 16, blocks);
        q.v = __builtin_amdgcn_raw_buffer_load_b128(src.ws, at, four * 16, kCached);
        q.more = __builtin_amdgcn_raw_buffer_load_b32(src.ws, offset_if(at + 16, 0, vshift), four * 16, kCached);
    };
    const auto store_scales = [&](const Scales& q, int four) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const uint32_t lo = (uint32_t)q.v[s], hi = (uint32_t)(s < 3 ? q.v[s < 3 ? s + 1 : 3] : q.more);
            const uint32_t d = __builtin_amdgcn_alignbyte(hi, lo, (uint32_t)vshift);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const bool in = four * 16 + s * 4 + b < blocks;  // bytes past the row are another row's
                ws_lds[four & 1][s][wave * 256 + (b * 16 + m) * 4 + vtile] = in ? (uint8_t)(d >> (8 * b)) : 0;
            }
        }
    };

    f32x4 acc[kMT][kNT];
#pragma unroll
    for (int j = 0; j < kMT; ++j)
#pragma unroll
        for (int i = 0; i < kNT; ++i) acc[j][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    constexpr int kHold = FP8 ? 1 : 4;  // row tiles read from LDS at a time
    const int rx0 = place(m, g), rx1 = place(m, FP8 ? g + 4 : g);
    const auto compute = [&](auto halves, const i32x4 (&w)[kNT], int buf, int step) {
        const int ws = *reinterpret_cast<const int*>(&ws_lds[(step >> 2) & 1][step & 3][wave * 256 + lane * 4]);
        // row tiles H .. H + kHold - 1
        const auto rows = [&](auto first) {
            constexpr int H = decltype(first)::value;
            XPiece<FP8> x[kHold], high[kHold];
#pragma unroll
            for (int j = 0; j < kHold; ++j) {
                x[j].v[0] = rows_lds[buf][0][rx0 + (H + j) * 16 * kChunks];
                if constexpr (FP8) {
                    x[j].v[1] = rows_lds[buf][0][rx1 + (H + j) * 16 * kChunks];
                    high[j].v[0] = rows_lds[buf][kParts - 1][rx0 + (H + j) * 16 * kChunks];
                    high[j].v[1] = rows_lds[buf][kParts - 1][rx1 + (H + j) * 16 * kChunks];
                }
            }
            if constexpr (FP8) {
                const float sc = *reinterpret_cast<const float*>(&xs_lds[buf][(m * kMT + H) * 4]);
                f32x4 r[kNT];
                const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
                r[0] = multiply<true, 0, 0>(w[0], ws, x[0], kUnit, zero);
                r[1] = multiply<true, 1, 0>(w[1], ws, x[0], kUnit, zero);
                r[2] = multiply<true, 2, 0>(w[2], ws, x[0], kUnit, zero);
                r[3] = multiply<true, 3, 0>(w[3], ws, x[0], kUnit, zero);
                r[0] = multiply<true, 0, 0>(w[0], ws, high[0], kUnit, r[0]);
                r[1] = multiply<true, 1, 0>(w[1], ws, high[0], kUnit, r[1]);
                r[2] = multiply<true, 2, 0>(w[2], ws, high[0], kUnit, r[2]);
                r[3] = multiply<true, 3, 0>(w[3], ws, high[0], kUnit, r[3]);
#pragma unroll
                for (int i = 0; i < kNT; ++i) {
                    const f32x4 o = acc[H][i];
                    acc[H][i] = f32x4{__builtin_fmaf(sc, r[i][0], o[0]), __builtin_fmaf(sc, r[i][1], o[1]),
                                      __builtin_fmaf(sc, r[i][2], o[2]), __builtin_fmaf(sc, r[i][3], o[3])};
                }
            } else {
                const int sc = *reinterpret_cast<const int*>(&xs_lds[buf][g * kTileRows + m * kMT + H]);
                const auto column = [&](auto i) {
                    constexpr int I = decltype(i)::value;
                    acc[H + 0][I] = multiply<false, I, 0>(w[I], ws, x[0], sc, acc[H + 0][I]);
                    acc[H + 1][I] = multiply<false, I, 1>(w[I], ws, x[1 % kHold], sc, acc[H + 1][I]);
                    acc[H + 2][I] = multiply<false, I, 2>(w[I], ws, x[2 % kHold], sc, acc[H + 2][I]);
                    acc[H + 3][I] = multiply<false, I, 3>(w[I], ws, x[3 % kHold], sc, acc[H + 3][I]);
                };
                column(Int<0>()), column(Int<1>()), column(Int<2>()), column(Int<3>());
            }
        };
        const auto half = [&](auto first) {
            constexpr int H = decltype(first)::value;
            rows(Int<H>());
            if constexpr (kHold == 1) rows(Int<H + 1>()), rows(Int<H + 2>()), rows(Int<H + 3>());
        };
        half(Int<0>());
        if constexpr (halves > 1) half(Int<4>());
    };

    Staged st[kXSets];
    i32x4 w[kWSets][kNT];
    Scales sc;
    load_scales(sc, 0);
    load_rows(st[0], 0);
#pragma unroll
    for (int i = 0; i + 1 < kWSets; ++i) load_weights(w[i], i);
    store_scales(sc, 0);
    store_rows(st[0], 0);
#pragma unroll
    for (int i = 1; i <= kXSets; ++i) load_rows(st[i % kXSets], i);
    // Step s: its rows and scales are in LDS when every wavefront is past the
    // barrier, and the other buffers are no longer read.  Four steps at a time,
    // without conditions: loads past the last step read zeros, which add
    // nothing, and each wait counts exactly what is in flight.
    const auto loop = [&](auto halves) {
        for (int s = 0; s < steps; s += 4) {
            const auto body = [&](auto phase) {
                constexpr int I = decltype(phase)::value;
                __syncthreads();
                __builtin_amdgcn_sched_barrier(0);
                if constexpr (I == 0) load_scales(sc, (s >> 2) + 1);
                store_rows(st[(I + 1) % kXSets], (I + 1) & 1);
                load_rows(st[(I + 1) % kXSets], s + I + 1 + kXSets);
                load_weights(w[(I + kWSets - 1) % kWSets], s + I + kWSets - 1);
                __builtin_amdgcn_sched_barrier(0);
                compute(halves, w[I % kWSets], I & 1, s + I);
                if constexpr (I == 3) store_scales(sc, (s >> 2) + 1);
            };
            body(Int<0>()), body(Int<1>()), body(Int<2>()), body(Int<3>());
        }
    };
    if (t.rows > 64) loop(Int<2>());
    else loop(Int<1>());

    // the sums are final here, with every lane active (the matrix instructions
    // must not move into the guarded stores below)
#pragma unroll
    for (int j = 0; j < kMT; ++j)
#pragma unroll
        for (int i = 0; i < kNT; ++i) asm volatile("" : "+v"(acc[j][i]));

    // lane (g, m): row 16 j + m, consecutive columns
#pragma unroll
    for (int j = 0; j < kMT; ++j) {
        const int row = j * 16 + m;
        const size_t yrow = (size_t)t.row0 + row;
        if constexpr (EPI == kPlain) {
            const int n = n0 + 16 * g;
            if (row < t.rows && n < N) {
                i32x4* to = reinterpret_cast<i32x4*>(static_cast<uint16_t*>(p.y) + yrow * N + n);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const f32x4 a = acc[j][2 * h], b = acc[j][2 * h + 1];
                    to[h] = i32x4{(int)pack_bf16x2(a[0], a[1]), (int)pack_bf16x2(a[2], a[3]),
                                  (int)pack_bf16x2(b[0], b[1]), (int)pack_bf16x2(b[2], b[3])};
                }
            }
        } else {
            const int n = n0 + 8 * g;
            f32x4 a, b;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                a[c] = gated(acc[j][0][c], acc[j][2][c]);
                b[c] = gated(acc[j][1][c], acc[j][3][c]);
            }
            if constexpr (EPI == kGated) {
                if (row < t.rows && n < N)
                    *reinterpret_cast<i32x4*>(static_cast<uint16_t*>(p.y) + yrow * N + n) =
                        i32x4{(int)pack_bf16x2(a[0], a[1]), (int)pack_bf16x2(a[2], a[3]),
                              (int)pack_bf16x2(b[0], b[1]), (int)pack_bf16x2(b[2], b[3])};
            } else {
                // the four lanes of a row hold a block of 32
                uint32_t x = 0u;
#pragma unroll
                for (int c = 0; c < 4; ++c) x = max(x, max(mag(a[c]), mag(b[c])));
                x = max(x, (uint32_t)__shfl_xor((int)x, 16, kWave));
                x = max(x, (uint32_t)__shfl_xor((int)x, 32, kWave));
                const uint32_t e = mx_scale(x);
                if (row < t.rows && n < N) {
                    *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.y) + (yrow * N + n) / 2) =
                        mx_codes4(a[0], a[1], a[2], a[3], e) | mx_codes4(b[0], b[1], b[2], b[3], e) << 16;
                    if (g == 0) p.ys[yrow * (N / 32) + n / 32] = (uint8_t)e;
                }
            }
        }
    }
}

// Launches one workgroup for every tile there can be (none where that many
// cannot be launched; no receive buffer this GPU holds gets there).
template <int BM, class Kernel>
hipError_t launch_tiles(Kernel kernel, const Product& p, long pairs, int cols, int threads, hipStream_t stream) {
    const int ntiles = (p.N + cols - 1) / cols;
    const long grid = (pairs / BM + (pairs < p.rows.E ? pairs : p.rows.E)) * ntiles;
    if (grid * threads >= 1L << 32) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL(kernel, dim3((uint32_t)grid), dim3(threads), 0, stream, p, ntiles);
    return hipGetLastError();
}

template <bool FP8, int EPI>
hipError_t launch_one(const Product& p, long pairs, hipStream_t stream) {
    if (pairs / p.rows.E < 32)
        return launch_tiles<16>(thin_kernel<FP8, EPI, 1, 4, 2>, p, pairs, kCols<EPI>, 256, stream);
    return launch_tiles<kTileRows>(tile_kernel<FP8, EPI>, p, pairs, kTileWaves * kCols<EPI>, kTileThreads, stream);
}

template <bool FP8>
hipError_t launch_epilogue(const Product& p, int epi, long pairs, hipStream_t stream) {
    if (epi == kPlain) return launch_one<FP8, kPlain>(p, pairs, stream);
    if (epi == kGated) return launch_one<FP8, kGated>(p, pairs, stream);
    return launch_one<FP8, kGatedMx>(p, pairs, stream);
}

}  // namespace

hipError_t launch_expert_product(const Shape& s, int cap, bool fp8, bool gate, bool mx_out, int K, int N,
                                 const uint8_t* x, const void* xs, const int32_t* list, const uint8_t* w,
                                 const uint8_t* ws, void* y, uint8_t* ys, hipStream_t stream) {
    const long pairs = (long)s.T * s.k;
    if (pairs == 0) return hipSuccess;
    const Product p{x, xs, w, ws, y, ys, Rows{list, cap, s.E, cap ? s.E * cap : (int)pairs}, K, N};
    const int epi = gate ? (mx_out ? kGatedMx : kGated) : kPlain;
    return fp8 ? launch_epilogue<true>(p, epi, pairs, stream) : launch_epilogue<false>(p, epi, pairs, stream);
}

}  // namespace ep
