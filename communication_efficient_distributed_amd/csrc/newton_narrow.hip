// newton_narrow.hip -- the matrix update for matrices whose shorter side m is
// at most 128 and whose longer one is eight times that or more (attention
// heads), fp16 products.
//
// Every step multiplies X by a polynomial of its Gram matrix, so all of them
// can be worked out on m x m matrices: with R = X X^T, for each (a, b, c)
//     P = a I + b R + c R R,   R <- P R P,   Q <- Q P
// and at the end O = Q X.  Only the first Gram matrix and the last product
// touch the long side; the steps between run in one workgroup per matrix with
// R and P in LDS.  Against three products of the long side for each step that
// is 4 launches instead of 17 and two passes over X instead of fifteen.
//
// The m x m products take operands as the sum of two fp16 values (22 bits) and
// their linear terms from fp32 registers: an error in R's small eigenvalues grows
// with them, which 11 bits would not survive.  X is fp16 as in the other way;
// Q, whose entries grow up to `growth`, multiplies it as two terms.
//
// Bound by latency: eight 8192 x 128 bf16 take 85 us, of which the steps on
// one compute unit each are 39 (VALU and LDS, writing pairs), the last product
// 23, the Gram matrices 15 with their join 6, the norms 6; the 34 MB in and
// out alone would take 5.
#include "newton.h"

namespace sl {
namespace {

constexpr int kSide = (int)kNarrow;
constexpr int kTileBytes = kSide * kSide * 2;            // one 128 x 128 fp16 array
constexpr float kScaleX = 8192.0f, kScaleR = 2048.0f, kScaleP = 512.0f;
constexpr int kTriangle = 10;                            // 32 x 32 tiles on and below the diagonal
constexpr float kMaxGrowth = 2048.0f;

// The 16-byte piece c of row r of a 128 x 128 array in LDS sits at position
// c ^ fold(r): 16 rows read at one piece, or pieces written down 16 rows that
// are 8 apart, meet all 64 banks.
__device__ __forceinline__ int fold(int r) { return (r ^ (r >> 3)) & 15; }
__device__ __forceinline__ int cell(int r, int c) { return r * kSide + ((c >> 3) ^ fold(r)) * 8 + (c & 7); }

__device__ __forceinline__ half8 fragment(const _Float16* lds, int block, int sub) {
    const int lane = lane_id(), r = block * 32 + (lane & 31);
    return *reinterpret_cast<const half8*>(lds + r * kSide + ((sub * 2 + (lane >> 5)) ^ fold(r)) * 8);
}

// Tile t of the triangle: (0,0) (1,0) (1,1) (2,0) ...
__device__ __forceinline__ void triangle_tile(int t, int* ti, int* tj) {
    int i = 0;
    while (t > i) t -= ++i;
    *ti = i;
    *tj = t;
}

struct NarrowArgs {
    Source s;
    int64_t rows, cols;
    bool vector;       // eight elements at a time are aligned
    int64_t m;         // the short side
    const double* partial;
    int n_partial;
    float eps;
};

// Eight values of u along a row, zero beyond the matrix.
__device__ __forceinline__ void load_row8(const NarrowArgs& a, int64_t matrix, int64_t r, int64_t c, float* u) {
    const Source& s = a.s;
    const int64_t at = matrix * s.stride + r * s.ld + c, am = (matrix * a.rows + r) * a.cols + c;
    const bool from_x = !s.momentum || s.nesterov;
    float m[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) u[e] = m[e] = 0;
    if (r < a.rows) {
        if (a.vector) {
            if (c < a.cols) {
                if (from_x) load_values8(s.x, s.type, at, u);
                if (s.momentum) load_values8(s.momentum, SL_F32, am, m);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (c + e < a.cols) {
                    if (from_x) u[e] = load_value(s.x, s.type, at + e);
                    if (s.momentum) m[e] = s.momentum[am + e];
                }
        }
    }
    if (s.momentum)
#pragma unroll
        for (int e = 0; e < 8; ++e) u[e] = s.nesterov ? __builtin_fmaf(s.decay, m[e], u[e] * s.grad_scale) : m[e];
}

// The tile of X from (r0, c0) of the matrix into LDS as fp16: ROWS x 128
// elements with rows as they are, or (TURN) 128 x ROWS with columns as rows.
// 256 threads.
template <int ROWS, bool TURN>
__device__ __forceinline__ void load_tile(const NarrowArgs& a, int64_t matrix, int64_t r0, int64_t c0, Scale scale,
                                          _Float16* lds) {
    if (TURN) {  // 8 x 8 elements per thread, turned in registers
        const int block = threadIdx.x % (ROWS / 8), row = threadIdx.x / (ROWS / 8);
        if (row >= 16) return;
        half8 h[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            float u[8];
            load_row8(a, matrix, r0 + row * 8 + k, c0 + block * 8, u);
#pragma unroll
            for (int e = 0; e < 8; ++e) h[e][k] = (_Float16)scale(u[e]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) *reinterpret_cast<half8*>(lds + cell(block * 8 + e, row * 8)) = h[e];
    } else {
        const int block = threadIdx.x & 15, row = threadIdx.x >> 4;
#pragma unroll
        for (int k = 0; k < ROWS / 16; ++k) {
            float u[8];
            load_row8(a, matrix, r0 + row + 16 * k, c0 + block * 8, u);
            half8 h;
#pragma unroll
            for (int e = 0; e < 8; ++e) h[e] = (_Float16)scale(u[e]);
            *reinterpret_cast<half8*>(lds + cell(row + 16 * k, block * 8)) = h;
        }
    }
}

// Sums of the Gram matrix over tiles slice, slice + slices, ... of the long
// side: part[(matrix * slices + slice) * 10 + tile][register / 4][lane].
template <bool TALL>
__global__ __launch_bounds__(256, 2) void narrow_gram_kernel(NarrowArgs a, int64_t long_tiles, float4* part) {
    __shared__ __attribute__((aligned(128))) _Float16 x[kSide * kSide];
    __shared__ double sums[4];
    const int64_t matrix = blockIdx.y;
    const int wave = uniform(threadIdx.x >> 6), lane = lane_id();
    const int blocks = (int)(a.m + 31) / 32, tiles = blocks * (blocks + 1) / 2;
    const Scale scale = start_scale(kScaleX, a.partial, a.n_partial, matrix, a.eps, sums);
    float16v acc[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) acc[k] = 0.0f;
    for (int64_t t = blockIdx.x; t < long_tiles; t += gridDim.x) {
        if constexpr (TALL)
            load_tile<kSide, true>(a, matrix, t * kSide, 0, scale, x);
        else
            load_tile<kSide, false>(a, matrix, 0, t * kSide, scale, x);
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            int ti, tj;
            if (wave + 4 * k < tiles) {
                triangle_tile(wave + 4 * k, &ti, &tj);
#pragma unroll
                for (int sub = 0; sub < 8; ++sub)
                    acc[k] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fragment(x, ti, sub), fragment(x, tj, sub), acc[k], 0, 0, 0);
            }
        }
        __syncthreads();
    }
    part += (matrix * gridDim.x + blockIdx.x) * (kTriangle * 4 * kWave) + lane;
#pragma unroll
    for (int k = 0; k < 3; ++k)
        if (wave + 4 * k < tiles)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                part[((wave + 4 * k) * 4 + r) * kWave] =
                    make_float4(acc[k][r * 4], acc[k][r * 4 + 1], acc[k][r * 4 + 2], acc[k][r * 4 + 3]);
}

// Adds up the slices of tile blockIdx.x of the triangle: the four wavefronts a
// quarter of the slices each, in order, then the quarters.
__global__ __launch_bounds__(256) void narrow_join_kernel(int slices, const float4* part, float4* gram) {
    __shared__ float4 quarters[3][4][kWave];
    const int lane = lane_id(), wave = uniform(threadIdx.x >> 6);
    const int64_t matrix = blockIdx.y;
    const int from = slices * wave / 4, to = slices * (wave + 1) / 4;
    part += ((matrix * slices + from) * kTriangle + blockIdx.x) * 4 * kWave + lane;
    float4 sum[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) sum[r] = make_float4(0, 0, 0, 0);
#pragma unroll 4
    for (int s = from; s < to; ++s, part += kTriangle * 4 * kWave)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float4 v = part[r * kWave];
            sum[r].x += v.x, sum[r].y += v.y, sum[r].z += v.z, sum[r].w += v.w;
        }
    if (wave)
#pragma unroll
        for (int r = 0; r < 4; ++r) quarters[wave - 1][r][lane] = sum[r];
    __syncthreads();
    if (wave) return;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
#pragma unroll
        for (int w = 0; w < 3; ++w) {
            const float4 v = quarters[w][r][lane];
            sum[r].x += v.x, sum[r].y += v.y, sum[r].z += v.z, sum[r].w += v.w;
        }
        gram[((matrix * kTriangle + blockIdx.x) * 4 + r) * kWave + lane] = sum[r];
    }
}

struct Steps {
    Quintic k[SL_MAX_STEPS];
    int n;
};

// One matrix per workgroup, one 32 x 32 tile of the triangle per wavefront:
// lane l, register r holds row 8 (r / 4) + 4 (l / 32) + r % 4, column l % 32 of
// the tile of every m x m matrix, in fp32.  Writes Q times scale_q as fp16
// pairs, hi then lo, rows of 128.
// BLOCKS: m in blocks of 32.
template <int BLOCKS>
__global__ __launch_bounds__(BLOCKS*(BLOCKS + 1) / 2 * kWave) void narrow_steps_kernel(const float4* gram, int slices, Steps steps,
                                                                                       float scale_q, _Float16* q_out) {
    __shared__ __attribute__((aligned(128))) _Float16 pool[4 * kSide * kSide];  // two pairs of 128 x 128
    _Float16* const first = pool;
    _Float16* const second = pool + 2 * kSide * kSide;
    const int lane = lane_id(), t = uniform(threadIdx.x >> 6);
    int ti, tj;
    triangle_tile(t, &ti, &tj);
    const int j = lane & 31, i4 = 4 * (lane >> 5);
    // Where the tile's rows of four go in a pair, and the elements of its mirror image.
    int direct[4], mirror[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        mirror[r] = cell(ti * 32 + (r >> 2) * 8 + i4 + (r & 3), tj * 32 + j);
        if ((r & 3) == 0) direct[r >> 2] = cell(tj * 32 + j, ti * 32 + (r >> 2) * 8 + i4);
    }
    const bool turned = ti != tj;
    // To a pair in LDS: hi is cut off towards zero, lo the rest (2^-21 of the
    // value at most stays behind), which takes half the instructions that two
    // rounded conversions would; those, not the products, bound the kernel.
    auto put = [&](_Float16* to, const float16v& v) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const half2 h0 = __builtin_bit_cast(half2, __builtin_amdgcn_cvt_pkrtz(v[r * 4], v[r * 4 + 1]));
            const half2 h1 = __builtin_bit_cast(half2, __builtin_amdgcn_cvt_pkrtz(v[r * 4 + 2], v[r * 4 + 3]));
            const half2 l0 = __builtin_bit_cast(
                half2, __builtin_amdgcn_cvt_pkrtz(__builtin_fmaf((float)h0[0], -1.0f, v[r * 4]), __builtin_fmaf((float)h0[1], -1.0f, v[r * 4 + 1])));
            const half2 l1 = __builtin_bit_cast(
                half2, __builtin_amdgcn_cvt_pkrtz(__builtin_fmaf((float)h1[0], -1.0f, v[r * 4 + 2]), __builtin_fmaf((float)h1[1], -1.0f, v[r * 4 + 3])));
            *reinterpret_cast<half4*>(to + direct[r]) = half4{h0[0], h0[1], h1[0], h1[1]};
            *reinterpret_cast<half4*>(to + direct[r] + kSide * kSide) = half4{l0[0], l0[1], l1[0], l1[1]};
            if (turned) {
                to[mirror[r * 4]] = h0[0], to[mirror[r * 4] + kSide * kSide] = l0[0];
                to[mirror[r * 4 + 1]] = h0[1], to[mirror[r * 4 + 1] + kSide * kSide] = l0[1];
                to[mirror[r * 4 + 2]] = h1[0], to[mirror[r * 4 + 2] + kSide * kSide] = l1[0];
                to[mirror[r * 4 + 3]] = h1[1], to[mirror[r * 4 + 3] + kSide * kSide] = l1[1];
            }
        }
    };
    // The product of two symmetric pairs that commute: symmetric too.
    auto product = [&](const _Float16* a, const _Float16* b, float scale) {
        float16v sum, cross;  // two chains of dependent instructions
#pragma unroll
        for (int r = 0; r < 16; ++r) sum[r] = cross[r] = 0;
#pragma unroll 4
        for (int sub = 0; sub < 2 * BLOCKS; ++sub) {
            const half8 ah = fragment(a, ti, sub), al = fragment(a + kSide * kSide, ti, sub);
            const half8 bh = fragment(b, tj, sub), bl = fragment(b + kSide * kSide, tj, sub);
            cross = __builtin_amdgcn_mfma_f32_32x32x16_f16(al, bh, cross, 0, 0, 0);
            sum = __builtin_amdgcn_mfma_f32_32x32x16_f16(ah, bh, sum, 0, 0, 0);
            cross = __builtin_amdgcn_mfma_f32_32x32x16_f16(ah, bl, cross, 0, 0, 0);
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) sum[r] = (sum[r] + cross[r]) * scale;
        return sum;
    };

    // R times kScaleR, P times kScaleP, Q times scale_q: powers of two, so that
    // registers and LDS hold the same values.
    float16v rr, q;
#pragma unroll
    for (int r = 0; r < 16; ++r) rr[r] = q[r] = 0;
    gram += ((int64_t)blockIdx.x * slices * kTriangle + t) * 4 * kWave + lane;
    for (int s = 0; s < slices; ++s, gram += kTriangle * 4 * kWave)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float4 v = gram[r * kWave];
            rr[r * 4] += v.x, rr[r * 4 + 1] += v.y, rr[r * 4 + 2] += v.z, rr[r * 4 + 3] += v.w;
        }
#pragma unroll
    for (int r = 0; r < 16; ++r) rr[r] *= kScaleR / (kScaleX * kScaleX);
    put(first, rr);
    for (int k = 0; k < steps.n; ++k) {
        const Quintic z = steps.k[k];
        __syncthreads();
        float16v p = product(first, first, z.c * (kScaleP / (kScaleR * kScaleR)));
        const float zb = z.b * (kScaleP / kScaleR);
#pragma unroll
        for (int r = 0; r < 16; ++r) p[r] = __builtin_fmaf(zb, rr[r], p[r]);
        if (!turned) {
            const float za = z.a * kScaleP;
#pragma unroll
            for (int r = 0; r < 16; ++r)
                if (j == (r >> 2) * 8 + i4 + (r & 3)) p[r] += za;
        }
        put(second, p);
        const bool last = k + 1 == steps.n;
        if (!last) {  // R <- (P R) P
            __syncthreads();
            const float16v pr = product(second, first, 1.0f / kScaleP);
            __syncthreads();
            put(first, pr);
            __syncthreads();
            rr = product(first, second, 1.0f / kScaleP);
        }
        if (k == 0) {
#pragma unroll
            for (int r = 0; r < 16; ++r) q[r] = p[r] * (scale_q / kScaleP);
        } else {  // Q <- Q P
            __syncthreads();
            put(first, q);
            __syncthreads();
            q = product(first, second, 1.0f / kScaleP);
        }
        if (!last) {
            __syncthreads();
            put(first, rr);
        }
    }
    __syncthreads();
    put(first, q);
    __syncthreads();
    // Straight rows to memory; what lies beyond m was never set and is zero here.
    _Float16* const out = q_out + (int64_t)blockIdx.x * 2 * kSide * kSide;
    constexpr int used = BLOCKS * 32;
    for (int at = threadIdx.x; at < 2 * kSide * kSide / 8; at += blockDim.x) {
        const int part_of = at / (kSide * kSide / 8), r = at / (kSide / 8) % kSide, c = at % (kSide / 8) * 8;
        half8 v = {0, 0, 0, 0, 0, 0, 0, 0};
        if (r < used && c < used) v = *reinterpret_cast<const half8*>(first + part_of * kSide * kSide + cell(r, c));
        *reinterpret_cast<half8*>(out + at * 8) = v;
    }
}

struct NarrowOut {
    MatrixView out;
    bool aligned;
    bool update;
    float keep, move;
    float scale;  // of the sums
};

constexpr int kApply = 64;  // of the long side at a time: two blocks' LDS fit a compute unit

// O = Q X over tiles along the long side, Q staying in LDS.  The four
// consecutive elements of a lane run along out's rows: the first operand is Q
// for a tall matrix and X for a wide one.
template <bool TALL>
__global__ __launch_bounds__(256, 2) void narrow_apply_kernel(NarrowArgs a, int64_t long_tiles, const _Float16* q_in, NarrowOut o) {
    __shared__ __attribute__((aligned(128))) _Float16 pool[(2 * kSide + kApply) * kSide];
    _Float16* const q = pool;  // hi, lo
    _Float16* const x = pool + 2 * kSide * kSide;
    const int64_t matrix = blockIdx.y;
    const int wave = uniform(threadIdx.x >> 6), lane = lane_id();
    // Four rows of 16 pieces with each instruction, each piece to its place.
    q_in += matrix * 2 * kSide * kSide;
#pragma unroll 2
    for (int k = 0; k < 16; ++k) {
        const int r4 = (k * 4 + wave) * 4, r = r4 + (lane >> 4);  // of hi and lo together
        load_to_lds(q_in + r * kSide + ((lane & 15) ^ fold(r)) * 8, q + r4 * kSide);
    }
    const Scale scale = start_scale(kScaleX, a.partial, a.n_partial, matrix, a.eps, reinterpret_cast<double*>(x));
    const int subs = (int)(a.m + 15) / 16;
    for (int64_t t = blockIdx.x; t < long_tiles; t += gridDim.x) {
        __syncthreads();
        if constexpr (TALL)
            load_tile<kApply, false>(a, matrix, t * kApply, 0, scale, x);
        else
            load_tile<kApply, true>(a, matrix, 0, t * kApply, scale, x);
        arrive();  // the copies of Q among the rest
        // This wavefront's two 32 x 32 blocks: i (rows of the first operand) from i0, j from j0.
        const int i0 = TALL ? wave >> 1 << 6 : 0, j0 = (TALL ? wave & 1 : wave) * 32;
        float16v acc[2];
        acc[0] = acc[1] = 0.0f;
        for (int sub = 0; sub < subs; ++sub) {
            if constexpr (TALL) {
                const half8 f = fragment(x, wave & 1, sub);
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const int block = (wave >> 1) * 2 + b;
                    acc[b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fragment(q + kSide * kSide, block, sub), f, acc[b], 0, 0, 0);
                    acc[b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fragment(q, block, sub), f, acc[b], 0, 0, 0);
                }
            } else {
                const half8 h = fragment(q, wave, sub), l = fragment(q + kSide * kSide, wave, sub);
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const half8 f = fragment(x, b, sub);
                    acc[b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f, l, acc[b], 0, 0, 0);
                    acc[b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f, h, acc[b], 0, 0, 0);
                }
            }
        }
        const int64_t row = (TALL ? t * kApply : 0) + j0 + (lane & 31);
        const int64_t col0 = (TALL ? 0 : t * kApply) + i0 + 4 * (lane >> 5);
        if (row >= a.rows) continue;
        const int64_t at = matrix * o.out.stride + row * o.out.ld;
        if (o.aligned) {  // cols a multiple of four
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int64_t col = col0 + b * 32 + r * 8;
                    if (col >= a.cols) continue;
                    float v[4], old[4];
                    if (o.update) load_values4(o.out.ptr, o.out.type, at + col, old);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        v[e] = acc[b][r * 4 + e] * o.scale;
                        if (o.update) v[e] = __builtin_fmaf(-o.move, v[e], old[e] * o.keep);
                    }
                    store_values4(o.out.ptr, o.out.type, at + col, v);
                }
        } else {  // element by element, the registers taking turns in one place
#pragma unroll 1
            for (int r = 0; r < 32; ++r) {
                const float sum = acc[0][0];
#pragma unroll
                for (int e = 0; e < 15; ++e) acc[0][e] = acc[0][e + 1];
                acc[0][15] = acc[1][0];
#pragma unroll
                for (int e = 0; e < 15; ++e) acc[1][e] = acc[1][e + 1];
                const int64_t col = col0 + (r >> 4) * 32 + (r >> 2 & 3) * 8 + (r & 3);
                if (col >= a.cols) continue;
                float v = sum * o.scale;
                if (o.update) v = __builtin_fmaf(-o.move, v, load_value(o.out.ptr, o.out.type, at + col) * o.keep);
                store_value(o.out.ptr, o.out.type, at + col, v);
            }
        }
    }
}

struct Layout {
    int64_t long_tiles;
    int slices;
    int64_t gram, q, total;
};

Layout layout_of(int64_t rows, int64_t cols, int64_t count) {
    Layout l;
    const int64_t n = rows > cols ? rows : cols;
    l.long_tiles = (n + kSide - 1) / kSide;
    // A block for every tile while 512 blocks are not enough to keep the chip
    // busy, and no more than 64 sums to join.
    const int64_t want = (512 + count - 1) / count, most = want < 8 ? 8 : want < 64 ? want : 64;
    l.slices = (int)(l.long_tiles < most ? l.long_tiles : most);
    const int64_t tile = kTriangle * 4 * kWave * sizeof(float4);
    l.gram = count * l.slices * tile;
    l.q = l.gram + count * tile;
    l.total = l.q + count * 2 * kTileBytes;
    return l;
}

template <int BLOCKS>
void run_steps(int64_t count, const float4* gram, int slices, const Steps& steps, float scale_q, _Float16* q, hipStream_t stream) {
    narrow_steps_kernel<BLOCKS><<<(unsigned)count, BLOCKS*(BLOCKS + 1) / 2 * kWave, 0, stream>>>(gram, slices, steps, scale_q, q);
}

}  // namespace

// Growth beyond kMaxGrowth would push Q's 22 bits into the result.  R's
// roundings are stretched where singular values are small, as they are unless
// the matrix is long: this way is up to 8e-3 off at 64 x 96 and 2e-3 at 128 x
// 192 where the other stays within 1.2e-3; at 128 x 512 4e-4 against 8e-4.
bool is_narrow(const UpdateArgs& u) {
    const int64_t m = u.rows < u.cols ? u.rows : u.cols, n = u.rows < u.cols ? u.cols : u.rows;
    return !u.split && m <= kNarrow && n >= 8 * m && n >= 512 && u.growth <= kMaxGrowth;
}

size_t narrow_workspace_bytes(int64_t rows, int64_t cols, int64_t count) { return (size_t)layout_of(rows, cols, count).total; }

hipError_t launch_narrow(const UpdateArgs& u, const Source& s, const double* partial, int n_partial, void* workspace,
                         hipStream_t stream) {
    const Layout l = layout_of(u.rows, u.cols, u.count);
    float4* part = static_cast<float4*>(workspace);
    _Float16* q = reinterpret_cast<_Float16*>(static_cast<char*>(workspace) + l.q);
    NarrowArgs a = {};
    a.s = s;
    a.rows = u.rows, a.cols = u.cols;
    const bool tall = u.rows > u.cols;
    a.vector = u.cols % 8 == 0 && u.x.ld % 8 == 0 && u.x.stride % 8 == 0 && reinterpret_cast<uintptr_t>(u.x.ptr) % 16 == 0;
    a.m = tall ? u.cols : u.rows;
    a.partial = partial, a.n_partial = n_partial, a.eps = u.eps;
    Steps steps = {};
    for (int k = 0; k < u.n_steps; ++k) steps.k[k] = u.steps[k];
    steps.n = u.n_steps;
    float scale_q = 16384.0f;  // times Q, which is at most growth
    for (float g = 1; g < u.growth; g *= 2) scale_q *= 0.5f;
    const dim3 gram_grid(l.slices, (unsigned)u.count);
    if (tall)
        narrow_gram_kernel<true><<<gram_grid, 256, 0, stream>>>(a, l.long_tiles, part);
    else
        narrow_gram_kernel<false><<<gram_grid, 256, 0, stream>>>(a, l.long_tiles, part);
    const int blocks = (int)(a.m + 31) / 32;
    const float4* gram = part;
    int slices = l.slices;
    if (slices > 4) {  // fewer are added up on the way in
        float4* sum = reinterpret_cast<float4*>(static_cast<char*>(workspace) + l.gram);
        narrow_join_kernel<<<dim3(blocks * (blocks + 1) / 2, (unsigned)u.count), 256, 0, stream>>>(l.slices, part, sum);
        gram = sum;
        slices = 1;
    }
    if (blocks == 1)
        run_steps<1>(u.count, gram, slices, steps, scale_q, q, stream);
    else if (blocks == 2)
        run_steps<2>(u.count, gram, slices, steps, scale_q, q, stream);
    else if (blocks == 3)
        run_steps<3>(u.count, gram, slices, steps, scale_q, q, stream);
    else
        run_steps<4>(u.count, gram, slices, steps, scale_q, q, stream);
    NarrowOut o = {};
    o.out = u.out;
    o.aligned = u.cols % 4 == 0 && u.out.ld % 4 == 0 && u.out.stride % 4 == 0 &&
                reinterpret_cast<uintptr_t>(u.out.ptr) % (4 * type_bytes(u.out.type)) == 0;
    o.update = u.momentum != nullptr;
    o.keep = u.keep, o.move = u.move;
    o.scale = 1.0f / (kScaleX * scale_q);
    const int64_t tiles = ((tall ? u.rows : u.cols) + kApply - 1) / kApply, room = (512 + u.count - 1) / u.count;
    const dim3 apply_grid((unsigned)(tiles < room ? tiles : room), (unsigned)u.count);
    if (tall)
        narrow_apply_kernel<true><<<apply_grid, 256, 0, stream>>>(a, tiles, q, o);
    else
        narrow_apply_kernel<false><<<apply_grid, 256, 0, stream>>>(a, tiles, q, o);
    return hipGetLastError();
}

}  // namespace sl
