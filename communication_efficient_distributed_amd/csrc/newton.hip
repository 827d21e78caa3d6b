// newton.hip -- Newton-Schulz orthogonalisation and the weight update that
// uses it (sl_orthogonalize, sl_muon_step).
//
// With X the m x n matrix (m <= n; a tall input is taken transposed), every
// step is three products on the matrix cores:
//     gram   A = X X^T                     symmetric, lower tiles computed, both halves written
//     poly   B = b A + c A A               symmetric likewise
//     step   X <- a X + B X
// All three are run as C = P Q^T with both operands stored along the summed
// index: gram reads X twice, poly A twice (A = A^T), step reads B and X^T.  X
// is therefore kept in both orientations, which the step's epilogue writes.
//
// Operands are fp16 (11 bits; bf16's 8 would leave 1e-2 in the result where
// fp16 leaves 5e-4 to 8e-4), or the sum of two fp16 values hi + lo (22 bits)
// multiplied as hi hi + hi lo + lo hi, which leaves about 1e-6.  Sums are fp32.
// The diagonals of A and B, which carry most of their weight once X is nearly
// orthogonal, are left out of the fp16 matrices and kept in fp32: rounding
// them cost more than all other entries together.  Powers of two keep fp16's
// range: X is stored times 2^13, A times 2^12, B times 2^11, for which the
// host refuses coefficients whose iterates could pass 3.8 (|X_ij| <= |X|_2,
// |A_ij| <= |X|_2^2) or 30 for |B|_2.
//
// Large matrices are bound by the matrix cores at the clock that their power
// leaves: 8192 x 8192 bf16 9.7 ms for 11 TFLOP (1.13 PFLOP/s; a library fp16
// product of that size runs at 1.34).  Small ones are bound by the latency of
// a chain of 17 to 36 launches.  Split products of matrices twice as long as
// wide, or more, go by the Gram matrix alone (run_by_gram), fp16 products of
// long matrices of up to 128 rows or columns by newton_narrow.hip.
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "newton.h"

namespace sl {
namespace {

constexpr float kScaleX = 8192.0f, kScaleA = 4096.0f, kScaleB = 2048.0f;
constexpr int kUnits = 256;       // compute units
constexpr int kSumBlocks = 1024;  // of all matrices' partial sums of squares, about

// ---------------------------------------------------------------------------
// The start: sums of squares (with the momentum update), then X and X^T.

// partial[i * gridDim.x + block] = the block's share of matrix i's sum of u^2
// in fp64 (no overflow or underflow for any finite fp32 values); momentum is
// updated on the way.  Blocks take pieces of 2048 columns of a row in turn, a
// thread eight columns of each: in one go where the rows' alignment allows it
// (VECTOR), else 256 apart.  Bound by memory: 8192 x 28672 fp32 with momentum
// (2.8 GB read and written) 0.60 ms, 4.7 TB/s.
template <bool VECTOR>
__global__ __launch_bounds__(256) void sum_squares_kernel(Source s, int64_t rows, int64_t cols, double* partial) {
    __shared__ double lds[4];
    const int64_t i = blockIdx.y;
    const int64_t pieces = (cols + 2047) / 2048;
    double acc = 0;
    for (int64_t t = blockIdx.x; t < rows * pieces; t += gridDim.x) {
        const int64_t r = rows == 1 ? 0 : t / pieces;
        const int64_t c0 = (t - r * pieces) * 2048 + (VECTOR ? threadIdx.x * 8 : threadIdx.x);
        const int64_t at = i * s.stride + r * s.ld;
        float* m = s.momentum ? s.momentum + (i * rows + r) * cols : nullptr;
        float u[8], old[8];
        if (VECTOR) {
            if (c0 >= cols) continue;
            load_values8(s.x, s.type, at + c0, u);
            if (m) load_values8(m, SL_F32, c0, old);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const bool in = c0 + e * 256 < cols;
                u[e] = in ? load_value(s.x, s.type, at + c0 + e * 256) : 0.0f;
                old[e] = in && m ? m[c0 + e * 256] : 0.0f;
            }
        }
        if (m) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float g = u[e] * s.grad_scale;
                old[e] = momentum_next(g, old[e], s.decay);
                u[e] = s.nesterov ? __builtin_fmaf(s.decay, old[e], g) : old[e];
            }
            if (VECTOR) {
                *reinterpret_cast<float4*>(m + c0) = make_float4(old[0], old[1], old[2], old[3]);
                *reinterpret_cast<float4*>(m + c0 + 4) = make_float4(old[4], old[5], old[6], old[7]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (c0 + e * 256 < cols) m[c0 + e * 256] = old[e];
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) acc = fma((double)u[e], (double)u[e], acc);
    }
    acc = block_sum(acc, lds);
    if (threadIdx.x == 0) partial[i * gridDim.x + blockIdx.x] = acc;
}

// X = u * 2^13 / (|u| + eps) as fp16 (hi, and lo if split) in both
// orientations, zero beyond the matrix: direct[r][c] (ld_direct) and
// turned[c][r] (ld_turned), 64 x 64 elements per block.  Bound by memory, by
// its writes of two bytes per lane: 8192 x 28672 with momentum, split (3.8 GB)
// 0.70 ms, 5.4 TB/s; 8192 x 8192 bf16 (0.4 GB) 0.15 ms.
template <bool SPLIT>
__global__ __launch_bounds__(256) void start_kernel(Source s, int64_t rows, int64_t cols, const double* partial,
                                                    int n_partial, float eps, _Float16* direct, int64_t ld_direct,
                                                    _Float16* turned, int64_t ld_turned, int64_t lo,
                                                    int64_t matrix_bytes) {
    __shared__ double sums[4];
    __shared__ float tile[64][65];
    const int64_t i = blockIdx.z;
    const int64_t r0 = (int64_t)blockIdx.y * 64, c0 = (int64_t)blockIdx.x * 64;
    const int tc = threadIdx.x & 63, tr = threadIdx.x >> 6;
    // The tile's values are on their way while the norm is summed.
    float u[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const int64_t r = r0 + tr + 4 * k;
        const bool in = r < rows && c0 + tc < cols;
        u[k] = in && !(s.momentum && !s.nesterov) ? load_value(s.x, s.type, i * s.stride + r * s.ld + c0 + tc) : 0.0f;
        if (s.momentum && in) {
            const float m = s.momentum[(i * rows + r) * cols + c0 + tc];
            u[k] = s.nesterov ? __builtin_fmaf(s.decay, m, u[k] * s.grad_scale) : m;
        }
    }
    const Scale scale = start_scale(kScaleX, partial, n_partial, i, eps, sums);
    direct = reinterpret_cast<_Float16*>(reinterpret_cast<char*>(direct) + i * matrix_bytes);
    turned = reinterpret_cast<_Float16*>(reinterpret_cast<char*>(turned) + i * matrix_bytes);
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const int r = tr + 4 * k;
        const float v = scale(u[k]);
        tile[r][tc] = v;
        _Float16 h, l;
        split_half(v, &h, &l);
        const int64_t at = (r0 + r) * ld_direct + c0 + tc;
        direct[at] = h;
        if (SPLIT) direct[at + lo] = l;
    }
    __syncthreads();
    for (int c = tr; c < 64; c += 4) {
        _Float16 h, l;
        split_half(tile[tc][c], &h, &l);
        const int64_t at = (c0 + c) * ld_turned + r0 + tc;
        turned[at] = h;
        if (SPLIT) turned[at + lo] = l;
    }
}

// ---------------------------------------------------------------------------
// The products.

// C from the sums S = P Q^T: kGram A, kPoly B, kStep X, kLast the output; and
// alpha S + beta old + gamma I: kSym symmetric, kFull (alpha S) in both
// orientations, kEnd (alpha S) to the output.
enum { kGram, kPoly, kStep, kLast, kSym, kFull, kEnd };
constexpr bool symmetric(int kind) { return kind == kGram || kind == kPoly || kind == kSym; }
constexpr bool to_output(int kind) { return kind == kLast || kind == kEnd; }

struct ProductArgs {
    const _Float16 *p, *q;  // operands: rows of ldp / ldq elements along the summed index
    int64_t ldp, ldq;
    int64_t lo;              // elements from any hi array to its lo array
    int64_t matrix_bytes;    // from one matrix's arrays to the next one's
    int32_t k_steps;         // summed index / 64
    int32_t tiles_i, tiles_j;
    int32_t whole;           // tiles done by one block each, before those that are sliced
    int32_t slices;          // of the summed index for the others, whose sums go to `part`
    float4* part;
    // epilogue
    const _Float16* old;     // poly: A; step, last: X, so that old[j * ldold + i] meets C[i][j]
    int64_t ldold;
    _Float16 *c, *ct;        // C[i * ldc + j] and its transpose ct[j * ldct + i]
    int64_t ldc, ldct;
    const float* diag_in;
    float* diag_out;
    Quintic k;
    float alpha, beta, gamma;
    // last
    MatrixView out;
    int64_t out_i, out_j;    // extent of out along i (its columns) and j (its rows)
    bool out_aligned;        // four elements of out along i can be moved at once
    bool diag_by_i;
    bool update;             // theta <- theta * keep - move * O
    float keep, move;
};

// Tile (ti, tj) of block t.  Symmetric products: the tiles with tj <= ti, in
// groups of 4 tile rows taken column by column, so that the tiles in flight on
// one XCD share few operand panels.
__device__ __forceinline__ void symmetric_tile(int t, int tiles, int* ti, int* tj) {
    int g = 0;
    for (;; ++g) {
        const int h = min(4, tiles - 4 * g);              // rows of this group
        const int n = h * 4 * g + h * (h + 1) / 2;
        if (t < n) {
            if (t < h * 4 * g) {
                *ti = 4 * g + t % h;
                *tj = t / h;
            } else {
                t -= h * 4 * g;
                int c = 0;
                while (t >= h - c) t -= h - c, ++c;
                *tj = 4 * g + c;
                *ti = 4 * g + c + t;
            }
            return;
        }
        t -= n;
    }
}

__device__ __forceinline__ void full_tile(int t, int tiles_i, int tiles_j, int* ti, int* tj) {
    const int per = 4 * tiles_j;
    const int g = t / per;
    const int h = min(4, tiles_i - 4 * g);
    t -= g * per;
    *ti = 4 * g + t % h;
    *tj = t / h;
}

// The dispatcher deals workgroups to the eight XCDs in turn; give each XCD a
// contiguous range of tiles, so that its L2 serves neighbours.
__device__ __forceinline__ int xcd_order(int b, int n) {
    const int x = b & 7, q = n >> 3, r = n & 7;
    return x * q + min(x, r) + (b >> 3);
}

constexpr int strip_pitch(int ti) { return 32 * ti + 4; }

// Finishes 32 columns of C for one wavefront: sums[a], as the matrix
// instructions leave them (lane l, register r: C[i][j] with
// i = 32 a + 8 (r / 4) + 4 (l / 32) + r % 4 and j = l % 32), rows from i0,
// columns from j0.  They pass through the wavefront's strip of LDS: rows of
// consecutive i from there meet the old values, the transpose ct and the
// output along memory; then (the finished values put back) columns give the
// rows of c.
template <int TI, bool SPLIT, int KIND>
__device__ __forceinline__ void finish_strip(const ProductArgs& g, int64_t matrix, int64_t i0, int64_t j0, bool on_diagonal,
                                             const float16v (&sums)[TI], float* strip) {
    constexpr int W = 32 * TI, kPitch = strip_pitch(TI);
    constexpr int kInFlight = 4 * TI < 8 ? 4 * TI : 8;  // loads in flight, within the register file
    const int lane = lane_id();
    const int64_t shift = matrix * (g.matrix_bytes / 2);
    constexpr bool kDirect = KIND <= kLast;  // with the diagonals apart
    const float* diag_in = KIND == kGram || !kDirect ? nullptr : g.diag_in + matrix * (g.matrix_bytes / 4);
    float* diag_out = kDirect && symmetric(KIND) ? g.diag_out + matrix * (g.matrix_bytes / 4) : nullptr;
    const bool has_old = KIND == kPoly || KIND == kStep || KIND == kLast || (KIND == kSym && g.old);
#pragma unroll
    for (int a = 0; a < TI; ++a)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float4 v = {sums[a][r * 4], sums[a][r * 4 + 1], sums[a][r * 4 + 2], sums[a][r * 4 + 3]};
            *reinterpret_cast<float4*>(&strip[(lane & 31) * kPitch + a * 32 + r * 8 + 4 * (lane >> 5)]) = v;
        }
    wave_sync();
#pragma unroll 1
    for (int it0 = 0; it0 < 4 * TI; it0 += kInFlight) {
        half4 oh[kInFlight], ol[kInFlight];
        if (has_old) {
#pragma unroll
            for (int it = 0; it < kInFlight; ++it) {
                const int at = (it0 + it) * 64 + lane;
                const _Float16* old = g.old + shift + (j0 + at / (8 * TI)) * g.ldold + i0 + at % (8 * TI) * 4;
                oh[it] = *reinterpret_cast<const half4*>(old);
                if (SPLIT) ol[it] = *reinterpret_cast<const half4*>(old + g.lo);
            }
        }
#pragma unroll
        for (int it = 0; it < kInFlight; ++it) {
            const int at = (it0 + it) * 64 + lane;
            const int jj = at / (8 * TI), ii = at % (8 * TI) * 4;
            const int64_t i = i0 + ii, j = j0 + jj;
            float4* cell = reinterpret_cast<float4*>(&strip[jj * kPitch + ii]);
            const float4 sum = *cell;
            float v[4] = {sum.x, sum.y, sum.z, sum.w}, w[4];
            if (has_old) {
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = (float)oh[it][e] + (SPLIT ? (float)ol[it][e] : 0.0f);
            }
            if (!kDirect) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[e] *= g.alpha;
                    if (KIND == kSym && has_old) v[e] = __builtin_fmaf(g.beta, w[e], v[e]);
                    if (KIND == kSym && i + e == j) v[e] += g.gamma;
                }
            } else if (KIND == kGram) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (i + e == j) {
                        diag_out[j] = v[e] * (1.0f / (kScaleX * kScaleX));
                        v[e] = 0;
                    }
                    v[e] *= kScaleA / (kScaleX * kScaleX);
                }
            } else if (KIND == kPoly) {
                // (A A)_ij with A = D + F: sum_k F_ik F_kj + (d_i + d_j) F_ij, and d_i^2 on the diagonal.
                const float dj = diag_in[j];
                const float4 di4 = *reinterpret_cast<const float4*>(diag_in + i);
                const float di[4] = {di4.x, di4.y, di4.z, di4.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float f = w[e] * (1.0f / kScaleA), sq = v[e] * (1.0f / (kScaleA * kScaleA));
                    if (i + e == j) {
                        diag_out[j] = g.k.b * dj + g.k.c * (dj * dj + sq);
                        v[e] = 0;
                    } else {
                        v[e] = kScaleB * (g.k.b * f + g.k.c * (sq + (di[e] + dj) * f));
                    }
                }
            } else {
                float4 d = {0, 0, 0, 0};
                if (KIND == kStep || g.diag_by_i)
                    d = *reinterpret_cast<const float4*>(diag_in + i);
                else
                    d.x = d.y = d.z = d.w = diag_in[j];
                const float dd[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = (g.k.a + dd[e]) * w[e] + v[e] * (1.0f / kScaleB);  // times kScaleX
            }
            if (to_output(KIND)) {
                if (KIND == kLast)
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] *= 1.0f / kScaleX;
                if (g.out_aligned && i + 4 <= g.out_i) {
                    if (j < g.out_j) {
                        const int64_t to = matrix * g.out.stride + j * g.out.ld + i;
                        if (g.update) {
                            float o[4];
                            load_values4(g.out.ptr, g.out.type, to, o);
#pragma unroll
                            for (int e = 0; e < 4; ++e) v[e] = __builtin_fmaf(-g.move, v[e], o[e] * g.keep);
                        }
                        store_values4(g.out.ptr, g.out.type, to, v);
                    }
                    continue;
                }
            } else {
                half4 h, l;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    _Float16 hh, ll;
                    split_half(v[e], &hh, &ll);
                    h[e] = hh;
                    l[e] = ll;
                }
                _Float16* ct = g.ct + shift + j * g.ldct + i;
                *reinterpret_cast<half4*>(ct) = h;
                if (SPLIT) *reinterpret_cast<half4*>(ct + g.lo) = l;
            }
            *cell = make_float4(v[0], v[1], v[2], v[3]);
        }
    }
    wave_sync();
    if (to_output(KIND)) {
        // What four at once did not reach: consecutive i, one element per lane.
        const int64_t done = g.out_aligned ? g.out_i & ~(int64_t)3 : 0;
        if (i0 + W > done)
#pragma unroll 4
            for (int it = 0; it < 16 * TI; ++it) {
                const int at = it * 64 + lane;
                const int64_t i = i0 + at % W, j = j0 + at / W;
                if (i >= done && i < g.out_i && j < g.out_j) {
                    const int64_t to = matrix * g.out.stride + j * g.out.ld + i;
                    float o = strip[(at / W) * kPitch + at % W];
                    if (g.update) o = __builtin_fmaf(-g.move, o, load_value(g.out.ptr, g.out.type, to) * g.keep);
                    store_value(g.out.ptr, g.out.type, to, o);
                }
            }
    } else if (!on_diagonal) {
#pragma unroll 4
        for (int it = 0; it < 4 * TI; ++it) {
            const int at = it * 64 + lane;
            const int ii = at >> 3, jj = (at & 7) * 4;
            half4 h, l;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                _Float16 hh, ll;
                split_half(strip[(jj + e) * kPitch + ii], &hh, &ll);
                h[e] = hh;
                l[e] = ll;
            }
            _Float16* c = g.c + shift + (i0 + ii) * g.ldc + j0 + jj;
            *reinterpret_cast<half4*>(c) = h;
            if (SPLIT) *reinterpret_cast<half4*>(c + g.lo) = l;
        }
    }
    wave_sync();
}

enum { kPlain, kInTurn, kPaired };

template <int V>
struct Constant {
    static constexpr int value = V;
};

// C = P Q^T over tiles of 64 TI x 64 TJ, four wavefronts of 32 TI x 32 TJ each
// (half the rows, half the columns).  Two stages of LDS, 64 columns of both
// operands each, filled from global memory without passing registers.  Split
// operands (TERMS) take the three products of the same columns one after
// another, or 32 columns of hi and of lo at a time and all three from those:
// less LDS traffic, but half lines from memory.  Measured on whole calls: one
// 1024 x 1024 409 against 345 us, three 1000 x 2731 867 against 830; but the
// Gram matrix of 1024 x 8192 35 against 45 us, and 256 x 256 tiles (8192 x
// 28672) 55.5 against 57.5 ms.  So: pairs for small tiles along the short
// side.  (Small tiles gained nothing from three or four stages, and lost the
// blocks per compute unit that their LDS takes: 8 x 1024 x 1024, 444 us in all
// with two stages, 460 with three, 512 with four.)
//
// 256 x 256 tiles are bound by the matrix cores: 8192 x 8192 x 8192 plain 0.92
// ms, 1.19 PFLOP/s with the cores busy 63% of the time at a clock that their
// power holds down; split 8192 x 28672 x 8192 8.8 ms, 1.31 PFLOP/s, 70%.
// Smaller tiles are bound by the latency of loads and the finish, all blocks
// running at once: split 8192 x 1024 x 1024 63 us, 0.82 PFLOP/s, 37%.
template <int TI, int TJ, int TERMS, int KIND>
__global__ __launch_bounds__(256, 1) void product_kernel(ProductArgs g) {
    constexpr bool SPLIT = TERMS != kPlain, PAIRED = TERMS == kPaired;
    constexpr int BI = 64 * TI, BJ = 64 * TJ, kStages = 2;
    __shared__ __attribute__((aligned(128))) _Float16 lds[kStages][(BI + BJ) * 64];
    const int lane = lane_id(), wave = uniform(threadIdx.x >> 6);
    const int wi = wave >> 1, wj = wave & 1;
    const int tiles = symmetric(KIND) ? g.tiles_i * (g.tiles_i + 1) / 2 : g.tiles_i * g.tiles_j;
    // Symmetric products: tiles by one block each first, then the sliced ones.
    const int whole = symmetric(KIND) ? g.whole : gridDim.x;
    const bool sliced = symmetric(KIND) && (int)blockIdx.x >= whole;
    const int slices = sliced ? g.slices : 1;
    const int block = sliced ? xcd_order(blockIdx.x - whole, gridDim.x - whole) : xcd_order(blockIdx.x, whole);
    const int slice = block % slices, t = (sliced ? whole : 0) + block / slices;
    const int64_t matrix = t / tiles;
    int ti, tj;
    if (symmetric(KIND))
        symmetric_tile(t % tiles, g.tiles_i, &ti, &tj);
    else
        full_tile(t % tiles, g.tiles_i, g.tiles_j, &ti, &tj);
    const int64_t shift = matrix * (g.matrix_bytes / 2);
    const int all = g.k_steps * (PAIRED ? 2 : SPLIT ? 3 : 1);
    const int from = all * slice / slices, steps = all * (slice + 1) / slices - from;

    // Loads: a wavefront instruction fills 8 rows of 64 elements.  The 16-byte
    // piece c of row r sits at position c ^ (r / 2 & 7), so that the 16 lanes
    // that read the LDS at once (one piece of 16 rows) meet all 64 banks.
    const int lr = lane >> 3, lc = (lane & 7) ^ ((wave & 1) * 4 + (lr >> 1));
    const int64_t piece = PAIRED ? (lc & 3) * 8 + (lc >> 2) * g.lo : lc * 8;  // pieces 0 to 3 of hi, then of lo
    const _Float16* p = g.p + shift + ((int64_t)ti * BI + wave * 8 + lr) * g.ldp + piece;
    const _Float16* q = g.q + shift + ((int64_t)tj * BJ + wave * 8 + lr) * g.ldq + piece;
    constexpr int kLoads = 2 * (TI + TJ);  // of a wavefront for one stage
    const int64_t hop_p = 32 * g.ldp, hop_q = 32 * g.ldq;
    auto load = [&](int s, int l) {
        _Float16* const stage = lds[s % kStages];
        int64_t kp, kq;
        if (SPLIT && !PAIRED) {
            const int k = (from + s) / 3, term = from + s - 3 * k;  // hi hi, hi lo, lo hi of the same columns
            kp = (int64_t)k * 64 + (term == 2 ? g.lo : 0);
            kq = (int64_t)k * 64 + (term == 1 ? g.lo : 0);
        } else {
            kp = kq = (int64_t)(from + s) * (PAIRED ? 32 : 64);
        }
        if (l < 2 * TI)
            load_to_lds(p + (kp + l * hop_p), stage + (l * 32 + wave * 8) * 64);
        else
            load_to_lds(q + (kq + (l - 2 * TI) * hop_q), stage + BI * 64 + ((l - 2 * TI) * 32 + wave * 8) * 64);
    };
    // A step is worked off 16 columns at a time; the fragments of the next 16
    // are read while the matrix cores work on the present ones.
    constexpr int kParts = PAIRED ? 2 : 4, kPair = PAIRED ? 2 : 1;
    half8 fp[2][kPair][TI], fq[2][kPair][TJ];
    constexpr int kReads = kPair * (TI + TJ), kMul = (PAIRED ? 3 : 1) * TI * TJ;
    const int row_p = wi * 32 * TI + (lane & 31), row_q = BI + wj * 32 * TJ + (lane & 31);
    auto fetch = [&](int s, int part, int into, int k) {
        const _Float16* const stage = lds[s % kStages];
        const int lo = k / (TI + TJ), f = k % (TI + TJ);
        const int pos = ((lo * 4 + part * 2 + (lane >> 5)) ^ ((lane >> 1) & 7)) * 8;
        if (f < TI)
            fp[into][lo][f] = *reinterpret_cast<const half8*>(stage + (row_p + f * 32) * 64 + pos);
        else
            fq[into][lo][f - TI] = *reinterpret_cast<const half8*>(stage + (row_q + (f - TI) * 32) * 64 + pos);
    };
    float16v acc[TJ][TI];
#pragma unroll
    for (int b = 0; b < TJ; ++b)
#pragma unroll
        for (int a = 0; a < TI; ++a) acc[b][a] = 0.0f;
    auto multiply = [&](int with, int first, int last) {
#pragma unroll
        for (int m = first; m < last; ++m) {
            const int a = m % (TI * TJ) / TJ, b = m % TJ, term = m / (TI * TJ);  // hi hi, hi lo, lo hi
            acc[b][a] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fp[with][term == 2][a], fq[with][term == 1][b], acc[b][a], 0, 0, 0);
        }
    };
    // A stage's loads go out as soon as it is free, in the last part of the
    // step that used it; large tiles leave half of them to the next step's
    // first parts, as one burst would hold up the products (8192 x
    // 8192: 11.4 ms against 11.7).
    constexpr bool kSpread = TI * TJ >= 8;
    constexpr int kFirst = kSpread ? kLoads / 2 : kLoads, kSecond = kSpread ? kLoads * 3 / 4 : kLoads;
    static_assert(!(kSpread && PAIRED), "two parts leave no third for the last loads");
    constexpr int kEarly = kSpread ? 4 : 0;  // products that cover the barrier
    // MAIN: the step s + 2 exists.
    auto step = [&](int s, auto main) {
        constexpr bool kMain = main.value;
#pragma unroll
        for (int sub = 0; sub < kParts - 1; ++sub) {
#pragma unroll
            for (int k = 0; k < kReads; ++k) {
                multiply(sub & 1, k * kMul / kReads, (k + 1) * kMul / kReads);
                fetch(s, sub + 1, (sub + 1) & 1, k);
                if (kSpread && (kMain || s + 1 < steps)) {
                    const int l0 = sub == 0 ? kFirst : kSecond, n = sub == 0 ? kSecond - kFirst : sub == 1 ? kLoads - kSecond : 0;
#pragma unroll
                    for (int l = l0 + k * n / kReads; l < l0 + (k + 1) * n / kReads; ++l) load(s + 1, l);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        // Every wavefront has its last fragments of this stage, and its own
        // loads of the next one have landed: after the barrier that holds for
        // all of them.
        multiply(1, 0, kEarly);
        __builtin_amdgcn_sched_barrier(0);
        arrive();
#pragma unroll
        for (int k = 0; k < kReads; ++k) {
            multiply(1, kEarly + k * (kMul - kEarly) / kReads, kEarly + (k + 1) * (kMul - kEarly) / kReads);
            if (kMain || s + 1 < steps) fetch(s + 1, 0, 0, k);
            if (kMain || s + 2 < steps)
#pragma unroll
                for (int l = k * kFirst / kReads; l < (k + 1) * kFirst / kReads; ++l) load(s + 2, l);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
#pragma unroll
    for (int l = 0; l < kLoads; ++l) load(0, l);
    arrive();
    if (steps > 1)
#pragma unroll
        for (int l = 0; l < kFirst; ++l) load(1, l);
#pragma unroll
    for (int k = 0; k < kReads; ++k) fetch(0, 0, 0, k);
    int s = 0;
    for (; s + 2 < steps; ++s) step(s, Constant<1>{});
    for (; s < steps; ++s) step(s, Constant<0>{});

    if (sliced) {
        float4* part = g.part + ((int64_t)(t - whole) * slices + slice) * (TI * TJ * 4 * 256) + threadIdx.x;
#pragma unroll
        for (int b = 0; b < TJ; ++b)
#pragma unroll
            for (int a = 0; a < TI; ++a)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    part[((b * TI + a) * 4 + r) * 256] =
                        make_float4(acc[b][a][r * 4], acc[b][a][r * 4 + 1], acc[b][a][r * 4 + 2], acc[b][a][r * 4 + 3]);
        return;
    }
    float* strip = reinterpret_cast<float*>(&lds[0][0]) + wave * ((BI + BJ) * 64 / 4);
    static_assert(32 * strip_pitch(TI) <= (BI + BJ) * 64 / 4, "a strip fits a quarter of the LDS");
#pragma unroll
    for (int b = 0; b < TJ; ++b)
        finish_strip<TI, SPLIT, KIND>(g, matrix, (int64_t)ti * BI + wi * 32 * TI, (int64_t)tj * BJ + wj * 32 * TJ + b * 32,
                                      symmetric(KIND) && ti == tj, acc[b], strip);
}

// Joins the slices of a symmetric product, 32 columns of a quarter tile per
// block.  Its SHARES wavefronts, one or four, add up equal parts of the slices,
// in order; the first adds those sums and finishes.  Four are taken for tiles
// up to 128 x 128 from eight slices on (300 x 4000: the whole update 193 ->
// 175 us); with fewer slices, or 256 x 256 tiles, the three that only read
// cost more than they save (1024 x 1024, plain: 204 -> 208 us).
template <int T, bool SPLIT, int KIND, int SHARES>
__global__ __launch_bounds__(SHARES * kWave) void join_kernel(ProductArgs g) {
    __shared__ __attribute__((aligned(16))) float strip[32 * strip_pitch(T)];
    __shared__ float4 others[SHARES > 1 ? SHARES - 1 : 1][T * 4][kWave];
    const int tiles = g.tiles_i * (g.tiles_i + 1) / 2;
    const int lane = lane_id(), share = SHARES > 1 ? uniform(threadIdx.x >> 6) : 0;
    const int b = blockIdx.x % T, wave = blockIdx.x / T % 4, sliced = blockIdx.x / (4 * T), t = g.whole + sliced;
    const int from = g.slices * share / SHARES, to = g.slices * (share + 1) / SHARES;
    const float4* part = g.part + ((int64_t)sliced * g.slices + from) * (T * T * 4 * 256) + b * T * 4 * 256 + wave * 64 + lane;
    float16v acc[T];
#pragma unroll
    for (int a = 0; a < T; ++a) acc[a] = 0.0f;
#pragma unroll 4
    for (int s = from; s < to; ++s, part += T * T * 4 * 256)
#pragma unroll
        for (int k = 0; k < T * 4; ++k) {
            const float4 v = part[k * 256];
            const int a = k / 4, r = k % 4 * 4;
            acc[a][r] += v.x, acc[a][r + 1] += v.y, acc[a][r + 2] += v.z, acc[a][r + 3] += v.w;
        }
    if (SHARES > 1) {
        if (share)
#pragma unroll
            for (int k = 0; k < T * 4; ++k) {
                const int a = k / 4, r = k % 4 * 4;
                others[share - 1][k][lane] = make_float4(acc[a][r], acc[a][r + 1], acc[a][r + 2], acc[a][r + 3]);
            }
        __syncthreads();
        if (share) return;
#pragma unroll
        for (int w = 0; w < SHARES - 1; ++w)
#pragma unroll
            for (int k = 0; k < T * 4; ++k) {
                const float4 v = others[w][k][lane];
                const int a = k / 4, r = k % 4 * 4;
                acc[a][r] += v.x, acc[a][r + 1] += v.y, acc[a][r + 2] += v.z, acc[a][r + 3] += v.w;
            }
    }
    int ti, tj;
    symmetric_tile(t % tiles, g.tiles_i, &ti, &tj);
    finish_strip<T, SPLIT, KIND>(g, t / tiles, (int64_t)ti * 64 * T + (wave >> 1) * 32 * T,
                                 (int64_t)tj * 64 * T + (wave & 1) * 32 * T + b * 32, ti == tj, acc, strip);
}

// ---------------------------------------------------------------------------
// Layout of the workspace and the launches.

struct Plan {
    int tile;              // 1, 2 or 4: tiles of 64, 128 or 256
    int64_t m, n;          // padded to the tile
    int64_t lo;            // elements between hi and lo arrays of one matrix
    int64_t x, xt0, xt1, a, b, da, db;  // byte offsets within one matrix's part
    bool by_gram;          // room for that way, with three more square matrices
    int64_t c[3];
    int64_t matrix_bytes;
    int64_t sums, part;    // byte offsets of the partial sums of squares and of sliced products
    int64_t total;
    int sum_blocks;
    int square;            // the tile of square products in the Gram matrix's way
    // Of Gram matrices, of polynomials step by step and of square products:
    // tiles that are not sliced, and slices of the others.
    int64_t gram_whole, poly_whole, square_whole;
    int gram_slices, poly_slices, square_slices;
};

// Four consecutive elements of a row, from a multiple of four on, lie in one aligned word.
bool aligned4(const MatrixView& v) {
    return v.ld % 4 == 0 && v.stride % 4 == 0 && reinterpret_cast<uintptr_t>(v.ptr) % (4 * type_bytes(v.type)) == 0;
}

int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// How many of `tiles` tiles of a symmetric product get a block each, the rest
// being sliced.  Small tiles: all or none.  256 x 256 tiles, one of which a
// compute unit holds: as many as fill the chip a whole number of times, if the
// rest would leave most of it idle (8192 x 8192: 512 of 528).
int64_t whole_of(int64_t tiles, int tile) {
    if (tile < 4) return 2 * tiles > (tile == 2 ? 512 : 1024) ? tiles : 0;
    return tiles % kUnits <= kUnits / 4 ? tiles - tiles % kUnits : tiles;
}

// Slices of each of `tiles` tiles that take `steps` steps: enough blocks to
// fill the chip, none so short that the join costs more than it saves, which
// it does sooner with more tiles.  Measured with slices of 6 / 10 / 16 steps
// and more: split 8 x 600 x 3000 658 / 658 / 556 us, 3 x 1000 x 2731 676 / 672
// / 648, 1024 x 1024 268 / 252 / 249; with fewer tiles 500 x 800 176 / 181 /
// 192, 400 x 16000 300 / 290 / 287.
int slices_of(int64_t tiles, int64_t steps, int tile) {
    if (tiles == 0) return 1;
    const int64_t room = tile == 4 ? kUnits : tile == 2 ? 512 : 1024;  // blocks that run at once
    const int64_t want = room / tiles, most = steps / (tiles < kUnits / 4 ? 10 : 16);
    return (int)(want < 2 || most < 2 ? 1 : want < most ? want : most);
}

Plan plan_of(int64_t rows, int64_t cols, int64_t count, bool split, bool update) {
    Plan p = {};
    const int64_t m = rows < cols ? rows : cols, n = rows < cols ? cols : rows;
    auto tiles = [&](int64_t t) { const int64_t k = (m + t - 1) / t; return count * k * (k + 1) / 2; };
    // Larger tiles do more products for each byte they read, smaller ones fill
    // the chip with less work and pad less.  Measured in all (256 / 128 / 64),
    // us: 4096 x 4096 1.85 / 1.95 / 2.42 ms, 3000 x 3000 1226 / 955 / 1118,
    // 2500 x 2500 811 / 598 / 692, 2048 x 2048 664 / 418 / 387, 16 of 700 x 900
    // 708 / 431 / 388; split 5000 x 5000 7.3 / 9.0 / 13.7 ms, 1024 x 8192 797 /
    // 638 / 782, 1000 x 1500 two of 708 / 407 / 418, 1024 x 1024 630 / 330 / 262.
    const double products = (double)count * m * m * n;
    p.tile = tiles(256) >= 128 ? 4 : products >= (split ? 2.5e9 : 1e10) ? 2 : 1;
    p.m = round_up(m, 64 * p.tile);
    p.n = round_up(n, 64 * p.tile);
    // All hi arrays, then all lo arrays in the same order.
    int64_t at = 0;
    auto take = [&](int64_t elements) { const int64_t was = at; at += round_up(elements * 2, 256); return was; };
    p.x = take(p.m * p.n);
    p.xt0 = take(p.m * p.n);
    p.xt1 = take(p.m * p.n);
    p.a = take(p.m * p.m);
    p.b = take(p.m * p.m);
    // That way takes about 9 square products more than the other, and 3 Gram
    // matrices and 3 products of the long side less.  Even at n = 2 m for 128 x
    // 128 tiles (3 x 1000 x 2000 591 us both, 3 x 1000 x 2731 812 -> 700, 1024 x
    // 8192 673 -> 514) and for 64 x 64 tiles if the square products fill a good
    // part of the chip (20 x 300 x 700 281 -> 250); if not, their latency wants
    // more (500 x 2000 186 -> 204, 300 x 4000 173 -> 166 us).  Below 256 rows the
    // result is less exact than fp32 arithmetic's, which a small m leaves at
    // 1e-6 (1.9e-6 against 1.1e-6), though faster.  With 256 x 256
    // tiles its result is less exact, about 1e-5 for singular values that span
    // decades, which a weight update does not see.
    const bool fills = tiles(64) >= 64 || n >= 8 * m;
    p.by_gram = split && (p.tile == 4 ? update && 2 * n >= 3 * m : m >= 256 && n >= 2 * m && (p.tile == 2 || fills));
    if (p.by_gram)
        for (int64_t& c : p.c) c = take(p.m * p.m);
    p.lo = at / 2;
    if (split) at *= 2;
    p.da = at;
    at += round_up(p.m * 4, 256);
    p.db = at;
    at += round_up(p.m * 4, 256);
    p.matrix_bytes = at;
    const int64_t narrow = !split && m <= kNarrow ? (int64_t)narrow_workspace_bytes(rows, cols, count) : 0;
    p.sums = count * at > narrow ? count * at : narrow;
    // A few pieces of 2048 elements for each block of the sums of squares, and
    // few enough blocks that the next kernel adds them up in no time.
    const int64_t pieces = (rows * cols + 2047) / 2048, most = round_up(kSumBlocks / count + 1, 64);
    p.sum_blocks = (int)(pieces < most ? pieces : most);
    p.part = p.sums + round_up(count * p.sum_blocks * 8, 256);
    // Square products by themselves fill less of the chip: smaller tiles up to
    // some size (600 x 9000 357 -> 312 us, 1024 x 8192 505 -> 490, 8 x 600 x
    // 3000 671 -> 660; 2 x 1000 x 5000 635 -> 645, 2048 x 8192 1355 -> 1539).
    p.square = p.by_gram && p.tile == 2 && (double)count * m * m * m <= 1.8e9 ? 1 : p.tile;
    const int64_t sym = tiles(64 * p.tile), square_sym = tiles(64 * p.square), per_step = split ? p.tile < 4 ? 2 : 3 : 1;
    p.gram_whole = p.poly_whole = whole_of(sym, p.tile);
    p.square_whole = whole_of(square_sym, p.square);
    p.gram_slices = slices_of(sym - p.gram_whole, (split ? 3 : 1) * p.n / 64, p.tile);
    p.poly_slices = slices_of(sym - p.poly_whole, per_step * p.m / 64, p.tile);
    p.square_slices = slices_of(square_sym - p.square_whole, per_step * p.m / 64, p.square);
    // The sums of squares lie behind what either way needs.
    auto parts = [](int64_t n, int64_t slices, int64_t tile) { return slices > 1 ? n * slices * tile * tile * 4 * 256 * 16 : 0; };
    p.total = p.part + std::max({parts(sym - p.gram_whole, p.gram_slices, p.tile),
                                 parts(sym - p.poly_whole, p.poly_slices, p.tile),
                                 parts(square_sym - p.square_whole, p.square_slices, p.square)});
    return p;
}

// The last product's output: the lanes' four consecutive elements run along i,
// out's columns.
void set_output(const UpdateArgs& u, ProductArgs* g) {
    g->out = u.out;
    g->out_i = u.cols;
    g->out_j = u.rows;
    g->out_aligned = aligned4(u.out);
    g->update = u.momentum != nullptr;
    g->keep = u.keep;
    g->move = u.move;
}

// A symmetric product, of whose tiles those after the first `whole` are sliced.
template <int T, int TERMS, int KIND>
void run_symmetric(ProductArgs g, int64_t whole, int slices, int64_t count, hipStream_t stream) {
    const int64_t tiles = count * g.tiles_i * (g.tiles_i + 1) / 2;
    g.whole = (int32_t)(slices > 1 ? whole : tiles);
    g.slices = slices;
    const int64_t rest = tiles - g.whole;
    product_kernel<T, T, TERMS, KIND><<<(unsigned)(g.whole + rest * slices), 256, 0, stream>>>(g);
    constexpr int kShares = T < 4 ? 4 : 1;
    const unsigned blocks = (unsigned)(rest * 4 * T);
    if (rest && kShares > 1 && slices >= 8)
        join_kernel<T, TERMS != kPlain, KIND, kShares><<<blocks, kShares * kWave, 0, stream>>>(g);
    else if (rest)
        join_kernel<T, TERMS != kPlain, KIND, 1><<<blocks, kWave, 0, stream>>>(g);
}

template <int T, bool SPLIT>
hipError_t run_products(const UpdateArgs& u, const Plan& p, char* ws, hipStream_t stream) {
    constexpr int B = 64 * T;
    // Split operands hold the diagonals well enough: they stay in the matrices,
    // with a I in B's, and the step needs no old X.
    constexpr int kGramTerms = SPLIT ? kInTurn : kPlain, kTerms = !SPLIT ? kPlain : T < 4 ? kPaired : kInTurn;
    constexpr int kGramKind = SPLIT ? kSym : kGram, kPolyKind = SPLIT ? kSym : kPoly;
    constexpr int kStepKind = SPLIT ? kFull : kStep, kLastKind = SPLIT ? kEnd : kLast;
    const bool tall = u.rows > u.cols;
    const int tm = (int)(p.m / B), tn = (int)(p.n / B);
    auto at = [&](int64_t o) { return reinterpret_cast<_Float16*>(ws + o); };
    ProductArgs g = {};
    g.lo = p.lo;
    g.matrix_bytes = p.matrix_bytes;
    g.part = reinterpret_cast<float4*>(ws + p.part);
    const unsigned full = (unsigned)(u.count * tm * tn);
    int64_t xt = p.xt0, xt_next = p.xt1;
    for (int s = 0; s < u.n_steps; ++s) {
        g.k = u.steps[s];
        g.tiles_i = g.tiles_j = tm;
        g.p = g.q = at(p.x);
        g.ldp = g.ldq = p.n;
        g.k_steps = (int)(p.n / 64);
        g.old = nullptr;
        g.c = g.ct = at(p.a);
        g.ldc = g.ldct = p.m;
        g.diag_in = nullptr;
        g.diag_out = reinterpret_cast<float*>(ws + p.da);
        g.alpha = kScaleA / (kScaleX * kScaleX), g.beta = g.gamma = 0;
        run_symmetric<T, kGramTerms, kGramKind>(g, p.gram_whole, p.gram_slices, u.count, stream);
        g.p = g.q = g.old = at(p.a);
        g.ldp = g.ldq = g.ldold = p.m;
        g.k_steps = (int)(p.m / 64);
        g.c = g.ct = at(p.b);
        g.diag_in = reinterpret_cast<const float*>(ws + p.da);
        g.diag_out = reinterpret_cast<float*>(ws + p.db);
        // a I + B times a power of two that keeps it within fp16's range
        float p_scale = 16384.0f;
        for (float f = 1; f < u.factors[s]; f *= 2) p_scale *= 0.5f;
        g.alpha = g.k.c * p_scale / (kScaleA * kScaleA), g.beta = g.k.b * p_scale / kScaleA, g.gamma = g.k.a * p_scale;
        run_symmetric<T, kTerms, kPolyKind>(g, p.poly_whole, p.poly_slices, u.count, stream);
        g.diag_in = reinterpret_cast<const float*>(ws + p.db);
        g.diag_out = nullptr;
        g.alpha = 1 / p_scale;
        if (s + 1 < u.n_steps) {
            g.tiles_j = tn;
            g.p = at(p.b);
            g.q = g.old = at(xt);
            g.c = at(p.x);
            g.ldc = p.n;
            g.ct = at(xt_next);
            product_kernel<T, T, kTerms, kStepKind><<<full, 256, 0, stream>>>(g);
            const int64_t was = xt;
            xt = xt_next;
            xt_next = was;
        } else {
            set_output(u, &g);
            g.alpha /= kScaleX;
            g.diag_by_i = tall;
            g.p = at(tall ? p.b : xt);
            g.q = at(tall ? xt : p.b);
            g.old = at(tall ? xt : p.x);
            g.ldold = tall ? p.m : p.n;
            g.tiles_i = tall ? tm : tn;
            g.tiles_j = tall ? tn : tm;
            product_kernel<T, T, kTerms, kLastKind><<<full, 256, 0, stream>>>(g);
        }
    }
    return hipGetLastError();
}

// The way by the Gram matrix.  Every step multiplies X by a polynomial of A,
// so a few steps together need one Gram matrix R = X X^T and one product of
// the long side, with square products in between:
//     P = a I + b R + c R R,  Q <- Q P,  R <- P R P       (Q = P at first)
// and X <- Q X in the end.  All of P, Q, R are symmetric and commute.

// Steps between two Gram matrices of X, and how much Q may grow over them.  A
// rounding of R is stretched by up to 11.9 with each step of the usual
// coefficients, against which a large m helps (the errors of R's entries are
// independent): where one singular value outweighs the others ten times, 300 x
// 4000 is 3.0e-6 off with three steps and 1.5e-6 with two (plain fp32 2.2e-6;
// 161 and 166 us), 1024 x 8192 2.4e-6 with three (plain fp32 3.6e-6).
int together_of(const Plan& p) { return p.m >= 512 ? 3 : 2; }
constexpr float kMaxGrowth = 256.0f;

// |Q|'s bound over the steps [from, to).
float growth_of(const UpdateArgs& u, int from, int to) {
    float most = 1, product = 1;
    for (int s = from; s < u.n_steps && s < to; ++s) {
        product *= u.factors[s];
        if (product > most) most = product;
        if (u.factors[s] > most) most = u.factors[s];
    }
    return most;
}

template <int T, int SQUARE>
hipError_t run_by_gram(const UpdateArgs& u, const Plan& p, char* ws, hipStream_t stream) {
    constexpr float kScaleR = 2048.0f;  // |R| and |P R| are at most 3.8^2
    constexpr int kTerms = T < 4 ? kPaired : kInTurn, kSquareTerms = SQUARE < 4 ? kPaired : kInTurn;
    const bool tall = u.rows > u.cols;
    const int tm = (int)(p.m / (64 * T)), tn = (int)(p.n / (64 * T));
    auto at = [&](int64_t o) { return reinterpret_cast<_Float16*>(ws + o); };
    ProductArgs g = {};
    g.lo = p.lo;
    g.matrix_bytes = p.matrix_bytes;
    g.part = reinterpret_cast<float4*>(ws + p.part);
    const unsigned full = (unsigned)(u.count * tm * tn);
    // to = alpha a b + beta old + gamma I, all m x m.
    auto square = [&](int64_t to, int64_t a, int64_t b, float alpha, int64_t old, float beta, float gamma) {
        g.tiles_i = g.tiles_j = tm * T / SQUARE;
        g.p = at(a), g.q = at(b);
        g.ldp = g.ldq = g.ldold = g.ldc = g.ldct = p.m;
        g.k_steps = (int)(p.m / 64);
        g.old = old < 0 ? nullptr : at(old);
        g.c = g.ct = at(to);
        g.alpha = alpha, g.beta = beta, g.gamma = gamma;
        run_symmetric<SQUARE, kSquareTerms, kSym>(g, p.square_whole, p.square_slices, u.count, stream);
    };
    const int64_t r = p.a, t = p.b;
    int64_t xt = p.xt0, xt_next = p.xt1;
    const int together = together_of(p);
    for (int from = 0; from < u.n_steps; from += together) {
        const int to = from + together < u.n_steps ? from + together : u.n_steps;
        float scale = 16384.0f;  // of P and Q
        for (float f = 1; f < growth_of(u, from, to); f *= 2) scale *= 0.5f;
        g.tiles_i = g.tiles_j = tm;
        g.p = g.q = at(p.x);
        g.ldp = g.ldq = p.n;
        g.ldc = g.ldct = p.m;
        g.k_steps = (int)(p.n / 64);
        g.old = nullptr;
        g.c = g.ct = at(r);
        g.alpha = kScaleR / (kScaleX * kScaleX), g.beta = g.gamma = 0;
        run_symmetric<T, kInTurn, kSym>(g, p.gram_whole, p.gram_slices, u.count, stream);
        int64_t poly = p.c[0], q = p.c[1], q_next = p.c[2];
        for (int s = from; s < to; ++s) {
            const Quintic& k = u.steps[s];
            square(poly, r, r, k.c * scale / (kScaleR * kScaleR), r, k.b * scale / kScaleR, k.a * scale);
            if (s + 1 < to) {
                square(t, poly, r, 1 / scale, -1, 0, 0);
                square(r, t, poly, 1 / scale, -1, 0, 0);
            }
            if (s == from) {
                const int64_t was = q;
                q = poly;
                poly = was;
            } else {
                square(q_next, q, poly, 1 / scale, -1, 0, 0);
                const int64_t was = q;
                q = q_next;
                q_next = was;
            }
        }
        g.old = nullptr;
        g.k_steps = (int)(p.m / 64);
        g.ldp = g.ldq = p.m;
        if (to < u.n_steps) {
            g.tiles_i = tm, g.tiles_j = tn;
            g.p = at(q), g.q = at(xt);
            g.c = at(p.x), g.ldc = p.n;
            g.ct = at(xt_next), g.ldct = p.m;
            g.alpha = 1 / scale;
            product_kernel<T, T, kTerms, kFull><<<full, 256, 0, stream>>>(g);
            const int64_t was = xt;
            xt = xt_next;
            xt_next = was;
        } else {
            set_output(u, &g);
            g.alpha = 1 / (scale * kScaleX);
            g.p = at(tall ? q : xt);
            g.q = at(tall ? xt : q);
            g.tiles_i = tall ? tm : tn;
            g.tiles_j = tall ? tn : tm;
            product_kernel<T, T, kTerms, kEnd><<<full, 256, 0, stream>>>(g);
        }
    }
    return hipGetLastError();
}

template <bool SPLIT>
hipError_t run(const UpdateArgs& u, const Plan& p, char* ws, hipStream_t stream) {
    Source s = {u.x.ptr, u.x.type, u.x.ld, u.x.stride, u.momentum, u.grad_scale, u.decay, u.nesterov};
    double* sums = reinterpret_cast<double*>(ws + p.sums);
    // Contiguous matrices are one long row.
    const bool flat = u.x.ld == u.cols;
    const int64_t sum_rows = flat ? 1 : u.rows, sum_cols = flat ? u.rows * u.cols : u.cols;
    const bool vector = sum_cols % 8 == 0 && (flat || u.x.ld % 8 == 0) && u.x.stride % 8 == 0 &&
                        reinterpret_cast<uintptr_t>(u.x.ptr) % 16 == 0;  // momentum is aligned and contiguous
    const dim3 sum_grid(p.sum_blocks, (unsigned)u.count);
    if (vector)
        sum_squares_kernel<true><<<sum_grid, 256, 0, stream>>>(s, sum_rows, sum_cols, sums);
    else
        sum_squares_kernel<false><<<sum_grid, 256, 0, stream>>>(s, sum_rows, sum_cols, sums);
    if (is_narrow(u)) return launch_narrow(u, s, sums, p.sum_blocks, ws, stream);
    const bool tall = u.rows > u.cols;
    const int64_t pr = tall ? p.n : p.m, pc = tall ? p.m : p.n;
    _Float16* direct = reinterpret_cast<_Float16*>(ws + (tall ? p.xt0 : p.x));
    _Float16* turned = reinterpret_cast<_Float16*>(ws + (tall ? p.x : p.xt0));
    start_kernel<SPLIT><<<dim3((unsigned)(pc / 64), (unsigned)(pr / 64), (unsigned)u.count), 256, 0, stream>>>(
        s, u.rows, u.cols, sums, p.sum_blocks, u.eps, direct, pc, turned, pr, p.lo, p.matrix_bytes);
    if (p.by_gram) {
        float most = 0;
        const int together = together_of(p);
        for (int from = 0; from < u.n_steps; from += together) most = fmaxf(most, growth_of(u, from, from + together));
        if (most <= kMaxGrowth)
            return p.tile == 4     ? run_by_gram<4, 4>(u, p, ws, stream)
                   : p.square == 2 ? run_by_gram<2, 2>(u, p, ws, stream)
                   : p.tile == 2   ? run_by_gram<2, 1>(u, p, ws, stream)
                                   : run_by_gram<1, 1>(u, p, ws, stream);
    }
    if (p.tile == 4) return run_products<4, SPLIT>(u, p, ws, stream);
    if (p.tile == 2) return run_products<2, SPLIT>(u, p, ws, stream);
    return run_products<1, SPLIT>(u, p, ws, stream);
}

}  // namespace

size_t update_workspace_bytes(int64_t rows, int64_t cols, int64_t count, bool split, bool update) {
    return (size_t)plan_of(rows, cols, count, split, update).total;
}

hipError_t launch_update(const UpdateArgs& u, void* workspace, hipStream_t stream) {
    const Plan p = plan_of(u.rows, u.cols, u.count, u.split, u.momentum != nullptr);
    char* ws = static_cast<char*>(workspace);
    return u.split ? run<true>(u, p, ws, stream) : run<false>(u, p, ws, stream);
}

}  // namespace sl
