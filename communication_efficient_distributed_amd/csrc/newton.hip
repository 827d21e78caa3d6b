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
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ops_internal.h"
#include "types.h"
#include "wave.h"

namespace sl {
namespace {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half4 __attribute__((ext_vector_type(4)));
typedef float float16v __attribute__((ext_vector_type(16)));

constexpr float kScaleX = 8192.0f, kScaleA = 4096.0f, kScaleB = 2048.0f;
constexpr int kSumBlocks = 512;  // partial sums of squares per matrix, at most

// ---------------------------------------------------------------------------
// The start: sums of squares (with the momentum update), then X and X^T.

// u of one element, before normalisation.
struct Source {
    const void* x;
    int32_t type;
    int64_t ld, stride;
    float* momentum;  // null: u = x
    float grad_scale, decay;
    bool nesterov;
};

__device__ __forceinline__ float momentum_next(float g, float m, float decay) { return __builtin_fmaf(decay, m, g); }

__device__ __forceinline__ double block_sum(double v, double* lds) {
    for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
    if (lane_id() == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    double s = 0;
    for (int w = 0; w < (int)(blockDim.x >> 6); ++w) s += lds[w];
    __syncthreads();
    return s;
}

// partial[i * gridDim.x + block] = the block's share of matrix i's sum of u^2
// in fp64 (no overflow or underflow for any finite fp32 values); momentum is
// updated on the way.  Blocks take pieces of 2048 columns of a row in turn.
__global__ __launch_bounds__(256) void sum_squares_kernel(Source s, int64_t rows, int64_t cols, double* partial) {
    __shared__ double lds[4];
    const int64_t i = blockIdx.y;
    const int64_t pieces = (cols + 2047) / 2048;
    double acc = 0;
    for (int64_t t = blockIdx.x; t < rows * pieces; t += gridDim.x) {
        const int64_t r = t / pieces, c0 = (t % pieces) * 2048;
        const int64_t at = i * s.stride + r * s.ld;
        float* m = s.momentum ? s.momentum + (i * rows + r) * cols : nullptr;
        for (int64_t c = c0 + threadIdx.x; c < cols && c < c0 + 2048; c += 256) {
            float u = load_value(s.x, s.type, at + c);
            if (m) {
                const float g = u * s.grad_scale;
                u = momentum_next(g, m[c], s.decay);
                m[c] = u;
                if (s.nesterov) u = __builtin_fmaf(s.decay, u, g);
            }
            acc = fma((double)u, (double)u, acc);
        }
    }
    acc = block_sum(acc, lds);
    if (threadIdx.x == 0) partial[i * gridDim.x + blockIdx.x] = acc;
}

__device__ __forceinline__ void split_half(float v, _Float16* hi, _Float16* lo) {
    *hi = (_Float16)v;
    *lo = (_Float16)(v - (float)*hi);
}

// X = u * 2^13 / (|u| + eps) as fp16 (hi, and lo if split) in both
// orientations, zero beyond the matrix: direct[r][c] (ld_direct) and
// turned[c][r] (ld_turned), 64 x 64 elements per block.
template <bool SPLIT>
__global__ __launch_bounds__(256) void start_kernel(Source s, int64_t rows, int64_t cols, const double* partial,
                                                    int n_partial, float eps, _Float16* direct, int64_t ld_direct,
                                                    _Float16* turned, int64_t ld_turned, int64_t lo,
                                                    int64_t matrix_bytes) {
    __shared__ double sums[4];
    __shared__ float tile[64][65];
    const int64_t i = blockIdx.z;
    double acc = 0;
    for (int k = threadIdx.x; k < n_partial; k += 256) acc += partial[i * n_partial + k];
    const double norm = sqrt(block_sum(acc, sums)) + (double)eps;
    const double scale = norm > 0 ? (double)kScaleX / norm : 0;
    direct = reinterpret_cast<_Float16*>(reinterpret_cast<char*>(direct) + i * matrix_bytes);
    turned = reinterpret_cast<_Float16*>(reinterpret_cast<char*>(turned) + i * matrix_bytes);
    const int64_t r0 = (int64_t)blockIdx.y * 64, c0 = (int64_t)blockIdx.x * 64;
    const int tc = threadIdx.x & 63, tr = threadIdx.x >> 6;
    for (int r = tr; r < 64; r += 4) {
        float v = 0;
        if (r0 + r < rows && c0 + tc < cols) {
            float u = load_value(s.x, s.type, i * s.stride + (r0 + r) * s.ld + c0 + tc);
            if (s.momentum) {
                const float m = s.momentum[(i * rows + r0 + r) * cols + c0 + tc];
                u = s.nesterov ? __builtin_fmaf(s.decay, m, u * s.grad_scale) : m;
            }
            v = (float)((double)u * scale);
        }
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

enum { kGram, kPoly, kStep, kLast };

struct ProductArgs {
    const _Float16 *p, *q;  // operands: rows of ldp / ldq elements along the summed index
    int64_t ldp, ldq;
    int64_t lo;              // elements from any hi array to its lo array
    int64_t matrix_bytes;    // from one matrix's arrays to the next one's
    int32_t k_steps;         // summed index / 64
    int32_t tiles_i, tiles_j;
    // epilogue
    const _Float16* old;     // poly: A; step, last: X, so that old[j * ldold + i] meets C[i][j]
    int64_t ldold;
    _Float16 *c, *ct;        // C[i * ldc + j] and its transpose ct[j * ldct + i]
    int64_t ldc, ldct;
    const float* diag_in;
    float* diag_out;
    Quintic k;
    // last
    MatrixView out;
    int64_t out_i, out_j;    // extent of out along i (its columns) and j (its rows)
    bool diag_by_i;
    bool update;             // theta <- theta * keep - move * O
    float keep, move;
};

// Copies 16 bytes per lane from global memory to LDS, lane l's to lds + 16 l.
__device__ __forceinline__ void load_to_lds(const _Float16* src, _Float16* lds) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) uint32_t*)src,
                                     (__attribute__((address_space(3))) uint32_t*)lds, 16, 0, 0);
}

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

struct Yes {
    static constexpr bool value = true;
};
struct No {
    static constexpr bool value = false;
};

// Orders the instructions of one quarter: a fragment read (and LOADS / 2 T
// loads to LDS) ahead of every T / 2 products, so that neither queue empties.
template <int T, int LOADS>
__device__ __forceinline__ void interleave() {
#pragma unroll
    for (int k = 0; k < 2 * T; ++k) {
        if constexpr (LOADS > 0) __builtin_amdgcn_sched_group_barrier(0x10, LOADS / (2 * T), 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x8, T * T >= 2 * T ? T / 2 : 1, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
}

// C = P Q^T over tiles of 64 T x 64 T, four wavefronts of 32 T x 32 T each.
template <int T, bool SPLIT, int KIND>
__global__ __launch_bounds__(256, 1) void product_kernel(ProductArgs g) {
    constexpr int B = 64 * T;
    __shared__ __attribute__((aligned(128))) _Float16 lds[2][2][B * 64];
    const int lane = lane_id(), wave = uniform(threadIdx.x >> 6);
    const int wi = wave >> 1, wj = wave & 1;
    const int tiles = (KIND == kGram || KIND == kPoly) ? g.tiles_i * (g.tiles_i + 1) / 2 : g.tiles_i * g.tiles_j;
    const int t = xcd_order(blockIdx.x, gridDim.x);
    const int64_t matrix = t / tiles;
    int ti, tj;
    if (KIND == kGram || KIND == kPoly)
        symmetric_tile(t % tiles, g.tiles_i, &ti, &tj);
    else
        full_tile(t % tiles, g.tiles_i, g.tiles_j, &ti, &tj);
    const int64_t shift = matrix * (g.matrix_bytes / 2);

    // Loads: a wavefront instruction fills 8 rows of 64 elements.  The 16-byte
    // piece c of row r sits at position c ^ (r & 7), so that the reads below,
    // same piece of 8 rows, meet 8 different positions.
    const int lr = lane >> 3, lc = (lane & 7) ^ lr;
    const _Float16* p = g.p + shift + ((int64_t)ti * B + wave * 8 + lr) * g.ldp + lc * 8;
    const _Float16* q = g.q + shift + ((int64_t)tj * B + wave * 8 + lr) * g.ldq + lc * 8;
    const int steps = SPLIT ? 3 * g.k_steps : g.k_steps;
    auto issue = [&](int s, int buf) {
        int64_t kp, kq;
        if (SPLIT) {
            const int k = s / 3, part = s - 3 * k;  // hi hi, hi lo, lo hi of the same 64 columns in turn
            kp = (int64_t)k * 64 + (part == 2 ? g.lo : 0);
            kq = (int64_t)k * 64 + (part == 1 ? g.lo : 0);
        } else {
            kp = kq = (int64_t)s * 64;
        }
#pragma unroll
        for (int a = 0; a < 2 * T; ++a) {
            load_to_lds(p + kp + a * 32 * g.ldp, &lds[buf][0][(a * 32 + wave * 8) * 64]);
            load_to_lds(q + kq + a * 32 * g.ldq, &lds[buf][1][(a * 32 + wave * 8) * 64]);
        }
    };
    half8 fp[2][T], fq[2][T];
    const int row_p = wi * 32 * T + (lane & 31), row_q = wj * 32 * T + (lane & 31);
    auto fetch = [&](int buf, int sub, int into) {
        const int pos = ((sub * 2 + (lane >> 5)) ^ (lane & 7)) * 8;
#pragma unroll
        for (int a = 0; a < T; ++a) {
            fp[into][a] = *reinterpret_cast<const half8*>(&lds[buf][0][(row_p + a * 32) * 64 + pos]);
            fq[into][a] = *reinterpret_cast<const half8*>(&lds[buf][1][(row_q + a * 32) * 64 + pos]);
        }
    };
    float16v acc[T][T];
#pragma unroll
    for (int a = 0; a < T; ++a)
#pragma unroll
        for (int b = 0; b < T; ++b) acc[a][b] = 0.0f;
    auto multiply = [&](int from) {
#pragma unroll
        for (int a = 0; a < T; ++a)
#pragma unroll
            for (int b = 0; b < T; ++b)
                acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fp[from][a], fq[from][b], acc[a][b], 0, 0, 0);
    };

    // One step: the fragments of each quarter of the 64 columns are fetched while
    // the matrix cores work on the quarter before.
    auto step = [&](int s, auto more, auto again) {
        const int buf = s & 1;
#pragma unroll
        for (int sub = 0; sub < 3; ++sub) {
            fetch(buf, sub + 1, (sub + 1) & 1);
            multiply(sub & 1);
            interleave<T, 0>();
        }
        // Every wavefront has its last fragments of this buffer and its own
        // loads of the next one have landed: after the barrier that holds for
        // all of them.
        __syncthreads();
        if constexpr (again.value) issue(s + 2, buf);
        if constexpr (more.value) fetch(buf ^ 1, 0, 0);
        multiply(1);
        if constexpr (again.value) interleave<T, 4 * T>();
    };
    issue(0, 0);
    __syncthreads();
    if (steps > 1) issue(1, 1);
    fetch(0, 0, 0);
    int s = 0;
    for (; s + 2 < steps; ++s) step(s, Yes{}, Yes{});
    if (s + 1 < steps) step(s++, Yes{}, No{});
    step(s, No{}, No{});

    // Lane l holds, for register r of block (a, b), C[i][j] with
    // i = 8 (r / 4) + 4 (l / 32) + r % 4 and j = l % 32 within the block.
    // Every wavefront passes its sums, 32 columns j at a time, through its own
    // quarter of the LDS: rows of consecutive i from there meet the old values,
    // the transpose ct and the output along memory, then (the finished values
    // put back) columns give the rows of c.
    constexpr int W = 32 * T, kPitch = W + 4;
    float* strip = reinterpret_cast<float*>(&lds[0][0][0]) + wave * (B * 64 / 2);
    static_assert(32 * kPitch <= B * 64 / 2, "a strip fits a quarter of the LDS");
    const int64_t i0 = (int64_t)ti * B + wi * W, j0 = (int64_t)tj * B + wj * W;
    const bool on_diagonal = (KIND == kGram || KIND == kPoly) && ti == tj;
    const float* diag_in = KIND == kGram ? nullptr : g.diag_in + matrix * (g.matrix_bytes / 4);
    float* diag_out = g.diag_out + matrix * (g.matrix_bytes / 4);
#pragma unroll
    for (int b = 0; b < T; ++b) {
        const int jb = b * 32;
#pragma unroll
        for (int a = 0; a < T; ++a)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float4 v = {acc[a][b][r * 4], acc[a][b][r * 4 + 1], acc[a][b][r * 4 + 2], acc[a][b][r * 4 + 3]};
                *reinterpret_cast<float4*>(&strip[(lane & 31) * kPitch + a * 32 + r * 8 + 4 * (lane >> 5)]) = v;
            }
        wave_sync();
        constexpr int kTogether = 4 * T < 8 ? 4 * T : 8;  // loads in flight, within the register file
#pragma unroll 1
        for (int it0 = 0; it0 < 4 * T; it0 += kTogether) {
        half4 oh[kTogether], ol[kTogether];
        if (KIND != kGram) {
#pragma unroll
            for (int it = 0; it < kTogether; ++it) {
                const int at = (it0 + it) * 64 + lane;
                const _Float16* old = g.old + shift + (j0 + jb + at / (8 * T)) * g.ldold + i0 + at % (8 * T) * 4;
                oh[it] = *reinterpret_cast<const half4*>(old);
                if (SPLIT) ol[it] = *reinterpret_cast<const half4*>(old + g.lo);
            }
        }
#pragma unroll
        for (int it = 0; it < kTogether; ++it) {
            const int at = (it0 + it) * 64 + lane;
            const int jj = at / (8 * T), ii = at % (8 * T) * 4;
            const int64_t i = i0 + ii, j = j0 + jb + jj;
            float4* cell = reinterpret_cast<float4*>(&strip[jj * kPitch + ii]);
            const float4 sum = *cell;
            float v[4] = {sum.x, sum.y, sum.z, sum.w}, w[4];
            if (KIND != kGram) {
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = (float)oh[it][e] + (SPLIT ? (float)ol[it][e] : 0.0f);
            }
            if (KIND == kGram) {
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
            if (KIND != kLast) {
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
        if (KIND == kLast) {
            // 64 consecutive i of one j at a time, whatever the output's type and alignment.
#pragma unroll 4
            for (int it = 0; it < 16 * T; ++it) {
                const int at = it * 64 + lane;
                const int64_t i = i0 + at % W, j = j0 + jb + at / W;
                if (i < g.out_i && j < g.out_j) {
                    const int64_t to = matrix * g.out.stride + j * g.out.ld + i;
                    float o = strip[(at / W) * kPitch + at % W] * (1.0f / kScaleX);
                    if (g.update) o = __builtin_fmaf(-g.move, o, load_value(g.out.ptr, g.out.type, to) * g.keep);
                    store_value(g.out.ptr, g.out.type, to, o);
                }
            }
        } else if (!on_diagonal) {
#pragma unroll 4
            for (int it = 0; it < 4 * T; ++it) {
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
                _Float16* c = g.c + shift + (i0 + ii) * g.ldc + j0 + jb + jj;
                *reinterpret_cast<half4*>(c) = h;
                if (SPLIT) *reinterpret_cast<half4*>(c + g.lo) = l;
            }
        }
        wave_sync();
    }
}

// ---------------------------------------------------------------------------
// Layout of the workspace and the launches.

struct Plan {
    int tile;              // 1, 2 or 4: tiles of 64, 128 or 256
    int64_t m, n;          // padded to the tile
    int64_t lo;            // elements between hi and lo arrays of one matrix
    int64_t x, xt0, xt1, a, b, da, db;  // byte offsets within one matrix's part
    int64_t matrix_bytes;
    int64_t sums;          // byte offset of the partial sums
    int64_t total;
    int sum_blocks;
};

int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

Plan plan_of(int64_t rows, int64_t cols, int64_t count, bool split) {
    Plan p = {};
    const int64_t m = rows < cols ? rows : cols, n = rows < cols ? cols : rows;
    auto tiles = [&](int64_t t) { const int64_t k = (m + t - 1) / t; return count * k * (k + 1) / 2; };
    p.tile = tiles(256) >= 192 ? 4 : tiles(128) >= 128 ? 2 : 1;
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
    p.lo = at / 2;
    if (split) at *= 2;
    p.da = at;
    at += round_up(p.m * 4, 256);
    p.db = at;
    at += round_up(p.m * 4, 256);
    p.matrix_bytes = at;
    p.sums = count * at;
    const int64_t pieces = rows * ((cols + 2047) / 2048);
    p.sum_blocks = (int)(pieces < kSumBlocks ? pieces : kSumBlocks);
    p.total = p.sums + round_up(count * p.sum_blocks * 8, 256);
    return p;
}

template <int T, bool SPLIT>
hipError_t run_products(const UpdateArgs& u, const Plan& p, char* ws, hipStream_t stream) {
    constexpr int B = 64 * T;
    const bool tall = u.rows > u.cols;
    const int tm = (int)(p.m / B), tn = (int)(p.n / B);
    auto at = [&](int64_t o) { return reinterpret_cast<_Float16*>(ws + o); };
    ProductArgs g = {};
    g.lo = p.lo;
    g.matrix_bytes = p.matrix_bytes;
    const unsigned sym = (unsigned)(u.count * (tm * (tm + 1) / 2)), full = (unsigned)(u.count * tm * tn);
    int64_t xt = p.xt0, xt_next = p.xt1;
    for (int s = 0; s < u.n_steps; ++s) {
        g.k = u.steps[s];
        g.tiles_i = g.tiles_j = tm;
        g.p = g.q = at(p.x);
        g.ldp = g.ldq = p.n;
        g.k_steps = (int)(p.n / 64);
        g.c = g.ct = at(p.a);
        g.ldc = g.ldct = p.m;
        g.diag_in = nullptr;
        g.diag_out = reinterpret_cast<float*>(ws + p.da);
        product_kernel<T, SPLIT, kGram><<<sym, 256, 0, stream>>>(g);
        g.p = g.q = g.old = at(p.a);
        g.ldp = g.ldq = g.ldold = p.m;
        g.k_steps = (int)(p.m / 64);
        g.c = g.ct = at(p.b);
        g.diag_in = reinterpret_cast<const float*>(ws + p.da);
        g.diag_out = reinterpret_cast<float*>(ws + p.db);
        product_kernel<T, SPLIT, kPoly><<<sym, 256, 0, stream>>>(g);
        g.diag_in = reinterpret_cast<const float*>(ws + p.db);
        g.diag_out = nullptr;
        if (s + 1 < u.n_steps) {
            g.tiles_j = tn;
            g.p = at(p.b);
            g.q = g.old = at(xt);
            g.c = at(p.x);
            g.ldc = p.n;
            g.ct = at(xt_next);
            product_kernel<T, SPLIT, kStep><<<full, 256, 0, stream>>>(g);
            const int64_t was = xt;
            xt = xt_next;
            xt_next = was;
        } else {
            // The lanes' four consecutive elements run along i: out's columns.
            g.out = u.out;
            g.out_i = u.cols;
            g.out_j = u.rows;
            g.update = u.momentum != nullptr;
            g.keep = u.keep;
            g.move = u.move;
            g.diag_by_i = tall;
            g.p = at(tall ? p.b : xt);
            g.q = at(tall ? xt : p.b);
            g.old = at(tall ? xt : p.x);
            g.ldold = tall ? p.m : p.n;
            g.tiles_i = tall ? tm : tn;
            g.tiles_j = tall ? tn : tm;
            product_kernel<T, SPLIT, kLast><<<full, 256, 0, stream>>>(g);
        }
    }
    return hipGetLastError();
}

template <bool SPLIT>
hipError_t run(const UpdateArgs& u, const Plan& p, char* ws, hipStream_t stream) {
    Source s = {u.x.ptr, u.x.type, u.x.ld, u.x.stride, u.momentum, u.grad_scale, u.decay, u.nesterov};
    double* sums = reinterpret_cast<double*>(ws + p.sums);
    sum_squares_kernel<<<dim3(p.sum_blocks, (unsigned)u.count), 256, 0, stream>>>(s, u.rows, u.cols, sums);
    const bool tall = u.rows > u.cols;
    const int64_t pr = tall ? p.n : p.m, pc = tall ? p.m : p.n;
    _Float16* direct = reinterpret_cast<_Float16*>(ws + (tall ? p.xt0 : p.x));
    _Float16* turned = reinterpret_cast<_Float16*>(ws + (tall ? p.x : p.xt0));
    start_kernel<SPLIT><<<dim3((unsigned)(pc / 64), (unsigned)(pr / 64), (unsigned)u.count), 256, 0, stream>>>(
        s, u.rows, u.cols, sums, p.sum_blocks, u.eps, direct, pc, turned, pr, p.lo, p.matrix_bytes);
    if (p.tile == 4) return run_products<4, SPLIT>(u, p, ws, stream);
    if (p.tile == 2) return run_products<2, SPLIT>(u, p, ws, stream);
    return run_products<1, SPLIT>(u, p, ws, stream);
}

}  // namespace

size_t update_workspace_bytes(int64_t rows, int64_t cols, int64_t count, bool split) {
    return (size_t)plan_of(rows, cols, count, split).total;
}

hipError_t launch_update(const UpdateArgs& u, void* workspace, hipStream_t stream) {
    const Plan p = plan_of(u.rows, u.cols, u.count, u.split);
    char* ws = static_cast<char*>(workspace);
    return u.split ? run<true>(u, p, ws, stream) : run<false>(u, p, ws, stream);
}

}  // namespace sl
