// logprobs.hip -- log probabilities of given tokens, entropies and the
// likeliest alternatives (sl_token_logprobs).
//
// One pass over the logits.  With y = x log2 e and R a reference near the
// largest y, each lane keeps over the values it meets
//     s = sum 2^(y - R),  t = sum 2^(y - R) (y - R);
// partial sums join after a shift to the larger R.  Then, whatever R is,
//     log p(x) = (y - R - log2 s) ln 2,  entropy = (log2 s - t / s) ln 2.
// y - R is one fused multiply-add with R the rounded m log2 e of the maximum
// m, so it carries one rounding however large x is.
//
// Alternatives come without a second pass over the row: the scan leaves the
// maximum of every tile of 1024 tokens, and the n_top likeliest tokens lie in
// the n_top tiles that come first by (maximum descending, position ascending),
// since each such tile's maximum precedes every token of the tiles after them.
// Only those tiles are read again.
//
// Enough rows (or a small vocabulary) give every row a block of its own, which
// scans and finishes it; few rows are split over the vocabulary and joined by a
// second kernel.
//
// Bound by memory where there are many rows: 1024 x 262208 bf16 88 us, 6.1
// TB/s; 4096 x 262208 with five alternatives 355 us, 6.05 TB/s.  One row is bound by
// latency: 20 us with 20 alternatives, 6 the scan and 12 the finish.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ops_internal.h"
#include "types.h"
#include "wave.h"

namespace sl {
namespace {

constexpr int kTile = 1024;           // tokens per tile: 16 per lane of a wavefront
constexpr int kPerLane = kTile / kWave;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kFar = -200.0f;       // 2^-200 is 0 in fp32
constexpr float kHuge = 1e38f;        // beyond it m log2 e may leave fp32's range
constexpr float kInf = __builtin_inff();

// The sums relative to the reference that goes with the maximum m.
struct Moments {
    float m, s, t;
};

// y - R for the value x and the maximum m (R = 0 while every value is -inf).
__device__ __forceinline__ float distance(float x, float m) {
    if (m == -kInf) m = 0;
    if (fabsf(m) > kHuge) return (x - m) * kLog2e;
    return __builtin_fmaf(x, kLog2e, -(m * kLog2e));
}

// From the reference of one maximum to that of a larger one.
__device__ __forceinline__ float shift_of(float from, float to) {
    if (from == -kInf) from = 0;
    if (to == -kInf) to = 0;
    const float d = fabsf(from) > kHuge || fabsf(to) > kHuge ? (from - to) * kLog2e : from * kLog2e - to * kLog2e;
    return fmaxf(d, kFar);
}

// a's sums relative to the new maximum m >= a.m.
__device__ __forceinline__ Moments rebase(Moments a, float m) {
    const float d = a.s > 0 ? shift_of(a.m, m) : 0.0f;  // empty sums stay 0; a NaN stays in s
    const float r = __builtin_amdgcn_exp2f(d);
    return {m, a.s * r, (a.t + d * a.s) * r};
}

__device__ __forceinline__ Moments join(Moments a, Moments b) {
    const float m = fmaxf(a.m, b.m);
    a = rebase(a, m);
    b = rebase(b, m);
    return {m, a.s + b.s, a.t + b.t};
}

__device__ __forceinline__ Moments shuffle_xor(Moments a, int o) {
    return {__shfl_xor(a.m, o), __shfl_xor(a.s, o), __shfl_xor(a.t, o)};
}

// A 32-bit key that orders floats (-0 as +0); -inf and below it nothing.
__device__ __forceinline__ uint32_t order_of(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
constexpr uint32_t kBannedOrder = 0x007fffffu;  // order_of(-inf)

__device__ __forceinline__ float value_of(uint32_t order) {
    return __uint_as_float(order ^ ((uint32_t)((int32_t)~order >> 31) | 0x80000000u));
}

// Larger for a larger value, then for a smaller place; 0 for a banned value.
__device__ __forceinline__ uint64_t key_of(float v, uint32_t place) {
    const uint32_t o = order_of(v);
    return o > kBannedOrder ? (uint64_t)o << 32 | (0xffffffffu - place) : 0;
}
__device__ __forceinline__ uint32_t place_of(uint64_t key) { return 0xffffffffu - (uint32_t)key; }

template <int CTRL, int ROW_MASK>
__device__ __forceinline__ uint64_t max_dpp(uint64_t v) {
    const uint64_t o = (uint64_t)dpp_or_zero<CTRL, ROW_MASK>((uint32_t)(v >> 32)) << 32 |
                       dpp_or_zero<CTRL, ROW_MASK>((uint32_t)v);
    return o > v ? o : v;
}

// The largest key of the wavefront, in every lane.
__device__ __forceinline__ uint64_t wave_max_key(uint64_t v) {
    v = max_dpp<kRowShr1, 0xf>(v);
    v = max_dpp<kRowShr2, 0xf>(v);
    v = max_dpp<kRowShr4, 0xf>(v);
    v = max_dpp<kRowShr8, 0xf>(v);
    v = max_dpp<kRowBcast15, 0xa>(v);
    v = max_dpp<kRowBcast31, 0xc>(v);
    return (uint64_t)read_lane((uint32_t)(v >> 32), kWave - 1) << 32 | read_lane((uint32_t)v, kWave - 1);
}

template <int TYPE>
struct Element;
template <>
struct Element<SL_F32> {
    typedef float type;
    static constexpr int kVector = 4;
    static __device__ __forceinline__ float value(float v) { return v; }
    static __device__ __forceinline__ void unpack(uint4 q, float* x) {
        x[0] = __uint_as_float(q.x), x[1] = __uint_as_float(q.y), x[2] = __uint_as_float(q.z), x[3] = __uint_as_float(q.w);
    }
};
template <>
struct Element<SL_BF16> {
    typedef uint16_t type;
    static constexpr int kVector = 8;
    static __device__ __forceinline__ float value(uint16_t v) { return bf16_value(v); }
    static __device__ __forceinline__ void unpack(uint4 q, float* x) {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
        for (int k = 0; k < 4; ++k) {
            x[2 * k] = __uint_as_float(w[k] << 16);
            x[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
        }
    }
};
template <>
struct Element<SL_F16> {
    typedef _Float16 type;
    static constexpr int kVector = 8;
    static __device__ __forceinline__ float value(_Float16 v) { return (float)v; }
    static __device__ __forceinline__ void unpack(uint4 q, float* x) {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
        for (int k = 0; k < 4; ++k) {
            x[2 * k] = (float)__builtin_bit_cast(_Float16, (uint16_t)w[k]);
            x[2 * k + 1] = (float)__builtin_bit_cast(_Float16, (uint16_t)(w[k] >> 16));
        }
    }
};

// Tiles are laid over the 16-byte line that holds the row's first token:
// position pos of the tiles is token pos - lead.
template <int TYPE>
__device__ __forceinline__ int lead_of(const typename Element<TYPE>::type* row) {
    return (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(*row));
}

// Positions [at, at + kVector) of a row: one aligned load inside the row,
// single tokens (and -inf beyond) at its ends.  ONCE: loads that pass the
// caches by, for the scan: 2048 rows of 131072 fp32 were read at 6.8 TB/s so
// and at 6.0 TB/s without.
typedef uint32_t uint4v __attribute__((ext_vector_type(4)));

template <int TYPE, bool ONCE>
__device__ __forceinline__ void load_vector(const typename Element<TYPE>::type* row, int lead, int64_t vocab, int64_t at,
                                            float* x) {
    typedef Element<TYPE> E;
    const int64_t token = at - lead;
    if (token >= 0 && token + E::kVector <= vocab) {
        const uint4v* p = reinterpret_cast<const uint4v*>(row + token);
        const uint4v q = ONCE ? __builtin_nontemporal_load(p) : *p;
        E::unpack(make_uint4(q.x, q.y, q.z, q.w), x);
    } else {
#pragma unroll
        for (int k = 0; k < E::kVector; ++k)
            x[k] = token + k >= 0 && token + k < vocab ? E::value(row[token + k]) : -kInf;
    }
}

constexpr int kMaxWaves = 8;     // of a scanning block
constexpr int kFinishWaves = 16; // of a block that finishes a split row: the chosen tiles' loads at once
constexpr int kUnitsPerLane = 8, kUnits = kWave * kUnitsPerLane;
constexpr int kListed = 512;     // candidates ranked against each other

// Writes row r's outputs from its joined moments.  Called by every thread of a
// block; maxima: the row's tile maxima in LDS (n_top > 0).
template <int TYPE>
__device__ void finish_row(const LogprobArgs& a, int64_t r, Moments all, const float* maxima, int n_tiles) {
    typedef Element<TYPE> E;
    constexpr int V = E::kVector;
    __shared__ int chosen[SL_MAX_ALTERNATIVES], n_chosen, n_listed;
    __shared__ uint32_t least;
    __shared__ uint64_t best[2][kFinishWaves], listed[kListed];
    const int lane = lane_id(), wave = uniform(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const typename E::type* row = static_cast<const typename E::type*>(a.logits) + r * a.ld;
    const bool bad = !(all.s >= 0);   // a NaN or +inf among the logits
    const float log_s = log2f(all.s);  // -inf for a row of banned tokens
    auto logprob_of = [&](float x) {
        // y would leave fp32's range; x - m, so far from 0, needs no reference
        if (fabsf(x) > kHuge) return (x - all.m) - log_s * kLn2;
        return (distance(x, all.m) - log_s) * kLn2;
    };
    if (threadIdx.x == blockDim.x - kWave) {  // of the last wavefront: the first has more to do
        if (a.logprob) {
            const int64_t token = a.targets[r];
            float v = 0;
            if (token >= 0 && token < a.vocab) {
                const float x = E::value(row[token]);
                v = bad ? __builtin_nanf("") : all.s == 0 ? -kInf : logprob_of(x);
            }
            a.logprob[r] = v;
        }
        if (a.entropy) a.entropy[r] = bad ? __builtin_nanf("") : all.s == 0 ? 0.0f : fmaxf((log_s - all.t / all.s) * kLn2, 0.0f);
    }
    if (a.n_top == 0) return;
    if (bad) {
        if ((int)threadIdx.x < a.n_top) {
            a.top_index[r * a.n_top + threadIdx.x] = -1;
            a.top_logprob[r * a.n_top + threadIdx.x] = __builtin_nanf("");
        }
        return;
    }

    // The n_top first units, each `unit` tiles in a row (one, up to 512 tiles).
    // Lane l of the first wavefront holds the units 8 l to 8 l + 7, so that of
    // equal maxima the lowest lane's, and there the lowest, is the first.
    const int unit = (n_tiles + kUnits - 1) / kUnits;
    if (wave == 0) {
        uint32_t held[kUnitsPerLane];
#pragma unroll
        for (int e = 0; e < kUnitsPerLane; ++e) {
            held[e] = kBannedOrder;
            const int t0 = (lane * kUnitsPerLane + e) * unit;
            for (int t = t0; t < min(t0 + unit, n_tiles); ++t) held[e] = max(held[e], order_of(maxima[t]));
        }
        uint32_t last = 0;
        int k = 0;
        for (; k < a.n_top; ++k) {
            uint32_t mine = held[0];
#pragma unroll
            for (int e = 1; e < kUnitsPerLane; ++e) mine = max(mine, held[e]);
            const uint32_t top = wave_max(mine);
            if (top == kBannedOrder) break;
            last = top;
            bool here = lane == __ffsll((unsigned long long)ballot(mine == top)) - 1;
            int where = 0;
#pragma unroll
            for (int e = 0; e < kUnitsPerLane; ++e) {
                const bool it = here && held[e] == top;
                if (it) held[e] = kBannedOrder, where = e + 1;
                here = here && !it;
            }
            if (where) chosen[k] = lane * kUnitsPerLane + where - 1;
        }
        // With units to spare every token counts, else those from the last maximum up.
        if (lane == 0) n_chosen = k, least = k < a.n_top ? kBannedOrder + 1 : last, n_listed = 0;
    }
    __syncthreads();

    // The alternatives are among the tokens of those units that are at least
    // the last unit's maximum, mostly a few more than n_top: list them and
    // rank each by counting the ones before it.
    const int lead = lead_of<TYPE>(row);
    const int tiles = n_chosen * unit;
    auto visit = [&](auto&& each) {  // each(value, token) for this lane's tokens of this wavefront's tiles
        for (int k = wave; k < tiles; k += waves) {
            const int64_t at = ((int64_t)chosen[k / unit] * unit + k % unit) * kTile + lane * kPerLane;
            float x[kPerLane];
#pragma unroll
            for (int u = 0; u < kPerLane / V; ++u) load_vector<TYPE, false>(row, lead, a.vocab, at + u * V, x + u * V);
#pragma unroll
            for (int e = 0; e < kPerLane; ++e) each(x[e], (uint32_t)(at - lead + e));
        }
    };
    auto write = [&](int k, uint64_t key) {
        a.top_index[r * a.n_top + k] = key ? (int)place_of(key) : -1;
        a.top_logprob[r * a.n_top + k] = key ? logprob_of(value_of((uint32_t)(key >> 32))) : -kInf;
    };
    const float floor_value = value_of(least);
    visit([&](float v, uint32_t token) {
        if (v >= floor_value) {
            const int at = atomicAdd(&n_listed, 1);
            if (at < kListed) listed[at] = key_of(v, token);
        }
    });
    __syncthreads();
    const int n = tiles ? n_listed : 0;
    if (n <= kListed) {
        for (int i = threadIdx.x; i < n; i += blockDim.x) {
            const uint64_t mine = listed[i];
            int rank = 0;
#pragma unroll 4
            for (int j = 0; j < n; ++j) rank += listed[j] > mine;
            if (rank < a.n_top) write(rank, mine);
        }
        if ((int)threadIdx.x >= n && (int)threadIdx.x < a.n_top) write(threadIdx.x, 0);
        return;
    }
    // Too many near the top (equal logits): one after another, each the
    // largest key below the one before.
    uint64_t before = ~(uint64_t)0;
    for (int k = 0; k < a.n_top; ++k) {
        uint64_t m = 0;
        visit([&](float v, uint32_t token) {
            const uint64_t key = key_of(v, token);
            if (key < before && key > m) m = key;
        });
        m = wave_max_key(m);
        if (lane == 0) best[k & 1][wave] = m;
        __syncthreads();  // the next round writes the other half, so one barrier a round is enough
        m = 0;
        for (int w = 0; w < waves; ++w) m = best[k & 1][w] > m ? best[k & 1][w] : m;
        if (threadIdx.x == 0) write(k, m);
        before = m;
    }
}

// Scans row blockIdx.y: of its tiles the wavefronts of all the row's blocks
// take one after another in turn.  WHOLE: the row is this block's alone, and
// is finished here; otherwise moments and tile maxima go to part and tile_max.
template <int TYPE, bool TOP, bool WHOLE>
__global__ __launch_bounds__(kMaxWaves * kWave) void scan_kernel(LogprobArgs a, int n_tiles, Moments* part, float* tile_max) {
    typedef Element<TYPE> E;
    constexpr int V = E::kVector, U = kPerLane / V;
    extern __shared__ float maxima[];
    __shared__ Moments joined[kMaxWaves];
    const int lane = lane_id(), wave = uniform(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int64_t r = blockIdx.y;
    const typename E::type* row = static_cast<const typename E::type*>(a.logits) + r * a.ld;
    const int lead = lead_of<TYPE>(row);
    float* const out = WHOLE ? maxima : tile_max + r * n_tiles;
    Moments acc = {-kInf, 0, 0};
    // Once a banned token, an infinity, a NaN or a value far beyond kHuge has
    // shown (t is a NaN or infinite then, as 0 times -inf is), the wavefront's
    // sums take care of them, at about twice the instructions.
    bool careful = false;
    for (int t = blockIdx.x * waves + wave; t < n_tiles; t += gridDim.x * waves) {
        float x[kPerLane];
#pragma unroll
        for (int u = 0; u < U; ++u)
            load_vector<TYPE, true>(row, lead, a.vocab, (int64_t)t * kTile + u * kWave * V + lane * V, x + u * V);
        float m = x[0];
#pragma unroll
        for (int k = 1; k < kPerLane; ++k) m = fmaxf(m, x[k]);
        if (TOP) {
            const uint32_t all = wave_max(order_of(m));
            if (lane == 0) out[t] = value_of(all);
        }
        acc = rebase(acc, fmaxf(acc.m, m));
        if (!careful) {
            const float ref = acc.m * kLog2e;
            float sum = acc.s, tsum = acc.t;
#pragma unroll
            for (int k = 0; k < kPerLane; ++k) {
                const float d = __builtin_fmaf(x[k], kLog2e, -ref);
                const float e = __builtin_amdgcn_exp2f(d);
                sum += e;
                tsum = __builtin_fmaf(e, d, tsum);
            }
            careful = ballot(!(fabsf(tsum) < kInf)) != 0;
            if (!careful) acc.s = sum, acc.t = tsum;
        }
        if (careful) {
#pragma unroll
            for (int k = 0; k < kPerLane; ++k) {
                const float d = distance(x[k], acc.m);
                const float e = __builtin_amdgcn_exp2f(d);
                acc.s += e;
                acc.t = __builtin_fmaf(e, fmaxf(d, kFar), acc.t);
            }
        }
    }
    for (int o = 32; o; o >>= 1) acc = join(acc, shuffle_xor(acc, o));
    if (lane == 0) joined[wave] = acc;
    __syncthreads();
    acc = joined[0];
    for (int w = 1; w < waves; ++w) acc = join(acc, joined[w]);
    if (WHOLE)
        finish_row<TYPE>(a, r, acc, maxima, n_tiles);
    else if (threadIdx.x == 0)
        part[r * gridDim.x + blockIdx.x] = acc;
}

// Joins the parts of row blockIdx.x and finishes it.
template <int TYPE>
__global__ __launch_bounds__(kFinishWaves * kWave) void finish_kernel(LogprobArgs a, int n_parts, int n_tiles,
                                                                   const Moments* part, const float* tile_max) {
    extern __shared__ float maxima[];
    const int64_t r = blockIdx.x;
    if (a.n_top)
        for (int t = threadIdx.x; t < n_tiles; t += blockDim.x) maxima[t] = tile_max[r * n_tiles + t];
    Moments all = {-kInf, 0, 0};
    for (int k = lane_id(); k < n_parts; k += kWave) all = join(all, part[r * n_parts + k]);
    for (int o = 32; o; o >>= 1) all = join(all, shuffle_xor(all, o));
    __syncthreads();
    finish_row<TYPE>(a, r, all, maxima, n_tiles);
}

constexpr int64_t kBlocks = 1024;

struct Plan {
    int n_tiles, n_parts, waves;
    int64_t maxima, total;  // byte offset of the tile maxima; bytes in all
};

Plan plan_of(int64_t rows, int64_t vocab, int32_t type, int32_t n_top) {
    Plan p = {};
    const int lead = 16 / type_bytes(type) - 1;  // at most
    p.n_tiles = (int)((vocab + lead + kTile - 1) / kTile);
    p.waves = p.n_tiles < kMaxWaves ? p.n_tiles : kMaxWaves;
    // Rows are split over the vocabulary, down to one tile per wavefront, until
    // kBlocks blocks share the work.
    const int64_t most = (p.n_tiles + p.waves - 1) / p.waves, want = kBlocks / (rows > 0 ? rows : 1);
    p.n_parts = (int)(want < 1 ? 1 : want < most ? want : most);
    if (p.n_parts == 1) return p;
    const int64_t part_bytes = rows * p.n_parts * (int64_t)sizeof(Moments);
    p.maxima = (part_bytes + 255) / 256 * 256;
    p.total = p.maxima + (n_top ? rows * p.n_tiles * 4 : 0);
    return p;
}

template <int TYPE, bool TOP>
hipError_t run(const LogprobArgs& a, const Plan& p, char* ws, hipStream_t stream) {
    Moments* part = reinterpret_cast<Moments*>(ws);
    float* maxima = reinterpret_cast<float*>(ws + p.maxima);
    const size_t lds = TOP ? (size_t)p.n_tiles * 4 : 0;
    // A grid's y extent is limited to 65535.
    for (int64_t r0 = 0; r0 < a.rows; r0 += 65535) {
        const int64_t rows = a.rows - r0 < 65535 ? a.rows - r0 : 65535;
        LogprobArgs b = a;
        b.logits = static_cast<const char*>(a.logits) + r0 * a.ld * type_bytes(TYPE);
        if (b.targets) b.targets += r0;
        if (b.logprob) b.logprob += r0;
        if (b.entropy) b.entropy += r0;
        if (b.top_logprob) b.top_logprob += r0 * a.n_top;
        if (b.top_index) b.top_index += r0 * a.n_top;
        const dim3 grid(p.n_parts, (unsigned)rows);
        if (p.n_parts == 1) {
            scan_kernel<TYPE, TOP, true><<<grid, p.waves * kWave, lds, stream>>>(b, p.n_tiles, nullptr, nullptr);
        } else {
            Moments* pt = part + r0 * p.n_parts;
            float* mx = maxima + r0 * p.n_tiles;
            scan_kernel<TYPE, TOP, false><<<grid, p.waves * kWave, 0, stream>>>(b, p.n_tiles, pt, mx);
            finish_kernel<TYPE><<<(unsigned)rows, (TOP ? kFinishWaves : 1) * kWave, lds, stream>>>(b, p.n_parts, p.n_tiles, pt, mx);
        }
    }
    return hipGetLastError();
}

template <int TYPE>
hipError_t run(const LogprobArgs& a, const Plan& p, char* ws, hipStream_t stream) {
    return a.n_top ? run<TYPE, true>(a, p, ws, stream) : run<TYPE, false>(a, p, ws, stream);
}

}  // namespace

size_t logprob_workspace_bytes(int64_t rows, int64_t vocab, int32_t type, int32_t n_top) {
    return (size_t)plan_of(rows, vocab, type, n_top).total;
}

hipError_t launch_logprobs(const LogprobArgs& a, void* workspace, hipStream_t stream) {
    const Plan p = plan_of(a.rows, a.vocab, a.type, a.n_top);
    char* ws = static_cast<char*>(workspace);
    if (a.type == SL_F32) return run<SL_F32>(a, p, ws, stream);
    if (a.type == SL_BF16) return run<SL_BF16>(a, p, ws, stream);
    return run<SL_F16>(a, p, ws, stream);
}

}  // namespace sl
