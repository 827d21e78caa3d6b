// logprobs.hip -- log probabilities of given tokens, entropies and the
// likeliest alternatives (sl_token_logprobs).
//
// One pass over the logits.  Each lane keeps, over the values x it meets,
//     m = max x,  s = sum exp(x - m),  t = sum exp(x - m) (x - m),
// and partial triples join as s = s1 exp(m1 - m) + s2 exp(m2 - m), t likewise
// with each part's t shifted by (m1 - m) s1.  Then lse = m + log s and
// entropy = log s - t / s.
//
// Alternatives come without a second pass over the row: the scan leaves the
// maximum of every tile of 1024 tokens, and the n_top likeliest tokens lie in
// the n_top tiles that come first by (maximum descending, position ascending),
// since each such tile's maximum precedes every token of the tiles after them.
// The finish kernel reads only those tiles again.
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
constexpr float kFar = -150.0f;       // exp(-150) is 0 in fp32
constexpr float kInf = __builtin_inff();

struct Moments {
    float m, s, t;
};

// The reference of exponentials: the maximum, or 0 while every value is -inf.
__device__ __forceinline__ float reference(float m) { return m == -kInf ? 0.0f : m; }

__device__ __forceinline__ float exp_of(float d) { return __builtin_amdgcn_exp2f(d * kLog2e); }

// a's sums relative to the new maximum m >= a.m.
__device__ __forceinline__ Moments rebase(Moments a, float m) {
    const float d = fmaxf(reference(a.m) - reference(m), kFar);
    const float r = a.s > 0 ? exp_of(d) : 0.0f;  // empty sums stay 0; a NaN stays in s
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

__device__ __forceinline__ float wave_fmax(float v) {
    for (int o = 32; o; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
    return v;
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
// single tokens (and -inf beyond) at its ends.
template <int TYPE>
__device__ __forceinline__ void load_vector(const typename Element<TYPE>::type* row, int lead, int64_t vocab, int64_t at,
                                            float* x) {
    typedef Element<TYPE> E;
    const int64_t token = at - lead;
    if (token >= 0 && token + E::kVector <= vocab) {
        E::unpack(*reinterpret_cast<const uint4*>(row + token), x);
    } else {
#pragma unroll
        for (int k = 0; k < E::kVector; ++k)
            x[k] = token + k >= 0 && token + k < vocab ? E::value(row[token + k]) : -kInf;
    }
}

// Row blockIdx.y, tiles blockIdx.x * 4 + wave, then every gridDim.x * 4th.
template <int TYPE, bool TOP>
__global__ __launch_bounds__(256) void scan_kernel(LogprobArgs a, int n_tiles, Moments* part, float* tile_max) {
    typedef Element<TYPE> E;
    constexpr int V = E::kVector, U = kPerLane / V;
    __shared__ Moments joined[4];
    const int lane = lane_id(), wave = threadIdx.x >> 6;
    const int64_t r = blockIdx.y;
    const typename E::type* row = static_cast<const typename E::type*>(a.logits) + r * a.ld;
    const int lead = lead_of<TYPE>(row);
    Moments acc = {-kInf, 0, 0};
    for (int t = blockIdx.x * 4 + wave; t < n_tiles; t += gridDim.x * 4) {
        float x[kPerLane];
#pragma unroll
        for (int u = 0; u < U; ++u)
            load_vector<TYPE>(row, lead, a.vocab, (int64_t)t * kTile + u * kWave * V + lane * V, x + u * V);
        float m = x[0];
#pragma unroll
        for (int k = 1; k < kPerLane; ++k) m = fmaxf(m, x[k]);
        if (TOP) {
            const float all = wave_fmax(m);
            if (lane == 0) tile_max[r * n_tiles + t] = all;
        }
        acc = rebase(acc, fmaxf(acc.m, m));
        const float ref = reference(acc.m);
#pragma unroll
        for (int k = 0; k < kPerLane; ++k) {
            const float d = x[k] - ref;
            const float e = exp_of(d);
            acc.s += e;
            acc.t = __builtin_fmaf(e, fmaxf(d, kFar), acc.t);
        }
    }
    for (int o = 32; o; o >>= 1) acc = join(acc, shuffle_xor(acc, o));
    if (lane == 0) joined[wave] = acc;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 4; ++w) acc = join(acc, joined[w]);
        part[r * gridDim.x + blockIdx.x] = acc;
    }
}

constexpr int kTilesPerWave = 2;  // of the n_top tiles read again

// One row per block of ceil(n_top / 2) wavefronts (one at least): joins the
// row's parts, then takes the alternatives one by one from the selected tiles,
// which the wavefronts hold in registers.
template <int TYPE>
__global__ __launch_bounds__(1024) void finish_kernel(LogprobArgs a, int n_parts, int n_tiles, const Moments* part,
                                                      const float* tile_max) {
    typedef Element<TYPE> E;
    constexpr int V = E::kVector;
    __shared__ int chosen[SL_MAX_ALTERNATIVES];
    __shared__ float best_value[16];
    __shared__ int best_token[16];
    const int lane = lane_id(), wave = uniform(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int64_t r = blockIdx.x;
    const typename E::type* row = static_cast<const typename E::type*>(a.logits) + r * a.ld;

    Moments all = {-kInf, 0, 0};
    for (int k = lane; k < n_parts; k += kWave) all = join(all, part[r * n_parts + k]);
    for (int o = 32; o; o >>= 1) all = join(all, shuffle_xor(all, o));
    const bool bad = !(all.s >= 0);  // a NaN or +inf among the logits
    const float log_s = logf(all.s);  // -inf for a row of banned tokens
    if (threadIdx.x == 0) {
        if (a.logprob) {
            const int64_t token = a.targets[r];
            float v = 0;
            if (token >= 0 && token < a.vocab) {
                const float x = E::value(row[token]);
                v = bad ? __builtin_nanf("") : all.s == 0 ? -kInf : (x - all.m) - log_s;
            }
            a.logprob[r] = v;
        }
        if (a.entropy) a.entropy[r] = bad ? __builtin_nanf("") : all.s == 0 ? 0.0f : fmaxf(log_s - all.t / all.s, 0.0f);
    }
    if (a.n_top == 0) return;

    // The n_top first tiles by (maximum descending, position ascending).  Lane l
    // holds the tiles [l c, (l + 1) c), so the lowest lane has the lowest tile.
    if (wave == 0) {
        const int c = (n_tiles + kWave - 1) / kWave;
        const float* maxima = tile_max + r * n_tiles;
        uint64_t taken = 0;  // of the lane's own tiles, c <= 64
        auto next = [&](float* v, int* which) {
            *v = -kInf;
            *which = -1;
            for (int k = 0; k < c; ++k) {
                const int t = lane * c + k;
                if (t >= n_tiles || (taken >> k & 1)) continue;
                const float x = maxima[t];
                if (x > *v) *v = x, *which = k;
            }
        };
        float v;
        int which;
        next(&v, &which);
        for (int k = 0; k < a.n_top; ++k) {
            const float top = wave_fmax(v);
            const uint64_t who = ballot(v == top && which >= 0);
            if (who == 0) {  // only banned tokens are left
                if (lane == 0) chosen[k] = -1;
                continue;
            }
            if (lane == __ffsll((unsigned long long)who) - 1) {
                chosen[k] = lane * c + which;
                taken |= (uint64_t)1 << which;
                next(&v, &which);
            }
        }
    }
    __syncthreads();

    // This wavefront's tiles, 16 consecutive tokens per lane.
    const int lead = lead_of<TYPE>(row);
    float x[kTilesPerWave][kPerLane];
    int64_t first[kTilesPerWave];
#pragma unroll
    for (int h = 0; h < kTilesPerWave; ++h) {
        const int k = wave * kTilesPerWave + h;
        const int t = k < a.n_top ? chosen[k] : -1;
        first[h] = (int64_t)t * kTile + lane * kPerLane;
        if (t >= 0) {
#pragma unroll
            for (int u = 0; u < kPerLane / V; ++u) load_vector<TYPE>(row, lead, a.vocab, first[h] + u * V, &x[h][u * V]);
        } else {
#pragma unroll
            for (int k2 = 0; k2 < kPerLane; ++k2) x[h][k2] = -kInf;
        }
    }
    // The wavefront's likeliest remaining token; ties go to the lower one.
    float value;
    int token;
    auto find = [&]() {
        value = -kInf;
        token = 0x7fffffff;
#pragma unroll
        for (int h = 0; h < kTilesPerWave; ++h) {
            float v = -kInf;
            int at = 0;
#pragma unroll
            for (int k = 0; k < kPerLane; ++k)
                if (x[h][k] > v) v = x[h][k], at = k;
            const float top = wave_fmax(v);
            const uint64_t who = ballot(v == top && v > -kInf);
            if (who == 0) continue;
            const int l = __ffsll((unsigned long long)who) - 1;
            const int tok = (int)__shfl((int)(first[h] - lead) + at, l);
            if (top > value || (top == value && tok < token)) value = top, token = tok;
        }
    };
    find();
    for (int k = 0; k < a.n_top; ++k) {
        if (lane == 0) best_value[wave] = value, best_token[wave] = token;
        __syncthreads();
        float v = lane < waves ? best_value[lane] : -kInf;
        int tok = lane < waves ? best_token[lane] : 0x7fffffff;
        const float top = wave_fmax(v);
        if (v != top) tok = 0x7fffffff;
        for (int o = 32; o; o >>= 1) tok = min(tok, __shfl_xor(tok, o));
        const bool none = top == -kInf || bad;
        if (threadIdx.x == 0) {
            a.top_index[r * a.n_top + k] = none ? -1 : tok;
            a.top_logprob[r * a.n_top + k] = bad ? __builtin_nanf("") : none ? -kInf : (top - all.m) - log_s;
        }
        if (tok == token && !none) {  // this wavefront's: strike it out
#pragma unroll
            for (int h = 0; h < kTilesPerWave; ++h)
#pragma unroll
                for (int k2 = 0; k2 < kPerLane; ++k2)
                    if (first[h] - lead + k2 == tok) x[h][k2] = -kInf;
            find();
        }
        __syncthreads();
    }
}

struct Plan {
    int n_tiles, n_parts;
    int64_t maxima, total;  // byte offset of the tile maxima; bytes in all
};

Plan plan_of(int64_t rows, int64_t vocab, int32_t type, int32_t n_top) {
    Plan p;
    const int lead = 16 / type_bytes(type) - 1;  // at most
    p.n_tiles = (int)((vocab + lead + kTile - 1) / kTile);
    // Few rows are split over the vocabulary, down to one tile per wavefront,
    // until about 1024 blocks share the work.
    const int64_t most = (p.n_tiles + 3) / 4, want = (1024 + rows - 1) / (rows > 0 ? rows : 1);
    p.n_parts = (int)(want < most ? want : most);
    const int64_t part_bytes = rows * p.n_parts * (int64_t)sizeof(Moments);
    p.maxima = (part_bytes + 255) / 256 * 256;
    p.total = p.maxima + (n_top ? rows * p.n_tiles * 4 : 0);
    return p;
}

template <int TYPE>
hipError_t run(const LogprobArgs& a, const Plan& p, char* ws, hipStream_t stream) {
    Moments* part = reinterpret_cast<Moments*>(ws);
    float* maxima = reinterpret_cast<float*>(ws + p.maxima);
    const int waves = a.n_top > kTilesPerWave ? (a.n_top + kTilesPerWave - 1) / kTilesPerWave : 1;
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
        Moments* pt = part + r0 * p.n_parts;
        float* mx = maxima + r0 * p.n_tiles;
        if (a.n_top)
            scan_kernel<TYPE, true><<<grid, 256, 0, stream>>>(b, p.n_tiles, pt, mx);
        else
            scan_kernel<TYPE, false><<<grid, 256, 0, stream>>>(b, p.n_tiles, pt, mx);
        finish_kernel<TYPE><<<(unsigned)rows, waves * kWave, 0, stream>>>(b, p.n_parts, p.n_tiles, pt, mx);
    }
    return hipGetLastError();
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
