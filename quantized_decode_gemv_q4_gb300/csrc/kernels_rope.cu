// RMSNorm of every query and key head and the rotary rotation of its first `rot` elements, in one pass.
//
//   y_i = x_i * r * gamma_i, r = 1 / sqrt(sum x^2 / D + eps);   a pair (a, b) of y turns to
//   (a cos - b sin, b cos + a sin) with the cos and sin of the token's position from a table.
//
// A group of lanes holds one head row: each lane two 16-byte vectors that contain both elements of its pairs (for the
// half-split order vectors rot/2 apart, for the interleaved order adjacent ones; behind the rotated part adjacent
// vectors pass unrotated), so the rotation needs no exchange and the only shuffles are the norm's sum. Sums and
// products are fp32, and the values are rounded once, when they are stored. A row is read whole before it is written,
// so the outputs may be the inputs.
#include <algorithm>

#include "kv_common.cuh"

namespace q4 {

namespace {

constexpr int kThreads = 256;
// Where there are many rows (three for each resident thread of the device) a lane takes 4 heads and the resident blocks
// walk over the tokens, else a lane takes a head. 8191 bf16 tokens of 32 + 8 heads of 128: 49 us with a head a lane, 37 us
// with 4 heads a lane and a block for every 256 lanes, 32 us so (26 us for the bytes). What is left is the latency of the
// table row behind the position, which is read an iteration ahead.
constexpr int kHeads = 4;
constexpr int kBlocks = 2;  // resident blocks of an SM
constexpr long long kManyLanes = 1LL << 20;

// 16 bytes of activations as they lie in memory, and as floats.
__device__ __forceinline__ void widen(uint4 w, float (&x)[4], float) {
    x[0] = __uint_as_float(w.x), x[1] = __uint_as_float(w.y), x[2] = __uint_as_float(w.z), x[3] = __uint_as_float(w.w);
}
template <typename T>
__device__ __forceinline__ void widen(uint4 w, float (&x)[8], T tag) {
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2(v[i], tag);
        x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
}

// LPR lanes per head row; each takes U heads of a token, query heads or key heads, whose loads are in flight together and
// which share the token's table entries and gamma.
template <typename T, int LPR, int U>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const RopeArgs p) {
    constexpr int V = Vec<T>::N;
    const int lane = threadIdx.x % LPR, q_groups = (p.Hq + U - 1) / U, groups = q_groups + (p.Hkv + U - 1) / U;
    const int pairs = p.rot / (2 * V);  // slots of two vectors that are rotated
    const bool turns = lane < pairs, inside = lane < p.D / (2 * V);
    const int ia = turns && !p.interleaved ? lane * V : 2 * lane * V;
    const int ib = turns && !p.interleaved ? p.rot / 2 + lane * V : ia + V;
    const unsigned step = gridDim.x * (kThreads / LPR), all = (unsigned)p.T * (unsigned)groups;
    unsigned idx = blockIdx.x * (kThreads / LPR) + threadIdx.x / LPR;  // (token, group of heads)
    // Query and key rows share warps: where only one of them has a norm, the lanes of the other sum along, so that a whole
    // warp meets in the shuffles.
    const bool norms = p.q_gamma != nullptr || p.k_gamma != nullptr;
    grid_dependency_wait();
    grid_launch_dependents();

    // the position is known an iteration ahead, so that the table is read along with the heads and not after it
    auto position = [&](unsigned i) { return pairs > 0 && i < all ? p.positions[i / (unsigned)groups] : 0; };
    int pos = position(idx);
    const unsigned rounds = (all + step - 1) / step;  // the same for every lane of a warp: they meet in the norm's shuffles
    for (unsigned round = 0; round < rounds; ++round, idx += step) {
    const int t = (int)(idx / (unsigned)groups), group = (int)(idx - (unsigned)t * (unsigned)groups);
    const bool is_q = group < q_groups;
    const int h0 = (is_q ? group : group - q_groups) * U, heads = min(U, (is_q ? p.Hq : p.Hkv) - h0);
    const bool there = idx < all && inside;
    const T* src = static_cast<const T*>(is_q ? p.q : p.k) + t * (is_q ? p.q_stride : p.k_stride) + (long long)h0 * p.D;
    T* dst = static_cast<T*>(is_q ? p.q_out : p.k_out) + t * (is_q ? p.q_out_stride : p.k_out_stride) + (long long)h0 * p.D;
    const float* gamma = is_q ? p.q_gamma : p.k_gamma;

    uint4 wa[U], wb[U];
    const int next = position(idx + step);
#pragma unroll
    for (int i = 0; i < U; ++i) {
        wa[i] = wb[i] = make_uint4(0u, 0u, 0u, 0u);
        if (there && i < heads) {
            wa[i] = *reinterpret_cast<const uint4*>(src + i * p.D + ia);
            wb[i] = *reinterpret_cast<const uint4*>(src + i * p.D + ib);
        }
    }
    float ga[V] = {}, gb[V] = {};
    if (gamma && there) {
        load_floats(gamma + ia, ga);
        load_floats(gamma + ib, gb);
    }
    const bool bad = there && pairs > 0 && (pos < 0 || pos >= p.max_pos);
    float c[V] = {}, s[V] = {};
    if (there && turns && !bad) {
        const float* table = p.cos_sin + (long long)pos * p.rot + lane * V;
        load_floats(table, c);
        load_floats(table + p.rot / 2, s);
    }
    if (bad && lane == 0) atomicOr(p.fault, (unsigned)kFaultBadPosition);
#pragma unroll
    for (int i = 0; i < U; ++i) {
        float a[V], b[V];
        widen(wa[i], a, T());
        widen(wb[i], b, T());
        if (norms) {
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < V; ++j) sum = fmaf(a[j], a[j], fmaf(b[j], b[j], sum));
#pragma unroll
            for (int o = LPR / 2; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (gamma) {
                const float r = rsqrtf(sum / (float)p.D + p.eps);
#pragma unroll
                for (int j = 0; j < V; ++j) a[j] = a[j] * r * ga[j], b[j] = b[j] * r * gb[j];
            }
        }
        if (!there || i >= heads) continue;
        float oa[V], ob[V];
        if (p.interleaved && turns) {
#pragma unroll
            for (int j = 0; j < V; j += 2) {
                oa[j] = a[j] * c[j / 2] - a[j + 1] * s[j / 2];
                oa[j + 1] = a[j + 1] * c[j / 2] + a[j] * s[j / 2];
                ob[j] = b[j] * c[(V + j) / 2] - b[j + 1] * s[(V + j) / 2];
                ob[j + 1] = b[j + 1] * c[(V + j) / 2] + b[j] * s[(V + j) / 2];
            }
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                oa[j] = turns ? a[j] * c[j] - b[j] * s[j] : a[j];
                ob[j] = turns ? b[j] * c[j] + a[j] * s[j] : b[j];
            }
        }
        if (bad) {  // no table row: the token's heads are NaN
#pragma unroll
            for (int j = 0; j < V; ++j) oa[j] = ob[j] = qnan();
        }
        store_floats(dst + i * p.D + ia, oa);
        store_floats(dst + i * p.D + ib, ob);
    }
    pos = next;
    }
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeArgs& a, int dtype, cudaStream_t s) {
    return with_dtype(dtype, [&](auto tag) {
        using T = decltype(tag);
        const int slots = a.D / (2 * Vec<T>::N);
        auto go = [&](auto lpr) {
            constexpr int LPR = decltype(lpr)::value, rows = kThreads / LPR;
            const long long heads = a.Hq + a.Hkv;
            const bool many = a.T * heads * LPR >= kManyLanes;
            const int u = many ? kHeads : 1;
            const long long groups = (long long)a.T * ((a.Hq + u - 1) / u + (a.Hkv + u - 1) / u);
            long long blocks = (groups + rows - 1) / rows;
            if (many) blocks = std::min<long long>(blocks, (long long)a.sm_count * kBlocks);
            const dim3 grid((unsigned)blocks);
            return many ? launch_grid(qk_norm_rope_kernel<T, LPR, kHeads>, grid, dim3(kThreads), 0, s, launch_overlap(), a)
                        : launch_grid(qk_norm_rope_kernel<T, LPR, 1>, grid, dim3(kThreads), 0, s, launch_overlap(), a);
        };
        if (slots <= 4) return go(std::integral_constant<int, 4>());
        if (slots <= 8) return go(std::integral_constant<int, 8>());
        if (slots <= 16) return go(std::integral_constant<int, 16>());
        return go(std::integral_constant<int, 32>());
    });
}

}  // namespace q4
