// A whole mixture-of-experts layer for a few tokens over planar Q4 experts, and its last part alone (the experts' down
// projections and their weighted sum).
//
//   xn = x, or x * r * gamma;  logits = Wr xn, top-k and softmax weights (the router's kernel);
//   h[t, s] = silu(Wg xn) * (Wu xn) and z[t, s] = Wd h[t, s] of expert e(t, s);
//   out[t] = residual[t] + sum over s of weight[t, s] * z[t, s].
#include <algorithm>
#include <mutex>

#include "block.h"
#include "kv_common.cuh"

namespace q4 {

namespace {

struct Carve {  // parts of a workspace, each 16-byte aligned
    uint8_t* base;
    size_t at = 0;
    template <typename T>
    T* take(size_t n) {
        T* p = reinterpret_cast<T*>(base + at);
        at += (n * sizeof(T) + 15) / 16 * 16;
        return base ? p : nullptr;
    }
};

struct PrepParams {
    const void* x;
    const float* gamma;
    float* xn;
    unsigned *x_max, *h_max;
    float eps;
    int K, topk;
    long long x_stride;
};

// xn[t] = x[t], or its norm, in fp32, and the bits of its largest size; the maxima of the token's h start from 0.
template <typename T>
__global__ void __launch_bounds__(256) moe_prep_kernel(const PrepParams p) {
    constexpr int V = Vec<T>::N;
    __shared__ float part[8];
    __shared__ unsigned part_max[8];
    const T* x = static_cast<const T*>(p.x) + (long long)blockIdx.x * p.x_stride;
    float* xn = p.xn + (long long)blockIdx.x * p.K;
    grid_dependency_wait();
    grid_launch_dependents();
    float r = 1.f;
    if (p.gamma) {
        float sum = 0.f;
        for (int k = threadIdx.x * V; k < p.K; k += 256 * V) {
            float v[V];
            load_floats(x + k, v);
#pragma unroll
            for (int j = 0; j < V; ++j) sum = fmaf(v[j], v[j], sum);
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
        __syncthreads();
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += part[i];
        r = rsqrtf(sum / (float)p.K + p.eps);
    }
    unsigned m = 0u;
    for (int k = threadIdx.x * V; k < p.K; k += 256 * V) {
        float v[V];
        load_floats(x + k, v);
        if (p.gamma) {
            float g[V];
            load_floats(p.gamma + k, g);
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] = v[j] * r * g[j];
        }
#pragma unroll
        for (int j = 0; j < V; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
#pragma unroll
        for (int j = 0; j < V; j += 4)
            *reinterpret_cast<float4*>(xn + k + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) part_max[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int i = 1; i < 8; ++i) m = max(m, part_max[i]);
        p.x_max[blockIdx.x] = m;
    }
    for (int i = threadIdx.x; i < p.topk; i += 256) p.h_max[blockIdx.x * p.topk + i] = 0u;
}


// ---- the experts' products -------------------------------------------------------------------------------------------
//
// One kernel for gate and up (with SwiGLU) and for down. Slots that go to the same expert form a segment of up to `cap`
// (8, or fewer where the vectors are long); long inputs of the down projection are cut into parts whose sums the join adds. A
// segment's rows are units of 32: 16 of gate and the same 16 of up, or 32 of down. All units lie on one line that is cut
// into equal pieces, one for each CTA (one CTA an SM), and a piece's chunks of 4 blocks (128 columns) are cut into equal
// pieces for its warps. So every weight is read once a segment, and a warp adds a unit's chunks in registers; a unit cut
// between warps is joined through shared memory in the order of its chunks, so that the same call gives the same bits.
//
// Products run on m16n8k16 matrix instructions with the weights as rows: ldmatrix brings a block's word to each lane, eight
// codes become eight exact f16 values code - 8 with nine instructions, and a block's fp32 sums are multiplied by the block's
// scale in fp32. The columns are the segment's vectors in two f16 parts (x = hi + lo to 2^-22), scaled by a power of two that
// puts a vector's largest element near 2^14: with up to 4 slots both parts share an instruction's 8 columns, with more each
// part has its own and both add into the same sums. The parts lie in shared memory in the order in which lanes take them.
constexpr int kWarps = 16, kThreads = kWarps * 32;
constexpr int kStages = 3;                       // of a warp's ring; 2 where the vectors leave no room
constexpr int kChunk = 4;                        // blocks of a chunk
constexpr uint32_t kScalesAt = 2048, kStageBytes = 2304;  // a stage: 32 rows x 64 bytes of codes, 32 x 4 scales
constexpr int kMaxSlots = 512;
constexpr int kMaxCap = 8;
constexpr int kPartBlocks = 88;                  // most blocks of a part: 8 slots' fit beside the ring

struct ExpertParams {
    const uint8_t *qs0, *qs1;  // gate and up, or down twice
    const uint16_t *d0, *d1;
    const float* in;
    const unsigned* in_max;    // bits of the largest size in an input row
    float* out;                // [parts][slots][rows]
    unsigned* out_max;         // as in_max, of the outputs (gate and up)
    const int32_t* ids;
    int E, rows, blocks, parts, slots, per_in, cap, stages, scale_bytes;  // slot s reads input row s / per_in
    uint32_t ring_at, deposits_at, frags_at;
};

struct Tables {
    int ids[kMaxSlots], seg_e[kMaxSlots];
    uint16_t list[kMaxSlots], list_base[kMaxSlots], seg_at[kMaxSlots];
    uint8_t seg_n[kMaxSlots];
    int warp_segs[kWarps], warp_slots[kWarps];
    float back[2][kMaxCap];
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1,
                                    const float (&c)[4]) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}
// 16, 8 or 4 bytes global -> shared, zeros instead where `bytes` is 0.
template <int SIZE>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, uint32_t bytes) {
    if constexpr (SIZE == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(SIZE), "r"(bytes) : "memory");
}
__device__ __forceinline__ uint32_t bits_of(__half2 h) {
    uint32_t w;
    memcpy(&w, &h, 4);
    return w;
}
__device__ __forceinline__ __half2 half2_of(uint32_t w) {
    __half2 h;
    memcpy(&h, &w, 4);
    return h;
}
template <uint32_t MASK>
__device__ __forceinline__ __half2 masked_or(uint32_t w, uint32_t or_) {
    uint32_t x;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(x) : "r"(w), "n"(MASK), "r"(or_));
    return half2_of(x);
}
// The eight codes of a word (bytes 4t .. 4t + 3 of a block) as f16 pairs code - 8: elements (4t, 4t + 2), (4t + 16, 4t + 18),
// (4t + 1, 4t + 3), (4t + 17, 4t + 19). 1024 + q and 1024 + 16 q are exact in f16, and so are q - 8 and (..) / 16 - 72.
__device__ __forceinline__ void codes_of(uint32_t w, uint32_t k1024, uint32_t (&x)[4]) {
    const __half2 lo = __floats2half2_rn(-1032.f, -1032.f), hi = __floats2half2_rn(-72.f, -72.f),
                  six = __floats2half2_rn(0.0625f, 0.0625f);
    x[0] = bits_of(__hadd2(masked_or<0x000f000fu>(w, k1024), lo));
    x[1] = bits_of(__hfma2(masked_or<0x00f000f0u>(w, k1024), six, hi));
    w >>= 8;
    x[2] = bits_of(__hadd2(masked_or<0x000f000fu>(w, k1024), lo));
    x[3] = bits_of(__hfma2(masked_or<0x00f000f0u>(w, k1024), six, hi));
}

// The power of two that takes a vector whose largest size has the bits `m` to at most 2^15, as its exponent.
__device__ __forceinline__ int vector_exponent(unsigned m) { return m == 0u ? 0 : min(141 - (int)(m >> 23), 126); }

// A warp's chunks of one segment and part: the items [at, end) of (unit, chunk), counted from the CTA's first unit there.
struct Cursor {
    int v, at, end;    // v: segment * parts + part
    int unit, chunk;   // of `at`
    int chunks, block0, blocks;  // of the part
};

template <bool GateUp>
__global__ void __launch_bounds__(kThreads, 1) moe_expert_kernel(const ExpertParams p) {
    extern __shared__ __align__(128) uint8_t smem[];
    Tables& tab = *reinterpret_cast<Tables*>(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t base = smem_addr(smem), ring = base + p.ring_at + (uint32_t)(warp * p.stages) * kStageBytes, frags = base + p.frags_at;
    float* deposits = reinterpret_cast<float*>(smem + p.deposits_at);

    grid_dependency_wait();
    grid_launch_dependents();

    // Segments: the slots of an expert in their order, `cap` at a time, experts in the order of their first slots.
    for (int s = tid; s < p.slots; s += kThreads) tab.ids[s] = p.ids[s];
    __syncthreads();
    int segs = 0;
    {
        const int s = tid;
        const bool in = s < p.slots;
        const int e = in ? tab.ids[s] : -1;
        const bool valid = e >= 0 && e < p.E;
        int first = s, rank = 0, total = 0;
        if (valid) {
            for (int o = p.slots - 1; o >= 0; --o) {
                const bool same = tab.ids[o] == e;
                total += same;
                rank += same && o < s;
                if (same) first = o;
            }
        }
        const bool leads = valid && rank == 0;
        const int mine = leads ? (total + p.cap - 1) / p.cap : 0, slots = leads ? total : 0;
        int a = mine, b = slots;  // inclusive sums over the warp
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
            if (lane >= o) a += x, b += y;
        }
        if (lane == 31) tab.warp_segs[warp] = a, tab.warp_slots[warp] = b;
        __syncthreads();
        int seg = a - mine, at = b - slots;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) seg += tab.warp_segs[w], at += tab.warp_slots[w];
            segs += tab.warp_segs[w];
        }
        if (leads) {
            tab.list_base[s] = (uint16_t)at;
            for (int i = 0; i < mine; ++i) {
                tab.seg_e[seg + i] = e;
                tab.seg_at[seg + i] = (uint16_t)(at + i * p.cap);
                tab.seg_n[seg + i] = (uint8_t)min(p.cap, total - i * p.cap);
            }
        }
        __syncthreads();
        if (valid) tab.list[tab.list_base[first] + rank] = (uint16_t)s;
        __syncthreads();
    }

    const int units = GateUp ? p.rows / 16 : (p.rows + 31) / 32;
    const long long all = (long long)segs * p.parts * units;
    const long long u_lo = all * blockIdx.x / gridDim.x, u_hi = all * (blockIdx.x + 1) / gridDim.x;
    if (u_lo >= u_hi) return;
    const int v_lo = (int)(u_lo / units), v_hi = (int)((u_hi - 1) / units);

    auto enter = [&](Cursor& c, int v) {
        const int ua = v == v_lo ? (int)(u_lo - (long long)v * units) : 0;
        const int ub = v == v_hi ? (int)(u_hi - (long long)v * units) : units;
        const int part = v % p.parts;
        const int per = ((p.blocks + p.parts - 1) / p.parts + kChunk - 1) / kChunk * kChunk;  // blocks of a part
        c.v = v;
        c.block0 = part * per;
        c.blocks = min(per, p.blocks - c.block0);
        c.chunks = (c.blocks + kChunk - 1) / kChunk;
        const int items = (ub - ua) * c.chunks;
        c.at = (int)((unsigned)items * (unsigned)warp / kWarps);
        c.end = (int)((unsigned)items * (unsigned)(warp + 1) / kWarps);
        const int unit = c.at / c.chunks;
        c.chunk = c.at - unit * c.chunks;
        c.unit = ua + unit;
    };

    // ---- the ring: stages are filled in the order in which they are used, across segments
    Cursor f = {};
    uint32_t fill_at = 0, use_at = 0;  // stages of the ring, as offsets
    const uint32_t ring_bytes = (uint32_t)p.stages * kStageBytes;
    const char *src0 = nullptr, *src1 = nullptr, *src_d = nullptr;  // of this lane, at the cursor's chunk 0
    bool row_a = true, row_b = true, row_c = true, row_d = true, row_s = true;
    auto aim = [&]() {  // a new unit
        const int e = tab.seg_e[f.v / p.parts];
        const int row = GateUp ? f.unit * 16 : f.unit * 32;
        const long long first = (long long)e * p.rows + row;
        const int r = lane >> 2, c = lane & 3;
        const long long second = GateUp ? first : first + 16;
        src0 = reinterpret_cast<const char*>(p.qs0) + ((first + r) * p.blocks + f.block0 + c) * 16;
        src1 = reinterpret_cast<const char*>(p.qs1) + ((second + r) * p.blocks + f.block0 + c) * 16;
        src_d = reinterpret_cast<const char*>(lane < 16 ? p.d0 : p.d1) +
                (((lane < 16 ? first : second) + (lane & 15)) * p.blocks + f.block0) * 2;
        if (!GateUp) {
            const int left = p.rows - row;
            row_a = r < left, row_b = r + 8 < left, row_c = r + 16 < left, row_d = r + 24 < left;
            row_s = (lane < 16 ? 0 : 16) + (lane & 15) < left;
        }
    };
    enter(f, v_lo);
    auto settle = [&]() {  // to the next item, if there is one
        while (f.at >= f.end && f.v < v_hi) enter(f, f.v + 1);
        if (f.at < f.end) aim();
    };
    settle();
    auto fill = [&]() {
        if (f.at < f.end) {
            const uint32_t dst = ring + fill_at;
            const int r = lane >> 2, c = lane & 3, left = f.blocks - f.chunk * kChunk;
            const uint32_t to = dst + r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
            const long long o = (long long)f.chunk * (kChunk * 16), eight = (long long)p.blocks * 128;
            const bool in = c < left;
            auto copy = [&](uint32_t at, const char* src, bool there) {
                copy_async<16>(at, there && in ? src : reinterpret_cast<const char*>(p.qs0), there && in ? 16u : 0u);
            };
            copy(to, src0 + o, row_a);
            copy(to + 512, src0 + o + eight, row_b);
            copy(to + 1024, src1 + o, row_c);
            copy(to + 1536, src1 + o + eight, row_d);
            const uint32_t to_d = dst + kScalesAt + lane * 8;
            const char* sd = src_d + f.chunk * (kChunk * 2);
            if (p.scale_bytes == 8) {
                copy_async<8>(to_d, row_s ? sd : reinterpret_cast<const char*>(p.qs0), row_s ? 8u : 0u);
            } else if (p.scale_bytes == 4) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const bool there = row_s && 2 * i < left;
                    copy_async<4>(to_d + 4 * i, there ? sd + 4 * i : reinterpret_cast<const char*>(p.qs0), there ? 4u : 0u);
                }
            } else {
                uint32_t h[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    h[i] = row_s && i < left ? (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(sd) + i) : 0u;
                asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(to_d), "r"(h[0] | h[1] << 16), "r"(h[2] | h[3] << 16)
                             : "memory");
            }
            ++f.at;
            if (++f.chunk == f.chunks) {
                f.chunk = 0;
                ++f.unit;
                if (f.at < f.end) aim();
            }
            if (f.at >= f.end) settle();
        }
        fill_at = fill_at + kStageBytes == ring_bytes ? 0u : fill_at + kStageBytes;
        cp_async_commit();
    };
    for (int i = 0; i < p.stages - 1; ++i) fill();

    uint32_t k1024;
    asm volatile("mov.b32 %0, 0x64006400;" : "=r"(k1024));
    const int g = lane >> 2, t4 = lane & 3;
    // ldmatrix: lane l gives the address of row l % 8 of matrix l / 8: rows 0-7 and 8-15 of a block, then of the next one
    const int lm_row = (lane & 7) + (lane & 8), lm_half = lane >> 4;

    Cursor c;
    for (int v = v_lo; v <= v_hi; ++v) {
        enter(c, v);
        const int seg = v / p.parts, n = tab.seg_n[seg], at = tab.seg_at[seg];
        const int np = n <= 1 ? 1 : n <= 2 ? 2 : n <= 4 ? 4 : 8;  // columns kept of each part
        const uint32_t per_block = (uint32_t)np * 128u;
        float* back = tab.back[v & 1];

        // ---- the segment's vectors, in two parts
        for (int j = 0; j < n; ++j) {
            const int row = tab.list[at + j] / p.per_in;
            const unsigned m = p.in_max[row];
            const int k = vector_exponent(m);
            const float scale = pow2i(k);
            if (tid == j) back[j] = m >= 0x7f800000u ? qnan() : pow2i(-k);
            const float* x = p.in + (long long)row * (p.blocks * 32) + (long long)c.block0 * 32;
            for (int i = tid; i < c.chunks * kChunk * 4; i += kThreads) {
                const int b = i >> 2, t = i & 3;
                float4 lo4 = make_float4(0.f, 0.f, 0.f, 0.f), hi4 = lo4;
                if (b < c.blocks) {
                    lo4 = *reinterpret_cast<const float4*>(x + b * 32 + t * 4);
                    hi4 = *reinterpret_cast<const float4*>(x + b * 32 + 16 + t * 4);
                }
                const float pair[4][2] = {{lo4.x, lo4.z}, {hi4.x, hi4.z}, {lo4.y, lo4.w}, {hi4.y, hi4.w}};
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float a = pair[q][0] * scale, b2 = pair[q][1] * scale;
                    const __half2 h = __floats2half2_rn(a, b2);
                    const float2 back2 = __half22float2(h);
                    hi[q] = bits_of(h);
                    lo[q] = bits_of(__floats2half2_rn(a - back2.x, b2 - back2.y));
                }
                const uint32_t to = frags + b * per_block + j * 64 + t * 16;
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(hi[0]), "r"(hi[1]), "r"(hi[2]), "r"(hi[3])
                             : "memory");
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to + np * 64), "r"(lo[0]), "r"(lo[1]), "r"(lo[2]),
                             "r"(lo[3])
                             : "memory");
            }
        }
        __syncthreads();

        // ---- products
        float acc[2][4];
        auto clear = [&]() {
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[m][i] = 0.f;
        };
        // A unit's sums leave: joined over the parts of the vectors, scaled back, and for gate and up as silu(g) * u.
        auto finish = [&](int unit) {
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (np <= 4) acc[m][i] += __shfl_xor_sync(0xffffffffu, acc[m][i], 2);
            const int part = v % p.parts;
            unsigned big[2] = {0u, 0u};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = 2 * t4 + (i & 1), r = g + (i >> 1) * 8;
                if (j >= n || (np <= 4 && t4 >= 2)) continue;
                const float b = back[j];
                const long long slot = tab.list[at + j];
                if (GateUp) {
                    const float h = silu(acc[0][i] * b) * (acc[1][i] * b);
                    p.out[slot * p.rows + unit * 16 + r] = h;
                    big[i & 1] = max(big[i & 1], __float_as_uint(h) & 0x7fffffffu);
                } else {
                    float* out = p.out + ((long long)part * p.slots + slot) * p.rows + unit * 32;
#pragma unroll
                    for (int m = 0; m < 2; ++m)
                        if (unit * 32 + m * 16 + r < p.rows) out[m * 16 + r] = acc[m][i] * b;
                }
            }
            if (GateUp) {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
#pragma unroll
                    for (int o = 4; o <= 16; o <<= 1) big[q] = max(big[q], __shfl_xor_sync(0xffffffffu, big[q], o));
                    const int j = 2 * t4 + q;
                    if (g == 0 && j < n && !(np <= 4 && t4 >= 2)) atomicMax(p.out_max + tab.list[at + j], big[q]);
                }
            }
            clear();
        };
        auto products = [&](auto wide, uint32_t stage, uint32_t fr) {
            constexpr bool Wide = decltype(wide)::value;
            const uint32_t part_bytes = (uint32_t)np * 64u;
            const uint32_t mine = fr + (Wide ? (uint32_t)g * 64u : (uint32_t)(g >> 2) * part_bytes + (uint32_t)(g & 3) * 64u) + t4 * 16;
            const bool column = Wide || (g & 3) < np;
            float2 d[2][2][2];  // scales of rows g and g + 8, blocks 0, 1 and 2, 3
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t a, b;
                    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                                 : "=r"(a), "=r"(b)
                                 : "r"(stage + kScalesAt + (m * 16 + h * 8 + g) * 8));
                    d[m][h][0] = __half22float2(half2_of(a));
                    d[m][h][1] = __half22float2(half2_of(b));
                }
#pragma unroll
            for (int pair = 0; pair < 2; ++pair) {
                uint32_t w[2][4];
#pragma unroll
                for (int m = 0; m < 2; ++m)
                    ldsm4(stage + m * 1024 + lm_row * 64 + (((2 * pair + lm_half) ^ ((lm_row >> 1) & 3)) << 4), w[m]);
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const uint32_t from = mine + (2 * pair + b) * per_block;
                    uint4 h = make_uint4(0u, 0u, 0u, 0u), l = h;
                    if (column) h = lds128(from);
                    if (Wide) l = lds128(from + part_bytes);
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        uint32_t ra[4], rb[4];
                        codes_of(w[m][2 * b], k1024, ra);
                        codes_of(w[m][2 * b + 1], k1024, rb);
                        const float zero[4] = {0.f, 0.f, 0.f, 0.f};
                        float s[4];
                        mma(s, ra[0], rb[0], ra[1], rb[1], h.x, h.y, zero);
                        mma(s, ra[2], rb[2], ra[3], rb[3], h.z, h.w, s);
                        if (Wide) {
                            mma(s, ra[0], rb[0], ra[1], rb[1], l.x, l.y, s);
                            mma(s, ra[2], rb[2], ra[3], rb[3], l.z, l.w, s);
                        }
                        const float da = b ? d[m][0][pair].y : d[m][0][pair].x, db = b ? d[m][1][pair].y : d[m][1][pair].x;
                        acc[m][0] = fmaf(da, s[0], acc[m][0]);
                        acc[m][1] = fmaf(da, s[1], acc[m][1]);
                        acc[m][2] = fmaf(db, s[2], acc[m][2]);
                        acc[m][3] = fmaf(db, s[3], acc[m][3]);
                    }
                }
            }
        };
        auto deposit = [&]() {
#pragma unroll
            for (int i = 0; i < 8; ++i) deposits[(warp * 8 + i) * 32 + lane] = acc[i >> 2][i & 3];
            clear();
        };
        clear();
        const int first_item = c.at;
        bool head = c.chunk != 0;  // the unit was begun by a warp before this one, which joins it
        while (c.at < c.end) {
            if (p.stages == kStages) cp_async_wait<kStages - 2>();
            else cp_async_wait<0>();
            __syncwarp();
            fill();
            const uint32_t stage = ring + use_at;
            const uint32_t fr = frags + (uint32_t)(c.chunk * kChunk) * per_block;
            if (np == 8) products(std::integral_constant<bool, true>(), stage, fr);
            else products(std::integral_constant<bool, false>(), stage, fr);
            use_at = use_at + kStageBytes == ring_bytes ? 0u : use_at + kStageBytes;
            ++c.at;
            if (++c.chunk == c.chunks) {
                if (head) deposit();
                else finish(c.unit);
                head = false;
                c.chunk = 0;
                ++c.unit;
            }
        }
        if (first_item < c.end && head) deposit();
        const bool tail = first_item < c.end && !head && c.chunk != 0;  // begun here, not done
        __syncthreads();
        if (tail) {
            const int unit_end = c.at - c.chunk + c.chunks;  // as items
            for (int w = warp + 1, end = c.end; w < kWarps && end < unit_end; ++w) {
                const unsigned items = (unsigned)((v == v_hi ? (int)(u_hi - (long long)v * units) : units) -
                                                  (v == v_lo ? (int)(u_lo - (long long)v * units) : 0)) * (unsigned)c.chunks;
                const int to = (int)(items * (unsigned)(w + 1) / kWarps);
                if (to == end) continue;
                end = to;
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[i >> 2][i & 3] += deposits[(w * 8 + i) * 32 + lane];
            }
            finish(c.unit);
        }
    }
}

// The launch shape of one matrix (or gate and up): parts, slots of a segment, shared memory.
struct ExpertPlan {
    int parts, cap, stages;
    uint32_t ring_at, deposits_at, frags_at, smem;
};
int moe_parts(int blocks) { return (blocks + kPartBlocks - 1) / kPartBlocks; }
ExpertPlan plan_experts(int blocks, bool cut, int max_smem) {
    ExpertPlan l;
    l.parts = cut ? moe_parts(blocks) : 1;
    const int per = ((blocks + l.parts - 1) / l.parts + kChunk - 1) / kChunk * kChunk;
    l.cap = 0;
    for (int stages = kStages; stages >= 2; --stages)
        for (int cap = kMaxCap; cap >= 1; cap /= 2) {
            l.cap = cap, l.stages = stages;
            l.ring_at = (sizeof(Tables) + 127) / 128 * 128;
            l.deposits_at = l.ring_at + (uint32_t)(kWarps * stages) * kStageBytes;
            l.frags_at = l.deposits_at + kWarps * 8 * 32 * 4;
            l.smem = l.frags_at + (uint32_t)per * cap * 128u;
            if (l.smem <= (uint32_t)max_smem) return l;
        }
    l.cap = 0;
    return l;
}

template <bool GateUp>
cudaError_t launch_experts(ExpertParams p, const DeviceInfo& di, bool overlap, cudaStream_t s) {
    const ExpertPlan l = plan_experts(p.blocks, !GateUp, di.max_smem_optin);
    if (l.cap == 0) return cudaErrorNotSupported;
    p.parts = l.parts, p.cap = l.cap, p.stages = l.stages;
    p.ring_at = l.ring_at, p.deposits_at = l.deposits_at, p.frags_at = l.frags_at;
    const uintptr_t d = reinterpret_cast<uintptr_t>(p.d0) | reinterpret_cast<uintptr_t>(p.d1);
    p.scale_bytes = p.blocks % 4 == 0 && d % 8 == 0 ? 8 : p.blocks % 2 == 0 && d % 4 == 0 ? 4 : 2;
    auto kern = moe_expert_kernel<GateUp>;
    static std::once_flag once[64];
    cudaError_t e = cudaSuccess;
    std::call_once(once[di.device & 63],
                   [&] { e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, di.max_smem_optin); });
    if (e != cudaSuccess) return e;
    return launch_grid(kern, dim3((unsigned)di.sm_count), dim3(kThreads), l.smem, s, overlap, p);
}

// The largest size in each row of [rows][cols], as its bits.
__global__ void __launch_bounds__(256) moe_max_kernel(const float* x, unsigned* out, int cols) {
    grid_dependency_wait();
    grid_launch_dependents();
    __shared__ unsigned part[8];
    const float* row = x + (long long)blockIdx.x * cols;
    unsigned m = 0u;
    for (int k = threadIdx.x * 4; k < cols; k += 1024) {
        float v[4];
        load_floats(row + k, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int i = 1; i < 8; ++i) m = max(m, part[i]);
        out[blockIdx.x] = m;
    }
}

struct JoinParams {
    void* out;
    const void* residual;
    const float *z, *weights;
    const int32_t* ids;
    int topk, E, rows, parts, slots;
    long long out_stride, residual_stride;
    int32_t* status;
    unsigned* fault;
};

// out[t] = residual[t] + sum_s weights[t][s] * z[t][s], in the order of the slots.
template <typename T>
__global__ void __launch_bounds__(128) moe_join_kernel(const JoinParams p) {
    const int t = blockIdx.y, n = (blockIdx.x * 128 + threadIdx.x) * 4;
    grid_dependency_wait();
    grid_launch_dependents();
    if (n >= p.rows) return;
    float v[4] = {};
    if (p.residual) {
        const T* r = static_cast<const T*>(p.residual) + t * p.residual_stride + n;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = (float)r[j];
    }
    bool bad = false;
    for (int s = 0; s < p.topk; ++s) {
        const long long slot = (long long)t * p.topk + s;
        const int e = p.ids[slot];
        if (e < 0 || e >= p.E) {
            bad = true;
            continue;
        }
        const float w = p.weights[slot];
        float z[4];
        load_floats(p.z + slot * p.rows + n, z);
        for (int q = 1; q < p.parts; ++q) {
            float more[4];
            load_floats(p.z + ((long long)q * p.slots + slot) * p.rows + n, more);
#pragma unroll
            for (int j = 0; j < 4; ++j) z[j] += more[j];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = fmaf(w, z[j], v[j]);
    }
    if (bad) {  // an expert that is not there: the token's row is NaN
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = qnan();
        if (n == 0) {
            if (p.status) *p.status = (int32_t)kFaultBadExpert;
            atomicOr(p.fault, (unsigned)kFaultBadExpert);
        }
    }
    T* out = static_cast<T*>(p.out) + t * p.out_stride + n;
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(out) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
        *reinterpret_cast<uint2*>(out) = make_uint2(pack2(v[0], v[1], T()), pack2(v[2], v[3], T()));
    }
}

cudaError_t launch_join(const JoinParams& p, int T, int dtype, bool overlap, cudaStream_t s) {
    return with_dtype(dtype, [&](auto tag) {
        const dim3 grid((unsigned)((p.rows + 511) / 512), (unsigned)T);
        return launch_grid(moe_join_kernel<decltype(tag)>, grid, dim3(128), 0, s, overlap, p);
    });
}

struct DownSpace {
    float* z;
    unsigned* h_max;
    DownSpace(Carve& c, int slots, int rows, int cols)
        : z(c.take<float>((size_t)moe_parts(cols / 32) * slots * rows)), h_max(c.take<unsigned>(slots)) {}
};

cudaError_t launch_down(const DownSpace& w, const float* h, const uint8_t* qs, const uint16_t* d, const int32_t* ids, int slots,
                        int E, int rows, int cols, const DeviceInfo& di, cudaStream_t s) {
    ExpertParams p = {};
    p.qs0 = p.qs1 = qs, p.d0 = p.d1 = d;
    p.in = h, p.in_max = w.h_max, p.out = w.z, p.ids = ids;
    p.E = E, p.rows = rows, p.blocks = cols / 32, p.slots = slots, p.per_in = 1;
    return launch_experts<false>(p, di, true, s);
}

}  // namespace

size_t moe_down_workspace_bytes(int T, int topk, int rows, int cols) {
    Carve c{nullptr};
    DownSpace(c, T * topk, rows, cols);
    return c.at;
}

cudaError_t launch_moe_down(const MoeDownArgs& a, int dtype, void* workspace, const DeviceInfo& di, cudaStream_t s) {
    Carve c{static_cast<uint8_t*>(workspace)};
    const int slots = a.T * a.topk;
    const DownSpace w(c, slots, a.rows, a.cols);
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)slots), cfg.blockDim = dim3(256), cfg.stream = s;
    cfg.attrs = attr, cfg.numAttrs = launch_overlap() ? 1 : 0;
    cudaError_t e = cudaLaunchKernelEx(&cfg, moe_max_kernel, a.h, w.h_max, a.cols);
    if (e != cudaSuccess) return e;
    if ((e = launch_down(w, a.h, a.qs, a.d, a.ids, slots, a.E, a.rows, a.cols, di, s)) != cudaSuccess) return e;
    const JoinParams join = {a.out, a.residual, w.z, a.weights, a.ids, a.topk, a.E, a.rows, moe_parts(a.cols / 32), slots,
                             a.out_stride, a.residual_stride, a.status, a.fault};
    return launch_join(join, a.T, dtype, true, s);
}

struct LayerSpace {
    float *xn, *h, *weights;
    int32_t* ids;
    unsigned* x_max;
    DownSpace down;
    LayerSpace(Carve& c, int T, int topk, int N, int K)
        : xn(c.take<float>((size_t)T * K)), h(c.take<float>((size_t)T * topk * N)), weights(c.take<float>(T * topk)),
          ids(c.take<int32_t>(T * topk)), x_max(c.take<unsigned>(T)), down(c, T * topk, K, N) {}
};

size_t moe_layer_workspace_bytes(int T, int topk, int N, int K) {
    Carve c{nullptr};
    LayerSpace(c, T, topk, N, K);
    return c.at;
}

cudaError_t launch_moe_layer(const MoeLayerArgs& a, int dtype, void* workspace, const DeviceInfo& di, cudaStream_t s) {
    Carve c{static_cast<uint8_t*>(workspace)};
    const int slots = a.T * a.topk, N = a.w.N, K = a.w.K, E = a.w.E;
    const LayerSpace w(c, a.T, a.topk, N, K);
    int32_t* ids = a.ids ? a.ids : w.ids;
    float* weights = a.weights ? a.weights : w.weights;
    const PrepParams prep = {a.x, a.gamma, w.xn, w.x_max, w.down.h_max, a.eps, K, a.topk, a.x_stride};
    cudaError_t e = with_dtype(dtype, [&](auto tag) {
        return launch_grid(moe_prep_kernel<decltype(tag)>, dim3((unsigned)a.T), dim3(256), 0, s, launch_overlap(), prep);
    });
    if (e != cudaSuccess) return e;
    if ((e = launch_moe_router(ids, weights, nullptr, a.w.router_qs, a.w.router_d, w.xn, a.T, E, K, a.topk, a.normalize != 0,
                               s)) != cudaSuccess)
        return e;
    ExpertParams up = {};
    up.qs0 = a.w.gate_qs, up.qs1 = a.w.up_qs, up.d0 = a.w.gate_d, up.d1 = a.w.up_d;
    up.in = w.xn, up.in_max = w.x_max, up.out = w.h, up.out_max = w.down.h_max, up.ids = ids;
    up.E = E, up.rows = N, up.blocks = K / 32, up.slots = slots, up.per_in = a.topk;
    if ((e = launch_experts<true>(up, di, true, s)) != cudaSuccess) return e;
    if ((e = launch_down(w.down, w.h, a.w.down_qs, a.w.down_d, ids, slots, E, K, N, di, s)) != cudaSuccess) return e;
    const JoinParams join = {a.out, a.residual, w.down.z, weights, ids, a.topk, E, K, moe_parts(N / 32), slots, a.out_stride,
                             a.residual_stride, nullptr, a.fault};
    return launch_join(join, a.T, dtype, true, s);
}

}  // namespace q4
