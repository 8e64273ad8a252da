// The experts' products of a mixture of experts over planar Q4: gate and up with SwiGLU, and down.
//
// Work. Slots that go to the same expert form a segment of up to `cap` (8, of vectors in one part 16, or fewer where the
// vectors are long); long inputs of the down projection are cut into parts whose sums the join adds. A segment's rows are
// units of 32: 16 of gate and the same 16 of up, or 32 of down. All units lie on one line, weighted by what they cost and cut
// into pieces, one for each CTA, and a piece's chunks of 4 blocks (128 columns) are cut into equal pieces for its warps. So
// every weight is read once a segment, and a warp adds a unit's chunks in registers; a unit cut between warps is joined through
// shared memory in the order of its chunks, so that the same call gives the same bits.
//
// Products run on m16n8k16 matrix instructions with the weights as rows: ldmatrix brings a block's word to each lane, eight
// codes become eight exact f16 values code - 8 with nine instructions, and a block's fp32 sums are multiplied by the block's
// scale in fp32. The columns are the segment's vectors in f16, scaled by a power of two that puts a vector's largest element
// near 2^14. A vector is held in two parts (x = hi + lo to 2^-22): with up to 4 slots both parts share an instruction's 8
// columns, with more each part has its own and both add into the same sums. A bf16 x that goes into gate and up as it is has
// 8 bits, which one part holds exactly down to 2^-32 of the vector's largest element and to 2^-39 of it below: twice the slots
// in an instruction (64 tokens over 64 experts of 1408 x 2048: 117 us in two parts, 105 us in one). What is fp32 (h, and x
// behind its norm) takes two parts whatever the layer's type: one part's 11 bits would show in the bf16 outputs, and h is the
// caller's. The parts lie in shared memory in the order in which lanes take them. tcgen05 is not used: its operands would have to
// be decoded into f16 tiles in shared memory first, which costs the instructions that bind here and the writes besides, and at
// these few columns the matrix unit is a sixth busy. For segments of 32 slots and more, of which one decode could serve many
// columns, it was not tried.
//
// Copies. Each warp streams its chunks by cp.async through a ring of three (or two) stages of its own, across units and segments
// (16-byte chunks XOR-swizzled so that ldmatrix is free of bank conflicts); the scales of two chunks travel together. Four
// stages: 8 tokens 61.6 us instead of 59.8.
//
// What bounds it (8 tokens, 42 experts, 137 MB of gate and up in 35 us, 25 us of them at 5.4 TB/s): between the starts and the
// ends, instructions. A chunk costs a warp about 360, of which 220 are the products themselves (144 decode, 16 matrix, 48 scale),
// where the copy rate would leave a scheduler about 400 issue slots. So loops are kept straight and branches uniform (69 -> 62
// us), and there are fewer warps than would fit, with more registers each: 6 and 6 in two CTAs an SM, or 12 in one (16: 8 tokens
// 60.5 us, a down projection of 14336 columns 60.5 instead of 57.4 us; 10 or 14: slower). Some 6 us go by from the kernel's
// inputs to the first products (ids, segments, the first copies and vectors) and about 4 us at its end, where CTAs that share
// an SM finish at different times; down hides most of its start behind the kernel before it.
#pragma once

#include <mutex>

#include "block.h"
#include "kv_common.cuh"

namespace q4 {

namespace {

constexpr int kChunk = 4;                        // blocks of a chunk
constexpr uint32_t kStageBytes = 2048;           // a stage: 32 rows x 64 bytes of codes
constexpr uint32_t kGroupBytes = 512;            // 32 rows x 8 scales: those of two chunks, in a ring of their own
constexpr uint32_t kSlotBytes = kStageBytes + kGroupBytes;
constexpr int kMaxSlots = 512;
constexpr int kStageLoads = 2;                   // of a thread that are in flight together; with 4, 8 tokens take 64 us, not 62
constexpr int kMaxCap = 16;

struct Tables {
    int seg_e[kMaxSlots];
    uint16_t list[kMaxSlots], seg_at[kMaxSlots];
    uint8_t seg_n[kMaxSlots];
    int8_t exponent[kMaxSlots];  // of a slot's vector: see vector_exponent; kNotFinite
    int warp_sums[16];
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
                  sixteenth = __floats2half2_rn(0.0625f, 0.0625f);
    x[0] = bits_of(__hadd2(masked_or<0x000f000fu>(w, k1024), lo));
    x[1] = bits_of(__hfma2(masked_or<0x00f000f0u>(w, k1024), sixteenth, hi));
    w >>= 8;
    x[2] = bits_of(__hadd2(masked_or<0x000f000fu>(w, k1024), lo));
    x[3] = bits_of(__hfma2(masked_or<0x00f000f0u>(w, k1024), sixteenth, hi));
}

// The power of two that takes a vector whose largest size has the bits `m` to at most 2^15, as its exponent.
constexpr int kNotFinite = 127;
__device__ __forceinline__ int vector_exponent(unsigned m) {
    return m == 0u ? 0 : m >= 0x7f800000u ? kNotFinite : min(141 - (int)(m >> 23), 126);
}

// PER: slots of a thread. Scales: bytes of a row's scales that one copy may move, 16 or 8 (rows of whole chunks then), or 0: see
// scale_bytes. kStages: of a warp's ring. What every warp works out for itself is kept short: at the start of a kernel it costs all warps issue slots.
template <bool GateUp, int Parts, int W, int PER, int Scales, int kStages>
__global__ void __launch_bounds__(W * 32, W == 6 ? 2 : 1) moe_expert_kernel(const ExpertParams p) {
    constexpr int kThreads = W * 32;
    constexpr int kNarrow = Parts == 2 ? 4 : 8;    // slots in one instruction's columns
    constexpr int kTiles = Parts == 2 ? 1 : 2;     // sums of 8 slots that a warp keeps
    // Cost of a unit of a segment whose columns fill one instruction, or two: 64 fp32 tokens over 64 experts take 119 us with
    // 4 : 5, 127 us with 4 : 6 and 139 us with 4 : 7; with x in one part 107 us with 4 : 5 and 105 us with 4 : 6.
    constexpr unsigned kNarrowCost = 4, kWideCost = Parts == 1 ? 6 : 5;
    constexpr bool kRoom = W == 6 && PER == 1;     // of two CTAs an SM: see launch_experts_of
    extern __shared__ __align__(128) uint8_t smem[];
    Tables& tab = *reinterpret_cast<Tables*>(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const uint32_t base = smem_addr(smem), ring = base + p.ring_at + (uint32_t)(warp * kStages) * kSlotBytes, frags = base + p.frags_at;
    float* deposits = reinterpret_cast<float*>(smem + p.deposits_at);

    // Segments: the slots of an expert in their order, `cap` at a time, experts in the order of their first slots, those with
    // more columns than one instruction's behind the others. A hash table of experts, each with the bits of its slots, lies where
    // the ring and the vectors lie later.
    const int words = (p.slots + 31) / 32, entries = 1 << p.table_bits;
    uint16_t* const list_base = reinterpret_cast<uint16_t*>(smem + p.ring_at);
    int* const keys = reinterpret_cast<int*>(list_base + kMaxSlots);
    uint32_t* const masks = reinterpret_cast<uint32_t*>(keys + entries);
    for (int i = tid; i < entries * (1 + words); i += kThreads) keys[i] = i < entries ? -1 : 0;
    __syncthreads();
    // The ids and the weights were written before the kernel before this one began (down: its producer waits for them
    // itself before it lets this kernel start), so everything up to the first vectors runs while it ends.
    if (GateUp) grid_dependency_wait();
    grid_launch_dependents();
    int narrows = 0, wides = 0;
    {
        int e[PER], entry[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int s = tid * PER + i;
            e[i] = s < p.slots ? __ldcg(p.ids + s) : -1;
            if (GateUp && s < p.slots) tab.exponent[s] = (int8_t)vector_exponent(__ldcg(p.in_max + (unsigned)s / (unsigned)p.per_in));
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int s = tid * PER + i;
            entry[i] = -1;
            if (e[i] >= 0 && e[i] < p.E) {
                int at = (int)(((unsigned)e[i] * 2654435769u) >> (32 - p.table_bits));
                for (;; at = (at + 1) & (entries - 1)) {  // at most half of the entries are ever used
                    const int was = atomicCAS(keys + at, -1, e[i]);
                    if (was == -1 || was == e[i]) break;
                }
                atomicOr(masks + at * words + (s >> 5), 1u << (s & 31));
                entry[i] = at;
            }
        }
        __syncthreads();
        int first[PER], rank[PER], total[PER], narrow = 0, wide = 0, slots = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int s = tid * PER + i;
            first[i] = s, rank[i] = 0, total[i] = 0;
            if (entry[i] >= 0) {
                for (int w = words - 1; w >= 0; --w) {
                    const uint32_t m = masks[entry[i] * words + w];
                    total[i] += __popc(m);
                    rank[i] += w < s >> 5 ? __popc(m) : w == s >> 5 ? __popc(m & ((1u << (s & 31)) - 1u)) : 0;
                    if (m) first[i] = w * 32 + __ffs(m) - 1;
                }
                if (rank[i] == 0) {
                    const int full = total[i] / p.cap, more = total[i] - full * p.cap;
                    wide += (p.cap > kNarrow ? full : 0) + (more > kNarrow);
                    narrow += (p.cap > kNarrow ? 0 : full) + (more > 0 && more <= kNarrow);
                    slots += total[i];
                }
            }
        }
        const int mine = narrow << 20 | wide << 10 | slots;  // sums up to 512 each
        int both = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, both, o);
            if (lane >= o) both += x;
        }
        if (lane == 31) tab.warp_sums[warp] = both;
        __syncthreads();
        int before = both - mine, sum = 0;
#pragma unroll 4
        for (int w = 0; w < W; ++w) {
            if (w < warp) before += tab.warp_sums[w];
            sum += tab.warp_sums[w];
        }
        narrows = sum >> 20, wides = sum >> 10 & 1023;
        int seg_narrow = before >> 20, seg_wide = narrows + (before >> 10 & 1023), at = before & 1023;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (total[i] == 0 || rank[i] != 0) continue;
            list_base[tid * PER + i] = (uint16_t)at;
#pragma unroll 1
            for (int o = 0; o < total[i]; o += p.cap) {
                const int count = min(p.cap, total[i] - o), seg = count > kNarrow ? seg_wide++ : seg_narrow++;
                tab.seg_e[seg] = e[i];
                tab.seg_at[seg] = (uint16_t)(at + o);
                tab.seg_n[seg] = (uint8_t)count;
            }
            at += total[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (total[i] != 0) tab.list[list_base[first[i]] + rank[i]] = (uint16_t)(tid * PER + i);
        __syncthreads();
    }

    // The CTA's piece of the line of units. What is the same in a warp is passed through a shuffle, so that branches on it
    // need no reconvergence.
    const unsigned per_segment = (unsigned)(p.parts * p.units);
    const unsigned narrow_units = (unsigned)__shfl_sync(0xffffffffu, narrows, 0) * per_segment;
    const unsigned cost_narrow = narrow_units * kNarrowCost;
    const unsigned cost = cost_narrow + (unsigned)__shfl_sync(0xffffffffu, wides, 0) * per_segment * kWideCost;
    const unsigned quotient = cost / gridDim.x, rest = cost - quotient * gridDim.x;
    auto cut = [&](unsigned i) {  // the first unit of piece i
        const unsigned at = quotient * i + rest * i / gridDim.x;
        return at <= cost_narrow ? at / kNarrowCost : narrow_units + (at - cost_narrow) / kWideCost;
    };
    const unsigned u_lo = cut(blockIdx.x), u_hi = cut(blockIdx.x + 1);
    if (u_lo >= u_hi) {
        if (!GateUp) grid_dependency_wait();
        return;
    }
    const unsigned units = (unsigned)p.units, v_lo = u_lo / units, v_hi = (u_hi - 1) / units;  // v: segment * parts + part
    auto first_unit = [&](unsigned v) { return v == v_lo ? u_lo - v * units : 0u; };
    auto unit_count = [&](unsigned v) { return (v == v_hi ? u_hi - v * units : units) - first_unit(v); };
    auto segment_of = [&](unsigned v) { return GateUp ? v : v / (unsigned)p.parts; };
    auto part_of = [&](unsigned v) { return GateUp ? 0u : v % (unsigned)p.parts; };
    // A warp's chunks of one segment and part: items of (unit, chunk), counted from the CTA's first unit there.
    struct Piece {
        unsigned at, end, chunks;
        int unit, chunk, block0, blocks;  // unit and chunk of `at`
    };
    auto piece_of = [&](unsigned v) {
        Piece c;
        c.block0 = (int)part_of(v) * p.part_blocks;
        c.blocks = min(p.part_blocks, p.blocks - c.block0);
        c.chunks = (unsigned)(c.blocks + kChunk - 1) / kChunk;
        const unsigned items = unit_count(v) * c.chunks;
        c.at = items * (unsigned)warp / W, c.end = items * (unsigned)(warp + 1) / W;
        const unsigned unit = c.at / c.chunks;
        c.chunk = c.at == c.end ? 0 : (int)(c.at - unit * c.chunks);
        c.unit = (int)(first_unit(v) + unit);
        return c;
    };

    // ---- the ring: stages are filled in the order in which they are used, across segments
    constexpr uint32_t kRing = kStages * kStageBytes, kGroups = kStages * kGroupBytes;
    constexpr int kRows = GateUp ? 16 : 32;  // of one matrix in a unit
    unsigned f_v = v_lo, f_left = 0;         // items left of the piece
    int f_chunk = 0, f_chunks = 0, f_blocks = 0;  // the next item's chunk
    uint32_t fill_at = 0, group_fill = 0;    // offsets in the two rings
    bool group = true;                       // the next item needs the scales of its two chunks
    const int r4 = lane >> 2, c4 = lane & 3;
    const uint32_t to_codes = ring + r4 * 64 + ((c4 ^ ((r4 >> 1) & 3)) << 4), to_scales = ring + kRing + lane * 16;
    const long long row_bytes = (long long)p.blocks * 16;
    const char *src0 = nullptr, *src1 = nullptr, *src_d = nullptr;  // of this lane, of the next item
    long long code_step = 0, scale_step = 0;  // from the last chunk of a unit to the next unit
    int rows_left = 32;                       // of the unit, all of them for gate and up
    auto next_piece = [&]() {  // f_v: the first that is not begun
        for (; f_left == 0 && f_v <= v_hi; ++f_v) {
            const Piece c = piece_of(f_v);
            f_left = c.end - c.at;
            if (f_left == 0) continue;
            f_chunk = c.chunk, f_chunks = (int)c.chunks, f_blocks = c.blocks;
            const int e = __shfl_sync(0xffffffffu, tab.seg_e[segment_of(f_v)], 0);
            const long long first = (long long)e * p.rows + c.unit * kRows, second = GateUp ? first : first + 16;
            const int block = c.block0 + c.chunk * kChunk, pair = block & ~(2 * kChunk - 1);
            src0 = reinterpret_cast<const char*>(p.qs0) + (first + r4) * row_bytes + (block + c4) * 16;
            src1 = reinterpret_cast<const char*>(p.qs1) + (second + r4) * row_bytes + (block + c4) * 16;
            src_d = reinterpret_cast<const char*>(lane < 16 ? p.d0 : p.d1) +
                    (((lane < 16 ? first : second) + (lane & 15)) * p.blocks + pair) * 2;
            code_step = kRows * row_bytes - (f_chunks - 1) * (kChunk * 16);
            scale_step = ((long long)kRows * p.blocks - (f_chunks - 1) / 2 * (2 * kChunk)) * 2;
            if (!GateUp) rows_left = p.rows - c.unit * 32;
            group = true;
        }
    };
    auto fill_edge = [&]() {  // past the last column or row: zeros
        const int left = f_blocks - f_chunk * kChunk;
        const char* none = reinterpret_cast<const char*>(p.qs0);
        const uint32_t to = to_codes + fill_at;
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
            const bool there = c4 < left && r4 + 8 * i < rows_left;
            const char* src = (i < 2 ? src0 : src1) + (i & 1) * 8 * row_bytes;
            copy_async<16>(to + 512 * i, there ? src : none, there ? 16u : 0u);
        }
        if (!group) return;
        const uint32_t to_d = to_scales + group_fill;
        const int valid = lane < rows_left ? min(f_blocks - (f_chunk & ~1) * kChunk, 8) : 0;
        if (p.scale_bytes == 2) {
#pragma unroll 1
            for (int i = 0; i < 8; ++i) {
                const uint16_t h = i < valid ? __ldg(reinterpret_cast<const uint16_t*>(src_d) + i) : (uint16_t)0;
                asm volatile("st.shared.u16 [%0], %1;" ::"r"(to_d + 2 * i), "h"(h) : "memory");
            }
        } else {
#pragma unroll 1
            for (int i = 0; i < 4; ++i) copy_async<4>(to_d + 4 * i, 2 * i < valid ? src_d + 4 * i : none, 2 * i < valid ? 4u : 0u);
        }
    };
    auto fill = [&]() {
        if (f_left != 0) {
            if (Scales >= 8 && (GateUp || rows_left >= 32)) {
                const uint32_t to = to_codes + fill_at, to_d = to_scales + group_fill;
                copy_async<16>(to, src0, 16u);
                copy_async<16>(to + 512, src0 + 8 * row_bytes, 16u);
                copy_async<16>(to + 1024, src1, 16u);
                copy_async<16>(to + 1536, src1 + 8 * row_bytes, 16u);
                if (group) {
                    if (Scales == 16) {
                        copy_async<16>(to_d, src_d, 16u);
                    } else {
                        const bool more = (f_chunk | 1) < f_chunks;
                        copy_async<8>(to_d, src_d, 8u);
                        copy_async<8>(to_d + 8, more ? src_d + 8 : src_d, more ? 8u : 0u);
                    }
                }
            } else {
                fill_edge();
            }
            if (group) group_fill = group_fill + kGroupBytes == kGroups ? 0u : group_fill + kGroupBytes;
            group = f_chunk & 1;
            if (++f_chunk == f_chunks) {  // on to the next unit
                src0 += code_step, src1 += code_step, src_d += scale_step;
                f_chunk = 0;
                group = true;
                if (!GateUp) rows_left -= 32;
            } else {
                src0 += kChunk * 16, src1 += kChunk * 16;
                if (group) src_d += 2 * kChunk * 2;
            }
            if (--f_left == 0) next_piece();
        }
        cp_async_commit();
    };
    next_piece();
#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i) {
        fill();
        fill_at += kStageBytes;
    }

    uint32_t k1024;
    asm volatile("mov.b32 %0, 0x64006400;" : "=r"(k1024));
    const int g = lane >> 2, t4 = lane & 3;
    // ldmatrix: lane l gives the address of row l % 8 of matrix l / 8: rows 0-7 and 8-15 of a block, then of the next one
    const int lm_row = (lane & 7) + (lane & 8);
    const uint32_t from_codes = ring + lm_row * 64 + (((lane >> 4) ^ ((lm_row >> 1) & 3)) << 4), from_scales = ring + kRing + g * 16;
    uint32_t use_at = 0, group_use = 0;
    const int sums = Parts == 1 && p.cap > kNarrow ? 16 : 8;  // that a warp may deposit
    float acc[kTiles][2][4] = {};
    int staged = -1;
#pragma unroll 1
    for (unsigned v = v_lo; v <= v_hi; ++v) {
        const Piece c = piece_of(v);
        unsigned max_bits[PER];
        if (!GateUp && v == v_lo) {
            grid_dependency_wait();
#pragma unroll
            for (int i = 0; i < PER; ++i) max_bits[i] = tid * PER + i < p.slots ? __ldcg(p.in_max + tid * PER + i) : 0u;
        }

        // ---- the segment's vectors, in their parts. Four lanes take a block of a vector; a thread's loads of two blocks are in
        // flight together, and what else there is to do before the first products is done while they are.
        const int seg = (int)segment_of(v);
        const int n = __shfl_sync(0xffffffffu, (int)tab.seg_n[seg], 0), at = __shfl_sync(0xffffffffu, (int)tab.seg_at[seg], 0);
        const int np = n <= 1 ? 1 : n <= 2 ? 2 : n <= 4 ? 4 : n <= 8 ? 8 : 16;  // columns kept of each part
        // With room for them, the columns of narrow segments lie at the distance of a full set.
        const uint32_t per_block = kRoom && np <= kNarrow ? 512u : (uint32_t)np * (Parts * 64u);
        const int only = GateUp && n == 1 ? (int)((unsigned)tab.list[at] / (unsigned)p.per_in) : -1;
        const bool fresh = only < 0 || only != staged;
        const int per_vector = (int)c.chunks * kChunk * 4;
        int j = fresh ? 0 : n, i = tid;
        float4 x[kStageLoads][2];
        int where[kStageLoads];  // vector and task within it, or -1
        auto load = [&]() {
#pragma unroll
            for (int u = 0; u < kStageLoads; ++u) {
                while (i >= per_vector) i -= per_vector, ++j;
                x[u][0] = x[u][1] = make_float4(0.f, 0.f, 0.f, 0.f);
                where[u] = -1;
                if (j < n) {
                    const int slot = tab.list[at + j], b = i >> 2, t = i & 3;
                    where[u] = j << 16 | i;
                    if (b < c.blocks) {
                        const int row = GateUp ? (int)((unsigned)slot / (unsigned)p.per_in) : slot;
                        const float* from = p.in + (long long)row * (p.blocks * 32) + (c.block0 + b) * 32 + t * 4;
                        x[u][0] = __ldcg(reinterpret_cast<const float4*>(from));
                        x[u][1] = __ldcg(reinterpret_cast<const float4*>(from + 16));
                    }
                }
                i += kThreads;
            }
        };
        load();
        if (v == v_lo) {
            if (!GateUp) {
#pragma unroll
                for (int q = 0; q < PER; ++q)
                    if (tid * PER + q < p.slots) tab.exponent[tid * PER + q] = (int8_t)vector_exponent(max_bits[q]);
                __syncthreads();
            }
        }
        float* const back = tab.back[v & 1];
        if (tid < n) {
            const int k = tab.exponent[tab.list[at + tid]];
            back[tid] = k == kNotFinite ? qnan() : pow2i(-k);
        }
#pragma unroll 1
        while (where[0] >= 0) {
#pragma unroll
            for (int u = 0; u < kStageLoads; ++u) {
                if (where[u] < 0) break;
                const int vector = where[u] >> 16, task = where[u] & 0xffff;
                const float scale = pow2i(tab.exponent[tab.list[at + vector]]);
                const float pair[4][2] = {{x[u][0].x, x[u][0].z}, {x[u][1].x, x[u][1].z}, {x[u][0].y, x[u][0].w}, {x[u][1].y, x[u][1].w}};
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float a = pair[q][0] * scale, b = pair[q][1] * scale;
                    const __half2 h = __floats2half2_rn(a, b);
                    const float2 f2 = __half22float2(h);
                    hi[q] = bits_of(h);
                    lo[q] = bits_of(__floats2half2_rn(a - f2.x, b - f2.y));
                }
                const uint32_t to = frags + (task >> 2) * per_block + vector * 64 + (task & 3) * 16;
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(hi[0]), "r"(hi[1]), "r"(hi[2]), "r"(hi[3])
                             : "memory");
                if (Parts == 2)
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to + (kRoom ? per_block / 2 : np * 64)), "r"(lo[0]), "r"(lo[1]), "r"(lo[2]),
                                 "r"(lo[3])
                                 : "memory");
            }
            load();
        }
        staged = only;
        __syncthreads();

        // ---- products
        auto deposit = [&]() {
#pragma unroll
            for (int i = 0; i < 8 * kTiles; ++i) {
                if (i >= 8 && np <= kNarrow) break;
                deposits[(warp * sums + i) * 32 + lane] = acc[i >> 3][i >> 2 & 1][i & 3];
                acc[i >> 3][i >> 2 & 1][i & 3] = 0.f;
            }
        };
        // A unit's sums leave: joined over the parts of the vectors, scaled back, for gate and up as silu(g) * u.
        auto finish = [&](int unit) {
            const bool joined = Parts == 2 && np <= kNarrow;  // columns 4 to 7 are the second part of columns 0 to 3
#pragma unroll
            for (int tile = 0; tile < kTiles; ++tile) {
                if (tile == 1 && np <= kNarrow) break;
                unsigned big[2] = {0u, 0u};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = tile * 8 + 2 * t4 + (i & 1), r = g + (i >> 1) * 8;
                    float u[2];
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        float& sum = acc[tile][m][i];
                        u[m] = Parts == 2 ? __shfl_xor_sync(0xffffffffu, sum, 2) : 0.f;
                        u[m] = joined ? sum + u[m] : sum;
                        sum = 0.f;
                    }
                    if (j >= n || (joined && t4 >= 2)) continue;
                    const float b = back[j];
                    const long long slot = tab.list[at + j];
                    if (GateUp) {
                        const float h = silu(u[0] * b) * (u[1] * b);
                        p.out[slot * p.rows + unit * 16 + r] = h;
                        big[i & 1] = max(big[i & 1], __float_as_uint(h) & 0x7fffffffu);
                    } else {
                        float* out = p.out + ((long long)part_of(v) * p.slots + slot) * p.rows + unit * 32;
#pragma unroll
                        for (int m = 0; m < 2; ++m)
                            if (unit * 32 + m * 16 + r < p.rows) out[m * 16 + r] = u[m] * b;
                    }
                }
                if (GateUp) {
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
#pragma unroll
                        for (int o = 4; o <= 16; o <<= 1) big[q] = max(big[q], __shfl_xor_sync(0xffffffffu, big[q], o));
                        const int j = tile * 8 + 2 * t4 + q;
                        if (g == 0 && j < n && !(joined && t4 >= 2)) atomicMax(p.out_max + tab.list[at + j], big[q]);
                    }
                }
            }
        };
        // A lane's column of a block: slot g of the first part, and of the second behind it; with up to 4 slots the second
        // part has columns 4 to 7, and with fewer the columns behind them repeat them.
        const uint32_t column = frags + (Parts == 1 || np == 8 ? g & (np - 1) : (g >> 2) * (kRoom ? 4 : np) + (g & (np - 1))) * 64 + t4 * 16;
        // A warp's chunks. What a chunk needs from shared memory is asked for before any of it is used (the second columns of
        // wide segments excepted, for which there are no registers).
        auto run = [&](auto wide) {
            constexpr bool Wide = decltype(wide)::value;  // 16 columns: two parts of 8 slots, or 16 slots
            const uint32_t step = !kRoom ? per_block : Wide ? 1024u : 512u;
            int chunk = c.chunk, unit = c.unit;
            bool head = chunk != 0;  // the unit was begun by a warp before this one, which joins it
            uint32_t vec = column + (uint32_t)chunk * (kChunk * step), sc = from_scales + group_use + ((chunk & 1) << 3);
#pragma unroll 1
            for (unsigned left = c.end - c.at; left != 0; --left) {
                cp_async_wait<kStages - 2>();
                __syncwarp();
                fill();
                const uint32_t codes = from_codes + use_at;
                uint32_t w[2][2][4], scale[2][2][2];  // codes of (pair of blocks, tile); scales of (tile, rows g or g + 8)
#pragma unroll
                for (int pair = 0; pair < 2; ++pair)
#pragma unroll
                    for (int m = 0; m < 2; ++m) ldsm4((pair ? codes ^ 32u : codes) + m * 1024, w[pair][m]);
                uint4 x[kChunk], y[kChunk];
#pragma unroll
                for (int b = 0; b < kChunk; ++b) {
                    x[b] = lds128(vec + b * (Wide ? 1024u : step));
                    if (Wide) y[b] = lds128(vec + b * 1024u + 512u);
                }
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                                     : "=r"(scale[m][h][0]), "=r"(scale[m][h][1])
                                     : "r"(sc + m * 256 + h * 128));
#pragma unroll
                for (int b = 0; b < kChunk; ++b) {
                    const uint4 l = Wide ? y[b] : x[b];
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        uint32_t ra[4], rb[4];
                        codes_of(w[b >> 1][m][2 * (b & 1)], k1024, ra);
                        codes_of(w[b >> 1][m][2 * (b & 1) + 1], k1024, rb);
                        const float zero[4] = {0.f, 0.f, 0.f, 0.f};
                        float s[4], s2[4];
                        mma(s, ra[0], rb[0], ra[1], rb[1], x[b].x, x[b].y, zero);
                        mma(s, ra[2], rb[2], ra[3], rb[3], x[b].z, x[b].w, s);
                        if (Wide) {
                            if (Parts == 1) {
                                mma(s2, ra[0], rb[0], ra[1], rb[1], l.x, l.y, zero);
                                mma(s2, ra[2], rb[2], ra[3], rb[3], l.z, l.w, s2);
                            } else {
                                mma(s, ra[0], rb[0], ra[1], rb[1], l.x, l.y, s);
                                mma(s, ra[2], rb[2], ra[3], rb[3], l.z, l.w, s);
                            }
                        }
                        const __half2 pa = half2_of(scale[m][0][b >> 1]), pb = half2_of(scale[m][1][b >> 1]);
                        const float da = (b & 1) ? __high2float(pa) : __low2float(pa), db = (b & 1) ? __high2float(pb) : __low2float(pb);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            acc[0][m][i] = fmaf(i < 2 ? da : db, s[i], acc[0][m][i]);
                            if (Wide && Parts == 1) acc[kTiles - 1][m][i] = fmaf(i < 2 ? da : db, s2[i], acc[kTiles - 1][m][i]);
                        }
                    }
                }
                fill_at = use_at;  // the stage that the next copies go to
                use_at = use_at + kStageBytes == kRing ? 0u : use_at + kStageBytes;
                const bool last = chunk + 1 == (int)c.chunks;
                if ((chunk & 1) || last || left == 1) {
                    group_use = group_use + kGroupBytes == kGroups ? 0u : group_use + kGroupBytes;
                    sc = from_scales + group_use;
                } else {
                    sc += 8;
                }
                ++chunk;
                vec += kChunk * step;
                if (last) {
                    if (head) deposit();
                    else finish(unit);
                    head = false;
                    chunk = 0;
                    vec = column;
                    ++unit;
                }
            }
            // a unit cut between warps is joined by the one that began it
            bool open = chunk != 0 && c.end != c.at;
            if (open && head) {
                deposit();
                open = false;
            }
            __syncthreads();
            if (open) {
                const unsigned items = unit_count(v) * c.chunks, unit_end = c.end - (unsigned)chunk + c.chunks;
#pragma unroll 1
                for (unsigned w = (unsigned)warp + 1, end = c.end; w < W && end < unit_end; ++w) {
                    const unsigned to = items * (w + 1) / W;
                    if (to == end) continue;
                    end = to;
#pragma unroll
                    for (int i = 0; i < 8 * kTiles; ++i) {
                        if (i >= 8 && np <= kNarrow) break;
                        acc[i >> 3][i >> 2 & 1][i & 3] += deposits[((int)w * sums + i) * 32 + lane];
                    }
                }
                finish(unit);
            }
        };
        if (np > kNarrow) run(std::true_type());
        else run(std::false_type());
    }
}

// The launch shape of one matrix (or gate and up): parts, slots of a segment, shared memory.
struct ExpertPlan {
    int parts, part_blocks, cap;
    uint32_t ring_at, deposits_at, frags_at, smem;
};
ExpertPlan plan_experts(int blocks, bool cut, int vector_parts, int warps, int stages, int max_smem) {
    ExpertPlan l;
    l.parts = cut ? moe_parts(blocks) : 1;
    const int per = l.part_blocks = ((blocks + l.parts - 1) / l.parts + 7) / 8 * 8;  // whole groups of scales
    for (l.cap = vector_parts == 1 ? 16 : 8; l.cap >= 1; l.cap /= 2) {
        l.ring_at = (sizeof(Tables) + 127) / 128 * 128;
        l.deposits_at = l.ring_at + (uint32_t)(warps * stages) * kSlotBytes;
        l.frags_at = l.deposits_at + (uint32_t)warps * (l.cap > 8 ? 16 : 8) * 32 * 4;
        l.smem = l.frags_at + (uint32_t)(per * l.cap * vector_parts) * 64u;
        if (l.smem <= (uint32_t)max_smem) break;
    }
    return l;  // cap 0: one vector does not fit
}

template <bool GateUp, int Parts, int W, int PER, int Scales, int Stages>
cudaError_t launch_experts_as(const ExpertParams& p, const ExpertPlan& l, int ctas, const DeviceInfo& di, bool overlap,
                              cudaStream_t s) {
    auto kern = moe_expert_kernel<GateUp, Parts, W, PER, Scales, Stages>;
    static std::once_flag once[64];
    cudaError_t e = cudaSuccess;
    std::call_once(once[di.device & 63],
                   [&] { e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, di.max_smem_optin); });
    if (e != cudaSuccess) return e;
    return launch_grid(kern, dim3((unsigned)(di.sm_count * ctas)), dim3(W * 32), l.smem, s, overlap, p);
}

// Two CTAs of 6 warps an SM where the experts get few slots each (a CTA's start, its vectors and its end overlap with the other
// one's products: 8 tokens over 64 experts 59.2 us, 61.0 us with 12 warps in one CTA; 1 token 25.7 and 27.4 us) and the vectors
// fit beside two rings; else one of 12.
template <bool GateUp, int Parts>
cudaError_t launch_experts_of(ExpertParams p, const DeviceInfo& di, bool overlap, cudaStream_t s) {
    const int half = di.max_smem_optin / 2 - 1024;  // of two CTAs an SM
    ExpertPlan l = plan_experts(p.blocks, !GateUp, Parts, 6, 3, half);
    const bool two = l.cap >= 8 / Parts && 2LL * p.slots <= (long long)l.cap * p.E && p.slots <= 192;
    if (!two) l = plan_experts(p.blocks, !GateUp, Parts, 12, 3, di.max_smem_optin);
    // Where experts get more slots than half a segment's, a ring of two stages may make room for twice the slots: 64 f16 tokens, 64
    // slots for each of 4 experts of 14336 x 4096, 900 us with 4 slots a segment, 653 us with 8; 32 bf16 tokens, 8 slots for
    // each of 8 such experts, 309 us with 4 and 268 us with 8, with x in one part 229 us with 8 and 224 us with 16. Down's parts
    // are short enough for full segments beside three stages.
    bool two_stages = false;
    if (GateUp && !two && 2LL * p.slots > (long long)l.cap * p.E) {
        const ExpertPlan s = plan_experts(p.blocks, !GateUp, Parts, 12, 2, di.max_smem_optin);
        two_stages = s.cap > l.cap;
        if (two_stages) l = s;
    }
    if (l.cap == 0) return cudaErrorNotSupported;
    p.units = GateUp ? p.rows / 16 : (p.rows + 31) / 32;
    p.parts = l.parts, p.part_blocks = l.part_blocks, p.cap = l.cap;
    p.table_bits = 1;
    while ((1 << p.table_bits) < 2 * p.slots) ++p.table_bits;
    p.ring_at = l.ring_at, p.deposits_at = l.deposits_at, p.frags_at = l.frags_at;
    const uintptr_t d = reinterpret_cast<uintptr_t>(p.d0) | reinterpret_cast<uintptr_t>(p.d1);
    p.scale_bytes = p.blocks % 8 == 0 && d % 16 == 0 ? 16 : p.blocks % 4 == 0 && d % 8 == 0 ? 8 : p.blocks % 2 == 0 && d % 4 == 0 ? 4 : 2;
    auto go = [&](auto scales) {
        constexpr int S = decltype(scales)::value;
        if (two) return launch_experts_as<GateUp, Parts, 6, 1, S, 3>(p, l, 2, di, overlap, s);
        if constexpr (GateUp)
            if (two_stages) return launch_experts_as<GateUp, Parts, 12, 2, S, 2>(p, l, 1, di, overlap, s);
        return launch_experts_as<GateUp, Parts, 12, 2, S, 3>(p, l, 1, di, overlap, s);
    };
    return p.scale_bytes == 16 ? go(std::integral_constant<int, 16>())
           : p.scale_bytes == 8 ? go(std::integral_constant<int, 8>())
                                : go(std::integral_constant<int, 0>());
}

}  // namespace

}  // namespace q4
