// smr_ffn.cu -- the experts' feed-forward behind the align: the gated product
// (act = silu(x Wg^T) * (x Wu^T)) and the product that follows it, whose rows
// are summed per token with the router's weights; operands in bf16 or MXFP4.
//
// The products are computed transposed: the tensor core's M rows are 128 rows
// of an expert's weights and its N columns are the routed rows of one aligned
// block (16 to 128, only as many as the block holds, in steps of 16; a pair of
// CTAs takes 256 weight rows and up to 256 columns from several blocks of an
// expert). From one token to a couple of thousand the time is the touched experts' weights out
// of HBM, whatever the tile; this orientation streams each weight tile once
// per block at full MMA width, and a block with three rows costs N = 16
// columns instead of A padded rows. The ragged dimension has the fine step.
//
// GB300 design: one persistent CTA per SM over (block, weight tile) items,
// tiles of one block next to each other (its rows stay in L2; blocks of one
// expert follow each other, so its weights do too). Warp roles: 0 loads the
// weights by TMA, 1 issues the MMAs, 2 reads the align's outputs ahead and
// hands out the work, from 3 on load the routed rows (and their block scales)
// with asynchronous 16-byte copies (a TMA gather takes 4 rows an instruction,
// too slow for 128 rows a k-block), the last eight drain TMEM. The stage ring runs across
// items; accumulators are double-buffered in TMEM, so the epilogue of one item
// runs under the loads and MMAs of the next.
// Every wait is bounded; a wait that gives up sets the workspace's error bit.
#include <cudaTypedefs.h>

#include "smr_device.cuh"
#include "smr_launch.h"

namespace smr {

// k-blocks a stage: two for blocks of 64 rows and for pairs in MXFP4, else one
// (a stage would be too large for a ring of them). A stage costs every role a
// few hundred cycles of barrier round trips whatever its size (MXFP4 up, 16384
// tokens: 210 us in stages of one, 187 in stages of two).
template <int SUB>
constexpr int kFfLoaders = SUB == 2 ? 4 : 6;     // warps that load the routed rows; at most the stages
constexpr int kFfDrains = 8;                     // warps of the epilogue, two for each quarter of TMEM's lanes
template <int SUB>
constexpr int kFfThreads = 32 * (3 + kFfLoaders<SUB> + kFfDrains);
constexpr int kFfRows = 128;                     // weight rows of a tile (the MMA's M)
constexpr int kFfRowBytes = 128;                 // one k-block of a row: 64 bf16 or 256 MXFP4
constexpr int kFfWBytes = kFfRows * kFfRowBytes;  // weight tile of a stage
constexpr int kFfMaxStages = 8;
// Pieces of work known ahead of the epilogue: with a short contraction (MXFP4,
// K = 512: two k-blocks a piece) these bound the weights in flight.
constexpr int kFfInfos = 8;
constexpr int kSfAtom = 512;                     // scales of 128 rows x 4 blocks (128 values of K)

// What the producer tells the other warps about a piece of work: one expert's
// columns of an item.
template <int COLS>
struct FfInfo {
    int n;     // MMA columns (16..COLS, a multiple of 16); -1: no more work
    int nt;    // weight tile of this CTA
    int e;     // expert
    int pad;
    int slot[COLS];  // flat slot of every column, -1: none
    // its row of x, -1: none. Such a column is neither loaded nor stored: what
    // the MMAs make of the old contents of shared memory stays in its column.
    // (Loading row 0 for it, 15 times a block in every CTA, would queue the
    // whole GPU up on one line of L2.)
    int row[COLS];
};
constexpr int kFfBars = 2 * kFfMaxStages + 4 + 2 * kFfInfos + 1;
constexpr int kFfBarBytes = (kFfBars * 8 + 8 + 15) / 16 * 16;
// Columns of a piece, at most. (A pair of MXFP4: 128, as two accumulators of
// 256 columns would leave no room in TMEM for the scales.)
template <bool MX, bool PAIR>
constexpr int kFfCols = PAIR && !MX ? 256 : 128;
template <bool MX, bool PAIR>
constexpr int kFfMiscBytes = kFfBarBytes + kFfInfos * (int)sizeof(FfInfo<kFfCols<MX, PAIR>>);

struct FfParams {
    int num_kb, last_steps;  // k-blocks; MMA steps of the last one (4 in the others)
    int feat, ntiles;        // output features; weight tiles
    const uint8_t *x;
    uint32_t x_row_bytes;    // between rows of x
    int x_bytes;             // of a row of x
    // row of x = slot / width (gated product), exact for slots below 2^30 as
    // slot * div_mul >> div_shift
    uint32_t div_mul, div_shift;
    int num_experts, A, stages;
    int acc_cols, tmem_cols; // TMEM columns of an accumulator, of the allocation
    int64_t sorted_cap;
    int numel, max_blocks;
    const int32_t *sorted, *eids, *npp;
    void *out;               // [numel, feat], fp32 or bf16
    const uint8_t *x_scales, *w_scales;  // MXFP4
    int num_chunks;          // MXFP4: K / 128
    int scale_bytes;         // MXFP4: rows of x_scales can be read 16, 8 or 4 bytes at a time
    uint32_t *err;
    uint32_t stage_bytes, b_bytes;
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar) : "memory");
}
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap *map, int c0, int c3, int c4,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %3, %4, %5}], [%6];"
        ::"r"(dst), "l"(map), "r"(c0), "r"(0), "r"(c3), "r"(c4), "r"(bar) : "memory");
}
// The same loads by a CTA of a pair; bar may be the other CTA's barrier.
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2,
                                                 uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar) : "memory");
}
__device__ __forceinline__ void tma_load_5d_pair(uint32_t dst, const CUtensorMap *map, int c0, int c3, int c4,
                                                 uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %3, %4, %5}], [%6];"
        ::"r"(dst), "l"(map), "r"(c0), "r"(0), "r"(c3), "r"(c4), "r"(bar) : "memory");
}
// Arrive on a barrier of either CTA of a pair (address from cluster_addr).
// What is handed over is in this CTA's own shared memory (made visible to the
// tensor core by a proxy fence before) or TMEM (read, and fenced), never in
// global memory, so the arrival needs no release beyond the CTA: with
// .release.cluster every one waits for the device-wide visibility of the
// thread's earlier writes, which costs more than pairs gain.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
template <bool PAIR>
__device__ __forceinline__ void ff_mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    if constexpr (PAIR) tc_mma_bf16_pair(d, a, b, idesc, accumulate);
    else tc_mma_bf16(d, a, b, idesc, accumulate);
}
// Arrival (in both CTAs of a pair) once the MMAs issued so far are done.
template <bool PAIR>
__device__ __forceinline__ void ff_commit(uint64_t *bar) {
    if constexpr (PAIR) tc_commit_pair(smem_u32(bar), 0x3);
    else tc_commit(smem_u32(bar));
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}
// Loads of 16 or 8 bytes where row >= 0, else the registers stay as they are.
__device__ __forceinline__ void ld_cg_16(uint32_t *v, const void *src, int row) {
    asm volatile("{\n .reg .pred q;\n setp.ge.s32 q, %5, 0;\n @q ld.global.cg.v4.u32 {%0, %1, %2, %3}, [%4];\n}"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]) : "l"(src), "r"(row));
}
__device__ __forceinline__ void ld_cg_8(uint32_t *v, const void *src, int row) {
    asm volatile("{\n .reg .pred q;\n setp.ge.s32 q, %3, 0;\n @q ld.global.cg.v2.u32 {%0, %1}, [%2];\n}"
                 : "+r"(v[0]), "+r"(v[1]) : "l"(src), "r"(row));
}
// Copies that happen where row >= 0 (predicated: a branch a row cost the
// large batches 15%). No memory clobber: what they write is read only behind
// the wait for them, and loads of row numbers may move ahead of them.
__device__ __forceinline__ void cp_async_4(uint32_t dst, const void *src, int row) {
    asm volatile("{\n .reg .pred q;\n setp.ge.s32 q, %2, 0;\n @q cp.async.ca.shared.global [%0], [%1], 4;\n}"
                 ::"r"(dst), "l"(src), "r"(row));
}
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void *src, int row) {
    asm volatile("{\n .reg .pred q;\n setp.ge.s32 q, %2, 0;\n @q cp.async.cg.shared.global [%0], [%1], 16;\n}"
                 ::"r"(dst), "l"(src), "r"(row));
}

// MXFP4 instruction descriptor (kind::mxf4): A and B E2M1 (bits 7-9, 10-11 =
// 1), scales UE8M0 (bit 23), N >> 3 in bits 17-22, M >> 7 in bits 27-28; the
// byte of a scale column where the step's two scales start (0 or 2) in bits
// 4-5 (B) and 29-30 (A).
__host__ __device__ constexpr uint32_t idesc_mxf4(int m, int n) {
    return (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | (1u << 23) | ((uint32_t)(m >> 7) << 27);
}
// D[tmem] (+)= (A * scale_A) (B * scale_B)^T, 4-bit operands, one scale per 32
// values of K, fp32 accumulation.
template <bool PAIR>
__device__ __forceinline__ void tc_mma_mxf4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
    if constexpr (PAIR)
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
            " tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}"
            ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate) : "memory");
    else
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
            " tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}"
            ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate) : "memory");
}
// 512 bytes of scales (32 rows of 16 bytes) into 4 TMEM columns, the same in
// every quarter of the lanes (of a pair: in each CTA from its own shared
// memory). Ordered before the MMAs that this thread issues next, and behind
// those that it issued.
template <bool PAIR>
__device__ __forceinline__ void tc_cp_scales(uint32_t taddr, uint32_t saddr) {
    // no swizzle, 8-row groups 128 bytes apart (stride byte offset >> 4 in
    // bits 32-45), descriptor version 1
    const uint64_t desc = (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(128u >> 4) << 32) | ((uint64_t)1 << 46);
    if constexpr (PAIR) asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
    else asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// silu(g) * u in fp32: with h = exp(-|g| / 2) = 2^(-|g| log2(e) / 2), silu(g) =
// g / (1 + h^2) for g >= 0 and g h^2 / (1 + h^2) below, one factor h going to g
// and one to u. The denominator stays in [1, 2] and h is a normal number down
// to g = -174, so that a small sigmoid beside a large u keeps its value (1 / (1
// + exp(-g)) overflows at g = -88); from there on the product is below 2^-115
// for every finite u and comes out as 0. Off by at most 4 + 1.2 |g| units of
// 2^-23 from the two powers (the rounding of their argument, 2 units each) and
// 5 from the rest.
__device__ __forceinline__ float swiglu(float g, float u) {
    float h, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(h) : "f"(fabsf(g) * -0.72134752f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fmaf(h, h, 1.0f)));
    const float t = g < 0.0f ? h : 1.0f;
    return g * t * r * (u * t);
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&b);
}
// Outputs in bf16 leave through shared memory, in whole lines. (Stored from
// registers, a warp reaches 64 bytes of a line at most, which halves the rate
// of scattered rows.) TMEM is read in the matrix-fragment shape, whose
// transposing store puts neighbouring features next to each other without a
// shuffle, and which gives a thread the gate and the up value of the same
// places.
template <bool UP>
constexpr int kOutBytes = UP ? 128 : 256;        // of a column: 64 or 128 features
template <bool UP>
constexpr int kOutPitch = kOutBytes<UP> + 16;    // 8 rows of a store in different banks
template <bool UP>
constexpr int kOutCols = UP ? 16 : 8;            // columns of a block: one matrix store of each warp
// Two blocks for each half of the epilogue's warps: one is filled while the
// other is read.
template <bool UP, bool F32>
constexpr int kFfOutBytes = F32 ? 0 : 2 * 2 * kOutCols<UP> * kOutPitch<UP>;

// 32 lanes x 16 columns as two fragments of 16 x 16: v[8 h + 4 u + 2 r + b] is
// lane 16 h + 8 r + (thread / 4), column 8 u + 2 (thread % 4) + b.
__device__ __forceinline__ void tmem_ld_frags_async(uint32_t taddr, uint32_t (&v)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "r"(taddr));
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
                 : "r"(taddr + (16u << 16)));
}
// The fragments' values in bf16, in the order of put_frags: the gated product's
// features of 16 columns, or twice 32 features of 8 columns.
template <bool UP>
__device__ __forceinline__ void pack_frags(const uint32_t (&v)[16], uint32_t (&o)[UP ? 4 : 8]) {
    float a[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) a[j] = __uint_as_float(v[j]);
#pragma unroll
    for (int j = 0; j < (UP ? 4 : 8); ++j) {
        const int k = UP ? 2 * j : 4 * (j >> 2) + 2 * (j & 1) + 8 * (j >> 1 & 1);
        o[j] = UP ? pack_bf16x2(swiglu(a[k], a[(k + 8) & 15]), swiglu(a[k + 1], a[(k + 9) & 15]))  // (gate, up rows)
                  : pack_bf16x2(a[k], a[k + 1]);
    }
}
// Four 8 x 8 matrices, transposed: the address is that of the row (thread % 8)
// of matrix (thread / 8) in shared memory, which gets a column's 8 features.
__device__ __forceinline__ void put_frags(uint32_t dst, const uint32_t *o) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared::cta.b16 [%0], {%1, %2, %3, %4};"
                 ::"r"(dst), "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3]) : "memory");
}
// Four warps meet; every one gets whether all of them came with ok.
__device__ __forceinline__ bool meet_if(int id, bool ok) {
    uint32_t all;
    asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 q, %1, 0;\n barrier.cta.red.and.pred p, %2, 128, q;\n"
                 " selp.u32 %0, 1, 0, p;\n}" : "=r"(all) : "r"((uint32_t)ok), "r"(id) : "memory");
    return all != 0;
}
__device__ __forceinline__ void meet(int id) { asm volatile("barrier.cta.sync %0, 128;" ::"r"(id) : "memory"); }

// Four lanes hold a feature each (a row of TMEM), c0..c3 its values in four
// columns; each returns the four features of column (lane & 3), so that fp32
// outputs leave in whole lines of 8 lanes.
__device__ __forceinline__ float4 quad_turn(float c0, float c1, float c2, float c3, int lane) {
    const bool odd = lane & 1, top = lane & 2;
    const float x = __shfl_xor_sync(0xffffffffu, odd ? c0 : c1, 1), y = __shfl_xor_sync(0xffffffffu, odd ? c2 : c3, 1);
    const float2 p = odd ? make_float2(x, c1) : make_float2(c0, x), q = odd ? make_float2(y, c3) : make_float2(c2, y);
    const float z0 = __shfl_xor_sync(0xffffffffu, top ? p.x : q.x, 2), z1 = __shfl_xor_sync(0xffffffffu, top ? p.y : q.y, 2);
    return top ? make_float4(z0, z1, q.x, q.y) : make_float4(p.x, p.y, z0, z1);
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(one));
    return one != 0;
}
// A bounded wait of every lane of a warp, and one answer.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort) {
    return __all_sync(0xffffffffu, mbar_wait_bounded(smem_u32(bar), parity, abort));
}
// Position in a ring of barriers: index and the parity of its current use.
struct RingPos {
    int i = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void next(int n) {
        if (++i == n) {
            i = 0;
            ph ^= 1u;
        }
    }
    __device__ __forceinline__ void skip(int by, int n) {
        for (i += by; i >= n; i -= n) ph ^= 1u;
    }
};

// Every error goes to the workspace's header and to one word per device, which
// outlives workspaces and which a caller without one can read.
static __device__ uint32_t g_expert_error;
__device__ __forceinline__ void ffn_error(uint32_t *err, uint32_t bits) {
    set_error(err, bits);
    set_error(&g_expert_error, bits);
}

// MX: MXFP4 operands, else bf16. UP: the gated product (a tile holds 64
// features: 16 gate rows and their 16 up rows in turn, so that both halves of
// a feature are in one warp's TMEM lanes), else 128 plain rows. PAIR: two CTAs
// on one 256-row tile and up to kCols columns (blocks of one expert next to
// each other together); each holds its own 128 weight rows (and their scales),
// half of the routed rows and all of these rows' scales, and drains its own
// lanes.
// F32: the outputs are fp32, else bf16 (a variant of its own, without the other
// epilogue's registers, so that blocks of the sum fit beside a CTA).
template <bool MX, bool UP, bool PAIR, int SUB, bool F32>
__global__ void __launch_bounds__(kFfThreads<SUB>, 1)
expert_ffn_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_s, const FfParams p) {
    constexpr int kCols = kFfCols<MX, PAIR>;
    using Info = FfInfo<kCols>;
    constexpr int kLoaders = kFfLoaders<SUB>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    const int ST = p.stages;
    uint8_t *misc = smem + (size_t)ST * p.stage_bytes;
    // full and acc_empty of a pair are the leader's, the others each CTA's own
    uint64_t *full = reinterpret_cast<uint64_t *>(misc);  // the stage's operands landed
    uint64_t *empty = full + kFfMaxStages;                 // the MMAs are done with the stage
    uint64_t *acc_full = empty + kFfMaxStages;             // a piece's accumulator is complete
    uint64_t *acc_empty = acc_full + 2;                    // it has been read
    uint64_t *info_full = acc_empty + 2;
    uint64_t *info_empty = info_full + kFfInfos;
    uint64_t *last = info_empty + kFfInfos;                // every MMA issued is done
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(last + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    Info *info = reinterpret_cast<Info *>(misc + kFfBarBytes);
    uint8_t *out_rows = misc + kFfMiscBytes<MX, PAIR>;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
    if (threadIdx.x == 0) {
        for (int s = 0; s < ST; ++s) {
            mbar_init(smem_u32(&full[s]), PAIR ? 3 : 2);  // the weights' bytes, the row loader (of each CTA)
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(smem_u32(&acc_full[s]), 1);
            mbar_init(smem_u32(&acc_empty[s]), (PAIR ? 2 : 1) * kFfDrains);
        }
        for (int s = 0; s < kFfInfos; ++s) {
            mbar_init(smem_u32(&info_full[s]), 1);
            mbar_init(smem_u32(&info_empty[s]), 2 + kLoaders + kFfDrains);  // every warp but the scout
        }
        mbar_init(smem_u32(last), 1);
        *abort_flag = 0;
        mbar_fence_init();
        prefetch_tensormap(&tm_w);
        if constexpr (MX && PAIR) prefetch_tensormap(&tm_s);
    }
    if (warp == 1) {
        if constexpr (PAIR) {
            tmem_alloc_pair(smem_u32(tmem_slot), (uint32_t)p.tmem_cols);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(smem_u32(tmem_slot), (uint32_t)p.tmem_cols);
            tmem_relinquish();
        }
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    griddep_wait();  // the align's outputs and x come from previous kernels
    // (only now: a kernel that follows may read what those wrote at once)
    griddep_launch_dependents();

    // a stage: [weights SUB][rows SUB][MXFP4: weights' scales 2 SUB][rows' scales 2 SUB]
    const uint32_t ring = smem_u32(smem);
    const uint32_t x_off = SUB * kFfWBytes, ws_off = x_off + SUB * p.b_bytes, xs_off = ws_off + 2 * SUB * kSfAtom;
    int issued = 0;  // stages whose weights were requested (warp 0)

    if (warp == 0) {
        // ---------------------------------------------------- weights ----
        const bool elected = elect_one();
        RingPos st, iq;
        bool ok = true;
        while (ok) {
            if (!(ok = warp_wait(&info_full[iq.i], iq.ph, abort_flag))) break;
            const volatile Info *inf = info + iq.i;
            const int n = inf->n, nt = inf->nt, e = inf->e;
            __syncwarp();
            if (elected) mbar_arrive(smem_u32(&info_empty[iq.i]));
            iq.next(kFfInfos);
            if (n < 0) break;
            const uint8_t *scales = nullptr;
            if constexpr (MX) scales = p.w_scales + ((int64_t)e * p.ntiles + nt) * p.num_chunks * kSfAtom;
            for (int kb = 0; kb < p.num_kb; kb += SUB) {
                if (!(ok = warp_wait(&empty[st.i], st.ph ^ 1u, abort_flag))) break;
                const uint32_t base = ring + (uint32_t)st.i * p.stage_bytes;
                const uint32_t bar = smem_u32(&full[st.i]);
                const int subs = SUB == 1 ? 1 : min(SUB, p.num_kb - kb);
                if (elected) {
                    if constexpr (PAIR) {
                        // both CTAs' bytes complete the leader's barrier
                        if (rank == 0) mbar_arrive_expect_tx(bar, 2 * (subs * kFfWBytes + (MX ? 2 * SUB * kSfAtom : 0)));
                        const uint32_t fb = cluster_addr(bar, 0u);
                        // (the last stage's box may reach into the next tile's scales; they are not used)
                        if constexpr (MX)
                            tma_load_2d_pair(base + ws_off, &tm_s, 0, (e * p.ntiles + min(nt, p.ntiles - 1)) * p.num_chunks + 2 * kb, fb);
#pragma unroll
                        for (int u = 0; u < SUB; ++u) {
                            if (u >= subs) break;
                            const int xk = (kb + u) * (MX ? kFfRowBytes : kFfRowBytes / 2);
                            if constexpr (UP) tma_load_5d_pair(base + u * kFfWBytes, &tm_w, xk, nt * 4, e, fb);
                            else tma_load_3d_pair(base + u * kFfWBytes, &tm_w, xk, nt * kFfRows, e, fb);
                        }
                    } else {
                        uint32_t sbytes = 0;
                        if constexpr (MX) sbytes = (uint32_t)min(2 * SUB, p.num_chunks - 2 * kb) * kSfAtom;
                        mbar_arrive_expect_tx(bar, subs * kFfWBytes + sbytes);
#pragma unroll
                        for (int u = 0; u < SUB; ++u) {
                            if (u >= subs) break;
                            const int xk = (kb + u) * (MX ? kFfRowBytes : kFfRowBytes / 2);
                            if constexpr (UP) tma_load_5d(base + u * kFfWBytes, &tm_w, xk, nt * 4, e, bar);
                            else tma_load_3d(base + u * kFfWBytes, &tm_w, xk, nt * kFfRows, e, bar);
                        }
                        if constexpr (MX) bulk_load(base + ws_off, scales + 2 * kb * kSfAtom, sbytes, bar);
                    }
                }
                ++issued;
                st.next(ST);
            }
        }
        __syncwarp();
    } else if (warp == 2) {
        // ------------------------------------------------------ scout ----
        // An item is a group of blocks of one expert (one block; PAIR: up to
        // kCols / A, counted from the expert's first) and a weight tile (PAIR:
        // two). Both CTAs of a pair walk the same items. CTAs take every
        // gridDim-th item: a block's tiles run next to each other in time
        // (its rows stay in L2), blocks of one expert too (its weights).
        const int A = p.A, G = PAIR ? kCols / A : 1;
        const int tiles = PAIR ? (p.ntiles + 1) / 2 : p.ntiles;
        const int ctas = PAIR ? gridDim.x >> 1 : gridDim.x, cta = PAIR ? blockIdx.x >> 1 : blockIdx.x;
        const int dgrp = ctas / tiles, dtile = ctas % tiles;
        int grp = cta / tiles, tile = cta % tiles;  // the item
        const int bo = 8 * lane / A, po = 8 * lane % A;  // this lane's 8 entries: block of the group, place in it
        const bool in = bo < G;
        const bool wide = (reinterpret_cast<uintptr_t>(p.sorted) & 15) == 0;
        // the entries and the block's expert (of blocks below `limit`),
        // requested kAhead items ahead (a round trip to L2 is longer than two
        // short items)
        auto fetch = [&](int b0, int limit, int (&ent)[8], int &e) {
            const int b = b0 + bo;
            if (!in || b0 < 0 || b >= limit) return;
            const int64_t at = (int64_t)b * A + po;
            e = __ldcg(p.eids + b);
            if (wide && at + 8 <= p.sorted_cap) {
                const int4 lo = __ldcg(reinterpret_cast<const int4 *>(p.sorted + at));
                const int4 hi = __ldcg(reinterpret_cast<const int4 *>(p.sorted + at) + 1);
                ent[0] = lo.x; ent[1] = lo.y; ent[2] = lo.z; ent[3] = lo.w;
                ent[4] = hi.x; ent[5] = hi.y; ent[6] = hi.z; ent[7] = hi.w;
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) ent[j] = at + j < p.sorted_cap ? __ldcg(p.sorted + at + j) : p.numel;
            }
        };
        auto step = [&](int &g, int &t) {
            g += dgrp;
            t += dtile;
            if (t >= tiles) {
                t -= tiles;
                ++g;
            }
        };
        constexpr int kAhead = 4;
        int ent[kAhead][8], e[kAhead], at[kAhead], slot[8];  // (at: first block of the item's group)
        int grp2 = grp, tile2 = tile;  // the item that is requested next
        const int npp = __ldcg(p.npp);
        // (requested with npp: of blocks past it, left out below)
        const int first_e = PAIR && lane < p.max_blocks ? __ldcg(p.eids + lane) : 0;
        if constexpr (!PAIR) {  // the first two at once with npp: what lies past it is left out below
            int g = grp, t = tile;
            fetch(g, p.max_blocks, ent[0], e[0]);
            step(g, t);
            fetch(g, p.max_blocks, ent[1], e[1]);
        }
        const int nblk = max(0, min(npp / A, p.max_blocks));
        // First block of group g (asked for in ascending order), -1 past the
        // last: 32 blocks at a time, a bit for every block that starts one,
        // which is every G-th block of an expert's segment.
        int scan_at = -32, scan_base = 0, last_e = 0, run = 0;  // (run: blocks of the segment before the 32)
        uint32_t starts = 0u;
        auto locate = [&](int g) {
            if constexpr (PAIR) {
                while (g - scan_base >= __popc(starts)) {
                    if (scan_at + 32 >= nblk) return -1;
                    scan_base += __popc(starts);
                    scan_at += 32;
                    const int b = scan_at + lane, eb = scan_at == 0 ? first_e : (b < nblk ? __ldcg(p.eids + b) : 0);
                    int before = __shfl_up_sync(0xffffffffu, eb, 1);
                    if (lane == 0) before = last_e;
                    const uint32_t first = __ballot_sync(0xffffffffu, b == 0 || eb != before);
                    const uint32_t upto = first & (0xffffffffu >> (31 - lane));
                    const int place = upto != 0u ? lane - (31 - __clz(upto)) : run + lane;
                    starts = __ballot_sync(0xffffffffu, b < nblk && place % G == 0);
                    last_e = __shfl_sync(0xffffffffu, eb, 31);
                    run = __shfl_sync(0xffffffffu, place, 31) + 1;
                }
                // the bit with g - scan_base others below it
                const bool hit = (starts >> lane & 1u) && __popc(starts & ((1u << lane) - 1u)) == g - scan_base;
                return scan_at + __ffs(__ballot_sync(0xffffffffu, hit)) - 1;
            } else {
                return g < nblk ? g : -1;
            }
        };
        RingPos iq;
        bool ok = true;
        auto post = [&](int n, int nt, int e, const int (&slot)[8]) {
            if (!(ok = warp_wait(&info_empty[iq.i], iq.ph ^ 1u, abort_flag))) return;
            Info *inf = info + iq.i;
            const int c = 8 * lane;
            if (c < n) {
                int row[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    row[j] = slot[j];
                    if (UP && slot[j] >= 0) row[j] = (int)((uint64_t)(uint32_t)slot[j] * p.div_mul >> p.div_shift);
                }
#pragma unroll
                for (int j = 0; j < 8; j += 4) {
                    *reinterpret_cast<int4 *>(inf->slot + c + j) = make_int4(slot[j], slot[j + 1], slot[j + 2], slot[j + 3]);
                    *reinterpret_cast<int4 *>(inf->row + c + j) = make_int4(row[j], row[j + 1], row[j + 2], row[j + 3]);
                }
            }
            if (lane == 0) *reinterpret_cast<int4 *>(inf) = make_int4(n, nt, e, 0);
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&info_full[iq.i]));
            iq.next(kFfInfos);
        };
        // every block's entries into L2, each line by one CTA
        for (int64_t i = ((int64_t)blockIdx.x * 32 + lane) * 32; i < min((int64_t)nblk * A, p.sorted_cap);
             i += (int64_t)gridDim.x * 32 * 32)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(p.sorted + i));
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            at[u] = locate(grp2);
            if (PAIR || u >= 2) fetch(at[u], nblk, ent[u], e[u]);
            step(grp2, tile2);
        }
        auto take = [&](int &at, int (&ent)[8], int &e) {
            // the item whose first block is `at`; then the one kAhead later is requested
            int top = 0;
            bool bad = false;
            const bool here = in && at + bo < nblk;
            const int ex = here ? e : -1;
            const int eg = __shfl_sync(0xffffffffu, ex, 0);
            int h = 1;  // blocks of the group
            while (h < G && at + h < nblk && __shfl_sync(0xffffffffu, ex, h * A / 8) == eg) ++h;
            const bool mine = here && bo < h;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int i = mine ? ent[j] : p.numel;
                const bool real = (uint32_t)i < (uint32_t)p.numel;
                bad |= !real && i != p.numel;
                slot[j] = real ? i : -1;
                if (real) top = 8 * lane + j + 1;
            }
            // neither a slot nor the sentinel: a corrupted align output
            if (bad) ffn_error(p.err, kErrBadSlot);
            __syncwarp();
            const int rows = (int)__reduce_max_sync(0xffffffffu, (unsigned)top);
            const int nt = PAIR ? 2 * tile + (int)rank : tile;
            at = locate(grp2);
            fetch(at, nblk, ent, e);
            step(grp, tile);
            step(grp2, tile2);
            if (rows == 0) return;
            if ((unsigned)eg >= (unsigned)p.num_experts) {  // only a corrupted align output gets here
                if (lane == 0) ffn_error(p.err, kErrBadId);
                __syncwarp();
                return;
            }
            post((rows + 15) & ~15, nt, eg, slot);
        };
        while (ok && at[0] >= 0) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (ok && at[u] >= 0) take(at[u], ent[u], e[u]);
        }
        if (ok) post(-1, 0, 0, slot);
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------- MMAs ----
        // The whole warp runs the loop, so that descriptors and addresses stay
        // in uniform registers; one elected lane issues (a pair's leader; its
        // peer only keeps up with the pieces).
        const bool elected = elect_one();
        RingPos st, iq, ac;
        uint32_t sf = tmem + (uint32_t)(2 * p.acc_cols);  // MXFP4: two sets of scale columns in turn: [A 8][B 8]
        bool ok = true;
        while (ok) {
            if (!(ok = warp_wait(&info_full[iq.i], iq.ph, abort_flag))) break;
            const int n = __shfl_sync(0xffffffffu, reinterpret_cast<volatile Info *>(info)[iq.i].n, 0);
            __syncwarp();
            if (elected) mbar_arrive(smem_u32(&info_empty[iq.i]));
            iq.next(kFfInfos);
            if (n < 0) break;
            if (rank != 0) continue;
            if (!(ok = warp_wait(&acc_empty[ac.i], ac.ph ^ 1u, abort_flag))) break;
            tc_fence_after();
            const uint32_t acc = tmem + (uint32_t)(ac.i * p.acc_cols);
            constexpr int kM = PAIR ? 2 * kFfRows : kFfRows;
            const uint32_t idesc = MX ? idesc_mxf4(kM, n) : idesc_bf16_f32(kM, n);
            for (int kb = 0; kb < p.num_kb; kb += SUB) {
                if (!(ok = warp_wait(&full[st.i], st.ph, abort_flag))) break;
                tc_fence_after();
                const uint32_t base = ring + (uint32_t)st.i * p.stage_bytes;
#pragma unroll
                for (int u = 0; u < SUB; ++u) {
                    if (SUB > 1 && kb + u >= p.num_kb) break;
                    // descriptors: + 2 per 32 bytes of K
                    const uint64_t da = smem_desc_sw<128>(base + u * kFfWBytes),
                                   db = smem_desc_sw<128>(base + x_off + u * p.b_bytes);
                    const int steps = kb + u + 1 == p.num_kb ? p.last_steps : 4;
                    const uint32_t more = kb + u != 0 ? 1u : 0u;
                    if constexpr (MX) {
                        const uint32_t sa = base + ws_off + 2 * u * kSfAtom, sb = base + xs_off + 2 * u * kSfAtom;
                        if (elected) {
                            tc_cp_scales<PAIR>(sf, sa);
                            tc_cp_scales<PAIR>(sf + 8, sb);
                            tc_mma_mxf4<PAIR>(acc, da, db, idesc, sf, sf + 8, more);
                            tc_mma_mxf4<PAIR>(acc, da + 2, db + 2, idesc | (1u << 30) | (1u << 5), sf, sf + 8, 1u);
                            if (steps == 4) {
                                tc_cp_scales<PAIR>(sf + 4, sa + kSfAtom);
                                tc_cp_scales<PAIR>(sf + 12, sb + kSfAtom);
                                tc_mma_mxf4<PAIR>(acc, da + 4, db + 4, idesc, sf + 4, sf + 12, 1u);
                                tc_mma_mxf4<PAIR>(acc, da + 6, db + 6, idesc | (1u << 30) | (1u << 5), sf + 4, sf + 12, 1u);
                            }
                        }
                        sf ^= 16u;
                    } else if (elected) {
                        if (steps == 4) {
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                ff_mma_bf16<PAIR>(acc, da + 2 * kk, db + 2 * kk, idesc, kk ? 1u : more);
                        } else {
                            for (int kk = 0; kk < steps; ++kk)
                                ff_mma_bf16<PAIR>(acc, da + 2 * kk, db + 2 * kk, idesc, kk ? 1u : more);
                        }
                    }
                }
                if (elected) ff_commit<PAIR>(&empty[st.i]);
                st.next(ST);
            }
            if (!ok) break;
            if (elected) ff_commit<PAIR>(&acc_full[ac.i]);
            ac.next(2);
        }
        // every MMA issued is done before TMEM is freed, also after an abort
        if (rank == 0) {
            if (elected) {
                if constexpr (PAIR) tc_commit_pair(smem_u32(last), 0x1);
                else tc_commit(smem_u32(last));
            }
            volatile int never = 0;
            if (!mbar_wait_bounded(smem_u32(last), 0u, &never)) *abort_flag = 1;
        }
        __syncwarp();
    } else if (warp < 3 + kLoaders) {
        // ------------------------------------------------ routed rows ----
        // Each loader warp fills every kLoaders-th stage, so that a stage is
        // waited for, copied, made visible to the tensor core (async proxy)
        // and announced by one warp, while the others' copies are in flight.
        // A row's k-block is eight 16-byte chunks; eight neighbouring lanes
        // copy a row's, chunk c of row r landing at r * 128 + ((c ^ (r & 7)) <<
        // 4), the 128-byte swizzle.
        // A parity wait tells a stage's last use from the one before only: a
        // warp that waits for stage j (counted over all uses) must know that
        // j - 2 * ST was consumed. It waited for j - kLoaders, so everything
        // up to j - kLoaders - ST was: hence kLoaders <= ST.
        const int c = lane & 7;
        RingPos st, iq;
        int next = warp - 3;  // this warp's next stage, counted from the piece's first
        st.skip(next, ST);
        bool ok = true;
        while (ok) {
            if (!(ok = warp_wait(&info_full[iq.i], iq.ph, abort_flag))) break;
            const Info *inf = info + iq.i;
            const int all = inf->n;
            // this CTA's rows are columns [col0, col0 + n)
            const int n = PAIR ? all / 2 : all, col0 = (int)rank * n;
            if (all >= 0) {
                const int count = (p.num_kb + SUB - 1) / SUB;
                for (; next < count; next += kLoaders) {
                    if (!(ok = warp_wait(&empty[st.i], st.ph ^ 1u, abort_flag))) break;
                    const uint32_t base = ring + (uint32_t)st.i * p.stage_bytes;
                    const int kb = next * SUB;
                    // MXFP4: this lane's columns' scales of the stage. Where rows
                    // can be read in wider pieces they pass through registers,
                    // requested before the rows are copied and stored after:
                    // a gather of 32 rows costs the load unit 32 cycles
                    // whatever its width, and 4-byte copies take four for the
                    // 16 bytes of a stage (MXFP4 up, 16384 tokens: a
                    // tenth longer with those than with 16-byte loads).
                    constexpr int kSets = MX ? kCols / 32 : 1, kWords = 2 * SUB;
                    uint32_t scale[kSets][kWords];
                    int srow[kSets];
                    if constexpr (MX) {
#pragma unroll
                        for (int j = 0; j < kSets; ++j) {
                            srow[j] = lane + 32 * j < all ? inf->row[lane + 32 * j] : -1;
#pragma unroll
                            for (int q = 0; q < kWords; ++q) scale[j][q] = 0u;
                        }
                        if (p.scale_bytes > 4) {
#pragma unroll
                            for (int j = 0; j < kSets; ++j) {
                                const uint32_t *src = reinterpret_cast<const uint32_t *>(p.x_scales) +
                                                      (uint64_t)(uint32_t)srow[j] * (uint32_t)p.num_chunks + 2 * kb;
                                if (kWords == 4 && p.scale_bytes == 16) {
                                    ld_cg_16(scale[j], src, srow[j]);
                                } else {
#pragma unroll
                                    for (int q = 0; q < kWords; q += 2)
                                        ld_cg_8(scale[j] + q, src + q, 2 * kb + q < p.num_chunks ? srow[j] : -1);
                                }
                            }
                        }
                    }
                    // (chunks past the row's end are not read by the last MMA steps)
                    const int off = kb * kFfRowBytes + c * 16, ends = p.x_bytes;
                    const uint8_t *x = p.x + off;
                    // 4 rows a step and group of eight lanes
#pragma unroll 4
                    for (int r = 4 * (lane >> 3); r < n; r += 16) {
                        const int4 at = *reinterpret_cast<const int4 *>(inf->row + col0 + r);
                        const int row[4] = {at.x, at.y, at.z, at.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint8_t *from = x + (uint64_t)(uint32_t)row[j] * p.x_row_bytes;
                            const uint32_t to = base + x_off + (uint32_t)((r + j) * kFfRowBytes + ((c ^ ((r + j) & 7)) << 4));
#pragma unroll
                            for (int u = 0; u < SUB; ++u)
                                cp_async_16(to + u * p.b_bytes, from + u * kFfRowBytes, off + u * kFfRowBytes < ends ? row[j] : -1);
                        }
                    }
                    if constexpr (MX) {
                        // scale of column r, block q of a 128-value piece: byte
                        // (r % 32) * 16 + (r / 32) * 4 + q of its 512
                        const uint32_t sd = base + xs_off + lane * 16;
                        const int pieces = min(kWords, p.num_chunks - 2 * kb);
                        if (p.scale_bytes > 4) {
#pragma unroll
                            for (int q = 0; q < kWords; ++q)  // (kSets = 4)
                                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                                             ::"r"(sd + q * kSfAtom), "r"(scale[0][q]), "r"(scale[1][q]),
                                               "r"(scale[2][q]), "r"(scale[3][q]) : "memory");
                        } else {
#pragma unroll
                            for (int j = 0; j < kSets; ++j) {
                                const uint8_t *src = p.x_scales + ((uint64_t)(uint32_t)srow[j] * (uint32_t)p.num_chunks + 2 * kb) * 4;
#pragma unroll
                                for (int q = 0; q < kWords; ++q)
                                    cp_async_4(sd + q * kSfAtom + j * 4, src + 4 * q, q < pieces ? srow[j] : -1);
                            }
                        }
                    }
                    asm volatile("cp.async.wait_all;" ::: "memory");
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) {
                        if constexpr (PAIR) mbar_arrive_cluster(cluster_addr(smem_u32(&full[st.i]), 0u));
                        else mbar_arrive(smem_u32(&full[st.i]));
                    }
                    st.skip(kLoaders, ST);
                }
                next -= count;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&info_empty[iq.i]));
            iq.next(kFfInfos);
            if (all < 0) break;
        }
        __syncwarp();
    } else {
        // --------------------------------------------------- epilogue ----
        // four warps, one a quarter of TMEM's lanes, take every other 16
        // columns, the other four the rest
        const int q = warp & 3, half = warp < 3 + kLoaders + 4 ? 0 : 1;
        RingPos iq, ac;
        // this half's blocks, and this thread's place in one for the four
        // matrices of a store: 16 features x 16 columns, or 32 x 8
        const uint32_t blocks = smem_u32(out_rows) + (uint32_t)(half * 2 * kOutCols<UP> * kOutPitch<UP>);
        const uint32_t put = UP ? (uint32_t)((8 * (lane >> 4) + (lane & 7)) * kOutPitch<UP> + q * 32 + ((lane >> 3) & 1) * 16)
                                : (uint32_t)((lane & 7) * kOutPitch<UP> + q * 64 + (lane >> 3) * 16);
        uint32_t buf = 0;
        while (true) {
            bool ok = warp_wait(&info_full[iq.i], iq.ph, abort_flag);
            const Info *inf = info + iq.i;
            const int n = ok ? inf->n : -1;
            if (n >= 0) ok = warp_wait(&acc_full[ac.i], ac.ph, abort_flag);
            // the four warps go on together, or none does
            if constexpr (!F32) ok = meet_if(1 + half, ok);
            if (!ok || n < 0) break;
            tc_fence_after();
            const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(ac.i * p.acc_cols);
            uint32_t v[16], next[16];
            if constexpr (F32) {
                if (16 * half < n) {
                    tmem_ld16_async(acc + (uint32_t)(16 * half), v);
                    tmem_wait_ld16(v);
                }
                // this lane's store: 4 features from f of column (lane & 3) of every four
                const int f = inf->nt * kFfRows + q * 32 + (lane & 28);
                const bool f_ok = f < p.feat;  // (feat is a multiple of 16)
                for (int c0 = 16 * half; c0 < n; c0 += 32) {
                    if (c0 + 32 < n) tmem_ld16_async(acc + (uint32_t)(c0 + 32), next);
                    int i[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) i[j] = inf->slot[c0 + 4 * j + (lane & 3)];
                    float4 s[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        s[j] = quad_turn(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1]),
                                         __uint_as_float(v[4 * j + 2]), __uint_as_float(v[4 * j + 3]), lane);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (i[j] >= 0 && f_ok)
                            *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + f + (int64_t)i[j] * p.feat) = s[j];
                    if (c0 + 32 < n) {
                        tmem_wait_ld16(next);
#pragma unroll
                        for (int j = 0; j < 16; ++j) v[j] = next[j];
                    }
                }
            } else {
                constexpr int kSteps = 16 / kOutCols<UP>;
                uint32_t o[UP ? 4 : 8];
                if (16 * half < n) {
                    tmem_ld_frags_async(acc + (uint32_t)(16 * half), v);
                    tmem_wait_ld16(v);
                    pack_frags<UP>(v, o);
                }
                // 16 bytes a lane: 4 columns of 128 bytes or 2 of 256
                constexpr int kLanes = kOutBytes<UP> / 16;
                const int col = 32 / kLanes * q + lane / kLanes;
                const int f = inf->nt * (kOutBytes<UP> / 2) + lane % kLanes * 8;
                const bool f_ok = f < p.feat;  // (feat is a multiple of 16)
                uint16_t *out = static_cast<uint16_t *>(p.out) + f;
                for (int c0 = 16 * half; c0 < n; c0 += 32) {
                    if (c0 + 32 < n) tmem_ld_frags_async(acc + (uint32_t)(c0 + 32), next);
                    uint4 w[kSteps];
                    int i[kSteps];
#pragma unroll
                    for (int b = 0; b < kSteps; ++b) {
                        const uint32_t at = blocks + buf * (kOutCols<UP> * kOutPitch<UP>);
                        put_frags(at + put, o + 4 * b);
                        meet(1 + half);  // (the four have also read the block before the last one)
                        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(w[b].x), "=r"(w[b].y), "=r"(w[b].z), "=r"(w[b].w)
                                     : "r"(at + (uint32_t)(col * kOutPitch<UP> + lane % kLanes * 16)) : "memory");
                        i[b] = inf->slot[c0 + b * kOutCols<UP> + col];
                        buf ^= 1u;
                    }
                    // the next columns are computed while these are on their way from shared memory
                    if (c0 + 32 < n) {
                        tmem_wait_ld16(next);
                        pack_frags<UP>(next, o);
                    }
#pragma unroll
                    for (int b = 0; b < kSteps; ++b)
                        if (i[b] >= 0 && f_ok) *reinterpret_cast<uint4 *>(out + (int64_t)i[b] * p.feat) = w[b];
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (PAIR) mbar_arrive_cluster(cluster_addr(smem_u32(&acc_empty[ac.i]), 0u));
                else mbar_arrive(smem_u32(&acc_empty[ac.i]));
                mbar_arrive(smem_u32(&info_empty[iq.i]));
            }
            ac.next(2);
            iq.next(kFfInfos);
        }
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    if (*abort_flag && warp == 0 && lane == 0) {
        // a wait gave up: the piece's outputs are not written; weights still in
        // flight land before the CTA leaves
        ffn_error(p.err, kErrWaitTimeout);
        if (rank == 0)
            for (int j = issued - ST > 0 ? issued - ST : 0; j < issued; ++j) {
                volatile int drain = 0;
                mbar_wait_bounded(smem_u32(&full[j % ST]), (uint32_t)(j / ST) & 1u, &drain);
            }
    }
    if constexpr (PAIR) {
        // no barrier of either CTA can still be signalled, both are done with TMEM
        __syncwarp();
        cluster_sync();
        if (warp == 1) {
            tc_fence_after();
            tmem_dealloc_pair(tmem, (uint32_t)p.tmem_cols);
        }
    } else if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, (uint32_t)p.tmem_cols);
    }
}

// ------------------------------------------------------------- combine --
//
// out[t] = sum over the token's slots s, in order, of w[t, s] * y[t, s], in
// fp32, rounded once. Bound by reading y (16384 tokens, 8 slots, 2048
// features: 82 us, 7.4 TB/s with the output). One thread per 8 features of one
// token, its slots' rows requested 8 at a time. A slot whose id no expert has
// contributes nothing (the align skipped it, so its row of y was not written).
// The ids and weights come from kernels before the product, which lets this
// grid start only after it waited for them: they are read while the product
// still runs.
// Y32: y is fp32, else bf16 (half the bytes, one more rounding of each term:
// the error against 64 bits grows from 0.0017 to 0.0024 of the result; a caller
// can have fp32 rows at any number of them).
// Blocks of 128 threads fit beside a CTA of every variant of the product, so
// that they are resident before it ends (pairs in MXFP4 leave 11776 of 65536
// registers, blocks of 128 rows and pairs in bf16 13312: 256 threads of 64 do
// not fit there). The whole second product in us with 128 and 256: one token
// 9.95 and 10.4, 8 tokens in MXFP4 20.1 and 20.6, 700 tokens in blocks of 64
// rows 74.8 and 75.3, of 128 rows 74.3 and 74.6 (MXFP4 28.3 and 28.6), 2000
// tokens over 512 experts of 4096 features 422 and 424 (MXFP4 171 and 172).
// (The kernel is compiled for 256 threads: for 128 the compiler keeps fewer of
// the fp32 rows' loads ahead, 512 tokens 88.0 us instead of 86.4.)
constexpr int kCombineThreads = 128;
template <bool Y32>
__global__ void __launch_bounds__(2 * kCombineThreads)
expert_combine_kernel(const void *__restrict__ y, const int32_t *__restrict__ ids, const float *__restrict__ wts,
                      uint16_t *__restrict__ out, int parts, int width, int H, int num_logical) {
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t t = blockIdx.x / (unsigned)parts;
    const int f = ((int)(blockIdx.x % (unsigned)parts) * (int)blockDim.x + (int)threadIdx.x) * 8;
    ids += t * width;
    wts += t * width;
    const uint8_t *row = static_cast<const uint8_t *>(y) + (t * width * H + f) * (Y32 ? 4 : 2);
    const int64_t next = (int64_t)H * (Y32 ? 4 : 2);
    constexpr int kAhead = Y32 ? 4 : 8;  // slots whose rows are requested at once
    float acc[8] = {};
    for (int s0 = 0; s0 < width; s0 += 32) {
        const int s = s0 + lane;
        const bool use = s < width && (uint32_t)__ldcg(ids + s) < (uint32_t)num_logical;
        const float w = use ? __ldcg(wts + s) : 0.0f;
        uint32_t left = __ballot_sync(0xffffffffu, use);
        if (s0 == 0) griddep_wait();
        while (left != 0u) {
            uint4 x[kAhead * (Y32 ? 2 : 1)];
            float wx[kAhead];
            int n = 0;
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int at = left != 0u ? __ffs(left) - 1 : -1;
                wx[j] = __shfl_sync(0xffffffffu, w, at < 0 ? 0 : at);
                const uint8_t *from = row + (int64_t)(s0 + at) * next;
                if (at >= 0 && f < H) {
                    if constexpr (Y32) {
                        x[2 * j] = ld_stream_rows_v4(from);
                        x[2 * j + 1] = ld_stream_rows_v4(from + 16);
                    } else {
                        x[j] = ld_stream_rows_v4(from);
                    }
                }
                n += at >= 0;
                left &= left - 1u;
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                if (j >= n || f >= H) break;
                float v[8];
                if constexpr (Y32) {
                    const uint4 a = x[2 * j], b = x[2 * j + 1];
                    const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(u[i]);
                } else {
                    unpack8(x[j], v);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[i] = fmaf(wx[j], v[i], acc[i]);
            }
        }
    }
    if (f >= H) return;
    uint32_t o[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) o[u] = pack_bf16x2(acc[2 * u], acc[2 * u + 1]);
    *reinterpret_cast<uint4 *>(out + t * H + f) = make_uint4(o[0], o[1], o[2], o[3]);
}

// ---------------------------------------------------------------- host --

// CTA pairs from this many rows an expert, on average: a pair halves the rows
// that each CTA loads and that its MMAs read, but has only half as many items
// to share out. With pairs and without (us on the device, 128 experts, tokens
// of 8 slots): gated product in bf16, 16384 tokens 500 and 799, 1024 skewed
// tokens (64 rows an expert) 135 and 157, evenly spread 136 and 136, 768 tokens
// (48 rows) 133 and 146, evenly spread 135 and 128; in MXFP4, 16384 tokens 187
// and 262, 1024 tokens 44.8 and 48.9 skewed, 41.1 and 40.8 evenly spread. Second
// product in bf16, 16384 tokens 395 and 560, 1024 skewed tokens 84.7 and 94.8;
// in MXFP4 (K = 768, where the loaders bound both) 340 and 334, 38.9 and 40.1.
constexpr int kPairRows = 48;
static bool use_pairs(int64_t numel, int num_experts) { return numel >= (int64_t)kPairRows * num_experts; }

// Few enough to stay in L2 (32 MB), and no more than a pair's worth of rows an
// expert (see smr_expert_down_workspace_size for what more of them cost).
bool expert_rows_fp32(int64_t numel, int num_experts, int H) {
    return numel * H <= (int64_t)1 << 23 && !use_pairs(numel, num_experts);
}

static int sm_count() {
    static std::atomic<int> cached[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
    int n = cached[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        cached[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

cudaError_t expert_error_word(void **ptr) { return cudaGetSymbolAddress(ptr, g_expert_error); }

// cuTensorMapEncodeTiled, looked up once (a function-local static).
static PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) !=
                cudaSuccess || q != cudaDriverEntryPointSuccess)
            ptr = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    }();
    return fn;
}

static bool encode(CUtensorMap *map, CUtensorMapDataType type, int rank, const void *ptr, const cuuint64_t *dims,
                   const cuuint64_t *strides, const cuuint32_t *box, CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
    const auto fn = tensor_map_encoder();
    const cuuint32_t unit[5] = {1, 1, 1, 1, 1};
    return fn && fn(map, type, (cuuint32_t)rank, const_cast<void *>(ptr), dims, strides, box, unit,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool MX, bool UP, bool PAIR, int SUB, bool F32 = false>
static cudaError_t launch_product(const FfnLaunch &a, int sms, cudaStream_t stream) {
    FfParams p{};
    const int per_block = MX ? 256 : 64, step = MX ? 64 : 16;  // values of K in a k-block, in an MMA
    p.num_kb = (a.K + per_block - 1) / per_block;
    p.last_steps = (a.K - (p.num_kb - 1) * per_block + step - 1) / step;
    p.feat = a.feat;
    p.ntiles = UP ? (a.feat + 63) / 64 : (a.feat + kFfRows - 1) / kFfRows;
    p.div_shift = 30;
    while ((1ll << (p.div_shift - 30)) < a.width) ++p.div_shift;
    p.div_mul = (uint32_t)(((1ull << p.div_shift) + (uint64_t)a.width - 1) / (uint64_t)a.width);
    p.num_experts = a.num_experts;
    p.A = a.A;
    p.numel = (int)a.numel;
    p.sorted_cap = a.sorted_cap;
    p.max_blocks = (int)((a.sorted_cap + a.A - 1) / a.A);
    p.sorted = a.sorted;
    p.eids = a.eids;
    p.npp = a.npp;
    p.out = a.out;
    p.x_scales = a.x_scales;
    p.w_scales = a.w_scales;
    p.num_chunks = a.K / 128;
    const uintptr_t scales_at = reinterpret_cast<uintptr_t>(a.x_scales) | (uintptr_t)(4 * p.num_chunks);
    p.scale_bytes = scales_at % 16 == 0 ? 16 : (scales_at % 8 == 0 ? 8 : 4);
    p.err = &reinterpret_cast<WsHeader *>(a.hdr)->error;
    constexpr int kCols = kFfCols<MX, PAIR>;
    p.b_bytes = (uint32_t)(PAIR ? kCols / 2 : a.A) * kFfRowBytes;
    p.stage_bytes = SUB * (kFfWBytes + p.b_bytes + (MX ? 4 * kSfAtom : 0));
    constexpr uint32_t kSmemMax = 232448;
    constexpr int kMisc = kFfMiscBytes<MX, PAIR> + kFfOutBytes<UP, F32>;
    p.stages = (int)((kSmemMax - 1024 - kMisc) / p.stage_bytes);
    if (p.stages > kFfMaxStages) p.stages = kFfMaxStages;
    if (p.stages < kFfLoaders<SUB>) return cudaErrorNotSupported;  // (see the row loaders; never with these sizes)
    p.acc_cols = PAIR ? kCols : a.A;
    const int cols = 2 * p.acc_cols + (MX ? 32 : 0);
    p.tmem_cols = cols <= 128 ? 128 : (cols <= 256 ? 256 : 512);
    const size_t smem = 1024 + (size_t)p.stages * p.stage_bytes + kMisc;

    const CUtensorMapDataType type = MX ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const cuuint64_t k_elems = (cuuint64_t)(MX ? a.K / 2 : a.K), k_bytes = MX ? k_elems : 2 * k_elems;
    const cuuint32_t box_k = MX ? kFfRowBytes : kFfRowBytes / 2;
    CUtensorMap mw;
    bool ok;
    if (UP) {
        const cuuint64_t I = (cuuint64_t)a.feat;
        const cuuint64_t dims[5] = {k_elems, 16, 2, I / 16, (cuuint64_t)a.num_experts};
        const cuuint64_t strides[4] = {k_bytes, I * k_bytes, 16 * k_bytes, 2 * I * k_bytes};
        const cuuint32_t box[5] = {box_k, 16, 2, 4, 1};
        ok = encode(&mw, type, 5, a.w, dims, strides, box);
    } else {
        const cuuint64_t dims[3] = {k_elems, (cuuint64_t)a.feat, (cuuint64_t)a.num_experts};
        const cuuint64_t strides[2] = {k_bytes, (cuuint64_t)a.feat * k_bytes};
        const cuuint32_t box[3] = {box_k, kFfRows, 1};
        ok = encode(&mw, type, 3, a.w, dims, strides, box);
    }
    // a weight's tiled scales: pieces of 512 bytes
    CUtensorMap ms{};
    if (MX && PAIR && ok) {
        const cuuint64_t dims[2] = {kSfAtom / 4, (cuuint64_t)a.num_experts * p.ntiles * p.num_chunks};
        const cuuint64_t strides[1] = {kSfAtom};
        const cuuint32_t box[2] = {kSfAtom / 4, 2 * SUB};
        ok = encode(&ms, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, a.w_scales, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE);
    }
    if (!ok) return cudaErrorInvalidValue;
    p.x = static_cast<const uint8_t *>(a.x);
    p.x_bytes = (int)k_bytes;
    p.x_row_bytes = MX ? (uint32_t)k_bytes : (uint32_t)(a.ld_x * 2);

    static std::atomic<bool> configured[kMaxDevices];
    const cudaError_t e = once_per_device(configured, [](int) {
        cudaError_t r = cudaFuncSetAttribute(expert_ffn_kernel<MX, UP, PAIR, SUB, F32>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)kSmemMax);
        if (r == cudaSuccess)
            r = cudaFuncSetAttribute(expert_ffn_kernel<MX, UP, PAIR, SUB, F32>, cudaFuncAttributePreferredSharedMemoryCarveout,
                                     cudaSharedmemCarveoutMaxShared);
        return r;
    });
    if (e != cudaSuccess) return e;
    // one CTA (pair) per item, at most one CTA per SM
    const int64_t most = (int64_t)p.max_blocks * (PAIR ? (p.ntiles + 1) / 2 * 2 : p.ntiles);
    const int room = PAIR ? sms / 2 * 2 : sms;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(most < room ? most : room), 1, 1);
    cfg.blockDim = dim3(kFfThreads<SUB>, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = PAIR ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, expert_ffn_kernel<MX, UP, PAIR, SUB, F32>, mw, ms, p);
}

template <bool MX, bool UP>
static cudaError_t launch_format(const FfnLaunch &a, int sms, cudaStream_t stream) {
    const bool pairs = use_pairs(a.numel, a.num_experts);
    if constexpr (!UP)
        if (a.out32 && pairs) return launch_product<MX, UP, true, MX ? 2 : 1, true>(a, sms, stream);
    if (pairs) return launch_product<MX, UP, true, MX ? 2 : 1>(a, sms, stream);
    if constexpr (!UP)
        if (a.out32)
            return a.A == 64 ? launch_product<MX, UP, false, 2, true>(a, sms, stream)
                             : launch_product<MX, UP, false, 1, true>(a, sms, stream);
    return a.A == 64 ? launch_product<MX, UP, false, 2>(a, sms, stream) : launch_product<MX, UP, false, 1>(a, sms, stream);
}

cudaError_t launch_expert_product(const FfnLaunch &a, cudaStream_t stream) {
    const int sms = sm_count();
    if (sms < 2) return cudaErrorInvalidDevice;
    if (a.x_scales != nullptr)
        return a.gated ? launch_format<true, true>(a, sms, stream) : launch_format<true, false>(a, sms, stream);
    return a.gated ? launch_format<false, true>(a, sms, stream) : launch_format<false, false>(a, sms, stream);
}

cudaError_t launch_expert_combine(const CombineLaunch &a, cudaStream_t stream) {
    const int vecs = a.H / 8, threads = vecs < kCombineThreads ? (vecs + 31) / 32 * 32 : kCombineThreads;
    const int parts = (vecs + threads - 1) / threads;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.T * (unsigned)parts, 1, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, a.y32 ? expert_combine_kernel<true> : expert_combine_kernel<false>, a.y, a.ids,
                              a.wts, a.out, parts, a.width, a.H, a.num_logical);
}

}  // namespace smr
