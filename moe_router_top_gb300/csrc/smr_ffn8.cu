// smr_ffn8.cu -- the experts' products on E4M3 operands with one fp32 scale per
// 128 values of a row and per 128 x 128 block of a weight.
//
// y[i] = sum over the blocks b of 128 values of K of xs[i, b] ws[n, b] P_b[i, n],
// P_b the products of the codes. The scales are no powers of two, so the tensor
// core cannot apply them: each P_b is an MMA chain of its own into TMEM, and the
// epilogue's warps add it, scaled, to sums in their registers.
//
// Two forms. With few rows an expert the weights' traffic counts, and the
// kernel of the other formats (smr_ffn.cuh: weights as the MMA's rows, the
// routed rows its columns) streams them once whatever the rows. With many the
// scaling counts: there a column's scale is different for every column, read
// from shared memory by all threads, and these reads bound the kernel (16384
// tokens, gated product: 787 us). So here the routed rows are the MMA's rows: a
// thread of the epilogue holds one row, its scale is one register, and a weight
// tile's is the same for all.
#include "smr_ffn.cuh"

namespace smr {

// Rows of K: 256 a CTA pair (blocks of one expert together), 256 weight rows,
// 128 of each in either CTA. 16 warps: 0 weights, 1 MMAs, 2 scout, 4 to 7 load
// the routed rows (32 each), the last 8 are the epilogue, two for each quarter
// of TMEM's lanes (128 columns each).
constexpr int kRowLoaders = 4, kRowThreads = 512, kRowInfos = 4, kRowAccs = 2;
constexpr int kRowStageBytes = 2 * kFfWBytes;
constexpr int kRowBars = 2 * kFfMaxStages + 2 * kRowAccs + 2 * kRowInfos + 1;
constexpr int kRowBarBytes = (kRowBars * 8 + 8 + 15) / 16 * 16;
// The epilogue's outputs leave through shared memory, 128 bytes of 32 rows a
// warp at a time, so that rows are written in whole lines.
constexpr int kRowOutBytes = 8 * 32 * 128;
constexpr int kRowMiscBytes = kRowBarBytes + kRowInfos * (int)sizeof(FfInfo<256>) + kRowOutBytes + 2 * 128 * 4;

enum RowOut : int { kRowBf16 = 0, kRowF32 = 1, kRowE4m3 = 2 };

// Two warps meet; both get whether both came with ok.
__device__ __forceinline__ bool meet_two_if(int id, bool ok) {
    uint32_t all;
    asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 q, %1, 0;\n barrier.cta.red.and.pred p, %2, 64, q;\n"
                 " selp.u32 %0, 1, 0, p;\n}" : "=r"(all) : "r"((uint32_t)ok), "r"(id) : "memory");
    return all != 0;
}

// 128 bytes of every lane's row (8 pieces of 16) to the warp's buffer, then out
// in whole lines: out[r] is row r's address, nullptr: none; bytes: how much of
// the 128 there is.
__device__ __forceinline__ void put_row_lines(uint32_t buffer, const uint32_t (&v)[32], uint8_t *out, int bytes) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int c = 0; c < 8; ++c)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                     ::"r"(buffer + (uint32_t)(lane * 128 + ((c ^ (lane & 7)) << 4))), "r"(v[4 * c]), "r"(v[4 * c + 1]),
                       "r"(v[4 * c + 2]), "r"(v[4 * c + 3]) : "memory");
    __syncwarp();
    const int c = lane & 7;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = 4 * i + (lane >> 3);
        uint4 w;
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                     : "r"(buffer + (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4))) : "memory");
        uint8_t *to = reinterpret_cast<uint8_t *>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(out), r));
        if (to != nullptr && 16 * c < bytes) *reinterpret_cast<uint4 *>(to + 16 * c) = w;
    }
    __syncwarp();
}

template <bool UP, int OUT>
__global__ void __launch_bounds__(kRowThreads, 1)
expert_rows_kernel(const __grid_constant__ CUtensorMap tm_w, const FfParams p) {
    using Info = FfInfo<256>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    const int ST = p.stages;
    uint8_t *misc = smem + (size_t)ST * kRowStageBytes;
    // full and acc_empty are the leader's, the others each CTA's own
    uint64_t *full = reinterpret_cast<uint64_t *>(misc);
    uint64_t *empty = full + kFfMaxStages;
    uint64_t *acc_full = empty + kFfMaxStages;
    uint64_t *acc_empty = acc_full + kRowAccs;
    uint64_t *info_full = acc_empty + kRowAccs;
    uint64_t *info_empty = info_full + kRowInfos;
    uint64_t *last = info_empty + kRowInfos;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(last + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    Info *info = reinterpret_cast<Info *>(misc + kRowBarBytes);
    uint8_t *out_rows = misc + kRowBarBytes + kRowInfos * sizeof(Info);
    float *amax_ex = reinterpret_cast<float *>(out_rows + kRowOutBytes);  // [2][128]

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    if (threadIdx.x == 0) {
        for (int s = 0; s < ST; ++s) {
            mbar_init(smem_u32(&full[s]), 1 + 2 * kRowLoaders);  // the weights' bytes, the row loaders of both CTAs
            mbar_init(smem_u32(&empty[s]), 1);
        }
        for (int s = 0; s < kRowAccs; ++s) {
            mbar_init(smem_u32(&acc_full[s]), 1);
            mbar_init(smem_u32(&acc_empty[s]), 2 * kFfDrains);
        }
        for (int s = 0; s < kRowInfos; ++s) {
            mbar_init(smem_u32(&info_full[s]), 1);
            mbar_init(smem_u32(&info_empty[s]), 2 + kRowLoaders + kFfDrains);
        }
        mbar_init(smem_u32(last), 1);
        *abort_flag = 0;
        mbar_fence_init();
        prefetch_tensormap(&tm_w);
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(tmem_slot), 512u);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    griddep_wait();  // the align's outputs and x come from previous kernels
    griddep_launch_dependents();

    const uint32_t ring = smem_u32(smem);  // a stage: [rows][weights]
    int issued = 0;
    // A thread of the epilogue holds 128 sums: its 8 warps get registers of the
    // other 8 (256 x 64 + 256 x 192 = the 512 x 128 of the launch, which the
    // launcher makes sure of).
    if (warp < 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        if (warp == 0) {
            // ------------------------------------------------ weights ----
            const bool elected = elect_one();
            RingPos st, iq;
            bool ok = true;
            while (ok) {
                if (!(ok = warp_wait(&info_full[iq.i], iq.ph, abort_flag))) break;
                const volatile Info *inf = info + iq.i;
                const int n = inf->n, nt = inf->nt, e = inf->e;
                __syncwarp();
                if (elected) mbar_arrive(smem_u32(&info_empty[iq.i]));
                iq.next(kRowInfos);
                if (n < 0) break;
                for (int kb = 0; kb < p.num_kb; ++kb) {
                    if (!(ok = warp_wait(&empty[st.i], st.ph ^ 1u, abort_flag))) break;
                    const uint32_t to = ring + (uint32_t)(st.i * kRowStageBytes + kFfWBytes), bar = smem_u32(&full[st.i]);
                    if (elected) {
                        // both CTAs' bytes complete the leader's barrier
                        if (rank == 0) mbar_arrive_expect_tx(bar, 2 * kFfWBytes);
                        const uint32_t fb = cluster_addr(bar, 0u);
                        if constexpr (UP) tma_load_5d_pair(to, &tm_w, kb * kFfRowBytes, nt * 4, e, fb);
                        else tma_load_3d_pair(to, &tm_w, kb * kFfRowBytes, nt * kFfRows, e, fb);
                    }
                    ++issued;
                    st.next(ST);
                }
            }
            __syncwarp();
        } else if (warp == 2) {
            ff_scout<UP, true, 256, kRowInfos, 2>(p, info, info_full, info_empty, abort_flag, rank);
            __syncwarp();
        } else if (warp == 1) {
            // --------------------------------------------------- MMAs ----
            const bool elected = elect_one();
            const uint32_t idesc = idesc_e4m3(2 * kFfRows, 256);
            RingPos st, iq, ac;
            bool ok = true;
            while (ok) {
                if (!(ok = warp_wait(&info_full[iq.i], iq.ph, abort_flag))) break;
                const int n = __shfl_sync(0xffffffffu, reinterpret_cast<volatile Info *>(info)[iq.i].n, 0);
                __syncwarp();
                if (elected) mbar_arrive(smem_u32(&info_empty[iq.i]));
                iq.next(kRowInfos);
                if (n < 0) break;
                if (rank != 0) continue;
                for (int kb = 0; kb < p.num_kb; ++kb) {
                    if (!(ok = warp_wait(&full[st.i], st.ph, abort_flag))) break;
                    if (!(ok = warp_wait(&acc_empty[ac.i], ac.ph ^ 1u, abort_flag))) break;
                    tc_fence_after();
                    const uint32_t base = ring + (uint32_t)(st.i * kRowStageBytes), acc = tmem + (uint32_t)(ac.i * 256);
                    const uint64_t da = smem_desc_sw<128>(base), db = smem_desc_sw<128>(base + kFfWBytes);
                    const int steps = kb + 1 == p.num_kb ? p.last_steps : 4;
                    if (elected) {
                        if (steps == 4) {
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk) tc_mma_e4m3<true>(acc, da + 2 * kk, db + 2 * kk, idesc, kk ? 1u : 0u);
                        } else {
                            for (int kk = 0; kk < steps; ++kk) tc_mma_e4m3<true>(acc, da + 2 * kk, db + 2 * kk, idesc, kk ? 1u : 0u);
                        }
                        ff_commit<true>(&empty[st.i]);
                        ff_commit<true>(&acc_full[ac.i]);
                    }
                    st.next(ST);
                    ac.next(kRowAccs);
                }
            }
            // every MMA issued is done before TMEM is freed, also after an abort
            if (rank == 0) {
                if (elected) tc_commit_pair(smem_u32(last), 0x1);
                volatile int never = 0;
                if (!mbar_wait_bounded(smem_u32(last), 0u, &never)) *abort_flag = 1;
            }
            __syncwarp();
        } else if (warp >= 4) {
            // -------------------------------------------- routed rows ----
            // A warp copies 32 of the CTA's rows for every stage: eight lanes
            // a row, a lane the same chunk of eight rows, whose addresses it
            // keeps for the whole item. Chunk c of row r lands at r * 128 +
            // ((c ^ (r & 7)) << 4), the 128-byte swizzle. Copies of as many
            // stages as are free are under way; the oldest is waited for, made
            // visible to the tensor core and announced when the next stage is
            // not free yet, or when all are under way.
            const int c = lane & 7, r0 = 32 * (warp - 4) + (lane >> 3);  // rows r0 + 4 i
            const uint32_t to0 = ring + (uint32_t)(r0 * kFfRowBytes + ((c ^ (lane >> 3)) << 4));
            const uint32_t to1 = ring + (uint32_t)(r0 * kFfRowBytes + ((c ^ (4 + (lane >> 3))) << 4));
            RingPos st, old, iq;  // the next stage, the oldest under way
            int pending = 0;
            auto announce = [&] {
                switch (pending) {  // (all but the oldest may stay under way)
                    case 1: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
                    case 2: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
                    case 3: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
                    default: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(cluster_addr(smem_u32(&full[old.i]), 0u));
                old.next(ST);
                --pending;
            };
            auto wait_for = [&](uint64_t *bar, uint32_t parity) {
                while (pending > 0 && !__all_sync(0xffffffffu, mbar_try_wait(smem_u32(bar), parity))) announce();
                return warp_wait(bar, parity, abort_flag);
            };
            bool ok = true;
            while (ok) {
                if (!(ok = wait_for(&info_full[iq.i], iq.ph))) break;
                const Info *inf = info + iq.i;
                const int all = inf->n;
                if (all >= 0) {
                    const int n = all / 2;  // this CTA's rows of the item
                    const uint8_t *from[8];
                    uint32_t copy = 0u;  // a bit a row that there is
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int row = r0 + 4 * i < n ? inf->row[(int)rank * n + r0 + 4 * i] : -1;
                        if (row >= 0) copy |= 1u << i;
                        from[i] = p.x + (uint64_t)(uint32_t)max(row, 0) * p.x_row_bytes + c * 16;
                    }
                    int left = p.x_bytes - c * 16;  // (pieces past the row's end are not read by the last MMA steps)
                    for (int kb = 0; kb < p.num_kb; ++kb) {
                        if (!(ok = wait_for(&empty[st.i], st.ph ^ 1u))) break;
                        const uint32_t base = (uint32_t)(st.i * kRowStageBytes);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            cp_async_16((i & 1 ? to1 : to0) + base + (uint32_t)(i * 4 * kFfRowBytes), from[i],
                                        left > 0 && (copy >> i & 1u) ? 0 : -1);
                            from[i] += kFfRowBytes;
                        }
                        asm volatile("cp.async.commit_group;" ::: "memory");
                        left -= kFfRowBytes;
                        st.next(ST);
                        if (++pending == 4) announce();
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&info_empty[iq.i]));
                iq.next(kRowInfos);
                if (all < 0) break;
            }
            while (pending > 0) announce();
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
        // ------------------------------------------------------ epilogue ----
        // one row a thread: row q 32 + lane of the CTA's, columns [128 half, +
        // 128): the weight tile 2 t + half, both CTAs having the same tiles.
        // sum[32 c + j]: of a gated tile 16 gate and their 16 up values in turn
        const int q = warp & 3, half = (warp - 8) >> 2;
        RingPos iq, ac;
        const uint32_t buffer = smem_u32(out_rows) + (uint32_t)((warp - 8) * 32 * 128);
        while (true) {
            bool ok = warp_wait(&info_full[iq.i], iq.ph, abort_flag);
            const Info *inf = info + iq.i;
            const int n = ok ? inf->n / 2 : -1;  // (-1 / 2 = 0: told apart by the next line)
            const bool more = ok && inf->n >= 0;
            float sum[128];
#pragma unroll
            for (int j = 0; j < 128; ++j) sum[j] = 0.0f;
            const int r = q * 32 + lane;
            int slot = -1, tile = 0;
            if (more) {
                if (r < n) slot = inf->slot[(int)rank * n + r];
                tile = (inf->nt & ~1) + half;
                const int xrow = r < n ? inf->row[(int)rank * n + r] : -1;
                const float *xs = reinterpret_cast<const float *>(p.x_scales) + (uint64_t)(uint32_t)max(xrow, 0) * (uint32_t)p.num_kb;
                const int wrow = min(tile, p.ntiles - 1) >> (UP ? 1 : 0);
                const float *ws = reinterpret_cast<const float *>(p.w_scales) + ((int64_t)inf->e * p.scale_rows + wrow) * p.num_kb;
                const float *wu = ws + (int64_t)(p.scale_rows >> 1) * p.num_kb;  // (UP)
                // this row's scales of four k-blocks, and the next four; lane l
                // holds the tile's of k-block l of 32
                uint32_t now[4] = {}, next[4];
                auto request = [&](int kb, uint32_t (&v)[4]) {
                    const uint32_t *src = reinterpret_cast<const uint32_t *>(xs) + kb;
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[j] = 0u;
                    if (kb >= p.num_kb) return;
                    if (p.scale_bytes == 16) {
                        ld_cg_16(v, src, xrow);
                    } else if (p.scale_bytes == 8) {
                        ld_cg_8(v, src, xrow);
                        ld_cg_8(v + 2, src + 2, kb + 2 < p.num_kb ? xrow : -1);
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (xrow >= 0 && kb + j < p.num_kb) v[j] = __ldcg(src + j);
                    }
                };
                float tg = 0.0f, tu = 0.0f;
                request(0, next);
                for (int kb = 0; kb < p.num_kb; ++kb) {
                    if ((kb & 31) == 0) {
                        if (kb + lane < p.num_kb) {
                            tg = __ldcg(ws + kb + lane);
                            if (UP) tu = __ldcg(wu + kb + lane);
                        }
                        __syncwarp();
                    }
                    if ((kb & 3) == 0) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) now[j] = next[j];
                        request(kb + 4, next);
                    }
                    const float sx = __uint_as_float(kb & 2 ? (kb & 1 ? now[3] : now[2]) : (kb & 1 ? now[1] : now[0]));
                    const float g = sx * __shfl_sync(0xffffffffu, tg, kb & 31);
                    const float u = UP ? sx * __shfl_sync(0xffffffffu, tu, kb & 31) : g;
                    if (!(ok = warp_wait(&acc_full[ac.i], ac.ph, abort_flag))) break;
                    tc_fence_after();
                    const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(ac.i * 256 + half * 128);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t v[32];
                        tmem_ld32_async(acc + 32 * c, v);
                        tmem_wait_ld(v);
                        if (c == 3) {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive_cluster(cluster_addr(smem_u32(&acc_empty[ac.i]), 0u));
                        }
#pragma unroll
                        for (int j = 0; j < 32; ++j) sum[32 * c + j] = fmaf(__uint_as_float(v[j]), j < 16 ? g : u, sum[32 * c + j]);
                    }
                    ac.next(kRowAccs);
                }
            }
            if constexpr (OUT == kRowE4m3) ok = meet_two_if(1 + q, ok);  // both warps of a row go on, or none does
            if (!ok || !more) break;
            if constexpr (UP) {
                const int f = tile * 64, width = min(128, 2 * max(p.feat - f, 0));  // bytes of this tile's features in bf16
                uint32_t o[32];
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        o[8 * c + j] = pack_bf16x2(swiglu(sum[32 * c + 2 * j], sum[32 * c + 16 + 2 * j]),
                                                   swiglu(sum[32 * c + 2 * j + 1], sum[32 * c + 17 + 2 * j]));
                if constexpr (OUT == kRowBf16) {
                    uint8_t *to = slot >= 0 ? static_cast<uint8_t *>(p.out) + ((int64_t)slot * p.feat + f) * 2 : nullptr;
                    put_row_lines(buffer, o, to, width);
                }
            } else {
                constexpr int kPer = OUT == kRowF32 ? 32 : 64;  // features of 128 bytes
#pragma unroll
                for (int c = 0; c < 128 / kPer; ++c) {
                    uint32_t o[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        o[j] = OUT == kRowF32 ? __float_as_uint(sum[kPer * c + (OUT == kRowF32 ? j : 0)])
                                              : pack_bf16x2(sum[kPer * c + (OUT == kRowF32 ? 0 : 2 * j)],
                                                            sum[kPer * c + (OUT == kRowF32 ? 0 : 2 * j + 1)]);
                    const int f = tile * 128 + kPer * c;
                    uint8_t *to = slot >= 0 ? static_cast<uint8_t *>(p.out) + ((int64_t)slot * p.feat + f) * (128 / kPer) : nullptr;
                    put_row_lines(buffer, o, to, max(p.feat - f, 0) * (128 / kPer));
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&info_empty[iq.i]));
            iq.next(kRowInfos);
        }
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    if (*abort_flag && warp == 0 && lane == 0) {
        // a wait gave up: the piece's outputs are not written; weights still in
        // flight land before the CTA leaves
        ffn_error(p, kErrWaitTimeout);
        if (rank == 0)
            for (int j = issued - ST > 0 ? issued - ST : 0; j < issued; ++j) {
                volatile int drain = 0;
                mbar_wait_bounded(smem_u32(&full[j % ST]), (uint32_t)(j / ST) & 1u, &drain);
            }
    }
    // no barrier of either CTA can still be signalled, both are done with TMEM
    __syncwarp();
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512u);
    }
}

template <bool UP, int OUT>
static cudaError_t launch_rows(const FfnLaunch &a, int sms, cudaStream_t stream) {
    FfParams p{};
    p.num_kb = (a.K + 127) / 128;
    p.last_steps = (a.K - (p.num_kb - 1) * 128 + 31) / 32;
    p.feat = a.feat;
    p.ntiles = UP ? (a.feat + 63) / 64 : (a.feat + kFfRows - 1) / kFfRows;
    if (const cudaError_t e = common_params(a, p)) return e;
    p.x = static_cast<const uint8_t *>(a.x);
    p.x_bytes = a.K;
    p.x_row_bytes = (uint32_t)a.ld_x;
    p.x_scales = static_cast<const uint8_t *>(a.x_scales);
    p.w_scales = static_cast<const uint8_t *>(a.w_scales);
    const uintptr_t scales_at = reinterpret_cast<uintptr_t>(a.x_scales) | (uintptr_t)(4 * p.num_kb);
    p.scale_bytes = scales_at % 16 == 0 ? 16 : (scales_at % 8 == 0 ? 8 : 4);
    constexpr uint32_t kSmemMax = 232448;
    p.stages = (int)((kSmemMax - 1024 - kRowMiscBytes) / kRowStageBytes);
    if (p.stages > kFfMaxStages) p.stages = kFfMaxStages;
    if (p.stages < 5) return cudaErrorNotSupported;  // (more than the loaders have under way; never with these sizes)
    const size_t smem = 1024 + (size_t)p.stages * kRowStageBytes + kRowMiscBytes;
    CUtensorMap mw;
    if (!encode_weight(&mw, a, CU_TENSOR_MAP_DATA_TYPE_UINT8, (cuuint64_t)a.K, (cuuint64_t)a.K, kFfRowBytes))
        return cudaErrorInvalidValue;

    static std::atomic<bool> configured[kMaxDevices];
    const cudaError_t e = once_per_device(configured, [](int) {
        cudaFuncAttributes at;
        cudaError_t r = cudaFuncGetAttributes(&at, expert_rows_kernel<UP, OUT>);
        // (with fewer registers at launch the epilogue's wait for more would never end)
        if (r == cudaSuccess && at.numRegs != 128) r = cudaErrorNotSupported;
        if (r == cudaSuccess)
            r = cudaFuncSetAttribute(expert_rows_kernel<UP, OUT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemMax);
        if (r == cudaSuccess)
            r = cudaFuncSetAttribute(expert_rows_kernel<UP, OUT>, cudaFuncAttributePreferredSharedMemoryCarveout,
                                     cudaSharedmemCarveoutMaxShared);
        return r;
    });
    if (e != cudaSuccess) return e;
    const int64_t most = (int64_t)p.max_blocks * ((p.ntiles + 1) / 2 * 2);
    const int room = sms / 2 * 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(most < room ? most : room), 1, 1);
    cfg.blockDim = dim3(kRowThreads, 1, 1);
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
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, expert_rows_kernel<UP, OUT>, mw, p);
}

constexpr int kRowsPerExpert = 128;

template <bool UP, bool F32>
static cudaError_t launch_columns(const FfnLaunch &a, int sms, cudaStream_t stream) {
    if (expert_pairs(a.numel, a.num_experts)) return launch_product<false, UP, true, 1, F32, true>(a, sms, stream);
    return a.A == 64 ? launch_product<false, UP, false, 2, F32, true>(a, sms, stream)
                     : launch_product<false, UP, false, 1, F32, true>(a, sms, stream);
}

cudaError_t launch_expert_product_fp8(const FfnLaunch &a, int sms, cudaStream_t stream) {
    const bool rows = a.numel >= (int64_t)kRowsPerExpert * a.num_experts;
    if (a.gated) return rows ? launch_rows<true, kRowBf16>(a, sms, stream) : launch_columns<true, false>(a, sms, stream);
    if (a.out32) return rows ? launch_rows<false, kRowF32>(a, sms, stream) : launch_columns<false, true>(a, sms, stream);
    return rows ? launch_rows<false, kRowBf16>(a, sms, stream) : launch_columns<false, false>(a, sms, stream);
}

}  // namespace smr
