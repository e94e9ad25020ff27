// smr_mxfp4.cu -- MXFP4: quantisation, its inverse, and the one-off layout of
// a weight's block scales for the block-scaled products.
//
// Format (OCP microscaling): blocks of 32 consecutive values of a row share a
// scale 2^e held as the byte e + 127 (E8M0); a value is a 4-bit code (E2M1:
// sign, then 0, 0.5, 1, 1.5, 2, 3, 4, 6), two to a byte, the even one in the
// low half. Here e is the smallest exponent with amax <= 6 * 2^e, so no value
// saturates ("vLLM #60833 --monokernel decode", Details: dynamic MXFP4 with
// scales rounded up). It is read off amax's own bits: amax = m * 2^p with m in
// [1, 2) gives e = p - 2 for m <= 1.5, else p - 1. Scaling by 2^-e is exact,
// so the one rounding is the code's (nearest, ties to the even code).
#include "smr_device.cuh"
#include "smr_launch.h"

namespace smr {

constexpr int kMxThreads = 256;
constexpr int kMxVecs = 4;  // 16-byte vectors a thread has in flight

// Two fp32 values to E2M1 codes in one byte, lo in the low half; nearest,
// ties to even.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
    uint32_t r;
    asm("{\n .reg .b8 b;\n cvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n cvt.u32.u8 %0, b;\n}" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Bound by memory: 2 bytes read and 17/32 written per value. One 16-byte load
// per 8 values, 4 neighbouring lanes share a block; kMxVecs independent loads
// a thread cover the latency. vecs_per_row: K / 8, 0 when the rows have no gap
// between them (ld == K). A block holding a NaN or an infinity gets the NaN scale (byte
// 255) and zero codes; zeros get byte 0 and codes +-0.
__global__ void __launch_bounds__(kMxThreads)
quantize_mxfp4_kernel(const uint16_t *__restrict__ x, int64_t ld, uint32_t vecs_per_row, uint32_t vecs,
                      uint8_t *__restrict__ codes, uint8_t *__restrict__ scales) {
    griddep_wait();
    griddep_launch_dependents();
    const uint32_t first = blockIdx.x * (kMxThreads * kMxVecs) + threadIdx.x;
    uint4 v[kMxVecs];
#pragma unroll
    for (int j = 0; j < kMxVecs; ++j) {
        const uint32_t i = first + j * kMxThreads;
        // rows without a gap between them are one long row
        const uint32_t row = vecs_per_row ? i / vecs_per_row : 0u;
        v[j] = i < vecs ? ld_stream_rows_v4(x + (int64_t)row * ld + (int64_t)(i - row * vecs_per_row) * 8)
                        : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int j = 0; j < kMxVecs; ++j) {
        const uint32_t i = first + j * kMxThreads;
        const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
        // the largest magnitude's bf16 bits: as unsigned integers magnitudes
        // order like their values, with infinities and NaN above all
        uint32_t m = 0u;
#pragma unroll
        for (int u = 0; u < 4; ++u) m = max(m, max(w[u] & 0x7FFFu, (w[u] >> 16) & 0x7FFFu));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        uint32_t byte = 0u;
        const bool bad = m >= 0x7F80u;
        if (bad) {
            byte = 255u;
        } else if (m >= 0x0080u) {  // normal: exponent field p + 127, 7 fraction bits
            const int e = (int)(m >> 7) - 127 - ((m & 0x7Fu) <= 0x40u ? 2 : 1);
            byte = (uint32_t)(max(e, -127) + 127);
        }  // a subnormal bf16 is below 2^-126 <= 6 * 2^-127
        // 2^-e, e in [-127, 126], as a float's bits (2^-126 at the least: normal)
        const float inv = __uint_as_float((254u - (bad ? 127u : byte)) << 23);
        uint32_t c = 0u;
#pragma unroll
        for (int u = 0; u < 4; ++u)
            c |= e2m1x2(__uint_as_float(w[u] << 16) * inv, __uint_as_float(w[u] & 0xFFFF0000u) * inv) << (8 * u);
        if (i < vecs) {
            reinterpret_cast<uint32_t *>(codes)[i] = bad ? 0u : c;
            if ((i & 3) == 0) scales[i >> 2] = (uint8_t)byte;
        }
    }
}

// Four E2M1 codes (16 bits) as two pairs of bf16: the eight magnitudes' high
// and low bytes are picked from tables by the codes' low three bits, the sign
// is moved over.
__device__ __forceinline__ uint2 e2m1x4_bf16(uint32_t c) {
    const uint32_t m = c & 0x7777u;
    const uint32_t hi = __byte_perm(0x3F3F3F00u, 0x40404040u, m), lo = __byte_perm(0xC0800000u, 0xC0804000u, m);
    const uint32_t s01 = (c << 12 & 0x8000u) | (c << 24 & 0x80000000u), s23 = (c << 4 & 0x8000u) | (c << 16 & 0x80000000u);
    return make_uint2(__byte_perm(lo, hi, 0x5140) | s01, __byte_perm(lo, hi, 0x7362) | s23);
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&a), *reinterpret_cast<const __nv_bfloat162 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// Bound by memory like the quantisation: 4 bytes of codes to 8 bf16 values a
// step, times the scale in bf16 (exact: a value has two significant bits, and
// the smallest, 2^-128, is still a subnormal bf16; byte 255 is NaN). Table
// look-ups and paired products, as the arithmetic of one fp32 product a value
// takes longer than the memory (16384 x 4096: 26.3 us, 6.4 TB/s).
__global__ void __launch_bounds__(kMxThreads)
dequantize_mxfp4_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales, uint32_t vecs,
                        uint16_t *__restrict__ out) {
    griddep_wait();
    griddep_launch_dependents();
    const uint32_t first = blockIdx.x * (kMxThreads * kMxVecs) + threadIdx.x;
    uint32_t c[kMxVecs], b[kMxVecs];
#pragma unroll
    for (int j = 0; j < kMxVecs; ++j) {
        const uint32_t i = first + j * kMxThreads;
        c[j] = i < vecs ? __ldcg(reinterpret_cast<const uint32_t *>(codes) + i) : 0u;
        b[j] = i < vecs ? __ldcg(scales + (i >> 2)) : 0u;
    }
#pragma unroll
    for (int j = 0; j < kMxVecs; ++j) {
        const uint32_t i = first + j * kMxThreads;
        if (i >= vecs) continue;
        const uint32_t h = b[j] == 255u ? 0x7FC0u : (b[j] == 0u ? 0x0040u : b[j] << 7), s = h | (h << 16);
        const uint2 lo = e2m1x4_bf16(c[j] & 0xFFFFu), hi = e2m1x4_bf16(c[j] >> 16);
        reinterpret_cast<uint4 *>(out)[i] =
            make_uint4(mul_bf16x2(lo.x, s), mul_bf16x2(lo.y, s), mul_bf16x2(hi.x, s), mul_bf16x2(hi.y, s));
    }
}

// Row-major scales [E, N, K / 32] to the products' order: per expert and tile
// of 128 weight rows, per 128 values of K a 512-byte piece, byte
// (r % 32) * 16 + (r / 32) * 4 + q = block q of tile row r, which is the layout
// that the tensor core's scale columns are filled from. gated: N = 2 I rows
// (gate, then up); a tile holds 64 features, tile row 32 g + 16 u + i = row
// u * I + 64 * tile + 16 g + i. Rows past the end: zero bytes (their weights
// are read as zeros). Run once per weight; one thread per 4 bytes.
__global__ void __launch_bounds__(kMxThreads)
tile_mxfp4_scales_kernel(const uint32_t *scales, int N, int chunks, int ntiles, int gated,
                         int64_t words, uint32_t *__restrict__ tiled) {
    griddep_wait();
    griddep_launch_dependents();
    const int64_t at = (int64_t)blockIdx.x * kMxThreads + threadIdx.x;
    if (at >= words) return;
    const int in = (int)(at & 127), r = (in & 3) * 32 + (in >> 2);
    const int64_t piece = at >> 7;
    const int c = (int)(piece % chunks);
    const int64_t et = piece / chunks;
    const int t = (int)(et % ntiles);
    const int64_t e = et / ntiles;
    int64_t row;
    bool ok;
    if (gated) {
        const int f = t * 64 + (r >> 5) * 16 + (r & 15), I = N / 2;
        ok = f < I;
        row = (int64_t)((r >> 4) & 1) * I + f;
    } else {
        row = (int64_t)t * 128 + r;
        ok = row < N;
    }
    tiled[at] = ok ? __ldcg(scales + (e * N + row) * chunks + c) : 0u;  // (may come from the kernel before)
}

template <typename... P, typename... Q>
static cudaError_t launch_flat(void (*kernel)(P...), int64_t blocks, cudaStream_t stream, Q... args) {
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks, 1, 1);
    cfg.blockDim = dim3(kMxThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

cudaError_t launch_quantize_mxfp4(const uint16_t *x, int64_t rows, int K, int64_t ld, uint8_t *codes, uint8_t *scales,
                                  cudaStream_t stream) {
    const int64_t vecs = rows * (K / 8);
    return launch_flat(quantize_mxfp4_kernel, (vecs + kMxThreads * kMxVecs - 1) / (kMxThreads * kMxVecs), stream, x, ld,
                       (uint32_t)(ld == K ? 0 : K / 8), (uint32_t)vecs, codes, scales);
}

cudaError_t launch_dequantize_mxfp4(const uint8_t *codes, const uint8_t *scales, int64_t rows, int K, uint16_t *out,
                                    cudaStream_t stream) {
    const int64_t vecs = rows * (K / 8);
    return launch_flat(dequantize_mxfp4_kernel, (vecs + kMxThreads * kMxVecs - 1) / (kMxThreads * kMxVecs), stream,
                       codes, scales, (uint32_t)vecs, out);
}

cudaError_t launch_tile_mxfp4_scales(const uint8_t *scales, int E, int N, int K, bool gated, uint8_t *tiled,
                                     cudaStream_t stream) {
    const int ntiles = mxfp4_weight_tiles(N, gated), chunks = K / 128;
    const int64_t words = (int64_t)E * ntiles * chunks * 128;
    return launch_flat(tile_mxfp4_scales_kernel, (words + kMxThreads - 1) / kMxThreads, stream,
                       reinterpret_cast<const uint32_t *>(scales), N, chunks, ntiles, gated ? 1 : 0, words,
                       reinterpret_cast<uint32_t *>(tiled));
}

}  // namespace smr
