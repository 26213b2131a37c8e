// The int8 K/V cache: writing it with a scale per token and head, widening
// whole pages back, and copying pages with their scales ("03. KV Cache：用显存换
// 计算", KV quantisation follow-up; [HB-07] Q025 append, Q028 copy-on-write).
//
// Codes: int8 pools [num_pages][H_kv][P][Dh]; scales: fp32
// [num_pages][H_kv][2][P] (K then V), so a (page, head) pair's scales are one
// run of 8 P bytes that a decode launch fetches with a single bulk copy.
// For a row x of Dh values with a = max |x|:
//   scale = a / 127, code = rint(x * (127 / a)),  read value = code * scale,
// with both divisions and the product rounded to fp32 on their own, so the
// stored bits are fully determined. A row with a < 2^-100 (127 / a would
// overflow) is stored as zeros with scale 0; a row holding a NaN or an
// infinity gets scale NaN: it reads back as NaN, never as numbers.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "decode_launch.cuh"
#include "kvpaged.h"
#include "rope.cuh"

namespace kvp {
namespace {

// Sixteen consecutive elements of a row of type DT as fp32.
template <int DT>
__device__ __forceinline__ void load16(const uint4* src, float (&x)[16]) {
    using V = RopeVec<DT>;
#pragma unroll
    for (int i = 0; i < 16 / V::kN; ++i) V::load(src[i], x + i * V::kN);
}

// Sixteen elements of a row -> their codes, and (the same for all lanes of the row) its scale. The Dh / 16 threads of a
// row are neighbouring lanes and agree on the row's largest magnitude by shuffles, so a row is read once. Magnitudes are
// compared as integers: the pattern of a NaN is above that of infinity, which is above every finite value, so both show
// in the maximum.
__device__ __forceinline__ uint4 quantise16(const float (&x)[16], int32_t cpr, unsigned mask, float& scale) {
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 16; ++k) top = max(top, __float_as_uint(x[k]) & 0x7fffffffu);
    for (int o = cpr >> 1; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(mask, top, o));
    const float amax = __uint_as_float(top);
    const bool finite = top < 0x7f800000u;
    const bool zero = amax < 7.888609052210118e-31f;  // 2^-100
    const float inv = finite && !zero ? __fdiv_rn(127.f, amax) : 0.f;
    scale = finite ? (zero ? 0.f : __fdiv_rn(amax, 127.f)) : __uint_as_float(0x7fc00000u);
    uint32_t out[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint32_t y[4];
        // adding 1.5 * 2^23 rounds to an integer (to even) and leaves its two's complement in the low bits
#pragma unroll
        for (int j = 0; j < 4; ++j)
            y[j] = finite ? __float_as_uint(__fadd_rn(__fmul_rn(x[4 * k + j], inv), 12582912.f)) : 0u;
        out[k] = __byte_perm(__byte_perm(y[0], y[1], 0x0040), __byte_perm(y[2], y[3], 0x0040), 0x5410);
    }
    return make_uint4(out[0], out[1], out[2], out[3]);
}

// One thread takes the same sixteen elements of a token's K and V row (one 16-byte vector of codes each): four loads in
// flight, issued beside that of the slot. Bound by memory: 8185 tokens of 8 heads of 128 (bf16) take 14.7 us, 3.4 TB/s (0.52
// of the measured copy rate, at a size where a launch's start and end weigh as much as its middle); 15.4 us with a thread
// per K or V vector and the slot read first. CTAs of 128: with 256 the append and the read-back behind it take 26.4 us for
// 25.9.
// No pointer in this file is __restrict__: the kernel before may still be writing what one reads here when it starts
// (programmatic launches), so everything is read by ordinary loads behind the wait.
constexpr int kAppendThreads = 128;
template <int DT>
__global__ void __launch_bounds__(kAppendThreads) kv_append_int8_kernel(
    uint4* k_pages, uint4* v_pages, float* scales, const uint4* k_new, const uint4* v_new, int64_t k_stride, int64_t v_stride,
    const int64_t* slots, int64_t per, int32_t H_kv, int32_t lg_cpr, int32_t P, int64_t num_slots, int* err) {
    constexpr int kVec = 16 / RopeVec<DT>::kN;  // source vectors per thread and row
    grid_dependency_wait();
    if (threadIdx.x == 0) grid_launch_dependents();
    const int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
    if (i >= per) return;  // whole rows: per is a multiple of the threads per row
    const int32_t cpr = 1 << lg_cpr;
    const int64_t row = i >> lg_cpr;
    const int32_t c = static_cast<int32_t>(i) & (cpr - 1);
    const int64_t b = row / H_kv;
    const int32_t h = static_cast<int32_t>(row - b * H_kv);
    float xk[16], xv[16];
    load16<DT>(k_new + b * k_stride + ((int64_t)h * cpr + c) * kVec, xk);
    load16<DT>(v_new + b * v_stride + ((int64_t)h * cpr + c) * kVec, xv);
    const int64_t slot = slots[b];
    if (slot < 0) return;
    if (slot >= num_slots) {
        if (h == 0 && c == 0 && err) atomicOr(err, KV_DEV_ERR_SLOT);
        return;
    }
    const int lane = threadIdx.x & 31;
    const unsigned mask = (cpr == 32 ? 0xffffffffu : (1u << cpr) - 1u) << (lane & ~(cpr - 1));
    const int64_t page = slot / P, off = slot - page * P;
    const int64_t dst = ((page * H_kv + h) * P + off) * cpr + c, sdst = (page * H_kv + h) * 2 * P + off;
    float ks, vs;
    k_pages[dst] = quantise16(xk, cpr, mask, ks);
    v_pages[dst] = quantise16(xv, cpr, mask, vs);
    if (c == 0) {
        scales[sdst] = ks;
        scales[sdst + P] = vs;
    }
}

// Sixteen codes -> sixteen values of type DT.
template <int DT>
__device__ __forceinline__ void widen16(const uint4& v, float s, uint4* dst) {
    using V = RopeVec<DT>;
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float x[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) x[k] = static_cast<float>(static_cast<int8_t>(w[k >> 2] >> (8 * (k & 3)))) * s;
#pragma unroll
    for (int i = 0; i < 16 / V::kN; ++i) dst[i] = V::store(x + i * V::kN);
}

// blockIdx.x: page pair; the units (16 codes) of that page's K and V codes run
// over the threads of the blockIdx.y CTAs, four to a thread with their loads
// issued together. Bound by memory (one read of the codes, one write of the
// values): the pages of 8185 tokens of 8 heads of 128 to bf16 in 13.3 us, 3.8
// TB/s.
template <int DT>
__global__ void __launch_bounds__(256) kv_dequant_pages_int8_kernel(
    uint4* k_out, uint4* v_out, const uint4* k_pages, const uint4* v_pages, const float* scales, const int32_t* src,
    const int32_t* dst, int32_t upp, int32_t cpr, int32_t P, int32_t num_pages, int32_t num_out, int* err) {
    constexpr int kVec = 16 / RopeVec<DT>::kN, kBatch = 4;
    grid_dependency_wait();
    if (threadIdx.x == 0) grid_launch_dependents();
    const int32_t i = blockIdx.x, s = src[i], d = dst[i];
    if (s < 0 || s >= num_pages || d < 0 || d >= num_out) {
        if (threadIdx.x == 0 && blockIdx.y == 0 && err) atomicOr(err, KV_DEV_ERR_PAGE_RANGE);
        return;
    }
    // upp = units of one pool's page; its (head, slot) row is unit / cpr
    const int32_t step = gridDim.y * blockDim.x;
    for (int32_t u0 = blockIdx.y * blockDim.x + threadIdx.x; u0 < 2 * upp; u0 += kBatch * step) {
        uint4 codes[kBatch];
        float sc[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int32_t u = u0 + k * step;
            if (u >= 2 * upp) break;
            const bool is_v = u >= upp;
            const int32_t w = is_v ? u - upp : u, hp = w / cpr, h = hp / P;
            codes[k] = (is_v ? v_pages : k_pages)[(int64_t)s * upp + w];
            sc[k] = scales[2 * ((int64_t)s * (upp / cpr) + (int64_t)h * P) + (is_v ? P : 0) + (hp - h * P)];
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int32_t u = u0 + k * step;
            if (u >= 2 * upp) break;
            const bool is_v = u >= upp;
            widen16<DT>(codes[k], sc[k], (is_v ? v_out : k_out) + ((int64_t)d * upp + (is_v ? u - upp : u)) * kVec);
        }
    }
}

// Page copy with scales: 16-byte words of the K codes, the V codes and the
// scales of every pair.
__global__ void __launch_bounds__(256) kv_copy_pages_int8_kernel(uint4* k_pages, uint4* v_pages, uint4* scales,
                                                                 const int32_t* src, const int32_t* dst, int32_t n,
                                                                 int32_t code_words, int32_t scale_words,
                                                                 int32_t num_pages, int* err) {
    grid_dependency_wait();
    if (threadIdx.x == 0) grid_launch_dependents();
    for (int32_t i = blockIdx.x; i < n; i += gridDim.x) {
        const int64_t s = src[i], d = dst[i];
        if (s < 0 || s >= num_pages || d < 0 || d >= num_pages) {
            if (threadIdx.x == 0 && err) atomicOr(err, KV_DEV_ERR_PAGE_RANGE);
            continue;
        }
        for (int32_t w = threadIdx.x; w < code_words; w += blockDim.x) {
            const uint4 k = k_pages[s * code_words + w], v = v_pages[s * code_words + w];
            k_pages[d * code_words + w] = k;
            v_pages[d * code_words + w] = v;
        }
        for (int32_t w = threadIdx.x; w < scale_words; w += blockDim.x)
            scales[d * scale_words + w] = scales[s * scale_words + w];
    }
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int real_bytes(int32_t dtype) {
    return dtype == KV_DTYPE_F32 ? 4 : (dtype == KV_DTYPE_BF16 || dtype == KV_DTYPE_F16) ? 2 : 0;
}

// 16-byte code vectors of one pool's page, as an int; 0 if a page is too large for one.
int32_t page_units(int32_t H_kv, int32_t Dh, int32_t P) {
    const int64_t u = static_cast<int64_t>(H_kv) * P * (Dh / 16);
    return u < (1LL << 28) ? static_cast<int32_t>(u) : 0;
}

}  // namespace
}  // namespace kvp

using namespace kvp;

extern "C" {

int kv_append_int8(void* k_pages, void* v_pages, float* kv_scales, const void* k_new, const void* v_new,
                   int64_t k_stride, int64_t v_stride, int32_t src_dtype, const int64_t* slot_mapping, int32_t B,
                   int32_t H_kv, int32_t Dh, int32_t page_size, int32_t num_pages, int* err_flag, void* stream) {
    const int eb = real_bytes(src_dtype);
    if (B < 0 || H_kv <= 0 || Dh <= 0 || page_size <= 0 || num_pages <= 0 || eb == 0) return KV_ERR_ARG;
    if (Dh % 16 != 0 || Dh > 512 || ((Dh / 16) & (Dh / 16 - 1)) != 0) return KV_ERR_UNSUPPORTED;  // whole lanes per row
    if (B == 0) return KV_OK;
    if (!k_pages || !v_pages || !kv_scales || !k_new || !v_new || !slot_mapping) return KV_ERR_ARG;
    if (!al16(k_pages) || !al16(v_pages) || !al16(kv_scales) || !al16(k_new) || !al16(v_new)) return KV_ERR_ARG;
    const int64_t N = 16 / eb, row = static_cast<int64_t>(H_kv) * Dh;
    if (k_stride % N != 0 || v_stride % N != 0 || k_stride < row || v_stride < row) return KV_ERR_ARG;
    int32_t lg = 0;
    while ((16 << lg) < Dh) ++lg;
    const int64_t per = static_cast<int64_t>(B) * H_kv << lg;
    const int64_t blocks = (per + kAppendThreads - 1) / kAppendThreads;
    if (blocks > 0x7fffffffLL) return KV_ERR_UNSUPPORTED;
    auto run = [&](auto kernel) {
        return launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)), dim3(kAppendThreads), 0, static_cast<cudaStream_t>(stream),
                          static_cast<uint4*>(k_pages), static_cast<uint4*>(v_pages), kv_scales,
                          static_cast<const uint4*>(k_new), static_cast<const uint4*>(v_new), k_stride / N, v_stride / N,
                          slot_mapping, per, H_kv, lg, page_size, static_cast<int64_t>(num_pages) * page_size, err_flag);
    };
    const cudaError_t e = src_dtype == KV_DTYPE_BF16  ? run(kv_append_int8_kernel<KV_DTYPE_BF16>)
                          : src_dtype == KV_DTYPE_F16 ? run(kv_append_int8_kernel<KV_DTYPE_F16>)
                                                      : run(kv_append_int8_kernel<KV_DTYPE_F32>);
    return e == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}

int kv_dequant_pages_int8(void* k_out, void* v_out, int32_t out_dtype, int32_t num_out_pages, const void* k_pages,
                          const void* v_pages, const float* kv_scales, const int32_t* src_pages,
                          const int32_t* dst_pages, int32_t n, int32_t H_kv, int32_t Dh, int32_t page_size,
                          int32_t num_pages, int* err_flag, void* stream) {
    if (n < 0 || H_kv <= 0 || Dh <= 0 || page_size <= 0 || num_pages <= 0 || num_out_pages <= 0 || real_bytes(out_dtype) == 0)
        return KV_ERR_ARG;
    if (Dh % 16 != 0) return KV_ERR_UNSUPPORTED;
    const int32_t upp = page_units(H_kv, Dh, page_size);
    if (upp == 0) return KV_ERR_UNSUPPORTED;
    if (n == 0) return KV_OK;
    if (!k_out || !v_out || !k_pages || !v_pages || !kv_scales || !src_pages || !dst_pages) return KV_ERR_ARG;
    if (!al16(k_out) || !al16(v_out) || !al16(k_pages) || !al16(v_pages) || !al16(kv_scales)) return KV_ERR_ARG;
    // four units per thread of a page's K and V
    const int32_t ny = std::min(64, std::max(1, (2 * upp + 1023) / 1024));
    const dim3 grid(static_cast<unsigned>(n), static_cast<unsigned>(ny));
    auto run = [&](auto kernel) {
        return launch_pdl(kernel, grid, dim3(256), 0, static_cast<cudaStream_t>(stream), static_cast<uint4*>(k_out),
                          static_cast<uint4*>(v_out), static_cast<const uint4*>(k_pages),
                          static_cast<const uint4*>(v_pages), kv_scales, src_pages, dst_pages, upp, Dh / 16, page_size,
                          num_pages, num_out_pages, err_flag);
    };
    const cudaError_t e = out_dtype == KV_DTYPE_BF16  ? run(kv_dequant_pages_int8_kernel<KV_DTYPE_BF16>)
                          : out_dtype == KV_DTYPE_F16 ? run(kv_dequant_pages_int8_kernel<KV_DTYPE_F16>)
                                                      : run(kv_dequant_pages_int8_kernel<KV_DTYPE_F32>);
    return e == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}

int kv_copy_pages_int8(void* k_pages, void* v_pages, float* kv_scales, const int32_t* src_pages,
                       const int32_t* dst_pages, int32_t n, int32_t H_kv, int32_t Dh, int32_t page_size,
                       int32_t num_pages, int* err_flag, void* stream) {
    if (n < 0 || H_kv <= 0 || Dh <= 0 || page_size <= 0 || num_pages <= 0) return KV_ERR_ARG;
    const int32_t upp = page_units(H_kv, Dh, page_size);
    if (Dh % 16 != 0 || upp == 0 || (static_cast<int64_t>(H_kv) * page_size) % 2 != 0) return KV_ERR_UNSUPPORTED;
    if (n == 0) return KV_OK;
    if (!k_pages || !v_pages || !kv_scales || !src_pages || !dst_pages) return KV_ERR_ARG;
    if (!al16(k_pages) || !al16(v_pages) || !al16(kv_scales)) return KV_ERR_ARG;
    const cudaError_t e = launch_pdl(kv_copy_pages_int8_kernel, dim3(static_cast<unsigned>(n)), dim3(256), 0,
                                     static_cast<cudaStream_t>(stream), static_cast<uint4*>(k_pages),
                                     static_cast<uint4*>(v_pages), reinterpret_cast<uint4*>(kv_scales), src_pages,
                                     dst_pages, n, upp, H_kv * page_size / 2, num_pages, err_flag);
    return e == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}

}  // extern "C"
