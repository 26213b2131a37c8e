// RMS norm of every query and key head, rotary embedding and KV append in one
// pass ("06 KV Cache、Prefix Cache、PagedAttention 与 vLLM", 6.1: q and k are
// rotated by the token's position before k and v are appended and q attends;
// the per-head norm before the rotation is the usual query / key norm):
//   y = x * w / sqrt(mean(x^2) + eps)   over the Dh elements of one head,
//   q', k' = rotate(y, pos),            rounded once to the storage type.
//
// Unit of work as in kv_rope_append: a thread owns one pair of 16-byte
// vectors of a row, so both elements of every rotated pair (either pairing)
// sit in one thread, and the Dh * sizeof / 32 threads of a row (a power of
// two, at most a warp) are neighbouring lanes: the sum of squares is a few
// shuffles and a row is read once and written once. The thread keeps its unit
// -- row, weights, pair indices -- and walks the tokens; the next token's
// vectors, position and slot are loaded before the current one is finished,
// which doubles the bytes in flight of a launch that is bound by memory.
// Everything between the load and the store is fp32.
// Measured, 32 query and 8 KV heads of 128 (fp16): 8192 tokens 45 us, 4.5 TB/s
// (0.69 of the measured copy rate, as kv_rope_append); 64 tokens 2.5 us, bound
// by the launch and one round trip to memory.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "decode_launch.cuh"
#include "kvpaged.h"
#include "rope.cuh"

namespace kvp {
namespace {

struct NormRopeParams {
    uint4 *k_pages, *v_pages, *q_out, *k_out;
    const uint4 *q, *k_new, *v_new;
    int64_t q_stride, k_stride, v_stride;  // per token, in 16-byte vectors
    const float *q_weight, *k_weight;
    const int64_t* slots;
    const int32_t* positions;
    const float* cos_sin;
    int* err;
    int64_t B, num_slots;
    float eps, inv_dh;
    int32_t max_pos, style, q_rows, H_kv, Dh, P;
};

// A 16-byte vector as pairs of fp32 values, and back (rounded to nearest even).
template <int DT, int H>
__device__ __forceinline__ void unpack(const uint4& v, float2 (&x)[H]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (DT == KV_DTYPE_F32) {
        x[0] = make_float2(__uint_as_float(w[0]), __uint_as_float(w[1]));
        x[1] = make_float2(__uint_as_float(w[2]), __uint_as_float(w[3]));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (DT == KV_DTYPE_BF16)
                x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
            else
                x[i] = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        }
    }
}
template <int DT, int H>
__device__ __forceinline__ uint4 pack(const float2 (&x)[H]) {
    if constexpr (DT == KV_DTYPE_F32)
        return make_uint4(__float_as_uint(x[0].x), __float_as_uint(x[0].y), __float_as_uint(x[1].x), __float_as_uint(x[1].y));
    else
        return make_uint4(pack2<DT == KV_DTYPE_BF16>(x[0].x, x[0].y), pack2<DT == KV_DTYPE_BF16>(x[1].x, x[1].y),
                          pack2<DT == KV_DTYPE_BF16>(x[2].x, x[2].y), pack2<DT == KV_DTYPE_BF16>(x[3].x, x[3].y));
}

constexpr int kNormRopeThreads = 384, kNormRopeCtas = 2;  // per CTA, per SM

template <int DT>
__global__ void __launch_bounds__(kNormRopeThreads, kNormRopeCtas) kv_norm_rope_append_kernel(const __grid_constant__ NormRopeParams p) {
    constexpr int N = RopeVec<DT>::kN;  // elements per 16-byte vector
    constexpr int H = N / 2;
    grid_dependency_wait();
    if (threadIdx.x == 0) grid_launch_dependents();
    const int32_t Dh = p.Dh;
    const int32_t vpr = Dh / N, upr = vpr / 2;  // vectors and units per row; upr is a power of two <= 32
    const int32_t k_rows = p.H_kv, v_rows = p.v_pages != nullptr ? p.H_kv : 0;
    const int32_t units = (p.q_rows + k_rows + v_rows) * upr;  // per token
    const int lane = threadIdx.x & 31;
    const unsigned row_mask = (upr == 32 ? 0xffffffffu : (1u << upr) - 1u) << (lane & ~(upr - 1));
    for (int32_t rem = threadIdx.x; rem < units; rem += blockDim.x) {
        const int32_t r = rem / upr, u = rem - r * upr;
        const bool is_q = r < p.q_rows;
        const bool is_v = !is_q && r >= p.q_rows + k_rows;
        const int32_t h = is_q ? r : r - p.q_rows - (is_v ? k_rows : 0);
        const int32_t va = p.style == KV_ROPE_HALF ? u : 2 * u;
        const int32_t vb = p.style == KV_ROPE_HALF ? u + upr : 2 * u + 1;
        const int32_t k0 = u * N;  // pairs k0 .. k0 + N - 1
        const uint4* src = (is_q ? p.q : (is_v ? p.v_new : p.k_new)) + (int64_t)h * vpr;
        const int64_t stride = is_q ? p.q_stride : (is_v ? p.v_stride : p.k_stride);
        const float* w = is_q ? p.q_weight : p.k_weight;
        float2 wa[H], wb[H];
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const bool weighted = !is_v && w != nullptr;
            wa[i] = weighted ? make_float2(w[va * N + 2 * i], w[va * N + 2 * i + 1]) : make_float2(1.f, 1.f);
            wb[i] = weighted ? make_float2(w[vb * N + 2 * i], w[vb * N + 2 * i + 1]) : make_float2(1.f, 1.f);
        }
        int64_t b = blockIdx.x;
        if (b >= p.B) continue;
        uint4 a = src[b * stride + va], c = src[b * stride + vb];
        int32_t pos = p.positions[b];
        int64_t slot = p.slots != nullptr ? p.slots[b] : -1;
        while (true) {
            const int64_t nb = b + gridDim.x;
            uint4 a_n, c_n;
            int32_t pos_n = 0;
            int64_t slot_n = -1;
            if (nb < p.B) {
                a_n = src[nb * stride + va];
                c_n = src[nb * stride + vb];
                pos_n = p.positions[nb];
                if (p.slots != nullptr) slot_n = p.slots[nb];
            }
            const bool pos_ok = pos >= 0 && pos < p.max_pos;
            const bool slot_ok = slot >= 0 && slot < p.num_slots;
            if (rem == 0 && p.err != nullptr) {
                if (!pos_ok) atomicOr(p.err, KV_DEV_ERR_POSITION);
                else if (slot >= p.num_slots && p.slots != nullptr) atomicOr(p.err, KV_DEV_ERR_SLOT);
            }
            // the row's page slot: K and V rows of a token that is appended
            int64_t cache_row = 0;
            if (slot_ok && !is_q) {
                const int64_t page = slot / p.P, off = slot - page * p.P;
                cache_row = ((page * p.H_kv + h) * p.P + off) * vpr;
            }
            if (pos_ok && is_v) {
                if (slot_ok) {
                    p.v_pages[cache_row + va] = a;
                    p.v_pages[cache_row + vb] = c;
                }
            } else if (pos_ok) {
                // pairs of neighbouring elements go through the packed fp32 operations
                float2 xa[H], xb[H], cs[H], sn[H];
                unpack<DT>(a, xa);
                unpack<DT>(c, xb);
                float2 sq = make_float2(0.f, 0.f);
#pragma unroll
                for (int i = 0; i < H; ++i) sq = ffma2(xa[i], xa[i], ffma2(xb[i], xb[i], sq));
                float ss = sq.x + sq.y;
                const float* crow = p.cos_sin + (int64_t)pos * Dh;
#pragma unroll
                for (int i = 0; i < H; i += 2) {
                    const float4 cc = __ldg(reinterpret_cast<const float4*>(crow + k0 + 2 * i));
                    const float4 si = __ldg(reinterpret_cast<const float4*>(crow + Dh / 2 + k0 + 2 * i));
                    cs[i] = make_float2(cc.x, cc.y), cs[i + 1] = make_float2(cc.z, cc.w);
                    sn[i] = make_float2(si.x, si.y), sn[i + 1] = make_float2(si.z, si.w);
                }
                for (int o = upr >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(row_mask, ss, o);
                const float rs = rsqrtf(ss * p.inv_dh + p.eps);
                // 1 / rms joins the angles' cosines and sines: one product fewer per element
                const float2 rs2 = make_float2(rs, rs);
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    xa[i] = fmul2(xa[i], wa[i]);
                    xb[i] = fmul2(xb[i], wb[i]);
                    cs[i] = fmul2(cs[i], rs2);
                    sn[i] = fmul2(sn[i], rs2);
                }
                if (p.style == KV_ROPE_HALF) {
                    // pair k0 + e = (element e of a, element e of b)
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        const float2 ns = make_float2(-sn[i].x, -sn[i].y);
                        const float2 t = ffma2(xa[i], cs[i], fmul2(xb[i], ns));
                        xb[i] = ffma2(xb[i], cs[i], fmul2(xa[i], sn[i]));
                        xa[i] = t;
                    }
                } else {
                    // a holds pairs k0 .. k0 + H - 1 as neighbours, b the next H
                    auto turn = [](float2 x, float c1, float s1) {
                        return ffma2(x, make_float2(c1, c1), fmul2(make_float2(x.y, x.x), make_float2(-s1, s1)));
                    };
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        xa[i] = turn(xa[i], i & 1 ? cs[i / 2].y : cs[i / 2].x, i & 1 ? sn[i / 2].y : sn[i / 2].x);
                        const int k = i + H;
                        xb[i] = turn(xb[i], k & 1 ? cs[k / 2].y : cs[k / 2].x, k & 1 ? sn[k / 2].y : sn[k / 2].x);
                    }
                }
                const uint4 ya = pack<DT>(xa), yb = pack<DT>(xb);
                if (is_q) {
                    uint4* dst = p.q_out + (b * p.q_rows + h) * vpr;
                    dst[va] = ya;
                    dst[vb] = yb;
                } else {
                    if (p.k_out != nullptr) {
                        uint4* dst = p.k_out + (b * p.H_kv + h) * vpr;
                        dst[va] = ya;
                        dst[vb] = yb;
                    }
                    if (slot_ok) {
                        p.k_pages[cache_row + va] = ya;
                        p.k_pages[cache_row + vb] = yb;
                    }
                }
            }
            if (nb >= p.B) break;
            b = nb;
            a = a_n;
            c = c_n;
            pos = pos_n;
            slot = slot_n;
        }
    }
}

// SMs of the current device (looked up once per device).
int sm_count_cached() {
    static std::atomic<int> cached[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return -1;
    int v = cached[dev & 63].load(std::memory_order_relaxed);
    if (v > 0) return v;
    if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return -1;
    cached[dev & 63].store(v, std::memory_order_relaxed);
    return v;
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace kvp

using namespace kvp;

extern "C" int kv_norm_rope_append(void* k_pages, void* v_pages, void* q_out, void* k_out, const void* q,
                                   const void* k_new, const void* v_new, int64_t q_stride, int64_t k_stride,
                                   int64_t v_stride, const float* q_weight, const float* k_weight, float eps,
                                   const int64_t* slot_mapping, const int32_t* positions, const float* cos_sin,
                                   int32_t max_pos, int32_t rope_style, int32_t B, int32_t H_q, int32_t H_kv, int32_t Dh,
                                   int32_t page_size, int32_t num_pages, int32_t dtype, int* err_flag, void* stream) {
    const int eb = dtype == KV_DTYPE_F32 ? 4 : (dtype == KV_DTYPE_BF16 || dtype == KV_DTYPE_F16) ? 2 : 0;
    if (B < 0 || H_kv <= 0 || Dh <= 0 || eb == 0 || max_pos <= 0 || !(eps >= 0.f) || std::isinf(eps)) return KV_ERR_ARG;
    if (rope_style != KV_ROPE_HALF && rope_style != KV_ROPE_INTERLEAVED) return KV_ERR_ARG;
    if ((q == nullptr) != (q_out == nullptr) || (q != nullptr && H_q <= 0)) return KV_ERR_ARG;
    const bool cache = k_pages != nullptr;
    if (cache && (page_size <= 0 || num_pages <= 0)) return KV_ERR_ARG;
    // a row is upr pairs of 16-byte vectors, one per lane: a power of two of them, at most a warp
    const int64_t row_bytes = static_cast<int64_t>(Dh) * eb;
    if (row_bytes % 32 != 0 || row_bytes > 1024 || ((row_bytes / 32) & (row_bytes / 32 - 1)) != 0) return KV_ERR_UNSUPPORTED;
    const int32_t vpr = static_cast<int32_t>(row_bytes / 16), N = 16 / eb;
    if (B == 0) return KV_OK;
    if (!k_new || !positions || !cos_sin || (!cache && !k_out)) return KV_ERR_ARG;
    if (cache ? (!v_pages || !v_new || !slot_mapping) : (v_pages || v_new || slot_mapping)) return KV_ERR_ARG;
    if (!al16(k_pages) || !al16(v_pages) || !al16(k_new) || !al16(v_new) || !al16(cos_sin) || !al16(q) || !al16(q_out) ||
        !al16(k_out))
        return KV_ERR_ARG;
    // token strides in elements: whole 16-byte vectors, rows of different tokens apart
    auto stride_ok = [&](int64_t s, int64_t heads) { return s % N == 0 && s >= heads * Dh; };
    if ((q && !stride_ok(q_stride, H_q)) || !stride_ok(k_stride, H_kv) || (cache && !stride_ok(v_stride, H_kv)))
        return KV_ERR_ARG;
    // in place only row by row: with a larger input stride the outputs of one token lie over the inputs of others
    if ((q && q == q_out && q_stride != static_cast<int64_t>(H_q) * Dh) ||
        (k_out && k_new == k_out && k_stride != static_cast<int64_t>(H_kv) * Dh))
        return KV_ERR_ARG;
    NormRopeParams p{};
    p.k_pages = static_cast<uint4*>(k_pages);
    p.v_pages = static_cast<uint4*>(v_pages);
    p.q_out = static_cast<uint4*>(q_out);
    p.k_out = static_cast<uint4*>(k_out);
    p.q = static_cast<const uint4*>(q);
    p.k_new = static_cast<const uint4*>(k_new);
    p.v_new = static_cast<const uint4*>(v_new);
    p.q_stride = q_stride / N;
    p.k_stride = k_stride / N;
    p.v_stride = v_stride / N;
    p.q_weight = q_weight;
    p.k_weight = k_weight;
    p.slots = slot_mapping;
    p.positions = positions;
    p.cos_sin = cos_sin;
    p.err = err_flag;
    p.B = B;
    p.num_slots = static_cast<int64_t>(num_pages) * page_size;
    p.eps = eps;
    p.inv_dh = 1.f / static_cast<float>(Dh);
    p.max_pos = max_pos;
    p.style = rope_style;
    p.q_rows = q != nullptr ? H_q : 0;
    p.H_kv = H_kv;
    p.Dh = Dh;
    p.P = page_size;
    const int64_t units = (static_cast<int64_t>(p.q_rows) + H_kv + (cache ? H_kv : 0)) * (vpr / 2);
    if (units > 0x7fffffffLL) return KV_ERR_UNSUPPORTED;
    const int threads = static_cast<int>(std::min<int64_t>(kNormRopeThreads, (units + 31) / 32 * 32));
    const int sms = sm_count_cached();
    if (sms <= 0) return KV_ERR_CUDA;
    const int64_t blocks = std::min<int64_t>(B, static_cast<int64_t>(sms) * std::max(1, kNormRopeThreads * kNormRopeCtas / threads));  // resident CTAs
    auto run = [&](auto kernel) {
        return launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)), dim3(threads), 0, static_cast<cudaStream_t>(stream),
                          p);
    };
    const cudaError_t e = dtype == KV_DTYPE_BF16  ? run(kv_norm_rope_append_kernel<KV_DTYPE_BF16>)
                          : dtype == KV_DTYPE_F16 ? run(kv_norm_rope_append_kernel<KV_DTYPE_F16>)
                                                  : run(kv_norm_rope_append_kernel<KV_DTYPE_F32>);
    return e == cudaSuccess ? KV_OK : KV_ERR_CUDA;
}
