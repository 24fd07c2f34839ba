// ep_norm.cu -- the norm in front of an expert layer: the residual's addition with the
// root-mean-square norm, to bf16 rows (for the router) and to E4M3 rows with 1x128 scales
// (for the FP8 dispatch), and its gradient.
#include "ep_common.cuh"
#include "ep_quant.cuh"

namespace {

using namespace ep;

constexpr int kMaxNormH = 16384;
constexpr int kBlock = 128;         // channels per E4M3 scale
constexpr int kMaxThreads = 1024;
constexpr int kMaxParts = 512;      // rows of dweight partial sums
constexpr int kReduceWarps = 8;     // warps of a dweight reduction CTA

// The residual stream's type decides how a row is laid over the threads: a thread holds
// vectors of kElems consecutive channels, so that a vector of the stream is 16 bytes and a
// warp reads whole lines of every array (bf16 stream: 8 channels; fp32 stream: 4, whose
// bf16 neighbours are 8 bytes).
struct CarryBf16 {
    static constexpr int kElems = 8;
};
struct CarryF32 {
    static constexpr int kElems = 4;
};

// N / 2 words of packed bf16 (N = 4: 8 bytes, N = 8: 16 bytes). Not the read-only path: an
// output may be the same array as an input, and a thread reads its part before it writes.
template <int N>
__device__ __forceinline__ void load_bf16_words(uint32_t (&w)[N / 2], const uint16_t* p) {
    if constexpr (N == 8) {
        const uint4 v = ld_inout_v4(p);
        w[0] = v.x;
        w[1] = v.y;
        w[2] = v.z;
        w[3] = v.w;
    } else {
        asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
    }
}

template <int N>
__device__ __forceinline__ void store_bf16(uint16_t* p, const float (&f)[N]) {
    if constexpr (N == 8) {
        st_v4(p, make_uint4(pack_bf16x2_rn(f[0], f[1]), pack_bf16x2_rn(f[2], f[3]), pack_bf16x2_rn(f[4], f[5]),
                            pack_bf16x2_rn(f[6], f[7])));
    } else {
        st_v2(p, pack_bf16x2_rn(f[0], f[1]), pack_bf16x2_rn(f[2], f[3]));
    }
}

template <int N>
__device__ __forceinline__ void unpack_bf16(float (&f)[N], const uint32_t (&w)[N / 2]) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
    }
}

// a vector of the stream: 16 bytes for either type
template <class Carry>
__device__ __forceinline__ void load_carry_words(uint32_t (&w)[4], const void* base, size_t at) {
    const uint4 v = ld_inout_v4(static_cast<const char*>(base) + at * (16 / Carry::kElems));
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
}

template <class Carry>
__device__ __forceinline__ void unpack_carry(float (&f)[Carry::kElems], const uint32_t (&w)[4]) {
    if constexpr (Carry::kElems == 8) {
        unpack_bf16(f, w);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(w[i]);
    }
}

template <class Carry>
__device__ __forceinline__ void store_carry(void* base, size_t at, const float (&f)[Carry::kElems]) {
    char* p = static_cast<char*>(base) + at * (16 / Carry::kElems);
    if constexpr (Carry::kElems == 8) {
        store_bf16(reinterpret_cast<uint16_t*>(p), f);
    } else {
        st_v4(p, make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                            __float_as_uint(f[3])));
    }
}

// N weights from channel h; they are read by every row, so they stay in L1
template <int N>
__device__ __forceinline__ void load_weights(float (&f)[N], const void* weight, bool f32, int h) {
    if (f32) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(weight) + h);
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const float4 v = __ldg(p + i);
            f[4 * i] = v.x;
            f[4 * i + 1] = v.y;
            f[4 * i + 2] = v.z;
            f[4 * i + 3] = v.w;
        }
    } else {
        uint32_t w[N / 2];
        const uint16_t* p = static_cast<const uint16_t*>(weight) + h;
        if constexpr (N == 8) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
            w[0] = v.x;
            w[1] = v.y;
            w[2] = v.z;
            w[3] = v.w;
        } else {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
            w[0] = v.x;
            w[1] = v.y;
        }
        unpack_bf16(f, w);
    }
}

// the sum over the warp, the same in every lane
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(kFullMask, v, off);
    return v;
}

// ---------------------------------------------------------------------------
// Forward
// ---------------------------------------------------------------------------

struct NormArgs {
    const uint16_t* x;     // nullable
    const void* residual;  // nullable, stream type
    const void* weight;
    int weight_f32;
    float eps, inv_h;
    int H;
    void* residual_out;  // nullable, stream type
    uint16_t* y;         // nullable
    uint8_t* y_q;        // nullable
    float* y_scales;
};

// The E4M3 codes of a thread's vector; the block's kBlock / N lanes hold its channels. A
// block whose largest magnitude is 0 has scale 0 and every value's own code (a signed zero,
// or NaN); NaNs do not take part in the maximum. Lanes past the row's end pass zeros.
template <int N>
__device__ __forceinline__ float quantise(const float (&v)[N], uint32_t (&code)[N / 4]) {
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) amax = fmaxf(amax, fabsf(v[i]));
#pragma unroll
    for (int off = kBlock / N / 2; off >= 1; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, off));
    const float scale = scale_of(amax);
    float q[N];
    if (scale >= 1.17549435e-38f && scale < __int_as_float(0x7f800000)) {
        const float rcp = __frcp_rn(scale);
#pragma unroll
        for (int i = 0; i < N; ++i) q[i] = quotient(v[i], scale, rcp);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) q[i] = amax == 0.0f ? v[i] : __fdiv_rn(v[i], scale);
    }
#pragma unroll
    for (int i = 0; i < N / 4; ++i) code[i] = pack_e4m3x4_rn_sat(q[4 * i], q[4 * i + 1], q[4 * i + 2], q[4 * i + 3]);
    return scale;
}

// One CTA per row, kVecs vectors per thread, vector i of thread t being vector i * threads
// + t of the row. The row stays in registers between the sum of squares and the outputs.
template <class Carry, int kVecs, bool kFp8>
__global__ void __launch_bounds__(kMaxThreads* Carry::kElems* kVecs / 8 <= 2048 ? kMaxThreads : 512)
    rmsnorm_kernel(NormArgs a) {
    constexpr int N = Carry::kElems;
    __shared__ float s_part[32];
    grid_dependency_wait();  // dependent launch: inputs are ready after this
    allow_dependents();
    const int tid = static_cast<int>(threadIdx.x);
    const int nt = static_cast<int>(blockDim.x);
    const size_t row = static_cast<size_t>(blockIdx.x) * a.H;

    uint32_t xw[kVecs][N / 2], rw[kVecs][4];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int h = (i * nt + tid) * N;
        if (h < a.H) {
            if (a.x != nullptr) load_bf16_words<N>(xw[i], a.x + row + h);
            if (a.residual != nullptr) load_carry_words<Carry>(rw[i], a.residual, row + h);
        }
    }
    float z[kVecs][N];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int h = (i * nt + tid) * N;
#pragma unroll
        for (int e = 0; e < N; ++e) z[i][e] = 0.0f;
        if (h < a.H) {
            if (a.x != nullptr) unpack_bf16(z[i], xw[i]);
            if (a.residual != nullptr) {
                float r[N];
                unpack_carry<Carry>(r, rw[i]);
#pragma unroll
                for (int e = 0; e < N; ++e) z[i][e] = a.x != nullptr ? z[i][e] + r[e] : r[e];
            }
            if (a.residual_out != nullptr) store_carry<Carry>(a.residual_out, row + h, z[i]);
        }
#pragma unroll
        for (int e = 0; e < N; ++e) ss = fmaf(z[i][e], z[i][e], ss);
    }
    ss = warp_sum(ss);
    if (nt > 32) {
        if ((tid & 31) == 0) s_part[tid >> 5] = ss;
        __syncthreads();
        ss = warp_sum((tid & 31) < (nt >> 5) ? s_part[tid & 31] : 0.0f);
    }
    const float rstd = rsqrtf(fmaf(ss, a.inv_h, a.eps));
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int h = (i * nt + tid) * N;
        const bool in = h < a.H;
        float v[N];
        if (in) load_weights<N>(v, a.weight, a.weight_f32 != 0, h);
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = in ? z[i][e] * rstd * v[e] : 0.0f;
        if (in && a.y != nullptr) store_bf16(a.y + row + h, v);
        if constexpr (kFp8) {
            uint32_t code[N / 4];
            const float scale = quantise<N>(v, code);
            if (in) {
                if constexpr (N == 8) st_v2(a.y_q + row + h, code[0], code[1]);
                else *reinterpret_cast<uint32_t*>(a.y_q + row + h) = code[0];
                if (h % kBlock == 0) a.y_scales[(row + h) / kBlock] = scale;
            }
        }
    }
}

// Threads of a row of `vecs` vectors when each takes `per` of them.
inline int row_threads(int vecs, int per) { return ((vecs + per - 1) / per + 31) / 32 * 32; }

template <class Carry, int kVecs>
ep_status_t launch_norm(const NormArgs& a, int T, cudaStream_t stream) {
    const int nt = row_threads(a.H / Carry::kElems, kVecs);
    auto kernel = a.y_q != nullptr ? rmsnorm_kernel<Carry, kVecs, true> : rmsnorm_kernel<Carry, kVecs, false>;
    return launch_dependent(kernel, dim3(static_cast<unsigned>(T)), dim3(nt), 0, stream, a);
}

template <class Carry>
ep_status_t launch_norm(const NormArgs& a, int T, cudaStream_t stream) {
    const int vecs = a.H / Carry::kElems;
    if (vecs >= 128) return launch_norm<Carry, 4>(a, T, stream);
    return launch_norm<Carry, 1>(a, T, stream);
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------

struct NormBwdArgs {
    const uint16_t* dy;
    const void* z;       // stream type
    const void* weight;
    int weight_f32;
    const void* dz_in;   // nullable, stream type
    float eps, inv_h;
    int T, H;
    void* dz;            // stream type
    uint16_t* dx;        // nullable
    float* parts;        // nullable: [gridDim.x][H] partial sums of dweight
};

// A CTA takes rows blockIdx.x, + gridDim.x, ... and keeps the sums of its rows' dweight
// terms in registers.
template <class Carry, int kVecs>
__global__ void __launch_bounds__(kMaxThreads* Carry::kElems* kVecs / 8 <= 2048 ? kMaxThreads : 512)
    rmsnorm_bwd_kernel(NormBwdArgs a) {
    constexpr int N = Carry::kElems;
    __shared__ float s_part[2][2][32];
    grid_dependency_wait();
    const int tid = static_cast<int>(threadIdx.x);
    const int nt = static_cast<int>(blockDim.x);
    float dw[kVecs][N];
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
#pragma unroll
        for (int e = 0; e < N; ++e) dw[i][e] = 0.0f;
    int parity = 0;
    for (int t = static_cast<int>(blockIdx.x); t < a.T; t += static_cast<int>(gridDim.x), parity ^= 1) {
        const size_t row = static_cast<size_t>(t) * a.H;
        uint32_t yw[kVecs][N / 2], zw[kVecs][4], iw[kVecs][4];
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int h = (i * nt + tid) * N;
            if (h < a.H) {
                load_bf16_words<N>(yw[i], a.dy + row + h);
                load_carry_words<Carry>(zw[i], a.z, row + h);
                if (a.dz_in != nullptr) load_carry_words<Carry>(iw[i], a.dz_in, row + h);
            }
        }
        float ss = 0.0f, sg = 0.0f;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int h = (i * nt + tid) * N;
            if (h < a.H) {
                float w[N], dy[N], z[N];
                load_weights<N>(w, a.weight, a.weight_f32 != 0, h);
                unpack_bf16(dy, yw[i]);
                unpack_carry<Carry>(z, zw[i]);
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    ss = fmaf(z[e], z[e], ss);
                    sg = fmaf(dy[e] * w[e], z[e], sg);
                }
            }
        }
        ss = warp_sum(ss);
        sg = warp_sum(sg);
        if (nt > 32) {
            const int lane = tid & 31;
            if (lane == 0) {
                s_part[parity][0][tid >> 5] = ss;
                s_part[parity][1][tid >> 5] = sg;
            }
            __syncthreads();  // the other parity's values are read before this and written after it
            ss = warp_sum(lane < (nt >> 5) ? s_part[parity][0][lane] : 0.0f);
            sg = warp_sum(lane < (nt >> 5) ? s_part[parity][1][lane] : 0.0f);
        }
        const float rstd = rsqrtf(fmaf(ss, a.inv_h, a.eps));
        const float c = sg * a.inv_h * rstd * rstd;  // mean(g z) / (mean(z^2) + eps)
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int h = (i * nt + tid) * N;
            if (h < a.H) {
                float w[N], dy[N], z[N], d[N];
                load_weights<N>(w, a.weight, a.weight_f32 != 0, h);
                unpack_bf16(dy, yw[i]);
                unpack_carry<Carry>(z, zw[i]);
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    d[e] = rstd * fmaf(-c, z[e], dy[e] * w[e]);
                    dw[i][e] = fmaf(dy[e] * rstd, z[e], dw[i][e]);
                }
                if (a.dz_in != nullptr) {
                    float in[N];
                    unpack_carry<Carry>(in, iw[i]);
#pragma unroll
                    for (int e = 0; e < N; ++e) d[e] += in[e];
                }
                store_carry<Carry>(a.dz, row + h, d);
                if (a.dx != nullptr) store_bf16(a.dx + row + h, d);
            }
        }
    }
    allow_dependents();
    if (a.parts != nullptr) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const int h = (i * nt + tid) * N;
            if (h < a.H) {
                float* p = a.parts + static_cast<size_t>(blockIdx.x) * a.H + h;
#pragma unroll
                for (int e = 0; e < N; e += 4)
                    *reinterpret_cast<float4*>(p + e) =
                        make_float4(dw[i][e], dw[i][e + 1], dw[i][e + 2], dw[i][e + 3]);
            }
        }
    }
}

// dweight[h] = the sum of the nparts partial sums of channel h, in a fixed order: a warp's
// lanes take 4 channels each, warp w the partial rows w, w + kReduceWarps, ...
__global__ void __launch_bounds__(32 * kReduceWarps) dweight_reduce_kernel(const float* parts, int nparts, int H,
                                                                         float* dweight) {
    __shared__ float4 s_sum[kReduceWarps][32];
    grid_dependency_wait();
    const int lane = lane_id();
    const int warp = static_cast<int>(threadIdx.x >> 5);
    const int h = (static_cast<int>(blockIdx.x) * 32 + lane) * 4;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (h < H) {
#pragma unroll 4
        for (int p = warp; p < nparts; p += kReduceWarps) {
            const float4 v = *reinterpret_cast<const float4*>(parts + static_cast<size_t>(p) * H + h);
            s.x += v.x;
            s.y += v.y;
            s.z += v.z;
            s.w += v.w;
        }
    }
    s_sum[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && h < H) {
        for (int w = 1; w < kReduceWarps; ++w) {
            const float4 v = s_sum[w][lane];
            s.x += v.x;
            s.y += v.y;
            s.z += v.z;
            s.w += v.w;
        }
        *reinterpret_cast<float4*>(dweight + h) = s;
    }
    allow_dependents();
}

template <class Carry, int kVecs>
ep_status_t launch_norm_bwd(const NormBwdArgs& a, cudaStream_t stream, int* grid_out) {
    const int nt = row_threads(a.H / Carry::kElems, kVecs);
    static std::atomic<int> cache[kMaxDevices][33];  // resident CTAs per SM, by warps
    const int dev = current_device();
    int per_sm = 0;
    const int warps = nt / 32;
    if (dev >= 0) per_sm = cache[dev][warps].load(std::memory_order_relaxed);
    if (per_sm == 0) {
        const cudaError_t err =
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, rmsnorm_bwd_kernel<Carry, kVecs>, nt, 0);
        if (err != cudaSuccess) return cuda_fail(err);
        if (per_sm < 1) per_sm = 1;
        if (dev >= 0) cache[dev][warps].store(per_sm, std::memory_order_relaxed);
    }
    int grid = sm_count() * per_sm;
    if (grid > kMaxParts) grid = kMaxParts;
    if (grid > a.T) grid = a.T;
    *grid_out = grid;
    return launch_dependent(rmsnorm_bwd_kernel<Carry, kVecs>, dim3(grid), dim3(nt), 0, stream, a);
}

template <class Carry>
ep_status_t launch_norm_bwd(const NormBwdArgs& a, cudaStream_t stream, int* grid_out) {
    const int vecs = a.H / Carry::kElems;
    if (vecs >= 128) return launch_norm_bwd<Carry, 4>(a, stream, grid_out);
    return launch_norm_bwd<Carry, 1>(a, stream, grid_out);
}

bool norm_common_ok(int T, int H, ep_dtype_t stream_dtype, ep_dtype_t weight_dtype, float eps) {
    return T >= 0 && H > 0 && H % 8 == 0 && H <= kMaxNormH &&
           (stream_dtype == EP_DTYPE_BF16 || stream_dtype == EP_DTYPE_F32) &&
           (weight_dtype == EP_DTYPE_BF16 || weight_dtype == EP_DTYPE_F32) && eps >= 0.0f;
}

}  // namespace

extern "C" ep_status_t ep_rmsnorm(const void* x, const void* residual, const void* weight, ep_dtype_t stream_dtype,
                                  ep_dtype_t weight_dtype, float eps, int32_t T, int32_t H, void* residual_out,
                                  void* y, uint8_t* y_q, float* y_scales, void* stream) {
    if (!norm_common_ok(T, H, stream_dtype, weight_dtype, eps)) return EP_ERR_INVALID;
    if ((y_q != nullptr) != (y_scales != nullptr) || (y_q != nullptr && H % kBlock != 0)) return EP_ERR_INVALID;
    if (T == 0) return EP_OK;
    if ((x == nullptr && residual == nullptr) || weight == nullptr) return EP_ERR_INVALID;
    if (residual_out == nullptr && y == nullptr && y_q == nullptr) return EP_ERR_INVALID;
    if (!aligned16_or_null(x) || !aligned16_or_null(residual) || !aligned16(weight) ||
        !aligned16_or_null(residual_out) || !aligned16_or_null(y) || !aligned16_or_null(y_q) ||
        !aligned16_or_null(y_scales))
        return EP_ERR_INVALID;
    const NormArgs a{static_cast<const uint16_t*>(x), residual, weight, weight_dtype == EP_DTYPE_F32, eps,
                     1.0f / static_cast<float>(H), H, residual_out, static_cast<uint16_t*>(y), y_q, y_scales};
    return stream_dtype == EP_DTYPE_F32 ? launch_norm<CarryF32>(a, T, as_stream(stream))
                                        : launch_norm<CarryBf16>(a, T, as_stream(stream));
}

extern "C" size_t ep_rmsnorm_bwd_workspace_size(int32_t T, int32_t H) {
    if (T < 0 || H <= 0 || H > kMaxNormH) return 0;
    return static_cast<size_t>(T < kMaxParts ? T : kMaxParts) * H * sizeof(float);
}

extern "C" ep_status_t ep_rmsnorm_bwd(const void* dy, const void* z, const void* weight, const void* dz_in,
                                      ep_dtype_t stream_dtype, ep_dtype_t weight_dtype, float eps, int32_t T,
                                      int32_t H, void* dz, void* dx, float* dweight, void* workspace,
                                      size_t workspace_bytes, void* stream) {
    if (!norm_common_ok(T, H, stream_dtype, weight_dtype, eps)) return EP_ERR_INVALID;
    if (!aligned16_or_null(dweight) || !aligned16_or_null(workspace)) return EP_ERR_INVALID;
    int parts = 0;
    if (T > 0) {
        if (dy == nullptr || z == nullptr || weight == nullptr || dz == nullptr) return EP_ERR_INVALID;
        if (!aligned16(dy) || !aligned16(z) || !aligned16(weight) || !aligned16_or_null(dz_in) || !aligned16(dz) ||
            !aligned16_or_null(dx))
            return EP_ERR_INVALID;
        if (dweight != nullptr &&
            (workspace == nullptr || workspace_bytes < ep_rmsnorm_bwd_workspace_size(T, H)))
            return EP_ERR_INVALID;
        const NormBwdArgs a{static_cast<const uint16_t*>(dy), z, weight, weight_dtype == EP_DTYPE_F32, dz_in, eps,
                            1.0f / static_cast<float>(H), T, H, dz, static_cast<uint16_t*>(dx),
                            dweight != nullptr ? static_cast<float*>(workspace) : nullptr};
        const ep_status_t st = stream_dtype == EP_DTYPE_F32 ? launch_norm_bwd<CarryF32>(a, as_stream(stream), &parts)
                                                            : launch_norm_bwd<CarryBf16>(a, as_stream(stream), &parts);
        if (st != EP_OK) return st;
    }
    if (dweight == nullptr) return EP_OK;
    return launch_dependent(dweight_reduce_kernel, dim3((H + 127) / 128), dim3(32 * kReduceWarps), 0,
                            as_stream(stream), static_cast<const float*>(workspace), parts, static_cast<int>(H), dweight);
}
