// ep_permute_bwd.cu -- gradients of the expert-major path: of the (weighted) return to
// token order (ep_combine_permuted) and of the sort into expert order
// (ep_dispatch_permuted). Row p of an entry (t, j) as in ep_permute.cu:
//   p = expert_offsets[e] - expert_offsets[r*(E/R)] + expert_slot[t][j].
// Both move rows and add or multiply a few numbers per element, so HBM bandwidth bounds
// them; there is no contraction for the tensor cores.
#include "ep_common.cuh"

namespace {

using namespace ep;

constexpr int kMaxTopk = 32;
constexpr int kWarps = 8;         // most warps of a CTA of the return's gradient
constexpr int kSortThreads = 128;  // most threads of a CTA of the sort's gradient
constexpr int kVecs = 4;   // 16-byte vectors of a row per thread and step (return)
constexpr int kBatch = 8;  // source rows whose vectors are loaded together (sort)

// Slab row r * max_rows + p of entry (t, j), -1 when the entry is not counted, -2 when its
// row lies past the slab's end (the forward pass dropped it).
__device__ __forceinline__ long long entry_row(const int64_t* topk_idx, const int32_t* offsets, const int32_t* eslot,
                                               size_t entry, int E, int epr, int max_rows) {
    const int32_t sl = eslot[entry];
    const int64_t e = topk_idx[entry];
    if (sl < 0 || e < 0 || e >= E) return -1;
    const int r = static_cast<int>(e) / epr;
    const int p = offsets[e] - offsets[r * epr] + sl;
    return p >= 0 && p < max_rows ? static_cast<long long>(r) * max_rows + p : -2;
}

__device__ __forceinline__ void unpack8(float (&f)[8], const uint4& v) {
    f[0] = bf16_lo(v.x);
    f[1] = bf16_hi(v.x);
    f[2] = bf16_lo(v.y);
    f[3] = bf16_hi(v.y);
    f[4] = bf16_lo(v.z);
    f[5] = bf16_hi(v.z);
    f[6] = bf16_lo(v.w);
    f[7] = bf16_hi(v.w);
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_bf16x2_rn(f[0], f[1]), pack_bf16x2_rn(f[2], f[3]), pack_bf16x2_rn(f[4], f[5]),
                      pack_bf16x2_rn(f[6], f[7]));
}

// ---------------------------------------------------------------------------
// Gradient of the return to token order
// ---------------------------------------------------------------------------

struct CombineBwdArgs {
    const uint16_t* dout;
    const uint16_t* y;    // read when dtopk_w is given
    const int64_t* topk_idx;
    const float* topk_w;  // nullable: unweighted
    const int32_t* offsets;
    const int32_t* eslot;
    int T, H, k, E, R, max_rows;
    uint16_t* dy;
    float* dtopk_w;       // nullable
    int32_t* status;
};

// One CTA per token, a warp per top-k slot (slots past kWarps go round again): the warp
// resolves its entry, then streams the entry's row of y and the token's dout -- which its
// sibling warps read at the same time, so that L1 serves them -- and writes dy's row =
// bf16(w * dout). The dot product is kept in fp32 in one sum per channel of a vector (at
// most H / 256 terms each), added across the vector and the lanes at the end. At 64
// registers four CTAs, 32 warps with 4 vectors of y each in flight, fit an SM: 4096 x 7168
// top-8 in 153.6 us (6.50 TB/s, 0.96 of a measured copy); with 72 registers or 2 vectors 157
// us, with a CTA's threads all on one entry after the other 155 us, and 777 x 1032 top-6 in
// 4.5 us instead of 10.9 us.
__global__ void __launch_bounds__(32 * kWarps, 4) combine_bwd_kernel(CombineBwdArgs a) {
    grid_dependency_wait();  // dependent launch: inputs are ready after this
    const int lane = lane_id();
    const int nwarps = static_cast<int>(blockDim.x >> 5);
    const int t = static_cast<int>(blockIdx.x);
    const int nvec = a.H / 8;
    const uint4* dout = reinterpret_cast<const uint4*>(a.dout) + static_cast<size_t>(t) * nvec;
    const bool dots = a.dtopk_w != nullptr;
    for (int j = static_cast<int>(threadIdx.x >> 5); j < a.k; j += nwarps) {
        const size_t entry = static_cast<size_t>(t) * a.k + j;
        const float w = a.topk_w != nullptr ? a.topk_w[entry] : 1.0f;
        const long long row = entry_row(a.topk_idx, a.offsets, a.eslot, entry, a.E, a.E / a.R, a.max_rows);
        if (row < 0) {
            if (lane == 0) {
                if (row == -2) raise_flag(a.status, EP_FLAG_CAPACITY);
                if (dots) a.dtopk_w[entry] = 0.0f;
            }
            continue;
        }
        const uint4* y = reinterpret_cast<const uint4*>(a.y) + row * nvec;
        uint4* dy = reinterpret_cast<uint4*>(a.dy) + row * nvec;
        float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int v0 = lane; v0 < nvec; v0 += 32 * kVecs) {
            uint4 g[kVecs], yv[kVecs];
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const int v = v0 + i * 32;
                if (v < nvec) {
                    if (dots) yv[i] = ld_inout_v4(y + v);
                    g[i] = __ldg(dout + v);
                }
            }
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const int v = v0 + i * 32;
                if (v >= nvec) continue;
                float d[8];
                unpack8(d, g[i]);
                if (dots) {
                    float f[8];
                    unpack8(f, yv[i]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) acc[e] = fmaf(d[e], f[e], acc[e]);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) d[e] *= w;
                st_v4(dy + v, pack8(d));
            }
        }
        if (dots) {
            float dot = ((acc[0] + acc[1]) + (acc[2] + acc[3])) + ((acc[4] + acc[5]) + (acc[6] + acc[7]));
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1) dot += __shfl_xor_sync(kFullMask, dot, off);
            if (lane == 0) a.dtopk_w[entry] = dot;
        }
    }
    allow_dependents();
}

// ---------------------------------------------------------------------------
// Gradient of the sort into expert order
// ---------------------------------------------------------------------------

struct DispatchBwdArgs {
    const uint16_t* dperm_x;
    const float* dperm_w;  // read when dtopk_w is given
    const uint16_t* dx_in;  // nullable
    const int64_t* topk_idx;
    const int32_t* offsets;
    const int32_t* eslot;
    int T, H, k, E, R, max_rows;
    uint16_t* dx;
    float* dtopk_w;  // nullable
    int32_t* status;
};

// One CTA per token: warp 0 lists the token's rows, then every thread adds its vectors of
// those rows in slot order, the addend first, with kBatch rows' vectors in flight. 16384 x
// 4096 top-8 with the addend: 202.6 us (6.64 TB/s, 0.98 of a measured copy) with CTAs of 128
// threads, 207 us with 256, 238 us with 512 (fewer, larger CTAs wait longer for their lists).
__global__ void __launch_bounds__(kSortThreads, 8) dispatch_bwd_kernel(DispatchBwdArgs a) {
    grid_dependency_wait();
    __shared__ long long s_row[kMaxTopk];
    __shared__ int s_n;
    const int tid = static_cast<int>(threadIdx.x);
    const int t = static_cast<int>(blockIdx.x);
    const int nvec = a.H / 8;
    if (tid < 32) {
        const size_t entry = static_cast<size_t>(t) * a.k + tid;
        long long row = -1;
        if (tid < a.k) {
            row = entry_row(a.topk_idx, a.offsets, a.eslot, entry, a.E, a.E / a.R, a.max_rows);
            if (a.dtopk_w != nullptr) a.dtopk_w[entry] = row >= 0 ? a.dperm_w[row] : 0.0f;
        }
        const uint32_t m = __ballot_sync(kFullMask, row >= 0);
        if (row >= 0) s_row[__popc(m & lanemask_lt())] = row * nvec;
        if (__any_sync(kFullMask, row == -2) && tid == 0) raise_flag(a.status, EP_FLAG_CAPACITY);
        if (tid == 0) s_n = __popc(m);
    }
    __syncthreads();
    const int n = s_n;
    const uint4* src = reinterpret_cast<const uint4*>(a.dperm_x);
    const uint4* in = reinterpret_cast<const uint4*>(a.dx_in) + static_cast<size_t>(t) * nvec;
    uint4* dx = reinterpret_cast<uint4*>(a.dx) + static_cast<size_t>(t) * nvec;
    for (int v = tid; v < nvec; v += static_cast<int>(blockDim.x)) {
        uint4 first = make_uint4(0, 0, 0, 0);
        if (a.dx_in != nullptr) first = ld_inout_v4(in + v);
        float acc[8];
        unpack8(acc, first);
        for (int d0 = 0; d0 < n; d0 += kBatch) {
            uint4 buf[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (d0 + i < n) buf[i] = ld_stream_v4(src + s_row[d0 + i] + v);
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                if (d0 + i >= n) continue;
                float f[8];
                unpack8(f, buf[i]);
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] += f[e];
            }
        }
        st_v4(dx + v, pack8(acc));
    }
    allow_dependents();
}

bool bwd_common_ok(int T, int H, int k, int E, int R, int max_rows) {
    return T >= 0 && H > 0 && H % 8 == 0 && k >= 1 && k <= kMaxTopk && R >= 1 && R <= 256 && E >= R && E % R == 0 &&
           E <= 8192 && max_rows >= 0 && static_cast<long long>(R) * max_rows <= 0x7fffffffLL;
}

}  // namespace

extern "C" ep_status_t ep_combine_permuted_bwd(const void* dout, const void* y, const int64_t* topk_idx,
                                               const float* topk_w, const int32_t* expert_offsets,
                                               const int32_t* expert_slot, int32_t T, int32_t H, int32_t k, int32_t E,
                                               int32_t R, int32_t max_rows, void* dy, float* dtopk_w, int32_t* status,
                                               void* stream) {
    if (!bwd_common_ok(T, H, k, E, R, max_rows)) return EP_ERR_INVALID;
    if (dtopk_w != nullptr && topk_w == nullptr) return EP_ERR_INVALID;
    if (T == 0) return EP_OK;
    if (dout == nullptr || topk_idx == nullptr || expert_offsets == nullptr || expert_slot == nullptr ||
        (max_rows > 0 && (dy == nullptr || (dtopk_w != nullptr && y == nullptr))))
        return EP_ERR_INVALID;
    if (!aligned16(dout) || !aligned16_or_null(y) || !aligned16(topk_idx) || !aligned16_or_null(topk_w) ||
        !aligned16(expert_offsets) || !aligned16(expert_slot) || !aligned16_or_null(dy) ||
        !aligned16_or_null(dtopk_w))
        return EP_ERR_INVALID;
    const CombineBwdArgs a{static_cast<const uint16_t*>(dout), static_cast<const uint16_t*>(y), topk_idx, topk_w,
                           expert_offsets, expert_slot, T, H, k, E, R, max_rows, static_cast<uint16_t*>(dy), dtopk_w,
                           status};
    return launch_dependent(combine_bwd_kernel, dim3(static_cast<unsigned>(T)), dim3(32 * (k < kWarps ? k : kWarps)),
                            0, as_stream(stream), a);
}

extern "C" ep_status_t ep_dispatch_permuted_bwd(const void* dperm_x, const float* dperm_w, const void* dx_in,
                                                const int64_t* topk_idx, const int32_t* expert_offsets,
                                                const int32_t* expert_slot, int32_t T, int32_t H, int32_t k,
                                                int32_t E, int32_t R, int32_t max_rows, void* dx, float* dtopk_w,
                                                int32_t* status, void* stream) {
    if (!bwd_common_ok(T, H, k, E, R, max_rows)) return EP_ERR_INVALID;
    if (T == 0) return EP_OK;
    if (topk_idx == nullptr || expert_offsets == nullptr || expert_slot == nullptr || dx == nullptr ||
        (max_rows > 0 && (dperm_x == nullptr || (dtopk_w != nullptr && dperm_w == nullptr))))
        return EP_ERR_INVALID;
    if (!aligned16_or_null(dperm_x) || !aligned16_or_null(dperm_w) || !aligned16_or_null(dx_in) ||
        !aligned16(topk_idx) || !aligned16(expert_offsets) || !aligned16(expert_slot) || !aligned16(dx) ||
        !aligned16_or_null(dtopk_w))
        return EP_ERR_INVALID;
    const DispatchBwdArgs a{static_cast<const uint16_t*>(dperm_x), dperm_w, static_cast<const uint16_t*>(dx_in),
                            topk_idx, expert_offsets, expert_slot, T, H, k, E, R, max_rows,
                            static_cast<uint16_t*>(dx), dtopk_w, status};
    const int threads = H / 8 < kSortThreads ? (H / 8 + 31) / 32 * 32 : kSortThreads;
    return launch_dependent(dispatch_bwd_kernel, dim3(static_cast<unsigned>(T)), dim3(threads), 0, as_stream(stream),
                            a);
}
