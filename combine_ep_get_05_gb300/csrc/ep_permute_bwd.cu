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
// Rows of the return's gradient up to this many channels, where there are many, go two to a
// warp: their positions are then resolved together (8000 x 1024 top-6 37.0 us instead of 38.7
// us; 1237 x 1592 top-9, too few, 17.2 us instead of 15.5 us).
constexpr int kShortRowH = 1024;
// Entries an SM below which the return's gradient puts four warps on each row (44 x 4176
// top-4: 2.6 us instead of 4.2 us; 777 x 1032 top-6, 31 an SM, 8.6 us instead of 4.6 us)
constexpr int kFewEntries = 8;
constexpr int kSortWarps = 16;  // most warps of a CTA of the sort's gradient
constexpr int kSortThreads = 64;  // threads of a token there, where tokens abound
constexpr int kSortFill = 768;    // threads an SM that fill the GPU
constexpr int kWarpRowH = 2048;   // rows up to this take a warp each
constexpr int kVecs = 4;   // 16-byte vectors of a row per thread and step (return)

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

// A CTA takes `count` consecutive entries (t, j), t * k + j in order, kLanes threads on an
// entry at a time. They resolve its row, then stream the row of y and the token's dout --
// which the warps of the token's other entries read at the same time, so that L1 serves them
// -- and write dy's row = bf16(w * dout). The dot product is kept in fp32 in one sum per
// channel of a vector (at most H / (8 kLanes) terms each), added across the vector, the lanes
// and the entry's warps at the end.
//
// At 64 registers 32 warps with 4 vectors of y each in flight fit an SM: 4096 x 7168 top-8 in
// 153 us (6.5 TB/s, 0.96 of a measured copy); 157 us with 72 registers or 2 vectors. Requesting
// dout before the row is known costs 2 %, two warps a row 3 %, the token's rows one after the
// other by a whole CTA 1 % (and 777 x 1032 top-6 then takes 10.9 us instead of 4.5 us).
template <int kLanes>
__global__ void __launch_bounds__(32 * kWarps, 4) combine_bwd_kernel(CombineBwdArgs a, int count) {
    constexpr int kSub = kLanes < 32 ? kLanes : 32;  // lanes of an entry in a warp
    constexpr int kSplit = kLanes / kSub;            // warps of an entry
    __shared__ float s_dot[kWarps];
    grid_dependency_wait();  // dependent launch: inputs are ready after this
    const int tid = static_cast<int>(threadIdx.x);
    const int first = tid % kLanes;
    const int at_once = static_cast<int>(blockDim.x) / kLanes;
    const long long entry0 = static_cast<long long>(blockIdx.x) * count;
    const long long entries = static_cast<long long>(a.T) * a.k;
    const int mine = entries - entry0 < count ? static_cast<int>(entries - entry0) : count;
    const int nvec = a.H / 8;
    const bool dots = a.dtopk_w != nullptr;
    // the entries of rounds 0, 1, ... of these lanes are resolved together, a lane each
    const int e_first = tid / kLanes;
    const int sub = tid % kSub;
    long long my_row = -1;
    float my_w = 1.0f;
    if (e_first + sub * at_once < mine) {
        const size_t entry = static_cast<size_t>(entry0 + e_first + sub * at_once);
        if (a.topk_w != nullptr) my_w = a.topk_w[entry];
        my_row = entry_row(a.topk_idx, a.offsets, a.eslot, entry, a.E, a.E / a.R, a.max_rows);
        if (my_row == -2) raise_flag(a.status, EP_FLAG_CAPACITY);
    }
    for (int r = 0; r * at_once < mine; ++r) {  // the same number of rounds for all threads
        const int e = e_first + r * at_once;
        const long long row = __shfl_sync(kFullMask, my_row, r, kSub);
        const float w = __shfl_sync(kFullMask, my_w, r, kSub);
        float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (row >= 0) {
            const uint4* dout = reinterpret_cast<const uint4*>(a.dout) + (entry0 + e) / a.k * nvec;
            const uint4* y = reinterpret_cast<const uint4*>(a.y) + row * nvec;
            uint4* dy = reinterpret_cast<uint4*>(a.dy) + row * nvec;
            for (int v0 = first; v0 < nvec; v0 += kLanes * kVecs) {
                uint4 g[kVecs], yv[kVecs];
                if (dots) {
#pragma unroll
                    for (int i = 0; i < kVecs; ++i)
                        if (v0 + i * kLanes < nvec) yv[i] = ld_inout_v4(y + v0 + i * kLanes);
                }
#pragma unroll
                for (int i = 0; i < kVecs; ++i)
                    if (v0 + i * kLanes < nvec) g[i] = __ldg(dout + v0 + i * kLanes);
#pragma unroll
                for (int i = 0; i < kVecs; ++i) {
                    const int v = v0 + i * kLanes;
                    if (v >= nvec) continue;
                    float d[8];
                    unpack8(d, g[i]);
                    if (dots) {
                        float f[8];
                        unpack8(f, yv[i]);
#pragma unroll
                        for (int c = 0; c < 8; ++c) acc[c] = fmaf(d[c], f[c], acc[c]);
                    }
#pragma unroll
                    for (int c = 0; c < 8; ++c) d[c] *= w;
                    st_v4(dy + v, pack8(d));
                }
            }
        }
        if (dots) {
            float dot = ((acc[0] + acc[1]) + (acc[2] + acc[3])) + ((acc[4] + acc[5]) + (acc[6] + acc[7]));
#pragma unroll
            for (int off = kSub / 2; off >= 1; off >>= 1) dot += __shfl_xor_sync(kFullMask, dot, off);
            if constexpr (kSplit > 1) {
                if (sub == 0) s_dot[tid >> 5] = dot;
                __syncthreads();
                if (first == 0) {
#pragma unroll
                    for (int i = 1; i < kSplit; ++i) dot += s_dot[(tid >> 5) + i];
                }
                __syncthreads();  // s_dot is written again in the next round
            }
            if (first == 0 && e < mine) a.dtopk_w[entry0 + e] = dot;
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

// the addend's vectors v0, v0 + stride, ... (kVec of them), zeros where there is none
template <int kVec>
__device__ __forceinline__ void load_addend(const DispatchBwdArgs& a, uint4 (&first)[kVec], const uint4* in, int nvec,
                                            int v0, int stride) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        first[i] = make_uint4(0, 0, 0, 0);
        if (a.dx_in != nullptr && v0 + i * stride < nvec) first[i] = ld_inout_v4(in + v0 + i * stride);
    }
}

// Adds the vectors tid, tid + stride, ... (kVec at a time) of a token's n rows, kRows rows at
// a time in flight, in slot order, the addend first.
template <int kVec, int kRows>
__device__ __forceinline__ void add_rows(const DispatchBwdArgs& a, const long long* rows, int n, const uint4* in,
                                         uint4* out, int nvec, uint4 (&first)[kVec], int tid, int stride) {
    const uint4* src = reinterpret_cast<const uint4*>(a.dperm_x);
    for (int v0 = tid; v0 < nvec; v0 += kVec * stride) {
        if (v0 != tid) load_addend<kVec>(a, first, in, nvec, v0, stride);
        float acc[kVec][8];
        for (int d0 = 0; d0 == 0 || d0 < n; d0 += kRows) {
            uint4 buf[kRows][kVec];
#pragma unroll
            for (int r = 0; r < kRows; ++r)
                if (d0 + r < n) {
                    const uint4* row = src + rows[d0 + r] + v0;
#pragma unroll
                    for (int i = 0; i < kVec; ++i)
                        if (v0 + i * stride < nvec) buf[r][i] = ld_stream_v4(row + i * stride);
                }
            if (d0 == 0) {
#pragma unroll
                for (int i = 0; i < kVec; ++i) unpack8(acc[i], first[i]);
            }
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                if (d0 + r >= n) continue;
#pragma unroll
                for (int i = 0; i < kVec; ++i) {
                    float f[8];
                    unpack8(f, buf[r][i]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) acc[i][e] += f[e];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            if (v0 + i * stride < nvec) st_v4(out + v0 + i * stride, pack8(acc[i]));
    }
}

// A token per CTA, or per warp where rows are short (per_warp): the first warp, or the token's,
// lists the token's rows, then every thread adds its vectors of them. kVec and kRows follow
// from k, so that about eight vectors are in flight per thread however few rows a token has
// (2170 x 4752 top-2: 15.4 us instead of 20 us with one vector at a time). CTAs of 64 threads:
// 16384 x 4096 top-8 with the addend in 202 us (6.67 TB/s, 0.98 of a measured copy), 207 us
// with 256 threads and 238 us with 512, which wait longer for their lists; a warp per row up
// to 2048 channels (8000 x 1024 top-6: 22.6 us instead of 24.9 us), not above (16384 x 4096:
// 217 us). Few tokens: more threads each (281 x 6320 top-9 9.4 us instead of 32.6 us; 20 x
// 4024 top-10 3.2 us instead of 6.2 us).
template <int kVec, int kRows>
__global__ void __maxnreg__((kVec == 1 ? 64 : 72)) dispatch_bwd_kernel(DispatchBwdArgs a, int per_warp) {
    grid_dependency_wait();
    __shared__ long long s_row[kSortWarps][kMaxTopk];
    __shared__ int s_n[kSortWarps];
    const int lane = lane_id();
    const int warp = static_cast<int>(threadIdx.x >> 5);
    const int nvec = a.H / 8;
    const int t = per_warp ? static_cast<int>(blockIdx.x * (blockDim.x >> 5)) + warp : static_cast<int>(blockIdx.x);
    const int mine = per_warp ? warp : 0;
    const uint4* const in = reinterpret_cast<const uint4*>(a.dx_in) + static_cast<size_t>(t) * nvec;
    const int first_v = per_warp ? lane : static_cast<int>(threadIdx.x);
    const int stride = per_warp ? 32 : static_cast<int>(blockDim.x);
    uint4 first[kVec];  // the addend's first vectors, requested before the token's rows are known
    load_addend<kVec>(a, first, in, t < a.T ? nvec : 0, first_v, stride);
    float dw = 0.0f;
    if (t < a.T && (per_warp || warp == 0)) {
        const size_t entry = static_cast<size_t>(t) * a.k + lane;
        long long row = -1;
        if (lane < a.k) {
            row = entry_row(a.topk_idx, a.offsets, a.eslot, entry, a.E, a.E / a.R, a.max_rows);
            if (a.dtopk_w != nullptr && row >= 0) dw = __ldg(a.dperm_w + row);  // stored after the rows
        }
        const uint32_t m = __ballot_sync(kFullMask, row >= 0);
        if (row >= 0) s_row[mine][__popc(m & lanemask_lt())] = row * nvec;
        if (__any_sync(kFullMask, row == -2) && lane == 0) raise_flag(a.status, EP_FLAG_CAPACITY);
        if (lane == 0) s_n[mine] = __popc(m);
        __syncwarp();
    }
    if (!per_warp) __syncthreads();
    if (t < a.T) {
        uint4* const out = reinterpret_cast<uint4*>(a.dx) + static_cast<size_t>(t) * nvec;
        add_rows<kVec, kRows>(a, s_row[mine], s_n[mine], in, out, nvec, first, first_v, stride);
        if ((per_warp || warp == 0) && lane < a.k && a.dtopk_w != nullptr)
            a.dtopk_w[static_cast<size_t>(t) * a.k + lane] = dw;
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
    const long long entries = static_cast<long long>(T) * k;
    // Few entries: enough warps on each row to fill the GPU (an SM holds 32 warps). Many: short
    // rows take part of a warp, so that its 4 vectors a lane are all of use (6933 x 192 top-7
    // 9.4 us instead of 17.6 us, 8000 x 512 top-6 20.1 us instead of 24.7 us). Otherwise a warp a
    // row, and CTAs of a token's entries or an even part of them.
    const long long per_sm = entries / sm_count();
    auto kernel = combine_bwd_kernel<32>;
    int lanes = 32, threads = 32 * kWarps;
    if (per_sm < kFewEntries) {
        kernel = combine_bwd_kernel<128>, lanes = 128;
    } else if (H <= 256) {
        kernel = combine_bwd_kernel<8>, lanes = 8;
    } else if (H <= 512) {
        kernel = combine_bwd_kernel<16>, lanes = 16;
    } else {
        const int parts = (k + kWarps - 1) / kWarps;
        threads = 32 * ((k + parts - 1) / parts);
    }
    // many short rows: two rounds a CTA
    const int rounds = H <= kShortRowH && entries * lanes >= 32LL * sm_count() * (4 * 4 * kWarps) ? 2 : 1;
    const int count = threads / lanes * rounds;
    const long long grid = (entries + count - 1) / count;
    if (grid > 0x7fffffffLL) return EP_ERR_INVALID;
    return launch_dependent(kernel, dim3(static_cast<unsigned>(grid)), dim3(threads), 0, as_stream(stream), a, count);
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
    auto kernel = k == 1 ? dispatch_bwd_kernel<4, 1> : k <= 4 ? dispatch_bwd_kernel<2, 4> : dispatch_bwd_kernel<1, 8>;
    const int vec = k == 1 ? 4 : k <= 4 ? 2 : 1;
    if (H <= kWarpRowH && T >= 16 * sm_count())
        return launch_dependent(kernel, dim3(static_cast<unsigned>(T / 4 + (T % 4 != 0))), dim3(128), 0,
                                as_stream(stream), a, 1);
    // as many threads as the row has vectors, no fewer than fill the GPU
    const int fill = (kSortFill * sm_count() / T + 31) / 32 * 32;
    const int most = fill < kSortThreads ? kSortThreads : fill < 32 * kSortWarps ? fill : 32 * kSortWarps;
    const int steps = (H / 8 - 1) / (vec * most) + 1;  // all steps with as many threads
    const int threads = ((H / 8 - 1) / (vec * steps) + 32) / 32 * 32;
    return launch_dependent(kernel, dim3(static_cast<unsigned>(T)), dim3(threads), 0, as_stream(stream), a, 0);
}
