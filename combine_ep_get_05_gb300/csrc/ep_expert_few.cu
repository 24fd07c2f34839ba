// ep_expert_few.cu -- the experts' products for a few rows (a decoded token, a small batch): the
// weights' stream from HBM is all that counts, and tiles of 256 channels are too few to fill the
// GPU with it.
//
// A unit of work is 32 output channels of an expert (in the gated product, 16 and their gate and
// up) by 8, 16 or 32 of its rows: m16n8k16 products with the weights as A. A warp takes every
// eighth 64 k of a unit; a thread loads 16 bytes of four weight rows and of one to four rows of x, 64 bytes a
// row over four lanes, and uses them as fragments as they are: the products of a sum may be taken
// in any order of k as long as A's and B's is the same. The sums of the eight warps are added in
// shared memory, in order.
//
// A thread's loads are asynchronous copies into its own places of a ring in shared memory, several
// steps ahead and across units, so that some 160 KB an SM are on their way at any time without a
// register; it waits for its own copies only.
#include "ep_expert.cuh"

namespace {

using namespace ep;

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kChannels = 16, kStep = 64;

// One warp's 64 k of a unit, in two parts of 32: weight rows g and g + 8 of its two halves of 16
// (gate and up, or the first and the last) and row g of each eight of x; g = lane / 4, k =
// 8 (lane % 4) and the next 7 of each part.
constexpr int kHalves = 2;

template <bool kGated, int kGroups>
struct Ring {
    static constexpr int kSlice = kGated ? kChannels : kHalves * kChannels;  // channels of a unit
    static constexpr int kRows = 8 * kGroups;
    static constexpr int kVectors = 2 * (2 * kHalves + kGroups);  // 16 bytes each, of a thread and step
    static constexpr int kStages = kGroups == 4 ? 3 : kGated && kGroups == 1 ? 5 : 4;
    static constexpr int kBytes = kStages * kVectors * kThreads * 16;
    // sums by turns, where there is room: the next need not wait for these to be read
    static constexpr int kTurns = !kGated && kGroups == 1 ? 2 : 1;
};
template <typename Ring>
struct Sums {
    float v[Ring::kTurns][kWarps][kHalves][kChannels][Ring::kRows + 1];
    int found[kWarps];
};

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Where a CTA is: a slice of an expert's channels, some of its rows, and the warp's 64 k.
struct Place {
    int expert, slice;  // the how manieth of those that have rows; of its slices
    int row0, step;
    int count;          // the expert's rows
    long long first;    // the first of them
    const uint16_t* w;  // its weights
};

__device__ __forceinline__ uint4 lds_v4(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
}
// 16 bytes into shared memory, or zeros
__device__ __forceinline__ void copy_or_zero(uint32_t to, const void* from, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16 : 0) : "memory");
}

template <bool kGated, int kGroups>
__global__ void __launch_bounds__(kThreads, 1) few_rows_kernel(FewRows g) {
    using Tr = Ring<kGated, kGroups>;
    constexpr int kRows = Tr::kRows, kVectors = Tr::kVectors;
    extern __shared__ __align__(16) unsigned char s_ring[];
    Sums<Tr>& s = *reinterpret_cast<Sums<Tr>*>(s_ring + Tr::kBytes);
    uint16_t* const s_expert = reinterpret_cast<uint16_t*>(&s + 1);  // [E] those that have rows
    const int tid = static_cast<int>(threadIdx.x), lane = tid % 32, warp = tid / 32;
    allow_dependents();
    grid_dependency_wait();  // dependent launch: inputs are ready after this

    int experts = 0;
    for (int e0 = 0; e0 < g.E; e0 += kThreads) {
        const int e = e0 + tid;
        bool has = false;
        if (e < g.E) {
            const ExpertRows r = expert_rows(g.offsets, e, g.epr, g.inv_epr, g.max_rows);
            if (r.dropped && blockIdx.x == 0) raise_flag(g.status, EP_FLAG_CAPACITY);
            has = r.count > 0;
        }
        const unsigned mask = __ballot_sync(kFullMask, has);
        if (lane == 0) s.found[warp] = __popc(mask);
        __syncthreads();
        int at = experts;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) at += s.found[w];
            experts += s.found[w];
        }
        if (has) s_expert[at + __popc(mask & lanemask_lt())] = static_cast<uint16_t>(e);
        __syncthreads();
    }

    const int C = g.C, K = g.K, across = (C + Tr::kSlice - 1) / Tr::kSlice;
    const int steps = ((K + kStep - 1) / kStep + kWarps - 1) / kWarps;  // of every warp
    const int row = lane / 4, part = lane % 4 * 8;
    const uint32_t mine = smem_addr(s_ring) + tid * 16;  // vector v of stage i: 16 kThreads (i kVectors + v) on
    // units are dealt to the CTAs in turn: so many experts and slices further each time
    const int over = static_cast<int>(gridDim.x) / across, rest = static_cast<int>(gridDim.x) - over * across;

    const auto enter = [&](Place& p) {  // an expert
        if (p.expert >= experts) return;
        const int e = s_expert[p.expert];
        const ExpertRows r = expert_rows(g.offsets, e, g.epr, g.inv_epr, g.max_rows);
        p.count = r.count;
        p.first = r.first;
        p.w = g.w + static_cast<size_t>(e) * (kGated ? 2 : 1) * C * K;
    };
    const auto advance = [&](Place& p) {
        if (++p.step < steps) return;
        p.step = 0;
        p.row0 += kRows;
        if (p.row0 < p.count) return;
        p.row0 = 0;
        const int carry = p.slice + rest >= across ? 1 : 0;
        p.slice += rest - carry * across;
        p.expert += over + carry;
        if (over + carry > 0) enter(p);
    };
    const auto load = [&](const Place& p, int stage) {
        if (p.expert < experts) {
            uint32_t to = mine + stage * (kVectors * kThreads * 16);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int k = (p.step * kWarps + warp) * kStep + 32 * i + part;
#pragma unroll
                for (int half = 0; half < kHalves; ++half)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int c = p.slice * Tr::kSlice + (kGated ? 0 : half * kChannels) + row + 8 * j;
                        const bool there = k < K && c < C;
                        const size_t line = static_cast<size_t>(kGated ? half * C : 0) + c;
                        copy_or_zero(to, there ? p.w + line * K + k : p.w, there);
                        to += kThreads * 16;
                    }
#pragma unroll
                for (int j = 0; j < kGroups; ++j) {
                    const int n = p.row0 + 8 * j + row;
                    const bool there = k < K && n < p.count;
                    copy_or_zero(to, there ? g.x + static_cast<size_t>(p.first + n) * K + k : g.x, there);
                    to += kThreads * 16;
                }
            }
        }
        cp_async_commit();  // an empty group past the end
    };

    Place here, front;
    here.expert = static_cast<int>(blockIdx.x) / across;
    here.slice = static_cast<int>(blockIdx.x) - here.expert * across;
    here.row0 = here.step = 0;
    enter(here);
    front = here;
    for (int i = 0; i < Tr::kStages - 1; ++i) {
        load(front, i);
        if (front.expert < experts) advance(front);
    }
    float sum[kHalves][kGroups][4] = {};
    int stage = 0, turn = 0;
    while (here.expert < experts) {
        cp_async_wait<Tr::kStages - 2>();
        const uint32_t from = mine + stage * (kVectors * kThreads * 16);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t at = from + i * (2 * kHalves + kGroups) * kThreads * 16;
            uint4 x[kGroups];
#pragma unroll
            for (int j = 0; j < kGroups; ++j) x[j] = lds_v4(at + (2 * kHalves + j) * kThreads * 16);
#pragma unroll
            for (int half = 0; half < kHalves; ++half) {
                const uint4 a = lds_v4(at + 2 * half * kThreads * 16), b = lds_v4(at + (2 * half + 1) * kThreads * 16);
#pragma unroll
                for (int j = 0; j < kGroups; ++j) {
                    mma(sum[half][j], a.x, b.x, a.y, b.y, x[j].x, x[j].y);
                    mma(sum[half][j], a.z, b.z, a.w, b.w, x[j].z, x[j].w);
                }
            }
        }
        // the stage before this one, read a step ago, is filled again
        load(front, stage == 0 ? Tr::kStages - 1 : stage - 1);
        if (front.expert < experts) advance(front);
        if (here.step == steps - 1) {
#pragma unroll
            for (int half = 0; half < kHalves; ++half)
#pragma unroll
                for (int j = 0; j < kGroups; ++j) {
                    float(*const to)[kRows + 1] = s.v[turn][warp][half];
                    float(&v)[4] = sum[half][j];
                    const int n = 8 * j + lane % 4 * 2;
                    to[row][n] = v[0];
                    to[row][n + 1] = v[1];
                    to[row + 8][n] = v[2];
                    to[row + 8][n + 1] = v[3];
                    v[0] = v[1] = v[2] = v[3] = 0.0f;
                }
            __syncthreads();
            const int c = tid % Tr::kSlice, channel = here.slice * Tr::kSlice + c;
            for (int r = tid / Tr::kSlice; r < kRows && here.row0 + r < here.count; r += kThreads / Tr::kSlice) {
                if (channel >= C) break;
                float v = 0.0f, up = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    v += s.v[turn][w][c / kChannels][c % kChannels][r];
                    if (kGated) up += s.v[turn][w][1][c][r];
                }
                if (kGated) v = v * (g.act == EP_ACT_GELU ? sigmoid_of<true>(v) : sigmoid_of<false>(v)) * up;
                g.out[static_cast<size_t>(here.first + here.row0 + r) * C + channel] =
                    static_cast<uint16_t>(pack_bf16x2_rn(v, 0.0f));
            }
            if (Tr::kTurns == 1)
                __syncthreads();
            else
                turn ^= 1;
        }
        advance(here);
        if (++stage == Tr::kStages) stage = 0;
    }
}

template <bool kGated, int kGroups>
ep_status_t launch(const FewRows& g, void* stream) {
    using Tr = Ring<kGated, kGroups>;
    static std::atomic<int> ready[kMaxDevices];
    constexpr size_t fixed = Tr::kBytes + sizeof(Sums<Tr>), most = fixed + 2 * (kGroups == 4 ? 8 : 8192);  // 32 at once: for one or two experts
    static_assert(most <= 227 * 1024);
    const ep_status_t st = ensure_dynamic_smem(ready, few_rows_kernel<kGated, kGroups>, static_cast<int>(most));
    if (st != EP_OK) return st;
    return launch_dependent(few_rows_kernel<kGated, kGroups>, dim3(static_cast<unsigned>(sm_count())), dim3(kThreads),
                            fixed + 2 * static_cast<size_t>(g.E), as_stream(stream), g);
}

}  // namespace

namespace ep {

int few_rows_at_once(int E, int R, int max_rows, long long weights, bool gated) {
    const long long all = static_cast<long long>(R) * max_rows, total = E * weights;
    if (max_rows <= 8) return 8;
    if (max_rows <= 64 && all <= 4ll * E && (!gated || all <= E || total <= 512 << 20)) return 8;
    if (E <= 3 && max_rows <= 16) return 16;
    if (E <= 2 && max_rows <= 32 && (gated || weights <= 4 << 20)) return 32;
    if (E <= 8 && max_rows <= 64 && all <= 16ll * E && total <= 8 << 20) return 16;
    return 0;
}

ep_status_t launch_few_rows(const FewRows& g, bool gated, int at_once, void* stream) {
    if (at_once == 32) return gated ? launch<true, 4>(g, stream) : launch<false, 4>(g, stream);
    if (at_once == 8) return gated ? launch<true, 1>(g, stream) : launch<false, 1>(g, stream);
    return gated ? launch<true, 2>(g, stream) : launch<false, 2>(g, stream);
}

}  // namespace ep
