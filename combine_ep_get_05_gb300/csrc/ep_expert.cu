// ep_expert.cu -- the experts' gated feed-forward block over the expert-major slabs: the
// products of every expert's rows with its weights, and their gradients (include/ep.h).
//
// One kernel for all five: C[i][j] = sum over k of A[i][k] * B[j][k] in fp32, i a row of the
// expert (of the weights, in their gradient), j an output channel, with the operator's
// arithmetic on the finished sums. A CTA takes 128 channels of an expert and walks the
// expert's rows 32 at a time: tiles of 16 k in shared memory, 16 sums a thread, a row's 128
// channels in one warp.
#include "ep_expert.cuh"

namespace {

using namespace ep;

enum Op { kGateUp, kDown, kDownBwd, kGateUpBwd, kWgrad };

constexpr int kRows = 32, kCols = 128, kStep = 16, kThreads = 256;

struct ExpertArgs {
    const uint16_t* a;  // rows (the output's gradient, in kWgrad)
    const uint16_t* b;  // weights (the rows, in kWgrad)
    const uint16_t* pre;
    const uint8_t* pre_q;
    const uint16_t* pre_scales;
    const int32_t* offsets;
    int act;
    int N, K;  // output channels (one half of them in kGateUp and kDownBwd); products of a sum
    int E, R, max_rows;
    uint16_t *out, *out_pre, *out_scales;
    uint8_t* out_q;
    int32_t* status;
};

__device__ __forceinline__ float bf16_at(const uint16_t* p, size_t i) {
    return __uint_as_float(static_cast<uint32_t>(p[i]) << 16);
}
__device__ __forceinline__ uint16_t bf16_rn(float v) { return static_cast<uint16_t>(pack_bf16x2_rn(v, 0.0f)); }

template <int kOp>
__global__ void __launch_bounds__(kThreads) expert_kernel(ExpertArgs g) {
    constexpr int kHalves = kOp == kGateUp ? 2 : 1;
    __shared__ float s_a[kStep][kRows + 1];
    __shared__ float s_b[kHalves][kStep][kCols + 1];
    const int e = static_cast<int>(blockIdx.y);
    const int col0 = static_cast<int>(blockIdx.x) * kCols;
    const int tid = static_cast<int>(threadIdx.x), tx = tid % 32, ty = tid / 32;
    const ExpertRows rows = expert_rows(g.offsets, e, g.E / g.R, g.max_rows);
    if (rows.dropped && blockIdx.x == 0 && tid == 0) raise_flag(g.status, EP_FLAG_CAPACITY);
    const int I = kOp == kWgrad ? g.K : rows.count;  // kWgrad: K is the number of its rows' channels
    const int K = kOp == kWgrad ? rows.count : g.K;
    const size_t N = static_cast<size_t>(g.N);
    for (int row0 = 0; row0 < I; row0 += kRows) {
        float c[kHalves][4][4] = {};
        for (int k0 = 0; k0 < K; k0 += kStep) {
            __syncthreads();
            for (int n = tid; n < kRows * kStep; n += kThreads) {
                const int i = n / kStep, k = n % kStep;
                float v = 0.0f;
                if (row0 + i < I && k0 + k < K) {
                    if (kOp == kWgrad)
                        v = bf16_at(g.a, static_cast<size_t>(rows.first + k0 + k) * I + row0 + i);
                    else
                        v = bf16_at(g.a, static_cast<size_t>(rows.first + row0 + i) * K + k0 + k);
                }
                s_a[k][i] = v;
            }
            for (int n = tid; n < kHalves * kCols * kStep; n += kThreads) {
                const int half = n / (kCols * kStep), m = n % (kCols * kStep);
                // consecutive threads along what is contiguous in memory
                const bool k_major = kOp == kGateUp || kOp == kDown;
                const int j = k_major ? m / kStep : m % kCols, k = k_major ? m % kStep : m / kCols;
                float v = 0.0f;
                if (col0 + j < g.N && k0 + k < K) {
                    size_t at;
                    if (kOp == kWgrad)
                        at = static_cast<size_t>(rows.first + k0 + k) * N + col0 + j;
                    else if (k_major)
                        at = ((static_cast<size_t>(e) * kHalves + half) * N + col0 + j) * K + k0 + k;
                    else
                        at = (static_cast<size_t>(e) * K + k0 + k) * N + col0 + j;
                    v = bf16_at(g.b, at);
                }
                s_b[half][k][j] = v;
            }
            __syncthreads();
            for (int k = 0; k < kStep; ++k)
                for (int half = 0; half < kHalves; ++half)
                    for (int i = 0; i < 4; ++i)
                        for (int j = 0; j < 4; ++j)
                            c[half][i][j] = fmaf(s_a[k][ty * 4 + i], s_b[half][k][tx + 32 * j], c[half][i][j]);
        }
        for (int i = 0; i < 4; ++i) {
            const int row = row0 + ty * 4 + i;
            if (row >= I) break;  // the whole warp
            const size_t at = kOp == kWgrad ? static_cast<size_t>(e) * I + row : static_cast<size_t>(rows.first + row);
            float rcp[kHalves], scale[kHalves];
            if (kOp == kGateUp && g.out_q != nullptr) {
                for (int half = 0; half < kHalves; ++half) {
                    float amax = 0.0f;
                    for (int j = 0; j < 4; ++j) amax = fmaxf(amax, fabsf(c[half][i][j]));
                    for (int d = 16; d > 0; d /= 2) amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, d));
                    scale[half] = checkpoint_scale(amax);
                    rcp[half] = checkpoint_rcp(scale[half]);
                    if (tx == 0)
                        g.out_scales[(at * 2 * N + half * N + col0) / kCols] = bf16_rn(scale[half]);
                }
            }
            for (int j = 0; j < 4; ++j) {
                const int col = col0 + tx + 32 * j;
                if (col >= g.N) continue;
                const float v = c[0][i][j];
                if (kOp == kGateUp) {
                    const float up = c[kHalves - 1][i][j];
                    g.out[at * N + col] = bf16_rn(v * gate_of(v, g.act).s * up);
                    for (int half = 0; half < kHalves; ++half) {
                        const size_t to = at * 2 * N + half * N + col;
                        if (g.out_pre != nullptr) g.out_pre[to] = bf16_rn(c[half][i][j]);
                        if (g.out_q != nullptr)
                            g.out_q[to] = static_cast<uint8_t>(pack_e4m3x2_rn_sat(
                                checkpoint_quotient(c[half][i][j], scale[half], rcp[half]), 0.0f));
                    }
                } else if (kOp == kDownBwd) {
                    float of[2];
                    for (int half = 0; half < 2; ++half) {
                        const size_t from = at * 2 * N + half * N + col;
                        if (g.pre != nullptr)
                            of[half] = bf16_at(g.pre, from);
                        else
                            of[half] = f16_to_f32(e4m3x2_to_f16x2(g.pre_q[from]) & 0xffffu) *
                                       bf16_at(g.pre_scales, from / kCols);
                    }
                    const Gate s = gate_of(of[0], g.act);
                    const float act = of[0] * s.s;
                    g.out_pre[at * 2 * N + col] = bf16_rn(v * of[1] * (s.s + act * (1.0f - s.s) * s.slope));
                    g.out_pre[at * 2 * N + N + col] = bf16_rn(v * act);
                    if (g.out != nullptr) g.out[at * N + col] = bf16_rn(act * of[1]);
                } else {
                    g.out[at * N + col] = bf16_rn(v);
                }
            }
        }
    }
}

bool valid(int E, int R, int max_rows) {
    return R >= 1 && R <= 256 && E >= 1 && E <= 8192 && E % R == 0 && max_rows >= 0 &&
           static_cast<long long>(R) * max_rows < (1ll << 31);
}
bool valid_width(int n, int most) { return n >= 8 && n <= most && n % 8 == 0; }
constexpr int kMostWidth = 65536;

template <int kOp>
ep_status_t launch(const ExpertArgs& g, void* stream) {
    const dim3 grid((g.N + kCols - 1) / kCols, g.E);
    expert_kernel<kOp><<<grid, kThreads, 0, as_stream(stream)>>>(g);
    return check_launch();
}

}  // namespace

extern "C" {

ep_status_t ep_expert_gate_up(const void* x, const void* w_gate_up, const int32_t* expert_offsets, ep_act_t act,
                              int32_t H, int32_t F, int32_t E, int32_t R, int32_t max_rows, void* h, void* pre,
                              uint8_t* pre_q, void* pre_scales, int32_t* status, void* stream) {
    if (!valid(E, R, max_rows) || !valid_width(H, kMostWidth) || !valid_width(F, kMostWidth)) return EP_ERR_INVALID;
    if (act != EP_ACT_SILU && act != EP_ACT_GELU) return EP_ERR_INVALID;
    if ((pre_q == nullptr) != (pre_scales == nullptr) || (pre_q != nullptr && F % 128 != 0)) return EP_ERR_INVALID;
    if (max_rows == 0) return EP_OK;
    if (x == nullptr || w_gate_up == nullptr || expert_offsets == nullptr || h == nullptr) return EP_ERR_INVALID;
    if (!aligned16(x) || !aligned16(w_gate_up) || !aligned16(expert_offsets) || !aligned16(h) ||
        !aligned16_or_null(pre) || !aligned16_or_null(pre_q) || !aligned16_or_null(pre_scales))
        return EP_ERR_INVALID;
    ExpertArgs g = {};
    g.a = static_cast<const uint16_t*>(x);
    g.b = static_cast<const uint16_t*>(w_gate_up);
    g.offsets = expert_offsets;
    g.act = act;
    g.N = F;
    g.K = H;
    g.E = E;
    g.R = R;
    g.max_rows = max_rows;
    g.out = static_cast<uint16_t*>(h);
    g.out_pre = static_cast<uint16_t*>(pre);
    g.out_q = pre_q;
    g.out_scales = static_cast<uint16_t*>(pre_scales);
    g.status = status;
    return launch<kGateUp>(g, stream);
}

ep_status_t ep_expert_down(const void* h, const void* w_down, const int32_t* expert_offsets, int32_t H, int32_t F,
                           int32_t E, int32_t R, int32_t max_rows, void* y, int32_t* status, void* stream) {
    if (!valid(E, R, max_rows) || !valid_width(H, kMostWidth) || !valid_width(F, kMostWidth)) return EP_ERR_INVALID;
    if (max_rows == 0) return EP_OK;
    if (h == nullptr || w_down == nullptr || expert_offsets == nullptr || y == nullptr) return EP_ERR_INVALID;
    if (!aligned16(h) || !aligned16(w_down) || !aligned16(expert_offsets) || !aligned16(y)) return EP_ERR_INVALID;
    ExpertArgs g = {};
    g.a = static_cast<const uint16_t*>(h);
    g.b = static_cast<const uint16_t*>(w_down);
    g.offsets = expert_offsets;
    g.N = H;
    g.K = F;
    g.E = E;
    g.R = R;
    g.max_rows = max_rows;
    g.out = static_cast<uint16_t*>(y);
    g.status = status;
    return launch<kDown>(g, stream);
}

ep_status_t ep_expert_down_bwd(const void* dy, const void* w_down, const void* pre, const uint8_t* pre_q,
                               const void* pre_scales, const int32_t* expert_offsets, ep_act_t act, int32_t H,
                               int32_t F, int32_t E, int32_t R, int32_t max_rows, void* dpre, void* h,
                               int32_t* status, void* stream) {
    if (!valid(E, R, max_rows) || !valid_width(H, kMostWidth) || !valid_width(F, kMostWidth)) return EP_ERR_INVALID;
    if (act != EP_ACT_SILU && act != EP_ACT_GELU) return EP_ERR_INVALID;
    if ((pre_q == nullptr) != (pre_scales == nullptr) || (pre_q != nullptr && F % 128 != 0)) return EP_ERR_INVALID;
    if (max_rows == 0) return EP_OK;
    if ((pre == nullptr) == (pre_q == nullptr)) return EP_ERR_INVALID;
    if (dy == nullptr || w_down == nullptr || expert_offsets == nullptr || dpre == nullptr) return EP_ERR_INVALID;
    if (!aligned16(dy) || !aligned16(w_down) || !aligned16(expert_offsets) || !aligned16(dpre) ||
        !aligned16_or_null(pre) || !aligned16_or_null(pre_q) || !aligned16_or_null(pre_scales) || !aligned16_or_null(h))
        return EP_ERR_INVALID;
    ExpertArgs g = {};
    g.a = static_cast<const uint16_t*>(dy);
    g.b = static_cast<const uint16_t*>(w_down);
    g.pre = static_cast<const uint16_t*>(pre);
    g.pre_q = pre_q;
    g.pre_scales = static_cast<const uint16_t*>(pre_scales);
    g.offsets = expert_offsets;
    g.act = act;
    g.N = F;
    g.K = H;
    g.E = E;
    g.R = R;
    g.max_rows = max_rows;
    g.out = static_cast<uint16_t*>(h);
    g.out_pre = static_cast<uint16_t*>(dpre);
    g.status = status;
    return launch<kDownBwd>(g, stream);
}

ep_status_t ep_expert_gate_up_bwd(const void* dpre, const void* w_gate_up, const int32_t* expert_offsets, int32_t H,
                                  int32_t F, int32_t E, int32_t R, int32_t max_rows, void* dx, int32_t* status,
                                  void* stream) {
    if (!valid(E, R, max_rows) || !valid_width(H, kMostWidth) || !valid_width(F, kMostWidth)) return EP_ERR_INVALID;
    if (max_rows == 0) return EP_OK;
    if (dpre == nullptr || w_gate_up == nullptr || expert_offsets == nullptr || dx == nullptr) return EP_ERR_INVALID;
    if (!aligned16(dpre) || !aligned16(w_gate_up) || !aligned16(expert_offsets) || !aligned16(dx))
        return EP_ERR_INVALID;
    ExpertArgs g = {};
    g.a = static_cast<const uint16_t*>(dpre);
    g.b = static_cast<const uint16_t*>(w_gate_up);
    g.offsets = expert_offsets;
    g.N = H;
    g.K = 2 * F;
    g.E = E;
    g.R = R;
    g.max_rows = max_rows;
    g.out = static_cast<uint16_t*>(dx);
    g.status = status;
    return launch<kGateUpBwd>(g, stream);
}

ep_status_t ep_expert_wgrad(const void* dout, const void* rows, const int32_t* expert_offsets, int32_t I, int32_t J,
                            int32_t E, int32_t R, int32_t max_rows, void* dw, int32_t* status, void* stream) {
    if (!valid(E, R, max_rows) || !valid_width(I, 2 * kMostWidth) || !valid_width(J, 2 * kMostWidth))
        return EP_ERR_INVALID;
    if (expert_offsets == nullptr || dw == nullptr || !aligned16(expert_offsets) || !aligned16(dw))
        return EP_ERR_INVALID;
    if (max_rows > 0 && (dout == nullptr || rows == nullptr || !aligned16(dout) || !aligned16(rows)))
        return EP_ERR_INVALID;
    ExpertArgs g = {};
    g.a = static_cast<const uint16_t*>(dout);
    g.b = static_cast<const uint16_t*>(rows);
    g.offsets = expert_offsets;
    g.N = J;
    g.K = I;
    g.E = E;
    g.R = R;
    g.max_rows = max_rows;
    g.out = static_cast<uint16_t*>(dw);
    g.status = status;
    return launch<kWgrad>(g, stream);
}

}  // extern "C"
