// ep_norm.cu -- the norm in front of an expert layer: the residual's addition with the
// root-mean-square norm, to bf16 rows (for the router) and to E4M3 rows with 1x128 scales
// (for the FP8 dispatch), and its gradient.
//
//   z = x + residual;  v = z * weight / sqrt(mean(z^2) + eps);  y = bf16(v), q = e4m3(v / scale)
//   d = rstd * (g - z * rstd^2 * mean(g z)) + dz_in,  g = dy * weight;  dweight = sum dy z rstd
//
// Each row is read once and each output written once, so HBM bandwidth is the bound (a copy
// of 265 MB runs at 6.75 TB/s here); there is no contraction for the tensor cores. Forward,
// a row per CTA with few registers (rmsnorm_kernel) comes closest, since the hardware hands
// rows to whichever SM is free: 4096 x 7168 with a bf16 residual, bf16 and E4M3 outputs in
// 40.5 us (6.55 TB/s, 0.96 of a measured copy) against 45 us for the same rows given to
// resident CTAs in turn. Where a row moves little, the weights and the CTAs' own start cost
// more than that: those rows take the resident kernel with a shared-memory ring
// (rmsnorm_ring_kernel; 8191 x 4104 bf16 without a residual in 22.1 us against 31 us).
// Sums are fp32; each output is rounded once.
#include "ep_common.cuh"
#include "ep_quant.cuh"

namespace {

using namespace ep;

constexpr int kMaxNormH = 16384;
constexpr int kBlock = 128;  // channels per E4M3 scale
constexpr int kMaxThreads = 1024;
constexpr size_t kMaxRingSmem = 200 * 1024;
// Rows that move fewer bytes than this, in and out, take the ring whatever they hold: a GPU
// starts about one CTA a nanosecond, in which HBM moves 7 KB (16384 x 264: 5.5 us against
// 16.9 us; 16384 x 1024, 8 KB a row: 22.1 us against 21.1 us).
constexpr int kRingRowBytes = 6144;
constexpr int kRingRows = 8;      // rows of a ring CTA where one warp holds a row
constexpr int kMaxParts = 512;    // rows of dweight partial sums
// Threads of a gradient CTA that has rows side by side: as many rows as fit, a CTA per SM
// (16384 x 4096 bf16: 84.0 us instead of 87.7 us with 448 threads, whose CTAs hold one such row;
// 16384 x 2048 with an fp32 stream 82.5 us instead of 100.5 us)
constexpr int kBwdThreads = 704;
// but fewer rows side by side where that leaves CTAs with less than a row for each of them:
// one per so many rows (127 x 1024, fp32 stream: 3.5 us instead of 4.4 us)
constexpr int kBwdRowsPerGroup = 64;
constexpr int kBwdRows = 6;       // rows of a gradient CTA that are worth its partial sums
constexpr int kMaxGroups = 15;    // rows side by side: a named barrier each
constexpr int kReduceRows = 32;   // partial sums a dweight reduction CTA adds at a time

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

// Arithmetic is on pairs of channels (f32x2: one instruction, two IEEE results), and the
// addresses of a thread's vectors differ by constants: at 35 instructions a channel, as in a
// plain form of these kernels, issue slots and not HBM would bound them; here it is about 20.
using f2 = unsigned long long;

__device__ __forceinline__ f2 pair(float lo, float hi) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ f2 both(float v) { return pair(v, v); }
__device__ __forceinline__ void split(float& lo, float& hi, f2 v) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 bf16_pair(uint32_t w) { return pair(bf16_lo(w), bf16_hi(w)); }
__device__ __forceinline__ uint32_t pack_pair(f2 v) {
    float lo, hi;
    split(lo, hi, v);
    return pack_bf16x2_rn(lo, hi);
}

constexpr uint32_t kMinusZeroBf16 = 0x80008000u;  // a pair of -0: what a missing addend reads as,
constexpr uint32_t kMinusZeroF32 = 0x80000000u;   // since v + -0 = v for every v, -0 included

// N / 2 words of packed bf16 (N = 4: 8 bytes, N = 8: 16 bytes). Not the read-only path: an
// output may be the same array as an input, and a thread reads its part before it writes.
template <int W>
__device__ __forceinline__ void load_words(uint32_t (&w)[W], const void* p) {
    if constexpr (W == 4) {
        const uint4 v = ld_inout_v4(p);
        w[0] = v.x;
        w[1] = v.y;
        w[2] = v.z;
        w[3] = v.w;
    } else {
        asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
    }
}

// N / 2 pairs as bf16
template <int P>
__device__ __forceinline__ void store_bf16(uint16_t* p, const f2 (&f)[P]) {
    if constexpr (P == 4) st_v4(p, make_uint4(pack_pair(f[0]), pack_pair(f[1]), pack_pair(f[2]), pack_pair(f[3])));
    else st_v2(p, pack_pair(f[0]), pack_pair(f[1]));
}

template <int P>
__device__ __forceinline__ void unpack_bf16(f2 (&f)[P], const uint32_t (&w)[P]) {
#pragma unroll
    for (int i = 0; i < P; ++i) f[i] = bf16_pair(w[i]);
}

// a thread's own words of a shared-memory ring, 8 or 16 bytes
__device__ __forceinline__ void load_shared(uint32_t (&w)[4], const unsigned char* p) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
}
__device__ __forceinline__ void load_shared(uint32_t (&w)[2], const unsigned char* p) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x;
    w[1] = v.y;
}

// byte offset of channel `at` of a stream array
template <class Carry>
__device__ __forceinline__ size_t carry_bytes(size_t at) {
    return at * (16 / Carry::kElems);
}

// a vector of the stream, 16 bytes for either type
template <class Carry>
__device__ __forceinline__ void unpack_carry(f2 (&f)[Carry::kElems / 2], const uint32_t (&w)[4]) {
    if constexpr (Carry::kElems == 8) {
        unpack_bf16(f, w);
    } else {
        f[0] = pair(__uint_as_float(w[0]), __uint_as_float(w[1]));
        f[1] = pair(__uint_as_float(w[2]), __uint_as_float(w[3]));
    }
}

template <class Carry>
__device__ __forceinline__ void store_carry(void* base, size_t at, const f2 (&f)[Carry::kElems / 2]) {
    char* p = static_cast<char*>(base) + carry_bytes<Carry>(at);
    if constexpr (Carry::kElems == 8) {
        store_bf16(reinterpret_cast<uint16_t*>(p), f);
    } else {
        float a, b, c, d;
        split(a, b, f[0]);
        split(c, d, f[1]);
        st_v4(p, make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d)));
    }
}

// A thread's kVecs * 2 P weights, kept as the words they come in: W per vector.
template <bool kF32, int P>
constexpr int kWeightWords = kF32 ? 2 * P : P;

template <bool kF32, int P, int W>
__device__ __forceinline__ void load_weight_words(uint32_t (&w)[W], const void* weight, int h) {
    const char* p = static_cast<const char*>(weight) + h * (kF32 ? 4 : 2);
    if constexpr (W == 2) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
        w[0] = v.x;
        w[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
            w[4 * i] = v.x;
            w[4 * i + 1] = v.y;
            w[4 * i + 2] = v.z;
            w[4 * i + 3] = v.w;
        }
    }
}

template <bool kF32, int P, int W>
__device__ __forceinline__ f2 weight_pair(const uint32_t (&w)[W], int e) {
    if constexpr (kF32) return pair(__uint_as_float(w[2 * e]), __uint_as_float(w[2 * e + 1]));
    else return bf16_pair(w[e]);
}

// the weights of a thread's vectors from channel h0 on, zero past the row's end
template <bool kF32, int P, int kVecs, int W>
__device__ __forceinline__ void load_weights(uint32_t (&w)[kVecs][W], const void* weight, int h0, int H) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
#pragma unroll
        for (int e = 0; e < W; ++e) w[i][e] = 0;
        const int h = h0 + i * 32 * 2 * P;
        if (h < H) load_weight_words<kF32, P>(w[i], weight, h);
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

// The E4M3 codes of a thread's vectors; G = kBlock / (2 P) lanes hold a block. A block whose
// scale is 0 (the largest magnitude is 0, or at most 224 * 2^-149, which over 448 rounds to 0)
// has every value's own code (a signed zero, or NaN); NaNs do not take part in the maximum.
// Lanes past the row's end pass zeros.
//
// The maxima of the kVecs vectors are reduced together: at each of the first log2(kVecs)
// steps a lane keeps half of its vectors and hands the other half to its partner, so that
// each lane ends up with the maximum of one vector (which one follows from its upper lane
// bits within the G) and computes one scale and one reciprocal, which the others then read.
//
// The quotient is the one of ep_quant.cuh, v / scale correctly rounded, with its sign turned:
// with n = -1 / scale rounded, p = RN(v n), e = RN(p scale + v) and RN(e n + p) =
// -RN(v / scale), zeros and their signs included, so the codes' sign bits are flipped at the end.
// The conversion's code of any NaN is 0x7F, so it leaves as 0xFF; turning the signs before the
// conversion instead gives 0x7F and takes longer (4096 x 7168 without a residual, E4M3 only,
// 23.9 us instead of 23.1 us; one token 2.11 us instead of 2.06 us).
// Scales that are not `corrected` take the division.
// Returns the scale of the lane's vector; `leads` is set in the lane that stores it, `mine`
// names the vector.
template <int kVecs, int P>
__device__ __forceinline__ float quantise(const f2 (&v)[kVecs][P], uint32_t (&code)[kVecs][P / 2], bool& leads,
                                          int& mine) {
    constexpr int G = kBlock / (2 * P);
    const int lane = lane_id();
    float amax[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        amax[i] = 0.0f;
#pragma unroll
        for (int e = 0; e < P; ++e) {
            float lo, hi;
            split(lo, hi, v[i][e]);
            amax[i] = fmaxf(amax[i], fmaxf(fabsf(lo), fabsf(hi)));
        }
    }
    mine = 0;
    int off = G / 2;
#pragma unroll
    for (int half = kVecs / 2; half >= 1; half >>= 1, off >>= 1) {
        const bool upper = (lane & off) != 0;
        mine = 2 * mine + upper;
#pragma unroll
        for (int c = 0; c < half; ++c) {
            const float keep = upper ? amax[c + half] : amax[c];
            const float give = upper ? amax[c] : amax[c + half];
            amax[c] = fmaxf(keep, __shfl_xor_sync(kFullMask, give, off));
        }
    }
    leads = (lane & (2 * off - 1)) == 0;
#pragma unroll
    for (; off >= 1; off >>= 1) amax[0] = fmaxf(amax[0], __shfl_xor_sync(kFullMask, amax[0], off));
    const float scale = scale_of(amax[0]);
    // a zero block: n = -1 and s = 1 return every value's own code
    const bool zero = scale == 0.0f;
    const float n1 = zero ? -1.0f : -__frcp_rn(scale), s1 = zero ? 1.0f : scale;
    const bool odd = !zero && !corrected(scale);
    const bool any_odd = __any_sync(kFullMask, odd);
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int from = (lane & ~(G - 1)) | (i * (G / kVecs));  // a lane of the block that holds vector i's
        const float ns = kVecs > 1 ? __shfl_sync(kFullMask, n1, from) : n1;
        const float ss = kVecs > 1 ? __shfl_sync(kFullMask, s1, from) : s1;
        const f2 n = both(ns), s = both(ss);
        float q[2 * P];
#pragma unroll
        for (int e = 0; e < P; ++e) {
            const f2 p = mul2(v[i][e], n);
            split(q[2 * e], q[2 * e + 1], fma2(fma2(p, s, v[i][e]), n, p));
        }
        if (any_odd) {  // rare: the division itself
#pragma unroll
            for (int e = 0; e < P; ++e) {
                float lo, hi;
                split(lo, hi, v[i][e]);
                q[2 * e] = -__fdiv_rn(lo, ss);
                q[2 * e + 1] = -__fdiv_rn(hi, ss);
            }
        }
#pragma unroll
        for (int e = 0; e < P / 2; ++e)
            code[i][e] = pack_e4m3x4_rn_sat(q[4 * e], q[4 * e + 1], q[4 * e + 2], q[4 * e + 3]) ^ 0x80808080u;
    }
    return scale;
}

// Words of a vector before its loads: a missing input reads as -0, the place past the row's
// end as 0.
template <class Carry>
__device__ __forceinline__ void no_words(uint32_t (&xw)[Carry::kElems / 2], uint32_t (&rw)[4], bool in) {
#pragma unroll
    for (int e = 0; e < Carry::kElems / 2; ++e) xw[e] = in ? kMinusZeroBf16 : 0u;
#pragma unroll
    for (int e = 0; e < 4; ++e) rw[e] = !in ? 0u : Carry::kElems == 8 ? kMinusZeroBf16 : kMinusZeroF32;
}

// z = x + residual of a vector from its words; returns sq plus the squares
template <class Carry>
__device__ __forceinline__ f2 add_residual(f2 (&z)[Carry::kElems / 2], const uint32_t (&xw)[Carry::kElems / 2],
                                           const uint32_t (&rw)[4], f2 sq) {
    constexpr int P = Carry::kElems / 2;
    f2 x[P], r[P];
    unpack_bf16(x, xw);
    unpack_carry<Carry>(r, rw);
#pragma unroll
    for (int e = 0; e < P; ++e) {
        z[e] = add2(x[e], r[e]);
        sq = fma2(z[e], z[e], sq);
    }
    return sq;
}

__device__ __forceinline__ float sum2(f2 v) {
    float lo, hi;
    split(lo, hi, v);
    return lo + hi;
}

// The sum over the CTA's nt threads, the same in every thread. s_part holds 32 values that
// nobody else reads or writes until the next barrier but one.
__device__ __forceinline__ float block_sum(float v, int nt, float* s_part) {
    v = warp_sum(v);
    if (nt > 32) {
        const int lane = lane_id();
        if (lane == 0) s_part[threadIdx.x >> 5] = v;
        __syncthreads();
        v = warp_sum(lane < (nt >> 5) ? s_part[lane] : 0.0f);
    }
    return v;
}

// Where a thread's vectors lie: a warp takes kVecs * 32 consecutive vectors of the row, vector
// i of lane l being number i * 32 + l of them, so that a warp's accesses are whole lines and
// all of a thread's vectors are at fixed distances from its first.
template <class Carry, int kVecs>
__device__ __forceinline__ int first_channel(int thread) {
    return ((thread >> 5) * (kVecs * 32) + (thread & 31)) * Carry::kElems;
}

// The row's outputs from its z (zero past the row's end) and reciprocal root mean square;
// at: the thread's first channel h0 of the row in the whole array.
template <class Carry, int kVecs, bool kFp8, bool kWF32, int W>
__device__ __forceinline__ void write_row(const NormArgs& a, size_t at, int h0, const uint32_t (&w)[kVecs][W],
                                          const f2 (&z)[kVecs][Carry::kElems / 2], float rstd) {
    constexpr int N = Carry::kElems, P = N / 2;
    const f2 r = both(rstd);
    f2 v[kVecs][P];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
#pragma unroll
        for (int e = 0; e < P; ++e) v[i][e] = mul2(mul2(z[i][e], r), weight_pair<kWF32, P>(w[i], e));
        if (a.y != nullptr && h0 + i * 32 * N < a.H) store_bf16(a.y + at + i * 32 * N, v[i]);
    }
    if constexpr (kFp8) {
        uint32_t code[kVecs][P / 2];
        bool leads;
        int mine;
        const float scale = quantise(v, code, leads, mine);
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            if (h0 + i * 32 * N < a.H) {
                uint8_t* const q = a.y_q + at + i * 32 * N;
                if constexpr (P == 4) st_v2(q, code[i][0], code[i][1]);
                else *reinterpret_cast<uint32_t*>(q) = code[i][0];
            }
        }
        if (leads && h0 + mine * 32 * N < a.H) a.y_scales[(at + mine * 32 * N) / kBlock] = scale;
    }
}

// One CTA per row; the row stays in registers between the sum of squares and the outputs.
// 4 vectors a thread at 72 registers keep four 7168-channel rows in flight on an SM; with 64 or
// 80 registers, or 2 vectors a thread, 4096 x 7168 takes 41 to 44 us instead of 40.5. One row
// of 7168 takes 2.0 us (2.1 us with a thread for every vector), 128 rows of an fp32 stream 2.4 us.
template <class Carry, int kVecs, bool kFp8, bool kWF32>
__global__ void __maxnreg__((Carry::kElems == 8 && kVecs == 4 ? 72 : 64)) rmsnorm_kernel(NormArgs a) {
    constexpr int N = Carry::kElems, P = N / 2;
    __shared__ float s_part[32];
    grid_dependency_wait();  // dependent launch: inputs are ready after this
    allow_dependents();
    const int h0 = first_channel<Carry, kVecs>(static_cast<int>(threadIdx.x));
    const size_t at = static_cast<size_t>(blockIdx.x) * a.H + h0;
    const char* const res = static_cast<const char*>(a.residual) + carry_bytes<Carry>(at);
    uint32_t xw[kVecs][P], rw[kVecs][4];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const bool in = h0 + i * 32 * N < a.H;
        no_words<Carry>(xw[i], rw[i], in);
        if (in && a.x != nullptr) load_words(xw[i], a.x + at + i * 32 * N);
        if (in && a.residual != nullptr) load_words(rw[i], res + i * 32 * 16);
    }
    uint32_t w[kVecs][kWeightWords<kWF32, P>];
    load_weights<kWF32, P>(w, a.weight, h0, a.H);
    f2 z[kVecs][P], sq = 0;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        sq = add_residual<Carry>(z[i], xw[i], rw[i], sq);
        if (h0 + i * 32 * N < a.H && a.residual_out != nullptr)
            store_carry<Carry>(a.residual_out, at + i * 32 * N, z[i]);
    }
    const float ss = block_sum(sum2(sq), static_cast<int>(blockDim.x), s_part);
    write_row<Carry, kVecs, kFp8, kWF32>(a, at, h0, w, z, rsqrtf(fmaf(ss, a.inv_h, a.eps)));
}

// Bytes of one row of a ring: per thread and vector 16 of each stream array and 2 per channel
// of a bf16 array.
template <class Carry>
inline size_t ring_row_bytes(int nt, int vecs, int streams) {
    return static_cast<size_t>(nt) * vecs * (16 * streams + 2 * Carry::kElems);
}

// Fills a thread's places of a ring's array that no copy ever writes: with `absent` where the
// array is missing, with zeros past the row's end.
template <int kBytes, int kVecs>
__device__ __forceinline__ void fill_ring(unsigned char* at, int stage_bytes, int stages, bool has, uint32_t absent,
                                          int vectors_in) {
    for (int s = 0; s < stages; ++s) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            const bool in = i < vectors_in;
            if (has && in) continue;
            uint32_t* to = reinterpret_cast<uint32_t*>(at + s * stage_bytes + i * 32 * kBytes);
#pragma unroll
            for (int e = 0; e < kBytes / 4; ++e) to[e] = in ? absent : 0u;
        }
    }
}

// Many rows: a CTA takes rows blockIdx.x, + gridDim.x, ... and every thread copies its
// vectors of the next kStages - 1 rows into its own places of a shared-memory ring while it
// works on the current one, so reads stay in flight through the sums and the stores. No
// barrier guards the ring: a thread reads only what it copied itself. A missing input's
// places hold -0 and those past the row's end 0, so the arithmetic has no cases. The weights
// stay in registers over all rows.
// A row that one warp holds (kMany) needs no barrier, and its CTA has kRingRows of them.
template <class Carry, int kVecs, int kStages, bool kFp8, bool kWF32, bool kMany>
__global__ void __maxnreg__(64) rmsnorm_ring_kernel(NormArgs a, int T) {
    constexpr int N = Carry::kElems, P = N / 2;
    extern __shared__ __align__(16) unsigned char s_all[];
    __shared__ float s_part[2][32];
    const int nt = kMany ? 32 : static_cast<int>(blockDim.x);  // threads of a row
    const int rows = kMany ? kRingRows : 1;                   // of the CTA
    const int group = kMany ? static_cast<int>(threadIdx.x) >> 5 : 0;
    const int h0 = first_channel<Carry, kVecs>(kMany ? lane_id() : static_cast<int>(threadIdx.x));
    const bool has_x = a.x != nullptr, has_r = a.residual != nullptr;
    const int r_bytes = kVecs * nt * 16;  // of a stage
    const int stage_bytes = r_bytes + kVecs * nt * 2 * N;
    unsigned char* const s_ring = s_all + group * (kStages * stage_bytes);
    unsigned char* const r_ring = s_ring + h0 * (16 / N);
    unsigned char* const x_ring = s_ring + r_bytes + h0 * 2;
    const int vectors_in = h0 < a.H ? (a.H - h0 + 32 * N - 1) / (32 * N) : 0;
    fill_ring<16, kVecs>(r_ring, stage_bytes, kStages, has_r, N == 8 ? kMinusZeroBf16 : kMinusZeroF32, vectors_in);
    fill_ring<2 * N, kVecs>(x_ring, stage_bytes, kStages, has_x, kMinusZeroBf16, vectors_in);
    grid_dependency_wait();
    auto issue = [&](uint32_t t, int st) {
        if (t < static_cast<uint32_t>(T)) {
            const size_t at = static_cast<size_t>(t) * a.H + h0;
            const uint16_t* const x = a.x + at;
            const char* const r = static_cast<const char*>(a.residual) + carry_bytes<Carry>(at);
            unsigned char* const xs = x_ring + st * stage_bytes;
            unsigned char* const rs = r_ring + st * stage_bytes;
            if (has_x) {
#pragma unroll
                for (int i = 0; i < kVecs; ++i)
                    if (h0 + i * 32 * N < a.H) {
                        if constexpr (N == 8) cp_async16(xs + i * 32 * 16, x + i * 32 * N);
                        else cp_async8(xs + i * 32 * 8, x + i * 32 * N);
                    }
            }
            if (has_r) {
#pragma unroll
                for (int i = 0; i < kVecs; ++i)
                    if (h0 + i * 32 * N < a.H) cp_async16(rs + i * 32 * 16, r + i * 32 * 16);
            }
        }
        cp_async_commit();  // an empty group past the end keeps the waits uniform
    };
    const uint32_t first = blockIdx.x * rows + group;
    const uint32_t step = gridDim.x * rows;  // T < 2^31: row numbers past the end stay below 2^32
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) issue(first + s * step, s);
    uint32_t w[kVecs][kWeightWords<kWF32, P>];
    load_weights<kWF32, P>(w, a.weight, h0, a.H);
    int st = 0, parity = 0;
    for (uint32_t t = first; t < static_cast<uint32_t>(T); t += step, parity ^= 1) {
        issue(t + (kStages - 1) * step, st == 0 ? kStages - 1 : st - 1);  // the stage read last time
        cp_async_wait<kStages - 1>();
        const size_t at = static_cast<size_t>(t) * a.H + h0;
        f2 z[kVecs][P], sq = 0;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            uint32_t xw[P], rw[4];
            load_shared(xw, x_ring + st * stage_bytes + i * 32 * 2 * N);
            load_shared(rw, r_ring + st * stage_bytes + i * 32 * 16);
            sq = add_residual<Carry>(z[i], xw, rw, sq);
        }
        if (a.residual_out != nullptr) {
#pragma unroll
            for (int i = 0; i < kVecs; ++i)
                if (h0 + i * 32 * N < a.H) store_carry<Carry>(a.residual_out, at + i * 32 * N, z[i]);
        }
        st = st + 1 == kStages ? 0 : st + 1;
        const float ss = block_sum(sum2(sq), nt, s_part[parity]);
        write_row<Carry, kVecs, kFp8, kWF32>(a, at, h0, w, z, rsqrtf(fmaf(ss, a.inv_h, a.eps)));
    }
    cp_async_wait<0>();  // only empty groups can be left
    allow_dependents();
}

// Threads of a row of `vecs` vectors when each takes `per` of them.
inline int row_threads(int vecs, int per) { return (vecs + 32 * per - 1) / (32 * per) * 32; }

// Resident CTAs per SM of a kernel at nt threads and smem bytes (kMaxRingSmem allowed), kept
// per device and number of warps; smem follows from nt and `kind`.
struct Residency {
    std::atomic<int> per_sm[kMaxDevices][33][2];
};

template <typename Kernel>
ep_status_t resident(Residency& cache, Kernel* kernel, int nt, int kind, size_t smem, int* out) {
    const int dev = current_device();
    std::atomic<int>* slot = dev >= 0 ? &cache.per_sm[dev][nt / 32][kind] : nullptr;
    int n = slot != nullptr ? slot->load(std::memory_order_acquire) : 0;
    if (n == 0) {
        cudaError_t err =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMaxRingSmem));
        if (err == cudaSuccess) err = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, nt, smem);
        if (err != cudaSuccess) return cuda_fail(err);
        if (n < 1) n = 1;
        if (slot != nullptr) slot->store(n, std::memory_order_release);
    }
    *out = n;
    return EP_OK;
}

template <class Carry, int kVecs, int kStages, bool kFp8, bool kWF32, bool kMany>
ep_status_t launch_norm_ring(const NormArgs& a, int T, cudaStream_t stream) {
    static Residency cache;
    const int rows = kMany ? kRingRows : 1;
    const int threads = rows * row_threads(a.H / Carry::kElems, kVecs);
    auto kernel = rmsnorm_ring_kernel<Carry, kVecs, kStages, kFp8, kWF32, kMany>;
    const size_t smem = kStages * ring_row_bytes<Carry>(threads, kVecs, 1);
    int per_sm = 1;
    const ep_status_t st = resident(cache, kernel, threads, 0, smem, &per_sm);
    if (st != EP_OK) return st;
    const int cap = sm_count() * per_sm;
    const int ctas = (T - 1) / rows + 1;
    return launch_dependent(kernel, dim3(ctas < cap ? ctas : cap), dim3(threads), smem, stream, a, T);
}

template <class Carry, int kVecs, bool kFp8, bool kWF32>
ep_status_t launch_norm_rows(const NormArgs& a, int T, cudaStream_t stream) {
    return launch_dependent(rmsnorm_kernel<Carry, kVecs, kFp8, kWF32>, dim3(static_cast<unsigned>(T)),
                            dim3(row_threads(a.H / Carry::kElems, kVecs)), 0, stream, a);
}

template <class Carry, bool kFp8, bool kWF32>
ep_status_t launch_norm(const NormArgs& a, int T, cudaStream_t stream) {
    const int vecs = a.H / Carry::kElems;
    const int streams = (a.residual != nullptr) + (a.residual_out != nullptr);
    const int row_bytes = a.H * (streams * (16 / Carry::kElems) + (a.x != nullptr ? 2 : 0) + (a.y != nullptr ? 2 : 0) +
                                 (kFp8 ? 1 : 0));
    // Rows with one input take the ring at any width: ring against a row per CTA, us, one input,
    // y alone / E4M3 alone, 4096 x 7168 bf16 with bf16 weights 19.7 / 23.2 against 20.6 / 21.6, with
    // fp32 weights 19.8 / 23.1 against 25.6 / 26.0; 4096 x 16384 bf16 43.7 / 51.2 against 70.6 / 72.2;
    // 8192 x 8192 fp32 65.3 / 71.7 against 65.9 / 72.8. It costs up to 9 % where only E4M3 is written
    // (16384 x 2048 fp32 34.1 against 31.8) and more where the CTAs get few rows (512 x 7168 bf16
    // 3.0 / 4.2 against 2.8 / 3.5).
    if (T > sm_count() && (row_bytes < kRingRowBytes || a.x == nullptr || a.residual == nullptr)) {
        if constexpr (Carry::kElems == 4) {  // 4 channels a vector: 1024 threads of 2 vectors cover 8192
            if (row_threads(vecs, 2) > kMaxThreads)
                return launch_norm_ring<Carry, 4, 2, kFp8, kWF32, false>(a, T, stream);
        }
        if (row_threads(vecs, 2) == 32) return launch_norm_ring<Carry, 2, 2, kFp8, kWF32, true>(a, T, stream);
        return launch_norm_ring<Carry, 2, 2, kFp8, kWF32, false>(a, T, stream);
    }
    return launch_norm_rows<Carry, 4, kFp8, kWF32>(a, T, stream);
}

template <class Carry>
ep_status_t launch_norm(const NormArgs& a, int T, cudaStream_t stream) {
    const bool f32 = a.weight_f32 != 0;
    if (a.y_q != nullptr)
        return f32 ? launch_norm<Carry, true, true>(a, T, stream) : launch_norm<Carry, true, false>(a, T, stream);
    return f32 ? launch_norm<Carry, false, true>(a, T, stream) : launch_norm<Carry, false, false>(a, T, stream);
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

// Resident CTAs with the same ring as the forward pass; the sums of dweight's terms stay in
// registers over all rows of a thread, and each CTA writes one row of partial sums (resident
// CTAs, because every further CTA would add one). Where rows are short (kMany), a CTA has
// several rows side by side, each with its own threads and named barrier, whose sums it adds
// before it writes: 16384 x 1024 in 25.5 us against 46.8 us with a CTA per row. Both passes
// over a row read it from the ring, so it costs no registers between them. 4096 x 7168 bf16
// with dz_in: 40.0 us (5.87 TB/s), 36.0 us of them without dweight. At 72 registers instead of
// 80, a CTA with rows side by side takes 1 to 3 % longer.
template <class Carry, int kVecs, int kStages, bool kWF32, bool kMany>
__global__ void __maxnreg__((kMany ? 80 : 64)) rmsnorm_bwd_kernel(NormBwdArgs a, int rows_at_once) {
    constexpr int N = Carry::kElems, P = N / 2;
    extern __shared__ __align__(16) unsigned char s_ring[];
    __shared__ float2 s_part[2][32];  // [parity][warp of the CTA]
    const int groups = kMany ? rows_at_once : 1;
    const int nt = static_cast<int>(blockDim.x) / groups;  // threads of a row
    const int group = kMany ? static_cast<int>(threadIdx.x) / nt : 0;
    const int tid = static_cast<int>(threadIdx.x) - group * nt;
    const int h0 = first_channel<Carry, kVecs>(tid);
    const bool has_in = a.dz_in != nullptr;
    const int z_bytes = kVecs * nt * 16;  // of a stage
    const int in_bytes = has_in ? z_bytes : 0;
    const int stage_bytes = z_bytes + in_bytes + kVecs * nt * 2 * N;
    unsigned char* const my_ring = s_ring + group * (kStages * stage_bytes);
    unsigned char* const z_ring = my_ring + h0 * (16 / N);
    unsigned char* const in_ring = z_ring + z_bytes;
    unsigned char* const dy_ring = my_ring + z_bytes + in_bytes + h0 * 2;
    const int vectors_in = h0 < a.H ? (a.H - h0 + 32 * N - 1) / (32 * N) : 0;
    fill_ring<16, kVecs>(z_ring, stage_bytes, kStages, true, 0u, vectors_in);
    fill_ring<2 * N, kVecs>(dy_ring, stage_bytes, kStages, true, 0u, vectors_in);
    grid_dependency_wait();
    auto issue = [&](uint32_t t, int st) {
        if (t < static_cast<uint32_t>(a.T)) {
            const size_t at = static_cast<size_t>(t) * a.H + h0;
            const char* const z = static_cast<const char*>(a.z) + carry_bytes<Carry>(at);
            const char* const in = static_cast<const char*>(a.dz_in) + carry_bytes<Carry>(at);
            const uint16_t* const dy = a.dy + at;
            unsigned char* const zs = z_ring + st * stage_bytes;
            unsigned char* const is = in_ring + st * stage_bytes;
            unsigned char* const ys = dy_ring + st * stage_bytes;
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                if (h0 + i * 32 * N < a.H) {
                    cp_async16(zs + i * 32 * 16, z + i * 32 * 16);
                    if constexpr (N == 8) cp_async16(ys + i * 32 * 16, dy + i * 32 * N);
                    else cp_async8(ys + i * 32 * 8, dy + i * 32 * N);
                }
            }
            if (has_in) {
#pragma unroll
                for (int i = 0; i < kVecs; ++i)
                    if (h0 + i * 32 * N < a.H) cp_async16(is + i * 32 * 16, in + i * 32 * 16);
            }
        }
        cp_async_commit();
    };
    f2 dw[kVecs][P];
#pragma unroll
    for (int i = 0; i < kVecs; ++i)
#pragma unroll
        for (int e = 0; e < P; ++e) dw[i][e] = 0;
    const uint32_t first = blockIdx.x * groups + group;
    const uint32_t step = gridDim.x * groups;  // T < 2^31: row numbers past the end stay below 2^32
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) issue(first + s * step, s);
    uint32_t w[kVecs][kWeightWords<kWF32, P>];
    load_weights<kWF32, P>(w, a.weight, h0, a.H);
    int st = 0, parity = 0;
    for (uint32_t t = first; t < static_cast<uint32_t>(a.T); t += step, parity ^= 1) {
        issue(t + (kStages - 1) * step, st == 0 ? kStages - 1 : st - 1);  // the stage read last time
        cp_async_wait<kStages - 1>();
        const size_t at = static_cast<size_t>(t) * a.H + h0;
        const unsigned char* const zs = z_ring + st * stage_bytes;
        const unsigned char* const ys = dy_ring + st * stage_bytes;
        const unsigned char* const is = in_ring + st * stage_bytes;
        // dy, z and g = dy * weight of a vector, read from the ring in both passes
        auto read = [&](int i, f2(&dy)[P], f2(&z)[P], f2(&g)[P]) {
            uint32_t yw[P], zw[4];
            load_shared(yw, ys + i * 32 * 2 * N);
            load_shared(zw, zs + i * 32 * 16);
            unpack_bf16(dy, yw);
            unpack_carry<Carry>(z, zw);
#pragma unroll
            for (int e = 0; e < P; ++e) g[e] = mul2(dy[e], weight_pair<kWF32, P>(w[i], e));
        };
        f2 sq = 0, sg2 = 0;
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            f2 dy[P], z[P], g[P];
            read(i, dy, z, g);
#pragma unroll
            for (int e = 0; e < P; ++e) {
                sq = fma2(z[e], z[e], sq);
                sg2 = fma2(g[e], z[e], sg2);
            }
        }
        float ss = warp_sum(sum2(sq)), sg = warp_sum(sum2(sg2));
        if (nt > 32) {
            const int lane = lane_id(), warps = nt >> 5;
            float2* const part = s_part[parity] + group * warps;
            if (lane == 0) part[tid >> 5] = make_float2(ss, sg);
            // the row's threads only; the other parity's values are read before this and written after it
            if constexpr (kMany) asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(nt) : "memory");
            else __syncthreads();
            const float2 v = lane < warps ? part[lane] : make_float2(0.0f, 0.0f);
            ss = warp_sum(v.x);
            sg = warp_sum(v.y);
        }
        const float rstd = rsqrtf(fmaf(ss, a.inv_h, a.eps));
        const f2 r = both(rstd);
        const f2 nc = both(-(sg * a.inv_h * rstd * rstd));  // -mean(g z) / (mean(z^2) + eps)
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            f2 dy[P], z[P], g[P], in[P], d[P];
            read(i, dy, z, g);
#pragma unroll
            for (int e = 0; e < P; ++e) {
                d[e] = fma2(nc, z[e], g[e]);
                dw[i][e] = fma2(mul2(dy[e], r), z[e], dw[i][e]);
            }
            if (h0 + i * 32 * N < a.H) {
                if (has_in) {
                    uint32_t iw[4];
                    load_shared(iw, is + i * 32 * 16);
                    unpack_carry<Carry>(in, iw);
#pragma unroll
                    for (int e = 0; e < P; ++e) d[e] = fma2(r, d[e], in[e]);
                } else {
#pragma unroll
                    for (int e = 0; e < P; ++e) d[e] = mul2(r, d[e]);
                }
                store_carry<Carry>(a.dz, at + i * 32 * N, d);
                if (a.dx != nullptr) store_bf16(a.dx + at + i * 32 * N, d);
            }
        }
        st = st + 1 == kStages ? 0 : st + 1;
    }
    cp_async_wait<0>();  // only empty groups can be left
    allow_dependents();
    if (a.parts == nullptr) return;
    // the CTA's partial sums: the groups' are added in order, through the ring's memory
    float* const part = a.parts + static_cast<size_t>(blockIdx.x) * a.H;
    float* const mine = reinterpret_cast<float*>(s_ring) + static_cast<size_t>(group) * a.H;
    if (groups > 1) __syncthreads();  // every group is past its last row
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const int h = h0 + i * 32 * N;
        if (h < a.H) {
            float* to = (groups > 1 ? mine : part) + h;
#pragma unroll
            for (int e = 0; e < P; e += 2) {
                float4 v;
                split(v.x, v.y, dw[i][e]);
                split(v.z, v.w, dw[i][e + 1]);
                *reinterpret_cast<float4*>(to + 2 * e) = v;
            }
        }
    }
    if (groups > 1) {
        __syncthreads();
        for (int h = static_cast<int>(threadIdx.x) * 4; h < a.H; h += static_cast<int>(blockDim.x) * 4) {
            const float* const sums = reinterpret_cast<const float*>(s_ring) + h;
            float4 s = *reinterpret_cast<const float4*>(sums);
            for (int g = 1; g < groups; ++g) {
                const float4 v = *reinterpret_cast<const float4*>(sums + static_cast<size_t>(g) * a.H);
                s.x += v.x;
                s.y += v.y;
                s.z += v.z;
                s.w += v.w;
            }
            *reinterpret_cast<float4*>(part + h) = s;
        }
    }
}

// dweight[h] = the sum of the nparts partial sums of channel h, in a fixed order: 8 threads
// take 4 channels each, kReduceRows of them take the partial rows in turn, and their sums
// are added as a tree.
__global__ void __launch_bounds__(8 * kReduceRows) dweight_reduce_kernel(const float* parts, int nparts, int H,
                                                                       float* dweight) {
    __shared__ float4 s_sum[kReduceRows][8];
    grid_dependency_wait();
    const int col = static_cast<int>(threadIdx.x & 7);
    const int row = static_cast<int>(threadIdx.x >> 3);
    const int h = (static_cast<int>(blockIdx.x) * 8 + col) * 4;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](const float4& v) {
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
    };
    if (h < H) {
#pragma unroll 8
        for (int p = row; p < nparts; p += kReduceRows)
            add(*reinterpret_cast<const float4*>(parts + static_cast<size_t>(p) * H + h));
    }
    s_sum[row][col] = s;
#pragma unroll
    for (int half = kReduceRows / 2; half >= 1; half >>= 1) {
        __syncthreads();
        if (row < half) {
            add(s_sum[row + half][col]);
            s_sum[row][col] = s;
        }
    }
    if (row == 0 && h < H) *reinterpret_cast<float4*>(dweight + h) = s;
    allow_dependents();
}

template <class Carry, int kVecs, int kStages, bool kWF32, bool kMany>
ep_status_t launch_norm_bwd(const NormBwdArgs& a, cudaStream_t stream, int* grid_out) {
    static Residency cache;
    auto kernel = rmsnorm_bwd_kernel<Carry, kVecs, kStages, kWF32, kMany>;
    const int nt = row_threads(a.H / Carry::kElems, kVecs);
    int groups = !kMany ? 1 : kBwdThreads / nt < kMaxGroups ? kBwdThreads / nt : kMaxGroups;
    const int useful = (a.T - 1) / kBwdRowsPerGroup + 1;
    if (useful < groups) groups = useful;
    const int streams = a.dz_in != nullptr ? 2 : 1;
    const size_t smem = groups * kStages * ring_row_bytes<Carry>(nt, kVecs, streams);
    int per_sm = 1;
    const ep_status_t st = resident(cache, kernel, groups * nt, streams - 1, smem, &per_sm);
    if (st != EP_OK) return st;
    // Each CTA writes a row of partial sums, so there are as few as fill the SMs evenly with
    // kBwdRows rows each (431 x 5984: 8.4 us instead of 9.5 us with a row or two each), and no
    // more than end with equal numbers of rows.
    const int rows = (a.T - 1) / groups + 1;
    const int wanted = (rows / kBwdRows + sm_count() - 1) / sm_count();
    int most = sm_count() * (wanted < 1 ? 1 : wanted < per_sm ? wanted : per_sm);
    if (most > kMaxParts) most = kMaxParts;
    const int turns = (rows - 1) / most + 1;
    *grid_out = (rows - 1) / turns + 1;
    return launch_dependent(kernel, dim3(*grid_out), dim3(groups * nt), smem, stream, a, groups);
}

template <class Carry, bool kWF32>
ep_status_t launch_norm_bwd(const NormBwdArgs& a, cudaStream_t stream, int* grid_out) {
    const int nt = row_threads(a.H / Carry::kElems, 2);
    if (2 * nt <= kBwdThreads) return launch_norm_bwd<Carry, 2, 2, kWF32, true>(a, stream, grid_out);
    if constexpr (Carry::kElems == 4) {  // 4 channels a vector: 1024 threads of 2 vectors cover 8192
        if (nt > kMaxThreads) return launch_norm_bwd<Carry, 4, 1, kWF32, false>(a, stream, grid_out);
    }
    return launch_norm_bwd<Carry, 2, 2, kWF32, false>(a, stream, grid_out);
}

template <class Carry>
ep_status_t launch_norm_bwd(const NormBwdArgs& a, cudaStream_t stream, int* grid_out) {
    return a.weight_f32 ? launch_norm_bwd<Carry, true>(a, stream, grid_out)
                        : launch_norm_bwd<Carry, false>(a, stream, grid_out);
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
    const float* const sums = static_cast<const float*>(workspace);
    return launch_dependent(dweight_reduce_kernel, dim3((H + 31) / 32), dim3(8 * kReduceRows), 0, as_stream(stream),
                            sums, parts, static_cast<int>(H), dweight);
}
