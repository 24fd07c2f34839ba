// ep_expert.cu -- the experts' gated feed-forward block over the expert-major slabs: the
// products of every expert's rows with its weights, and their gradients (include/ep.h).
//
// One kernel for all five. The operand with the output's channels (the weights; in their own
// gradient, the rows that were multiplied with them) lies along the tensor cores' 256 lanes
// of a pair of CTAs, the expert's rows along the columns, of which a product takes any
// multiple of 32: an expert with 140 rows costs 160 columns, not two tiles of 128 rows. A tile
// is 256 channels by up to 256 rows, K long: 128 flops a byte that comes from L2.
//
// The grid is persistent, a CTA an SM. In a CTA two warps copy tensor boxes into a ring of 4 to 11
// stages of 64 k (3 in the gated product of more than 2048 experts, whose plan takes the place of one),
// one (of the pair) multiplies them into tensor memory, one plans tiles ahead, and sixteen finish the
// sums of one tile while the next is multiplied: 32 lanes by 16 columns at a time as fragments of 8 x 8,
// through a patch of shared memory into rows of 16-byte vectors.
//
// With few rows an expert the weights' stream bounds it, with many the tensor cores' power: 4096
// tokens top-8 of 256 experts of 7168 x 2048, gated with the 8-bit checkpoint 2.34 ms (6.7 TB/s), down
// 1.19 ms (6.8), back through the activation 1.24 ms (6.9); 16384 tokens of 128 uneven experts of
// 4096 x 2048 2.1 to 2.5 ms a product (1.75 to 2.1 PFLOP/s). With few rows and few tiles the warp that
// multiplies bounds it, 146 ns for 64 k.
#include "ep_expert.cuh"
#include "ep_mma.cuh"

namespace {

using namespace ep;

enum Op { kGateUp, kDown, kDownBwd, kGateUpBwd, kWgrad };

// Warps: two that copy the operands in, one that multiplies, one that clears tails, one that plans
// tiles, and four groups of four (32 lanes of the sums each) that finish them.
constexpr int kProducer = 0, kMultiplier = 1, kTail = 2, kScheduler = 3, kFinish = 4, kGroups = 4;
constexpr int kFinishWarps = 4 * kGroups, kLastFinish = kFinish + kFinishWarps - 1;
constexpr uint32_t kTmemColumns = 512;
constexpr uint32_t kSlotColumns = 256;  // of tensor memory: two tiles at a time
constexpr int kMostStages = 12;
constexpr int kTiles = 4;  // that are planned ahead
constexpr int kMostNLog = 8, kMostN = 1 << kMostNLog;  // rows of an expert a tile
constexpr size_t kSmemMost = 227 * 1024;

template <int kOp>
struct Traits {
    static constexpr bool kGated = kOp == kGateUp;
    static constexpr bool kAAcross = kOp == kDownBwd || kOp == kGateUpBwd || kOp == kWgrad;
    static constexpr bool kBAcross = kOp == kWgrad;
    static constexpr uint32_t kABytes = (kGated ? 2 : 1) * 128 * kBlockK * 2;
    static constexpr uint32_t kBBytes = kMostN / 2 * kBlockK * 2;
    // of one CTA, with tiles of up to kMostN >> choice rows
    static constexpr __host__ __device__ uint32_t stage_bytes(int choice) { return kABytes + (kBBytes >> choice); }
    static constexpr int kPatches = kOp == kWgrad ? 2 : 1;      // a finishing warp (kWgrad: four of a pair)
    // the second warp that copies in: the tails' place where there are none (20 warps leave 96
    // registers a thread, 21 no more than 80)
    static constexpr int kColumnProducer = kOp == kWgrad ? kLastFinish + 1 : kTail;
    static constexpr int kThreads = 32 * (kOp == kWgrad ? kLastFinish + 2 : kLastFinish + 1);
};

struct ExpertArgs {
    const int32_t* offsets;
    int act;
    int C;  // output channels, along the lanes (one half of them in kGateUp and kDownBwd)
    int K;  // products of a sum (kWgrad: output rows, along the columns)
    int E, R, max_rows;
    int epr;        // experts a rank
    float inv_epr;  // 1 / epr
    uint32_t ring;    // bytes of the stages
    uint32_t stages;  // a byte a choice of rows a tile (Planned): how many
    const uint16_t* pre;
    const uint8_t* pre_q;
    const uint16_t* pre_scales;
    uint16_t *out, *out_pre, *out_scales;
    uint8_t* out_q;
    int32_t* status;
};

// A tile: 256 channels (128 a CTA), or the last 128 or fewer (64 a CTA), of up to kMostN rows of an
// expert; in kWgrad, of up to kMostN rows of its gradient.
struct Tile {
    long long row;  // first row of the slabs; kWgrad: the expert's
    int e;          // -1: there are no more tiles
    int rows;       // rows that are there (columns of the sums that are kept)
    int m, n;       // lanes of the pair, 256 or 128; columns that are multiplied, a multiple of 32
    int channel;    // first of the pair's
    int column;     // kWgrad: first row of dw[e]
    int k;          // products of a sum
};

struct Planned {
    // a stage's bytes have come (CTA 0: both CTAs'), its products are done; a last stage of
    // kWgrad: the CTA's own bytes have come, both CTAs have cleared its tail
    uint64_t full[kMostStages], empty[kMostStages], part[kMostStages], ready[kMostStages];
    uint64_t sums_full[2], sums_empty[2], tile_full[kTiles], tile_empty[kTiles], drain;
    Tile tile[kTiles];
    uint32_t tmem;
    Watch watch;
    int choice;  // kMostN >> choice rows a tile, of this call
    int scan[4][32];  // of the plan: a warp's tiles, for each choice
};

// The reciprocals of the scales of 16 rows' gates and, from 16 on, up-projections, a warp's own.
struct Reciprocals {
    float high[2 * kChunk], low[2 * kChunk];
};

template <int kOp>
struct Shared : Planned {  // behind the stages
    alignas(1024) unsigned char patch[kFinishWarps * Traits<kOp>::kPatches][kPatchBytes];
    float amax[kOp == kGateUp ? kGroups * 2 * 4 : 1][2 * kChunk];  // [group, buffer, warp][gate and up]
    alignas(8) Reciprocals rcp[kOp == kGateUp ? kFinishWarps : 1];
    int prefix[1];  // [E + 1] tiles of rows before each expert's (but kWgrad)
};

// The stages. What a tile's rows leave of one goes to further ones: with few tiles the bytes on their way
// bound the copies (one expert of 7168 x 2048, 96 rows, gated: 38 us with 4 stages, 31 with 6).
template <int kOp>
struct Ring {
    uint32_t bytes;  // of a stage
    int stages;
    __device__ __forceinline__ Ring(const ExpertArgs& g, const Planned& s) {
        const int choice = kOp == kWgrad ? 0 : uniform(s.choice);
        bytes = Traits<kOp>::stage_bytes(choice);
        stages = static_cast<int>(g.stages >> 8 * choice & 255);
    }
};

// A wait gave up: every other one of the CTA ends soon, and the caller hears of it.
__device__ __forceinline__ void give_up(const ExpertArgs& g, Planned& s) {
    s.watch.stop = 1;
    raise_flag(g.status, EP_FLAG_TIMEOUT);
}

// The tiles of a role, in order, for a whole warp. next() is false where there are no more, or a wait
// gave up (`ok`); taken(), by one thread after all of the role's have read the tile, lets its place be used
// again. kUniform: with a tile that the compiler knows to be the same for the warp.
struct Tiles {
    uint32_t at = kTiles - 1, phase = 1;
    bool ok = true;
    template <bool kUniform = false>
    __device__ __forceinline__ bool next(Planned& s, Tile* t) {
        if (++at == kTiles) at = 0, phase ^= 1;
        ok = warp_wait(&s.tile_full[at], phase, &s.watch);
        if (!ok) return false;
        *t = s.tile[at];
        if (kUniform) {
            t->row = uniform(t->row);
            t->rows = uniform(t->rows);
            t->e = uniform(t->e);
            t->m = uniform(t->m);
            t->n = uniform(t->n);
            t->channel = uniform(t->channel);
            t->column = uniform(t->column);
            t->k = uniform(t->k);
        }
        return t->e >= 0;
    }
    __device__ __forceinline__ void taken(Planned& s) { mbar_arrive(&s.tile_empty[at]); }
};

// Tiles of an expert's rows, of most_n = kMostN >> choice rows at most, and rows of each: even
// tiles, not full ones and a rest. (With tiles - 1 of them not all rows are reached: the rows of
// each are at most most_n, and (tiles - 1) * most_n < count.)
__device__ __forceinline__ int row_tiles(int count, int choice) {
    return static_cast<int>((static_cast<uint32_t>(count) + (kMostN >> choice) - 1) >> (kMostNLog - choice));
}
// The choice for one expert. A gated tile of more than 128 rows has all of tensor memory, and its sums
// are finished before the next one's can begin; two of 128 rows take turns, but read the weights
// twice (from L2). Short sums cost less than their finish, so they take turns. us with tiles of up to
// 128 rows, of up to 256, 16 experts of 2048 rows, F = 2048, the 8-bit checkpoint: H = 512 137, 186, 1024
// 190, 254, 2048 336, 386, 4096 645, 680; 128 uneven ones of H = 4096 1995, 2002, with the bf16 checkpoint
// 2075, 2020; 256 of 128 rows on average, H = 7168 2534, 2362.
template <int kOp>
__device__ __forceinline__ int choice_of(const ExpertArgs& g, int count, int choice) {
    const bool turns = g.K <= 1024 || (g.K <= 2048 && count > kMostN);
    return kOp == kGateUp && choice == 0 && turns ? 1 : choice;
}
__device__ __forceinline__ int rows_each(int count, int tiles) {
    const uint32_t n = static_cast<uint32_t>(tiles);
    return static_cast<int>(((static_cast<uint32_t>(count) + n - 1) / n + 31) & ~31u);
}

// Lanes of a tile: the last 128 channels or fewer take 128, half of the copies, products and sums (64
// experts of 104 channels, gated, 8192 tokens 137 us instead of 168; their gradient of weights, 512
// tokens, 22.5 instead of 33.4; 16 experts of 128 channels 97 instead of 102). Not with the 8-bit
// checkpoint, whose blocks of 128 channels have to be one CTA's.
__device__ __forceinline__ int lanes_of(const ExpertArgs& g, int channel) {
    return g.C - channel <= 128 && g.out_q == nullptr ? 128 : 256;
}

// Tile l of an expert that has r.count rows. Eight tiles of rows with all channels, then the next
// eight: the rows that are at work at a time, and the weights that they share, stay in L2.
template <int kOp>
__device__ __forceinline__ void tile_of(const ExpertArgs& g, int choice, int e, const ExpertRows& r, uint32_t l,
                                        Tile* tile) {
    const int tiles = row_tiles(r.count, choice_of<kOp>(g, r.count, choice));
    tile->row = r.first;
    tile->rows = r.count;
    tile->channel = static_cast<int>(l * 256);
    if (tiles > 1) {
        const int each = rows_each(r.count, tiles);
        uint32_t before = 0, width = tiles;
        if (tiles > 8) {
            const uint32_t across = (static_cast<uint32_t>(g.C) + 255) / 256, group = l / (8 * across);
            l -= group * 8 * across;
            before = group * 8;
            width = tiles - before < 8 ? tiles - before : 8;
        }
        const uint32_t slice = l / width;
        const int i = static_cast<int>(before + l - slice * width);
        tile->row += static_cast<long long>(i) * each;
        tile->rows = r.count - i * each < each ? r.count - i * each : each;
        tile->channel = static_cast<int>(slice * 256);
    }
    tile->e = e;
    tile->m = lanes_of(g, tile->channel);
    tile->n = (tile->rows + 31) / 32 * 32;
    tile->column = 0;
    tile->k = g.K;
}

// Tile t of the call; false where there are not so many.
template <int kOp>
__device__ __forceinline__ bool tile_at(const ExpertArgs& g, const Shared<kOp>& s, uint32_t t, Tile* tile) {
    const uint32_t across = (static_cast<uint32_t>(g.C) + 255) / 256;
    if (kOp == kWgrad) {
        const uint32_t down = (static_cast<uint32_t>(g.K) + 255) / 256;
        if (t >= static_cast<uint32_t>(g.E) * across * down) return false;
        const int e = static_cast<int>(t / (across * down));
        const uint32_t l = t - e * (across * down);
        const ExpertRows r = expert_rows(g.offsets, e, g.epr, g.inv_epr, g.max_rows);
        tile->e = e;
        tile->row = r.first;
        tile->k = r.count;
        tile->channel = static_cast<int>(l % across * 256);
        tile->column = static_cast<int>(l / across * 256);
        tile->rows = g.K - tile->column < 256 ? g.K - tile->column : 256;
        tile->m = lanes_of(g, tile->channel);
        tile->n = (tile->rows + 31) / 32 * 32;
        return true;
    }
    if (t >= static_cast<uint32_t>(s.prefix[g.E]) * across) return false;
    int lo = 0, hi = g.E;  // the last expert whose tiles begin at or before t
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (static_cast<uint32_t>(s.prefix[mid]) * across <= t)
            lo = mid;
        else
            hi = mid;
    }
    tile_of<kOp>(g, s.choice, lo, expert_rows(g.offsets, lo, g.epr, g.inv_epr, g.max_rows), t - s.prefix[lo] * across, tile);
    return true;
}

// The number of tiles of rows before each expert's, by all threads, and the pair's first tile, by
// the thread that meets it. A tile has 256 rows at most, or 128, 64 or 32 where all tiles are at work
// at once even then: more of them draw more, but a second round costs as much as the first (one expert
// of 7168 x 2048, 512 rows, gated: 64 tiles 39 us, 128 of half the rows 66; 96 rows back through the
// up-projection: 56 tiles 17 us, 84 26).
template <int kOp>
__device__ __forceinline__ void plan_tiles(const ExpertArgs& g, Shared<kOp>& s, uint32_t pair, uint32_t pairs) {
    const int tid = static_cast<int>(threadIdx.x), lane = tid % 32, warp = tid / 32;
    constexpr int kThreads = Traits<kOp>::kThreads;
    const int per = (g.E + kThreads - 1) / kThreads, first = tid * per;
    const int last = first + per < g.E ? first + per : g.E;
    const uint32_t across = (static_cast<uint32_t>(g.C) + 255) / 256;
    ExpertRows r = {0, 0, false};
    int sum[4] = {0, 0, 0, 0};
    for (int e = first; e < last; ++e) {
        r = expert_rows(g.offsets, e, g.epr, g.inv_epr, g.max_rows);
        if (r.dropped && blockIdx.x == 0) raise_flag(g.status, EP_FLAG_CAPACITY);
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] += row_tiles(r.count, choice_of<kOp>(g, r.count, i));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int n = static_cast<int>(__reduce_add_sync(kFullMask, static_cast<unsigned>(sum[i])));
        if (lane == 0) s.scan[i][warp] = n;
    }
    __syncthreads();
    // lane w of every warp has warp w's sum of the choice
    static_assert(kThreads <= 32 * 32);
    int others[4], choice = 0;
    uint32_t total[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) others[i] = lane < kThreads / 32 ? s.scan[i][lane] : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) total[i] = __reduce_add_sync(kFullMask, static_cast<unsigned>(others[i]));
    int mine = sum[0], theirs = others[0];
    uint32_t tiles = total[0];
#pragma unroll
    for (int i = 1; i < 4; ++i)
        if (total[i] * across <= pairs) choice = i, mine = sum[i], theirs = others[i], tiles = total[i];
    int before = static_cast<int>(__reduce_add_sync(kFullMask, static_cast<unsigned>(lane < warp ? theirs : 0)));
    int upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int v = __shfl_up_sync(kFullMask, upto, d);
        if (lane >= d) upto += v;
    }
    before += upto - mine;
    for (int e = first; e < last; ++e) {
        if (per > 1) r = expert_rows(g.offsets, e, g.epr, g.inv_epr, g.max_rows);
        const uint32_t begin = static_cast<uint32_t>(before) * across;
        s.prefix[e] = before;
        before += row_tiles(r.count, choice_of<kOp>(g, r.count, choice));
        if (begin <= pair && pair < before * across) {
            Tile t;
            tile_of<kOp>(g, choice, e, r, pair - begin, &t);
            s.tile[0] = t;
        }
        if (e == g.E - 1) s.prefix[g.E] = before;
    }
    if (tid == 0) {
        s.choice = choice;
        if (pair >= tiles * across) s.tile[0].e = -1;
    }
}

// ---------------------------------------------------------------------------- finishing a tile

// 16 rows of 32 channels, of which `rows` and, 8 at a time, `channels` are there: 16-byte vectors of
// bf16, 8-byte ones of codes, four neighbouring lanes a row.
struct Window {
    int rows, channels;
    __device__ __forceinline__ bool has(int q, int lane) const {
        return 8 * q + lane / 4 < rows && lane % 4 * 8 < channels;
    }
};

__device__ __forceinline__ void store_rows(uint16_t* to, size_t stride, const uint32_t (&w)[8], const Window& win,
                                           uint32_t patch, int lane) {
    __syncwarp();  // what was in the patch has been read
    patch_put(patch, w, lane);
    __syncwarp();
    to += lane / 4 * stride + lane % 4 * 8;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const uint4 v = ld_shared_v4(row_place(patch, q, lane));
        if (win.has(q, lane)) st_v4(to + 8 * q * stride, v);
    }
}
__device__ __forceinline__ void load_rows(uint4 (&v)[2], const uint16_t* from, size_t stride, const Window& win,
                                          int lane) {
    from += lane / 4 * stride + lane % 4 * 8;
#pragma unroll
    for (int q = 0; q < 2; ++q)
        v[q] = win.has(q, lane) ? ld_stream_v4(from + 8 * q * stride) : make_uint4(0, 0, 0, 0);
}
// rows into fragments
__device__ __forceinline__ void spread(uint32_t (&w)[8], const uint4 (&v)[2], uint32_t patch, int lane) {
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 2; ++q) st_shared_v4(row_place(patch, q, lane), v[q]);
    __syncwarp();
    patch_get(w, patch, lane);
}
__device__ __forceinline__ void pack(uint32_t (&w)[8], const float (&v)[16]) {
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int i = fragment(q, b);
            w[4 * q + b] = pack_bf16x2_rn(v[i], v[i + 1]);
        }
}

// codes of v0, v1 by their reciprocals
__device__ __forceinline__ uint32_t pair_codes(float v0, float v1, const float2& high, const float2& low) {
    float q0, q1;
    asm("{\n .reg .b64 v, h, l;\n mov.b64 v, {%2, %3};\n mov.b64 h, {%4, %5};\n mov.b64 l, {%6, %7};\n"
        " mul.rn.f32x2 l, v, l;\n fma.rn.f32x2 v, v, h, l;\n mov.b64 {%0, %1}, v;\n}\n"
        : "=f"(q0), "=f"(q1)
        : "f"(v0), "f"(v1), "f"(high.x), "f"(high.y), "f"(low.x), "f"(low.y));
    return pack_e4m3x2_rn_sat(q0, q1);
}
// Codes of 16 rows of one block of 128 channels, of which the warp has 32, by the reciprocals from `side`
// on. They go through the patch as 16-bit values.
__device__ __forceinline__ void store_codes(uint8_t* to, size_t stride, const float (&v)[16], const Reciprocals& rcp,
                                            int side, const Window& win, uint32_t patch, int lane) {
    uint32_t w[8];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int row = side + 8 * q + lane % 4 * 2;  // and the next
        const float2 high = *reinterpret_cast<const float2*>(rcp.high + row);
        const float2 low = *reinterpret_cast<const float2*>(rcp.low + row);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int i = fragment(q, b);
            w[4 * q + b] = __byte_perm(pair_codes(v[i], v[i + 1], high, low), 0, 0x4140);
        }
    }
    __syncwarp();
    patch_put(patch, w, lane);
    __syncwarp();
    to += lane / 4 * stride + lane % 4 * 8;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const uint4 c = ld_shared_v4(row_place(patch, q, lane));
        if (win.has(q, lane))
            st_v2(to + 8 * q * stride, __byte_perm(c.x, c.y, 0x6420), __byte_perm(c.z, c.w, 0x6420));
    }
}
__device__ __forceinline__ void load_codes(uint4 (&v)[2], const uint8_t* from, size_t stride, const Window& win,
                                           int lane) {
    from += lane / 4 * stride + lane % 4 * 8;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const uint2 c = win.has(q, lane) ? __ldg(reinterpret_cast<const uint2*>(from + 8 * q * stride))
                                         : make_uint2(0, 0);
        v[q].x = c.x;
        v[q].y = c.y;
    }
}
// codes into fragments of fp16 (every code is one)
__device__ __forceinline__ void spread_codes(uint32_t (&w)[8], const uint4 (&c)[2], uint32_t patch, int lane) {
    uint4 f[2];
#pragma unroll
    for (int q = 0; q < 2; ++q)
        f[q] = make_uint4(e4m3x2_to_f16x2(c[q].x), e4m3x2_to_f16x2(c[q].x >> 16), e4m3x2_to_f16x2(c[q].y),
                          e4m3x2_to_f16x2(c[q].y >> 16));
    spread(w, f, patch, lane);
}

// max |v| of every column over the warp's lanes, NaN apart, into to[column]; NaN where there is nothing else
__device__ __forceinline__ void column_max(float* to, const float (&v)[16], int lane) {
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float m = fmaxf(fmaxf(fabsf(v[4 * q + i]), fabsf(v[4 * q + 2 + i])),
                            fmaxf(fabsf(v[8 + 4 * q + i]), fabsf(v[8 + 4 * q + 2 + i])));
#pragma unroll
            for (int d = 4; d < 32; d *= 2) m = fmaxf(m, __shfl_xor_sync(kFullMask, m, d));
            if (lane < 4) to[8 * q + 2 * lane + i] = m;
        }
}

template <bool kGelu>
__device__ __forceinline__ void activate(float (&v)[16], const float (&up)[16]) {
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = v[j] * sigmoid_of<kGelu>(v[j]) * up[j];
}
// dh, gate and up (fragments of bf16, or of fp16 times their rows' scales, of which lane j has row j's)
// into dgate, dup and h, packed
template <bool kGelu, bool kCodes>
__device__ __forceinline__ void activate_bwd(uint32_t (&dgate)[8], uint32_t (&dup)[8], uint32_t (&h)[8],
                                             const float (&dh)[16], const uint32_t (&gates)[8],
                                             const uint32_t (&ups)[8], float gate_scale, float up_scale, int lane) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        float gs[2], us[2];
        if (kCodes) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                gs[j] = __shfl_sync(kFullMask, gate_scale, 8 * q + lane % 4 * 2 + j);
                us[j] = __shfl_sync(kFullMask, up_scale, 8 * q + lane % 4 * 2 + j);
            }
        }
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const uint32_t wg = gates[4 * q + b], wu = ups[4 * q + b];
            float dg[2], du[2], hh[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float gate, up;
                if (kCodes) {
                    gate = f16_to_f32(j == 0 ? wg & 0xffffu : wg >> 16) * gs[j];
                    up = f16_to_f32(j == 0 ? wu & 0xffffu : wu >> 16) * us[j];
                } else {
                    gate = j == 0 ? bf16_lo(wg) : bf16_hi(wg);
                    up = j == 0 ? bf16_lo(wu) : bf16_hi(wu);
                }
                const float d = dh[fragment(q, b) + j];
                const float sig = sigmoid_of<kGelu>(gate), act = gate * sig;
                dg[j] = d * up * slope_of<kGelu>(gate, act, sig);
                du[j] = d * act;
                hh[j] = act * up;
            }
            dgate[4 * q + b] = pack_bf16x2_rn(dg[0], dg[1]);
            dup[4 * q + b] = pack_bf16x2_rn(du[0], du[1]);
            h[4 * q + b] = pack_bf16x2_rn(hh[0], hh[1]);
        }
    }
}

// true in all 128 threads of a group of finishing warps, or in none
__device__ __forceinline__ bool group_agrees(bool ok, int group) {
    int r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n barrier.cta.red.and.pred q, %2, 128, p;\n"
        " selp.s32 %0, 1, 0, q;\n}\n"
        : "=r"(r)
        : "r"(static_cast<int>(ok)), "r"(1 + group)
        : "memory");
    return r != 0;
}

// What the gradient reads of 16 rows of the checkpoint, on its way.
struct Kept {
    uint4 gate[2], up[2];        // bf16, or codes in x and y,
    float gate_scale, up_scale;  // and lane j's row's scales
};
__device__ __forceinline__ void load_kept(Kept& kept, const ExpertArgs& g, size_t row, int channel, const Window& win,
                                          int lane) {
    const size_t C = static_cast<size_t>(g.C), at = row * 2 * C + channel;
    if (g.pre != nullptr) {
        load_rows(kept.gate, g.pre + at, 2 * C, win, lane);
        load_rows(kept.up, g.pre + at + C, 2 * C, win, lane);
    } else {
        load_codes(kept.gate, g.pre_q + at, 2 * C, win, lane);
        load_codes(kept.up, g.pre_q + at + C, 2 * C, win, lane);
        const bool there = lane < kChunk && lane < win.rows && win.channels > 0;
        const uint16_t* scales = g.pre_scales + (row + lane) * (2 * C / 128) + channel / 128;
        kept.gate_scale = there ? __uint_as_float(static_cast<uint32_t>(__ldg(scales)) << 16) : 0.0f;
        kept.up_scale = there ? __uint_as_float(static_cast<uint32_t>(__ldg(scales + C / 128)) << 16) : 0.0f;
    }
}

// all 64 threads of two neighbouring finishing warps
__device__ __forceinline__ void pair_sync(int warp) {
    asm volatile("barrier.cta.sync %0, 64;" ::"r"(1 + kGroups + (warp - kFinish) / 2) : "memory");
}
// Two neighbouring warps' 64 channels leave together, 16 rows at a time, as one tensor copy from one
// of two patches that are filled in turn: rows and channels past the map's ends are left out. (A
// patch a warp, rows of 64 bytes, took twice as long, and plain 16-byte stores longer still: a copy's
// rows cost alike whatever their length.) `turn` outlives a tile: a patch is filled again when all
// copies but the newest, which is the other's, have read theirs.
struct Outlet {
    unsigned char* patches;  // two of 16 rows of 128 bytes, the pair's
    int turn = 0;

    __device__ __forceinline__ unsigned char* patch() const { return patches + turn * 2 * kPatchBytes; }
    __device__ __forceinline__ void fill(const uint32_t (&w)[8], int warp, int lane) const {
        pair_sync(warp);
#pragma unroll
        for (int q = 0; q < 2; ++q)
            matrices_put(wide_matrix_place(smem_addr(patch()), q, warp % 2, lane), w, q);
        fence_proxy_async_smem();
        pair_sync(warp);
    }
    // one chunk, from row y on
    __device__ __forceinline__ void send(const CUtensorMap& map, int x, int y, int z, const uint32_t (&w)[8], int warp,
                                         int lane) {
        const bool sends = warp % 2 == 0 && lane == 0;
        if (sends) bulk_wait_read<1>();
        fill(w, warp, lane);
        if (sends) {
            tma_store_3d(map, x, y, z, patch());
            bulk_commit();
        }
        turn ^= 1;
    }
    // zeros, every kGroups-th chunk of the rows from y to y_end
    __device__ __forceinline__ void send_zeros(const CUtensorMap& map, int x, int y, int y_end, int z, int warp,
                                               int lane) {
        const bool sends = warp % 2 == 0 && lane == 0;
        if (sends) bulk_wait_read_all();
        const uint32_t none[8] = {};
        fill(none, warp, lane);
        if (sends) {
            for (; y < y_end; y += kGroups * kChunk) tma_store_3d(map, x, y, z, patch());
            bulk_commit();
        }
        turn ^= 1;
    }
};

// One warp's part of a tile: 32 channels, every fourth 16 columns. `ready`, called before the sums
// are read, waits for them; false: give up.
template <int kOp, typename Ready>
__device__ __forceinline__ bool finish_tile(const ExpertArgs& g, const CUtensorMap& out_map, Shared<kOp>& s, const Tile& t,
                                            uint32_t sums, uint32_t ups, int rank, int warp, int lane, Outlet& outlet, Ready ready) {
    const int group = (warp - kFinish) / 4, quarter = warp % 4;
    // the warp's first channel; its columns of tensor memory and the first of the tile's that they are
    const bool narrow = t.m == 128;
    const int channel = t.channel + (narrow ? rank * 64 + quarter % 2 * 32 : rank * 128 + quarter * 32);
    const int columns = narrow ? t.n / 2 : t.n, from = narrow ? quarter / 2 * columns : 0;
    const size_t C = static_cast<size_t>(g.C);
    const uint32_t patch = smem_addr(s.patch[warp - kFinish]);
    sums += static_cast<uint32_t>(quarter * 32) << 16;
    ups += static_cast<uint32_t>(quarter * 32) << 16;
    const int pair_channel = channel & ~63;
    if constexpr (kOp == kWgrad) {
        if (t.k == 0) {  // an expert without rows
            const int first = from + group * kChunk, end = t.rows < from + columns ? t.rows : from + columns;
            if (pair_channel < g.C && first < end)
                outlet.send_zeros(out_map, pair_channel, t.column + first, t.column + end, t.e, warp, lane);
            return true;
        }
    }
    Kept kept;
    if constexpr (kOp == kDownBwd)  // on its way while the sums are made
        load_kept(kept, g, static_cast<size_t>(t.row) + from + group * kChunk, channel,
                  {t.rows - from - group * kChunk, g.C - channel}, lane);
    if (!ready()) return false;
    int buffer = 0;
    for (int c0 = group * kChunk; c0 < columns; c0 += kGroups * kChunk) {
        const Window win = {t.rows - from - c0, g.C - channel};
        const size_t row = static_cast<size_t>(t.row) + from + c0;
        uint32_t w[8];
        float v[16];
        if (t.k > 0) {
            tmem_load(v, sums + c0);
            tmem_load_wait(v);
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = 0.0f;
        }
        if constexpr (kOp == kGateUp) {
            float up[16];
            if (t.k > 0) {
                tmem_load(up, ups + c0);
                tmem_load_wait(up);
            } else {
#pragma unroll
                for (int j = 0; j < 16; ++j) up[j] = 0.0f;
            }
            if (g.out_pre != nullptr) {
                pack(w, v);
                store_rows(g.out_pre + row * 2 * C + channel, 2 * C, w, win, patch, lane);
                pack(w, up);
                store_rows(g.out_pre + row * 2 * C + C + channel, 2 * C, w, win, patch, lane);
            }
            if (g.out_q != nullptr) {
                float(*const amax)[2 * kChunk] = &s.amax[(group * 2 + buffer) * 4];
                buffer ^= 1;
                column_max(amax[quarter], v, lane);
                column_max(amax[quarter] + kChunk, up, lane);
                asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + group) : "memory");
                float a = 0.0f;  // lanes 0 .. 15 have the gate's rows, 16 .. 31 the up-projection's
#pragma unroll
                for (int i = 0; i < 4; ++i) a = fmaxf(a, amax[i][lane]);
                a = checkpoint_scale(a);
                if (quarter == 0 && lane % kChunk < win.rows && win.channels > 0)
                    g.out_scales[(row + lane % kChunk) * (2 * C / 128) + lane / kChunk * (C / 128) + channel / 128] =
                        static_cast<uint16_t>(__float_as_uint(a) >> 16);
                Reciprocals& rcp = s.rcp[warp - kFinish];
                checkpoint_rcp(a, rcp.high[lane], rcp.low[lane]);
                __syncwarp();
                store_codes(g.out_q + row * 2 * C + channel, 2 * C, v, rcp, 0, win, patch, lane);
                store_codes(g.out_q + row * 2 * C + C + channel, 2 * C, up, rcp, kChunk, win, patch, lane);
            }
            if (g.act == EP_ACT_GELU)
                activate<true>(v, up);
            else
                activate<false>(v, up);
            pack(w, v);
            store_rows(g.out + row * C + channel, C, w, win, patch, lane);
        } else if constexpr (kOp == kDownBwd) {
            uint32_t gates[8], ups[8], dup[8], h[8];
            const bool gelu = g.act == EP_ACT_GELU;
            if (g.pre != nullptr) {
                spread(gates, kept.gate, patch, lane);
                spread(ups, kept.up, patch, lane);
                if (gelu)
                    activate_bwd<true, false>(w, dup, h, v, gates, ups, 1.0f, 1.0f, lane);
                else
                    activate_bwd<false, false>(w, dup, h, v, gates, ups, 1.0f, 1.0f, lane);
            } else {
                spread_codes(gates, kept.gate, patch, lane);
                spread_codes(ups, kept.up, patch, lane);
                if (gelu)
                    activate_bwd<true, true>(w, dup, h, v, gates, ups, kept.gate_scale, kept.up_scale, lane);
                else
                    activate_bwd<false, true>(w, dup, h, v, gates, ups, kept.gate_scale, kept.up_scale, lane);
            }
            uint16_t* const dpre = g.out_pre + row * 2 * C + channel;
            store_rows(dpre, 2 * C, w, win, patch, lane);
            store_rows(dpre + C, 2 * C, dup, win, patch, lane);
            if (g.out != nullptr) store_rows(g.out + row * C + channel, C, h, win, patch, lane);
            if (c0 + kGroups * kChunk < columns)
                load_kept(kept, g, row + kGroups * kChunk, channel, {win.rows - kGroups * kChunk, win.channels}, lane);
        } else if constexpr (kOp == kWgrad) {
            pack(w, v);
            if (win.rows > 0 && pair_channel < g.C)
                outlet.send(out_map, pair_channel, t.column + from + c0, t.e, w, warp, lane);
        } else {
            pack(w, v);
            store_rows(g.out + row * C + channel, C, w, win, patch, lane);
        }
    }
    return true;
}

// ---------------------------------------------------------------------------- the kernel

// whether the last k of a stage do not fill their 16 (kWgrad, where k are rows)
__device__ __forceinline__ bool has_tail(int left) { return left < kBlockK && left % 16 != 0; }

// Tensor memory of a tile: one of two slots, gate and up side by side; a gated tile of more than
// 128 rows takes both.
template <int kOp>
__device__ __forceinline__ uint32_t slots_of(const Tile& t) {
    return Traits<kOp>::kGated && t.n > static_cast<int>(kSlotColumns / 2) ? 2 : 1;
}
__device__ __forceinline__ uint32_t up_sums(uint32_t tmem, uint32_t first, uint32_t slots) {
    return slots == 2 ? tmem + (first + 1) % 2 * kSlotColumns : tmem + first % 2 * kSlotColumns + kSlotColumns / 2;
}

// bytes of a CTA's part of the operand along the lanes of a tile, m / 2 lines or rows, as far as they lie
// before the last channel
template <int kOp>
__device__ __forceinline__ uint32_t a_bytes(int channels, int m) {
    if (channels <= 0) return 0;
    if (!Traits<kOp>::kAAcross) return m == 256 ? Traits<kOp>::kABytes : Traits<kOp>::kABytes / 2;
    return m == 256 && channels > 64 ? 2 * kCrossBlock : kCrossBlock;
}

// `a`: the operand along the lanes, in boxes of 128 rows, or of 64 lines of k, and `a64` in boxes of 64
// rows; `b64` and `b16`: the one along the columns, in boxes of 64 rows (or lines of k) and of 16; in
// kWgrad, `b16` is the output, in boxes of two warps' patch.
template <int kOp>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Traits<kOp>::kThreads, 1)
    expert_kernel(const __grid_constant__ CUtensorMap a_map, const __grid_constant__ CUtensorMap a64_map,
                  const __grid_constant__ CUtensorMap b64_map, const __grid_constant__ CUtensorMap b16_map,
                  ExpertArgs g) {
    using Tr = Traits<kOp>;
    extern __shared__ __align__(1024) unsigned char s_stages[];
    Shared<kOp>& s = *reinterpret_cast<Shared<kOp>*>(s_stages + g.ring);
    const int tid = static_cast<int>(threadIdx.x), lane = tid % 32, warp = uniform(tid / 32);
    const int rank = static_cast<int>(cluster_rank());
    const uint32_t pair = blockIdx.x / 2, pairs = gridDim.x / 2;

    // The next kernel may settle as places become free: it takes none from this one, whose CTAs have all
    // begun by then.
    allow_dependents();
    // by warps that have few experts to plan, while the others ask for theirs
    if (tid == (kLastFinish - 1) * 32) {
        for (int i = 0; i < kMostStages; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
            if (kOp == kWgrad) {
                mbar_init(&s.part[i], 1);
                mbar_init(&s.ready[i], 2);
            }
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.sums_full[i], 1);
            mbar_init(&s.sums_empty[i], 2 * kFinishWarps);  // of both CTAs
        }
        for (int i = 0; i < kTiles; ++i) {
            mbar_init(&s.tile_full[i], 1);
            // both producers, the finishing warps; the multiplier in CTA 0; the tail's warp
            mbar_init(&s.tile_empty[i], 2 + kFinishWarps + (rank == 0 ? 1 : 0) + (kOp == kWgrad ? 1 : 0));
        }
        mbar_init(&s.drain, 1);
        mbar_init_fence();
        s.watch = {0, 0};
    }
    if (warp == kLastFinish) tmem_alloc_pair(&s.tmem, kTmemColumns);
    if (tid == (kLastFinish - 2) * 32) {
        prefetch_tensor_map(a_map);
        prefetch_tensor_map(b64_map);
        prefetch_tensor_map(b16_map);
    }
    __syncwarp();
    cluster_arrive();  // the other CTA waits for these barriers while the tiles are planned
    grid_dependency_wait();  // dependent launch: inputs are ready after this
    if constexpr (kOp == kWgrad) {
        if (tid == 0) {
            Tile first;
            if (!tile_at<kOp>(g, s, pair, &first)) first.e = -1;
            s.tile[0] = first;
        }
        if (blockIdx.x == 0)
            for (int e = tid; e < g.E; e += Tr::kThreads)
                if (expert_rows(g.offsets, e, g.epr, g.inv_epr, g.max_rows).dropped) raise_flag(g.status, EP_FLAG_CAPACITY);
    } else {
        plan_tiles<kOp>(g, s, pair, pairs);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_wait();
    tc_fence_after();
    const uint32_t tmem = uniform(s.tmem);

    Tile t;
    Tiles tiles;
    if (warp == kScheduler) {
        if (lane == 0) {
            bool more = s.tile[0].e >= 0;  // the first tile is there
            mbar_arrive(&s.tile_full[0]);
            uint32_t at = 1, phase = 0;
            for (uint32_t i = pair + pairs; more; i += pairs) {
                more = tile_at<kOp>(g, s, i, &t);
                if (!more) t.e = -1;
                if (!mbar_wait(&s.tile_empty[at], phase ^ 1, &s.watch)) {
                    give_up(g, s);
                    break;
                }
                s.tile[at] = t;
                mbar_arrive(&s.tile_full[at]);
                if (++at == kTiles) at = 0, phase ^= 1;
            }
        }
    } else if (warp == kProducer || warp == Tr::kColumnProducer) {
        // One warp copies the operand along the lanes (and counts the bytes of both), the other the one
        // along the columns: one thread issued a stage's copies in 440 to 670 cycles, and they are
        // multiplied in 512. The whole warp keeps the books, so that they stay uniform; one lane issues.
        const bool leader = elected(), lanes = warp == kProducer;
        int stage = 0;
        uint32_t empty = ~0u, full = 0, part = 0, last_part = 0;  // a bit a stage: parities; its last use
        uint32_t issued = 0;
        const Ring<kOp> ring(g, s);
        const uint32_t counted = peer_addr(&s.full[0], 0);
        bool ok = true;
        while (ok && tiles.next<true>(s, &t)) {
            __syncwarp();
            if (leader) tiles.taken(s);
            const int half = t.n / 2;
            const int b_first = rank * half;
            // Bytes of a half of a stage: whole boxes, also where they hang over an end. Boxes that lie
            // past the last channel are left out: the sums of what is in their place are not kept.
            const uint32_t b_bytes = kOp == kWgrad ? (half + 63) / 64 * kCrossBlock
                                                   : static_cast<uint32_t>(half) * kBlockK * 2;
            const int c = t.channel + rank * (t.m / 2), row = static_cast<int>(t.row) + (kOp == kWgrad ? 0 : b_first);
            const uint32_t mine = a_bytes<kOp>(g.C - c, t.m);
            const uint32_t both = a_bytes<kOp>(g.C - t.channel, t.m) + a_bytes<kOp>(g.C - t.channel - t.m / 2, t.m) +
                                  2 * b_bytes;
            for (int k = 0; k < t.k; k += kBlockK) {
                ok = warp_wait(&s.empty[stage], empty >> stage & 1, &s.watch);
                if (!ok) break;
                empty ^= 1u << stage;
                const uint32_t to = smem_addr(s_stages) + stage * ring.bytes;
                const uint32_t b_to = to + Tr::kABytes;
                const bool tail = kOp == kWgrad && has_tail(t.k - k);
                // a tail's bytes each CTA counts itself, since it clears them; others CTA 0 counts for both
                const uint32_t bar = tail ? smem_addr(&s.part[stage]) : counted + stage * 8;
                if (leader && lanes) {
                    if (tail)
                        mbar_arrive_expect_tx(&s.part[stage], mine + b_bytes);
                    else if (rank == 0)
                        mbar_arrive_expect_tx(&s.full[stage], both);
                    if constexpr (kOp == kGateUp) {
                        const CUtensorMap& map = t.m == 256 ? a_map : a64_map;
                        if (mine > 0) {
                            tma_load_pair_3d(to, map, k, c, 2 * t.e, bar);
                            tma_load_pair_3d(to + 128 * kBlockK * 2, map, k, c, 2 * t.e + 1, bar);
                        }
                    } else if constexpr (kOp == kDown) {
                        if (mine > 0) tma_load_pair_3d(to, t.m == 256 ? a_map : a64_map, k, c, t.e, bar);
                    } else if constexpr (kOp == kWgrad) {
                        if (mine > 0) tma_load_pair_2d(to, a_map, c, row + k, bar);
                        if (mine > kCrossBlock) tma_load_pair_2d(to + kCrossBlock, a_map, c + 64, row + k, bar);
                    } else {
                        if (mine > 0) tma_load_pair_3d(to, a_map, c, k, t.e, bar);
                        if (mine > kCrossBlock) tma_load_pair_3d(to + kCrossBlock, a_map, c + 64, k, t.e, bar);
                    }
                } else if (leader) {
                    if constexpr (kOp == kWgrad) {
                        tma_load_pair_2d(b_to, b64_map, t.column + b_first, row + k, bar);
                        if (half > 64)
                            tma_load_pair_2d(b_to + kCrossBlock, b64_map, t.column + b_first + 64, row + k, bar);
                    } else {
                        int j = 0;
                        for (; j + 64 <= half; j += 64)
                            tma_load_pair_2d(b_to + j * kBlockK * 2, b64_map, k, row + j, bar);
                        for (; j < half; j += 16) tma_load_pair_2d(b_to + j * kBlockK * 2, b16_map, k, row + j, bar);
                    }
                }
                if (tail) {
                    part ^= 1u << stage;
                    last_part |= 1u << stage;
                } else {
                    full ^= 1u << stage;
                    last_part &= ~(1u << stage);
                }
                ++issued;
                if (leader && lanes) *static_cast<volatile uint32_t*>(&s.watch.stages) = issued;
                if (++stage == ring.stages) stage = 0;
            }
        }
        ok = ok && tiles.ok;
        if (!ok) give_up(g, s);
        // The last use of every stage is waited for: by its release, or where something gave up, by
        // its bytes, so that no copy and no arrival is on its way when the CTA ends.
        const int used = issued < static_cast<uint32_t>(ring.stages) ? static_cast<int>(issued) : ring.stages;
        for (int i = 0; i < used; ++i) {
            stage = stage == 0 ? ring.stages - 1 : stage - 1;
            if (ok && !mbar_wait(&s.empty[stage], empty >> stage & 1, &s.watch)) ok = false;
            if (ok) continue;
            if (last_part >> stage & 1)
                mbar_wait(&s.part[stage], (part >> stage & 1) ^ 1, nullptr);
            else if (rank == 0)
                mbar_wait(&s.full[stage], (full >> stage & 1) ^ 1, nullptr);
        }
        if (!ok) give_up(g, s);
    } else if (warp == kMultiplier) {
        if (rank == 0) {
            const bool leader = elected();
            int stage = 0;
            uint32_t full = 0, ready = 0, slot = 0;
            const Ring<kOp> ring(g, s);
            constexpr uint32_t kUp = 128 * kBlockK * 2 >> 4;
            const uint32_t first_a = operand_low(smem_addr(s_stages), Tr::kAAcross);
            const uint32_t first_b = operand_low(smem_addr(s_stages) + Tr::kABytes, Tr::kBAcross);
            bool ok = true;
            constexpr uint32_t kAStep = Tr::kAAcross ? kStepAcross : kStepAlong;
            constexpr uint32_t kBStep = Tr::kBAcross ? kStepAcross : kStepAlong;
            while (ok && tiles.next<true>(s, &t)) {
                __syncwarp();
                if (leader) tiles.taken(s);
                if (t.k == 0) continue;
                const uint32_t first = slot, slots = slots_of<kOp>(t);
                for (uint32_t i = 0; ok && i < slots; ++i)
                    ok = __all_sync(kFullMask, mbar_wait<true>(&s.sums_empty[(slot + i) % 2],
                                                               ((slot + i) / 2 % 2) ^ 1, &s.watch));
                if (!ok) break;
                slot += slots;
                tc_fence_after();
                const uint32_t desc = product_desc(t.m, t.n, Tr::kAAcross, Tr::kBAcross);
                const uint32_t sums = tmem + first % 2 * kSlotColumns, ups = up_sums(tmem, first, slots);
                // Whole stages without a branch between their products, on values that the compiler knows to
                // be uniform: 64 k take 146 ns (N = 32; products 70, barriers and loop 76), and took 229 with
                // branches and values of each lane's own.
                int k = 0;
                for (; k + kBlockK <= t.k; k += kBlockK) {
                    ok = warp_wait(&s.full[stage], full >> stage & 1, &s.watch);
                    if (!ok) break;
                    full ^= 1u << stage;
                    tc_fence_after();
                    const uint32_t a = first_a + stage * (ring.bytes >> 4);
                    const uint32_t b = first_b + stage * (ring.bytes >> 4);
                    if (leader) {
#pragma unroll
                        for (int j = 0; j < kBlockK / 16; ++j) {
                            mma_pair(sums, a + j * kAStep, b + j * kBStep, desc, j > 0 || k > 0);
                            if (Tr::kGated) mma_pair(ups, a + kUp + j * kAStep, b + j * kBStep, desc, j > 0 || k > 0);
                        }
                        mma_commit_pair(&s.empty[stage]);
                    }
                    if (++stage == ring.stages) stage = 0;
                }
                if (ok && k < t.k) {  // the rest
                    if (kOp == kWgrad && has_tail(t.k - k)) {
                        ok = warp_wait<true>(&s.ready[stage], ready >> stage & 1, &s.watch);
                        ready ^= 1u << stage;
                    } else {
                        ok = warp_wait(&s.full[stage], full >> stage & 1, &s.watch);
                        full ^= 1u << stage;
                    }
                    if (!ok) break;
                    tc_fence_after();
                    uint32_t a = first_a + stage * (ring.bytes >> 4), b = first_b + stage * (ring.bytes >> 4);
                    if (leader) {
                        for (; k < t.k; k += 16, a += kAStep, b += kBStep) {
                            mma_pair(sums, a, b, desc, k > 0);
                            if (Tr::kGated) mma_pair(ups, a + kUp, b, desc, k > 0);
                        }
                        mma_commit_pair(&s.empty[stage]);
                    }
                    if (++stage == ring.stages) stage = 0;
                }
                if (!ok) break;
                if (leader)
                    for (uint32_t i = 0; i < slots; ++i) mma_commit_pair(&s.sums_full[(first + i) % 2]);
            }
            ok = ok && tiles.ok;
            // the other CTA's last arrivals must not come when this one has ended
            for (uint32_t i = slot < 2 ? 0 : slot - 2; ok && i < slot; ++i)
                ok = __all_sync(kFullMask, mbar_wait<true>(&s.sums_empty[i % 2], i / 2 % 2, &s.watch));
            if (!ok) {  // the products that were begun still read shared memory
                give_up(g, s);
                if (leader) mma_commit(&s.drain);
                mbar_wait(&s.drain, 0, nullptr);
            }
        }
    } else if (warp == kTail) {
        if constexpr (kOp == kWgrad) {
            // k is an expert's rows: what lies behind the last of them in their last 16, other experts'
            // rows or whatever a slab's end holds, is cleared before it is multiplied
            const Ring<kOp> ring(g, s);
            uint32_t blocks = 0, part = 0;
            bool ok = true;
            while (ok && tiles.next(s, &t)) {
                __syncwarp();
                if (lane == 0) tiles.taken(s);
                blocks += static_cast<uint32_t>((t.k + kBlockK - 1) / kBlockK);
                const int left = t.k % kBlockK;
                if (!has_tail(left)) continue;
                const uint32_t stage = (blocks - 1) % static_cast<uint32_t>(ring.stages);
                ok = __all_sync(kFullMask, mbar_wait(&s.part[stage], part >> stage & 1, &s.watch));
                if (!ok) break;
                part ^= 1u << stage;
                unsigned char* const at = s_stages + static_cast<size_t>(stage) * ring.bytes;
                const int end = (left + 15) / 16 * 16, blocks_here = 2 + (t.n / 2 + 63) / 64;
                for (int block = 0; block < blocks_here; ++block)
                    for (int line = left + lane / 8; line < end; line += 4)
                        *reinterpret_cast<uint4*>(at + block * kCrossBlock + line * 128 + lane % 8 * 16) =
                            make_uint4(0, 0, 0, 0);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(peer_addr(&s.ready[stage], 0));
            }
            if (!ok || !tiles.ok) give_up(g, s);
        }
    } else {
        const int group = (warp - kFinish) / 4;
        uint32_t slot = 0;
        // The first pass has no rows, while the first sums are made: it brings the code in, which takes
        // longer than a small tile itself (and is there once: 16 experts of 1024 x 512, 127 tokens back
        // through the activation 8.45 us, with a second copy of the code for this pass 9.2).
        Outlet outlet = {s.patch[(warp - kFinish) / 2 * 2 * Tr::kPatches]};
        t = {0, 0, 0, 256, 64, 0, 0, 0};
        for (bool begun = false;; begun = true) {
            if (begun) {
                const bool more = tiles.next<true>(s, &t);
                if (!group_agrees(tiles.ok, group)) {
                    give_up(g, s);
                    break;
                }
                if (!more) break;
                if (lane == 0) tiles.taken(s);
            }
            const uint32_t first = slot, slots = slots_of<kOp>(t);
            const auto ready = [&] {
                if (t.k == 0) return true;
                bool ok = true;
                for (uint32_t i = 0; ok && i < slots; ++i)
                    ok = mbar_wait(&s.sums_full[(first + i) % 2], (first + i) / 2 % 2, &s.watch);
                ok = group_agrees(ok, group);
                tc_fence_after();
                return ok;
            };
            if (!finish_tile<kOp>(g, b16_map, s, t, tmem + first % 2 * kSlotColumns, up_sums(tmem, first, slots),
                                  rank, warp, lane, outlet, ready)) {
                give_up(g, s);
                break;
            }
            if (t.k > 0) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    for (uint32_t i = 0; i < slots; ++i)
                        mbar_arrive_cluster_relaxed(peer_addr(&s.sums_empty[(first + i) % 2], 0));
                slot += slots;
            }
        }
        if (kOp == kWgrad && lane == 0) bulk_wait_all();
    }
    __syncwarp();
    tc_fence_before();
    cluster_sync_relaxed();  // neither CTA's shared or tensor memory is used by the other any more
    if (warp == kLastFinish) {
        tc_fence_after();
        tmem_free_pair(tmem, kTmemColumns);
    }
}

// Rows of all slabs, so that 32 bits hold a row, the end of a stage or of a tile of rows that begins there,
// and the last coordinate of a box of its copies.
constexpr long long kMostRows = (1ll << 31) - 512;
bool valid(int E, int R, int max_rows) {
    return R >= 1 && R <= 256 && E >= 1 && E <= 8192 && E % R == 0 && max_rows >= 0 &&
           static_cast<long long>(R) * max_rows <= kMostRows;
}
bool valid_width(int n, int most) { return n >= 8 && n <= most && n % 8 == 0; }
constexpr int kMostWidth = 65536;

ep_status_t zero_fill(void* p, size_t bytes, void* stream) {
    const cudaError_t err = cudaMemsetAsync(p, 0, bytes, as_stream(stream));
    return err == cudaSuccess ? EP_OK : cuda_fail(err);
}

// A map of bf16 `dims` (innermost first, dense), in boxes of 64 values by `lines`, swizzled for the
// tensor cores.
ep_status_t map_of(CUtensorMap* map, const void* base, uint64_t d0, uint64_t d1, uint64_t d2, uint32_t lines) {
    const uint64_t dims[3] = {d0, d1, d2}, strides[2] = {d0 * 2, d0 * d1 * 2};
    const uint32_t box[3] = {64, lines, 1};
    return encode_tensor_map(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, d2 == 0 ? 2 : 3, base, dims, strides, box,
                             CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int kOp>
ep_status_t launch(ExpertArgs g, const CUtensorMap& a, const CUtensorMap& a64, const CUtensorMap& b64,
                   const CUtensorMap& b16, void* stream) {
    using Tr = Traits<kOp>;
    static std::atomic<int> ready[kMaxDevices];
    g.epr = g.E / g.R;
    g.inv_epr = 1.0f / static_cast<float>(g.epr);
    const size_t behind = sizeof(Shared<kOp>) + (kOp == kWgrad ? 0 : sizeof(int) * static_cast<size_t>(g.E));
    g.ring = static_cast<uint32_t>((kSmemMost - behind) / 1024 * 1024);
    g.stages = 0;
    for (int i = 0; i < 4; ++i) {
        const uint32_t n = g.ring / Traits<kOp>::stage_bytes(i);
        g.stages |= (n < kMostStages ? n : kMostStages) << 8 * i;
    }
    const ep_status_t st = ensure_dynamic_smem(ready, expert_kernel<kOp>, static_cast<int>(kSmemMost));
    if (st != EP_OK) return st;
    const dim3 grid(static_cast<unsigned>(sm_count() / 2 * 2));
    return launch_dependent(expert_kernel<kOp>, grid, dim3(Tr::kThreads), g.ring + behind,
                            as_stream(stream), a, a64, b64, b16, g);
}

// Slabs without any rows: all that is left of a call is the flag, if an expert has rows.
__global__ void no_room_kernel(const int32_t* offsets, int E, int epr, float inv_epr, int32_t* status) {
    allow_dependents();
    grid_dependency_wait();
    for (int e = static_cast<int>(threadIdx.x); e < E; e += static_cast<int>(blockDim.x))
        if (expert_rows(offsets, e, epr, inv_epr, 0).dropped) raise_flag(status, EP_FLAG_CAPACITY);
}
ep_status_t no_room(const int32_t* offsets, int E, int R, int32_t* status, void* stream) {
    if (status == nullptr) return EP_OK;
    if (offsets == nullptr || !aligned16(offsets)) return EP_ERR_INVALID;
    const int epr = E / R;
    return launch_dependent(no_room_kernel, dim3(1), dim3(256), 0, as_stream(stream), offsets, E, epr,
                            1.0f / static_cast<float>(epr), status);
}

FewRows few(const ExpertArgs& g, const void* x, const void* w) {
    return {static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(w), g.offsets, g.act, g.C, g.K, g.E,
            g.max_rows, g.E / g.R, 1.0f / static_cast<float>(g.E / g.R), g.out, g.status};
}

// Rows of the slabs as the operand along the columns: in boxes of 64 rows and of 16.
ep_status_t row_maps(CUtensorMap* b64, CUtensorMap* b16, const void* rows, uint64_t width, const ExpertArgs& g) {
    const uint64_t n = static_cast<uint64_t>(g.R) * g.max_rows;
    const ep_status_t st = map_of(b64, rows, width, n, 0, 64);
    return st != EP_OK ? st : map_of(b16, rows, width, n, 0, 16);
}

}  // namespace

extern "C" {

ep_status_t ep_expert_gate_up(const void* x, const void* w_gate_up, const int32_t* expert_offsets, ep_act_t act,
                              int32_t H, int32_t F, int32_t E, int32_t R, int32_t max_rows, void* h, void* pre,
                              uint8_t* pre_q, void* pre_scales, int32_t* status, void* stream) {
    if (!valid(E, R, max_rows) || !valid_width(H, kMostWidth) || !valid_width(F, kMostWidth)) return EP_ERR_INVALID;
    if (act != EP_ACT_SILU && act != EP_ACT_GELU) return EP_ERR_INVALID;
    if ((pre_q == nullptr) != (pre_scales == nullptr) || (pre_q != nullptr && F % 128 != 0)) return EP_ERR_INVALID;
    if (max_rows == 0) return no_room(expert_offsets, E, R, status, stream);
    if (x == nullptr || w_gate_up == nullptr || expert_offsets == nullptr || h == nullptr) return EP_ERR_INVALID;
    if (!aligned16(x) || !aligned16(w_gate_up) || !aligned16(expert_offsets) || !aligned16(h) ||
        !aligned16_or_null(pre) || !aligned16_or_null(pre_q) || !aligned16_or_null(pre_scales))
        return EP_ERR_INVALID;
    ExpertArgs g = {};
    g.offsets = expert_offsets;
    g.act = act;
    g.C = F;
    g.K = H;
    g.E = E;
    g.R = R;
    g.max_rows = max_rows;
    g.out = static_cast<uint16_t*>(h);
    g.out_pre = static_cast<uint16_t*>(pre);
    g.out_q = pre_q;
    g.out_scales = static_cast<uint16_t*>(pre_scales);
    g.status = status;
    const int few_at_once = pre == nullptr && pre_q == nullptr ? few_rows_at_once(E, R, max_rows, 1ll * H * F, true) : 0;
    if (few_at_once > 0) return launch_few_rows(few(g, x, w_gate_up), true, few_at_once, stream);
    CUtensorMap a, a64, b64, b16;
    ep_status_t st = map_of(&a, w_gate_up, H, F, 2ull * E, 128);
    if (st == EP_OK) st = map_of(&a64, w_gate_up, H, F, 2ull * E, 64);
    if (st == EP_OK) st = row_maps(&b64, &b16, x, H, g);
    return st != EP_OK ? st : launch<kGateUp>(g, a, a64, b64, b16, stream);
}

ep_status_t ep_expert_down(const void* h, const void* w_down, const int32_t* expert_offsets, int32_t H, int32_t F,
                           int32_t E, int32_t R, int32_t max_rows, void* y, int32_t* status, void* stream) {
    if (!valid(E, R, max_rows) || !valid_width(H, kMostWidth) || !valid_width(F, kMostWidth)) return EP_ERR_INVALID;
    if (max_rows == 0) return no_room(expert_offsets, E, R, status, stream);
    if (h == nullptr || w_down == nullptr || expert_offsets == nullptr || y == nullptr) return EP_ERR_INVALID;
    if (!aligned16(h) || !aligned16(w_down) || !aligned16(expert_offsets) || !aligned16(y)) return EP_ERR_INVALID;
    ExpertArgs g = {};
    g.offsets = expert_offsets;
    g.C = H;
    g.K = F;
    g.E = E;
    g.R = R;
    g.max_rows = max_rows;
    g.out = static_cast<uint16_t*>(y);
    g.status = status;
    const int few_at_once = few_rows_at_once(E, R, max_rows, 1ll * H * F, false);
    if (few_at_once > 0) return launch_few_rows(few(g, h, w_down), false, few_at_once, stream);
    CUtensorMap a, a64, b64, b16;
    ep_status_t st = map_of(&a, w_down, F, H, E, 128);
    if (st == EP_OK) st = map_of(&a64, w_down, F, H, E, 64);
    if (st == EP_OK) st = row_maps(&b64, &b16, h, F, g);
    return st != EP_OK ? st : launch<kDown>(g, a, a64, b64, b16, stream);
}

ep_status_t ep_expert_down_bwd(const void* dy, const void* w_down, const void* pre, const uint8_t* pre_q,
                               const void* pre_scales, const int32_t* expert_offsets, ep_act_t act, int32_t H,
                               int32_t F, int32_t E, int32_t R, int32_t max_rows, void* dpre, void* h,
                               int32_t* status, void* stream) {
    if (!valid(E, R, max_rows) || !valid_width(H, kMostWidth) || !valid_width(F, kMostWidth)) return EP_ERR_INVALID;
    if (act != EP_ACT_SILU && act != EP_ACT_GELU) return EP_ERR_INVALID;
    if ((pre_q == nullptr) != (pre_scales == nullptr) || (pre_q != nullptr && F % 128 != 0)) return EP_ERR_INVALID;
    if (max_rows == 0) return no_room(expert_offsets, E, R, status, stream);
    if ((pre == nullptr) == (pre_q == nullptr)) return EP_ERR_INVALID;
    if (dy == nullptr || w_down == nullptr || expert_offsets == nullptr || dpre == nullptr) return EP_ERR_INVALID;
    if (!aligned16(dy) || !aligned16(w_down) || !aligned16(expert_offsets) || !aligned16(dpre) ||
        !aligned16_or_null(pre) || !aligned16_or_null(pre_q) || !aligned16_or_null(pre_scales) || !aligned16_or_null(h))
        return EP_ERR_INVALID;
    ExpertArgs g = {};
    g.pre = static_cast<const uint16_t*>(pre);
    g.pre_q = pre_q;
    g.pre_scales = static_cast<const uint16_t*>(pre_scales);
    g.offsets = expert_offsets;
    g.act = act;
    g.C = F;
    g.K = H;
    g.E = E;
    g.R = R;
    g.max_rows = max_rows;
    g.out = static_cast<uint16_t*>(h);
    g.out_pre = static_cast<uint16_t*>(dpre);
    g.status = status;
    CUtensorMap a, b64, b16;
    ep_status_t st = map_of(&a, w_down, F, H, E, 64);
    if (st == EP_OK) st = row_maps(&b64, &b16, dy, H, g);
    return st != EP_OK ? st : launch<kDownBwd>(g, a, a, b64, b16, stream);
}

ep_status_t ep_expert_gate_up_bwd(const void* dpre, const void* w_gate_up, const int32_t* expert_offsets, int32_t H,
                                  int32_t F, int32_t E, int32_t R, int32_t max_rows, void* dx, int32_t* status,
                                  void* stream) {
    if (!valid(E, R, max_rows) || !valid_width(H, kMostWidth) || !valid_width(F, kMostWidth)) return EP_ERR_INVALID;
    if (max_rows == 0) return no_room(expert_offsets, E, R, status, stream);
    if (dpre == nullptr || w_gate_up == nullptr || expert_offsets == nullptr || dx == nullptr) return EP_ERR_INVALID;
    if (!aligned16(dpre) || !aligned16(w_gate_up) || !aligned16(expert_offsets) || !aligned16(dx))
        return EP_ERR_INVALID;
    ExpertArgs g = {};
    g.offsets = expert_offsets;
    g.C = H;
    g.K = 2 * F;
    g.E = E;
    g.R = R;
    g.max_rows = max_rows;
    g.out = static_cast<uint16_t*>(dx);
    g.status = status;
    CUtensorMap a, b64, b16;
    ep_status_t st = map_of(&a, w_gate_up, H, 2ull * F, E, 64);
    if (st == EP_OK) st = row_maps(&b64, &b16, dpre, 2ull * F, g);
    return st != EP_OK ? st : launch<kGateUpBwd>(g, a, a, b64, b16, stream);
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
    g.offsets = expert_offsets;
    g.C = J;
    g.K = I;
    g.E = E;
    g.R = R;
    g.max_rows = max_rows;
    g.out = static_cast<uint16_t*>(dw);
    g.status = status;
    if (max_rows == 0) {
        const ep_status_t st = zero_fill(dw, static_cast<size_t>(E) * I * J * 2, stream);
        return st != EP_OK ? st : no_room(expert_offsets, E, R, status, stream);
    }
    const uint64_t n = static_cast<uint64_t>(R) * max_rows;
    CUtensorMap a, b, out;
    ep_status_t st = map_of(&a, rows, J, n, 0, 64);
    if (st == EP_OK) st = map_of(&b, dout, I, n, 0, 64);
    if (st == EP_OK) st = map_of(&out, dw, J, I, E, 16);
    return st != EP_OK ? st : launch<kWgrad>(g, a, a, b, out, stream);
}

}  // extern "C"
