// paged_attention.hip -- attention of one new token per sequence over a
// paged key/value cache, split over the cache's length and joined.
//
// Mathematics.  With s_j = scale q . k_j over the visible tokens j,
//   out = sum_j 2^(t_j - M) v_j / sum_j 2^(t_j - M),  t_j = s_j log2(e),
// for any reference M: the sums are kept relative to a running M that is
// raised (and the sums scaled down) only when a score exceeds it by more
// than 2^8, so a tile rarely costs a rescale, and a weight is at most 2^8.
// Parts with their own M are joined by weighting each with 2^(M_part - M).
//
// Bound: HBM.  Every visible row of K and V is read once; per byte there is
// one multiply-add per query head of the group, far below the matrix cores'
// rate.  Eight sequences of 32768 tokens, 8 key heads, both launches: bf16
// heads of 128 194 us (5.5 TB/s; heads of 64 5.3, of 192 5.1, of 256 5.7),
// int8 heads of 128 111 us (5.0; of 256 4.9).  48 sequences of up to 9001
// tokens, 100000 in all, int8: 52 to 57 us (3.9 TB/s; 43 where the Infinity Cache
// holds them): the blocks that find nothing to do leave at about 100 a us, and the
// last ones run alone.  A short sequence is bound by latency, the chain lens ->
// table -> K -> V and the join: one of 1000 tokens 6.7 us.
//
// A block takes one sequence, one key head (up to 16 of its query heads,
// one matrix tile) and a chunk of the visible tokens.  Its threads first
// turn the chunk's tokens into row offsets in LDS (page lookup, window and
// sinks, the bounds check of the page), so the main loop knows nothing of
// pages.  Then each wave walks its own tiles of 32 tokens, K and V rows
// copied straight into its part of LDS, the next tile's K while this one's
// softmax and V product run and the next V during the next K product: no
// barrier until the waves' sums meet at the end.
//
// Products (16 x 16 x 32): K rows are the first operand and the queries the
// second, so S^T lands with lane 16 G + i holding tokens 4 G + r of two
// 16-token tiles for head i.  These eight are one lane's K elements of the
// next product's second operand (the order of the 32 tokens is free as long
// as V's is the same), so the weights pass from one product to the other in
// registers.  The first operand, V^T, comes out of row-major LDS by
// transposing reads of the same tokens.  Weights enter as 16-bit parts, each
// the rounded rest that those before it left: three of bf16, which hold p to
// fp32's own 2^-24 (two would leave 2^-16, which shows where values cancel),
// and four of fp16.  fp16 ends at 2^-24, so its last two parts are 2^23 times
// finer and have sums of their own: a weight is held to 2^-22 of itself or
// 2^-54 of the largest one.  (With the first two alone, light tokens beside a
// heavy one of little value were 0.2 % off at 2^-24 of it and lost at 2^-32.)
// The matrix cores have the time: 4 x 131072 bf16 tokens take 394 us with two
// parts and with three, 8 x 32768 fp16 ones 194 us with two and with four.
//
// The keys of an int8 cache are multiplied in fp16: codes are exact in it,
// and cost five operations for four (byte | 0x6400 is 1024 + byte).  A head's
// query is scaled by a power of two to the range of fp16 (exact for bf16
// elements down to 2^-31 of its largest and fp16 ones down to 2^-28; lost below
// 2^-38), and the scale of a key row is applied to its score.  Values are multiplied in bf16 (six operations for
// four codes): a row's scale is applied to its weight, and the product has to
// hold what a light token's row or a row of a small scale contributes beside a
// heavy one or one of a large scale.  (In fp16, whose parts end at 2^-24, the
// rows whose product lay 2^26 below the largest were 4 % off and those 2^32
// below were lost; 48 ragged sequences took 53.3 us so, 55.1 in bf16.)  Scales are
// taken relative to a power of two near the chunk's largest, so that the
// product neither overflows nor is subnormal.

struct AttnArgs {
    const uint16_t* q;
    uint16_t* out;
    const int32_t* table;
    const int32_t* lens;
    float* part;                         // [batch * hq * splits][d] weighted values
    float2* part_ml;                     // [batch * hq * splits] (M, sum)
    const uint8_t* ck;
    const uint8_t* cv;
    const float* cks;
    const float* cvs;
    int64_t q_bs, q_hs, o_bs, o_hs, table_stride, c_ps, c_hs, c_ts, s_ps, s_hs, s_ts;
    int64_t pages, capacity;             // capacity: tokens a table row can name
    int64_t window, sinks;
    float scale;
    int hq, hk, group, row_blocks, page_shift, splits, chunk;
};

// The visible tokens of a sequence, counted from 0: the first `head` are
// tokens 0 .. head - 1, the others follow from token `gap` + index on.
struct Visible {
    int64_t count, head, gap;
    __device__ __forceinline__ int64_t token(int64_t i) const { return i < head ? i : i + gap; }
};

__device__ __forceinline__ Visible visible(const AttnArgs& a, int64_t len)
{
    const int64_t n = min(max(len, (int64_t)0), a.capacity);
    if (a.window <= 0 || n <= a.window) return {n, n, 0};
    const int64_t lo = n - a.window, head = min(a.sinks, lo);
    return {head + a.window, head, lo - head};
}

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kAttnTile = 32;            // tokens per tile
constexpr int kAttnChunk = 1024;         // most tokens per block
constexpr float kAttnSlack = 8.0f;       // a score may exceed M by this (base 2)
// M before any score: the lowest finite value, so that a score of -inf has
// the weight 0 under every M, and a row of nothing else ends as 0 / 0.
constexpr float kAttnLow = -3.402823466e38f;

constexpr int gcd_c(int a, int b) { return b == 0 ? a : gcd_c(b, a % b); }

// Sizes for rows of RB bytes: a wave holds one tile of K and one of V, and a
// block has as many waves as fit 64 KiB, so that two blocks share a CU (one
// hides the other's start and end).  Persistent blocks, two a CU, that walk
// a list of the chunks that exist took 60 us for the 54 us above, and 421 us
// for 394 us at 4 sequences of 131072 tokens.
template <int RB>
struct AttnShape {
    static constexpr int tile = kAttnTile * RB;          // bytes of a K (or V) tile
    static constexpr int loads = tile / 1024;            // 1 KiB loads per tile
    static constexpr int fit = 65536 / (2 * tile);
    static constexpr int waves = fit >= 8 ? 8 : fit >= 4 ? 4 : 2;
    static constexpr int chunks = RB / 16;               // 16-byte pieces of a row
    // Rows repeat their place among the 256 bytes of banks every `period`
    // rows; within a place, pieces are exchanged by xor so that the 16 rows
    // (8 rows of two pieces) that a read touches at once land apart.
    static constexpr int span = gcd_c(RB, 256);
    static constexpr int period = 256 / span;
    __device__ static constexpr int swz(int row) { return (row / period) & (span / 16 - 1); }
    __device__ static constexpr int swz2(int row) { return ((row / period) & (span / 32 - 1)) << 1; }
};

__device__ __forceinline__ void dma16_at(const uint8_t* p, uint32_t lds)
{
    asm volatile("global_load_lds_dwordx4 %0, off" : : "v"(p), "{m0}"(lds) : "memory");
}

// Four int8 codes to fp16, exactly: byte + 128 in the low bits of 1024.
__device__ __forceinline__ void codes_f16(uint32_t w, uint32_t& lo, uint32_t& hi)
{
    const uint32_t u = w ^ 0x80808080u;
    const f16x2 off = {(_Float16)-1152.0f, (_Float16)-1152.0f};
    lo = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, u, 0x04010400u)) + off);
    hi = __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, u, 0x04030402u)) + off);
}

__device__ __forceinline__ v4i codes8_f16(uint2 w)
{
    uint32_t o[4];
    codes_f16(w.x, o[0], o[1]);
    codes_f16(w.y, o[2], o[3]);
    return v4i{(int)o[0], (int)o[1], (int)o[2], (int)o[3]};
}

// Four int8 codes to bf16, exactly: the upper halves of their fp32 values.
__device__ __forceinline__ void codes_bf16(uint32_t w, uint32_t& lo, uint32_t& hi)
{
    float f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = (float)(int8_t)(w >> (8 * i));
    lo = __builtin_amdgcn_perm(__float_as_uint(f[1]), __float_as_uint(f[0]), 0x07060302u);
    hi = __builtin_amdgcn_perm(__float_as_uint(f[3]), __float_as_uint(f[2]), 0x07060302u);
}

__device__ __forceinline__ v4i codes8_bf16(uint2 w)
{
    uint32_t o[4];
    codes_bf16(w.x, o[0], o[1]);
    codes_bf16(w.y, o[2], o[3]);
    return v4i{(int)o[0], (int)o[1], (int)o[2], (int)o[3]};
}

template <int DT>
__device__ __forceinline__ f32x4v mfma16(const v4i& a, const v4i& b, const f32x4v& c)
{
    if constexpr (DT == CK_DT_FP16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Transposing LDS reads, per 16 lanes: lanes 4 r .. 4 r + 3 point at 16
// two-byte columns of row r, and lane i gets column i of rows 0 .. 3; or
// lanes 2 r, 2 r + 1 at 16 one-byte columns of row r, lane i column i of
// rows 0 .. 7.
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint2 read_tr16(const uint8_t* p)
{
    return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(p)));
}

__device__ __forceinline__ uint2 read_tr8(const uint8_t* p)
{
    return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr8_b64_v2i32((__attribute__((address_space(3))) i32x2*)(p)));
}

// The types of the products and how a weight enters the second one: PARTS
// parts of 16 bits, in NA sums.  The parts of fp16 are kept 2^6 higher, at most
// 2^14, and those of the second sum hold `fine` times what the first ones left,
// at most 2^14 too.
template <int DT, bool I8, int PARTS>
struct AttnKind {
    static constexpr int KT = I8 ? CK_DT_FP16 : DT;
    static constexpr int VT = I8 ? CK_DT_BF16 : DT;
    static constexpr int NA = VT == CK_DT_FP16 ? 2 : 1;
    static constexpr int each = PARTS / NA;                  // parts of a sum
    static constexpr float lift = VT == CK_DT_FP16 ? 6.0f : 0.0f;
    static constexpr float fine = each == 2 ? 8388608.0f : 2048.0f;
};

// Where a lane reads K and V of a tile, whose rows begin at kr and vr in LDS: what
// of its places does not follow from the others by a constant.
template <bool I8, int D>
struct AttnLane {
    static constexpr int RB = D * (I8 ? 1 : 2), KK = D / 32, DB = D / 16;
    using Sh = AttnShape<RB>;
    static constexpr int kstep = I8 ? 2 : 4, vstep = I8 ? 1 : 2;             // 16-byte pieces of a K step, of 16 columns of V
    static constexpr int least(int x, int y) { return x < y ? (x < 1 ? 1 : x) : y; }
    static constexpr int KN = least(Sh::span / 16 / kstep, KK), VN = least(Sh::span / 16 / vstep, DB);
    const uint8_t *k[KN], *v[VN];

    __device__ __forceinline__ AttnLane(const uint8_t* kr, const uint8_t* vr, int lane)
    {
        const int G = lane >> 4, i16 = lane & 15;
#pragma unroll
        for (int i = 0; i < KN; ++i) {
            const int piece = 4 * i + G;                     // int8: of eight codes
            k[i] = kr + i16 * RB + (I8 ? (((piece >> 1) ^ Sh::swz(i16)) << 4) + (piece & 1) * 8 : (piece ^ Sh::swz(i16)) << 4);
        }
        // transposing reads; int8: row r of the eight is token 4 G + r of the first tile or 4 G + r - 4 of the second
        const int r = i16 >> 1, row = I8 ? 4 * G + (r & 3) + 16 * (r >> 2) : 4 * G + (i16 >> 2);
#pragma unroll
        for (int i = 0; i < VN; ++i)
            v[i] = vr + row * RB + ((I8 ? i ^ Sh::swz(row) : (2 * i + ((i16 >> 1) & 1)) ^ Sh::swz2(row)) << 4) + (i16 & 1) * 8;
    }
    // (rows 16 apart have the same place among the banks)
    __device__ __forceinline__ const uint8_t* k_at(int u, int kk) const { return k[kk % KN] + 16 * u * RB + kk / KN * (KN * kstep * 16); }
    __device__ __forceinline__ const uint8_t* v_at(int u, int d) const { return v[d % VN] + 16 * u * RB + d / VN * (VN * vstep * 16); }
};

// One tile of 32 tokens for MB blocks of 16 rows of queries: `at` are this
// lane's places in the tile's K and V, `off` bytes on; kscale and vscale (int8)
// are the tokens' scales, and `limit` is the number of its tokens that count.
// M, L and acc are the rows' running reference, sums of weights and weighted
// values; `empty`: the sums are still zero.  k_read(), v_ready() and v_read() are
// called when K has been read, before V is read and after.  FOLD: a score is
// scaled in the step that takes the reference off, one rounding for two; V,
// which has to be there, is read before the weights are made where there are
// registers for it; a wave in its products goes before one in its weights; and K
// is read some pieces ahead of its products, which the compiler, short of
// registers, does not do by itself (128 sequences behind 65536 tokens, 64/8 heads
// of 128, with two parts of a weight: 453 us, 421, 408 and 402; 471 with three).
template <int DT, bool I8, int D, int MB, int PARTS, bool FOLD, class KRead, class VReady, class VRead>
__device__ __forceinline__ void attn_tile(const AttnLane<I8, D>& at, int off, const v4i (&qf)[MB][D / 32],
                                          const float (&sc)[MB], const float* kscale, const float* vscale, int ve,
                                          int limit, bool empty, float (&M)[MB], float (&L)[MB],
                                          f32x4v (&acc)[MB][AttnKind<DT, I8, PARTS>::NA][D / 16], KRead k_read,
                                          VReady v_ready, VRead v_read)
{
    constexpr int KK = D / 32, DB = D / 16;
    using Kind = AttnKind<DT, I8, PARTS>;
    constexpr int KT = Kind::KT, VT = Kind::VT, NA = Kind::NA;
    constexpr bool AHEAD = FOLD && MB * NA < 4;
    const int G = (threadIdx.x & 63) >> 4;
    f32x4v s[MB][2];
    if constexpr (FOLD) __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int b = 0; b < MB; ++b) s[b][u] = f32x4v{0.0f, 0.0f, 0.0f, 0.0f};
    using Raw = std::conditional_t<I8, uint2, v4i>;
    auto read_k = [&](int u, int kk) { return *reinterpret_cast<const Raw*>(at.k_at(u, kk) + off); };
    auto score = [&](int u, int kk, const Raw& raw) {
        v4i kf;
        if constexpr (I8) kf = codes8_f16(raw);
        else kf = raw;
#pragma unroll
        for (int b = 0; b < MB; ++b) s[b][u] = mfma16<KT>(kf, qf[b][kk], s[b][u]);
    };
    if constexpr (AHEAD) {
        constexpr int N = KK % 2 == 0 ? 4 : 2, groups = 2 * KK / N;
        Raw raw[2][N];
#pragma unroll
        for (int g = 0; g <= groups; ++g) {
            if (g < groups) {
#pragma unroll
                for (int x = 0; x < N; ++x) raw[g & 1][x] = read_k((g * N + x) / KK, (g * N + x) % KK);
            }
            __builtin_amdgcn_sched_barrier(0);
            if (g > 0) {
#pragma unroll
                for (int x = 0; x < N; ++x) score(((g - 1) * N + x) / KK, ((g - 1) * N + x) % KK, raw[(g - 1) & 1][x]);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    } else {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) score(u, kk, read_k(u, kk));
    }
    k_read();
    if constexpr (FOLD) __builtin_amdgcn_s_setprio(0);
    constexpr bool EARLY = FOLD && MB * (NA * DB + KK) <= 24;
    uint2 vr[EARLY ? DB : 1][2];
    auto read_v = [&](int d, uint2 (&v)[2]) {
        if constexpr (I8) {
            v[0] = read_tr8(at.v_at(0, d) + off);
        } else {
            v[0] = read_tr16(at.v_at(0, d) + off);
            v[1] = read_tr16(at.v_at(1, d) + off);
        }
    };
    if constexpr (EARLY) {
#pragma unroll
        for (int d = 0; d < DB; ++d) read_v(d, vr[d]);
    }
    v4i part[MB][PARTS];                                     // the weights are their sum
#pragma unroll
    for (int b = 0; b < MB; ++b) {
        float p[8], by[8];                                   // by: what a score is multiplied by
#pragma unroll
        for (int e = 0; e < 8; ++e) by[e] = sc[b];
        if constexpr (I8 && FOLD) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const float4 ks = *reinterpret_cast<const float4*>(&kscale[4 * G + 16 * u]);
                by[4 * u] *= ks.x; by[4 * u + 1] *= ks.y; by[4 * u + 2] *= ks.z; by[4 * u + 3] *= ks.w;
            }
        }
        auto hide = [&]() {
            if (limit < kAttnTile) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (4 * G + 16 * (e >> 2) + (e & 3) >= limit) p[e] = -INFINITY;
            }
        };
        auto highest = [&]() {
            return fmaxf(fmaxf(fmaxf(p[0], p[1]), fmaxf(p[2], p[3])), fmaxf(fmaxf(p[4], p[5]), fmaxf(p[6], p[7])));
        };
        auto raise = [&](float top) {                        // M to at least `top` of any lane of the row
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            const float m = fmaxf(M[b], top);
            const float f = __builtin_amdgcn_exp2f(M[b] - m);
            M[b] = m;
            L[b] *= f;
            if (!empty) {
#pragma unroll
                for (int i = 0; i < NA; ++i)
#pragma unroll
                    for (int d = 0; d < DB; ++d) acc[b][i][d] = acc[b][i][d] * f;
            }
        };
        float sum = 0.0f;
        if constexpr (FOLD) {
            auto less = [&]() {                              // the exponents of the weights
                const float ref = M[b] - Kind::lift;
#pragma unroll
                for (int e = 0; e < 8; ++e) p[e] = __builtin_fmaf(s[b][e >> 2][e & 3], by[e], -ref);
                hide();
            };
            less();
            if (__any(highest() > kAttnSlack + Kind::lift)) {
#pragma unroll
                for (int e = 0; e < 8; ++e) p[e] = s[b][e >> 2][e & 3] * by[e];
                hide();
                raise(highest());
                less();
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                p[e] = __builtin_amdgcn_exp2f(p[e]);
                sum += p[e];
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) p[e] = s[b][e >> 2][e & 3] * sc[b];
            if constexpr (I8) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float4 ks = *reinterpret_cast<const float4*>(&kscale[4 * G + 16 * u]);
                    p[4 * u] *= ks.x; p[4 * u + 1] *= ks.y; p[4 * u + 2] *= ks.z; p[4 * u + 3] *= ks.w;
                }
            }
            hide();
            const float top = highest();
            if (__any(top > M[b] + kAttnSlack)) raise(top);
            const float ref = M[b] - Kind::lift;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                p[e] = __builtin_amdgcn_exp2f(p[e] - ref);
                sum += p[e];
            }
        }
        L[b] += sum;
        if constexpr (I8) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const float4 vs = *reinterpret_cast<const float4*>(&vscale[4 * G + 16 * u]);
                const float v[4] = {vs.x, vs.y, vs.z, vs.w};
#pragma unroll
                for (int r = 0; r < 4; ++r) p[4 * u + r] *= __builtin_amdgcn_ldexpf(v[r], -ve);
            }
        }
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            float x = p[2 * w], y = p[2 * w + 1];
#pragma unroll
            for (int i = 0; i < PARTS; ++i) {
                const uint32_t h = narrow2<VT>(x, y);
                part[b][i][w] = (int)h;
                if (i + 1 == PARTS) break;
                const float2 back = widen2<VT>(h);
                x -= back.x;
                y -= back.y;
                if (NA == 2 && i == Kind::each - 1) {
                    x *= Kind::fine;
                    y *= Kind::fine;
                }
            }
        }
    }
    v_ready();
    if constexpr (FOLD) __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int d = 0; d < DB; ++d) {
        if constexpr (!EARLY) read_v(d, vr[0]);
        const uint2 (&v)[2] = vr[EARLY ? d : 0];
        v4i vf;
        if constexpr (I8) vf = codes8_bf16(v[0]);
        else vf = v4i{(int)v[0].x, (int)v[0].y, (int)v[1].x, (int)v[1].y};
#pragma unroll
        for (int i = 0; i < PARTS; ++i)
#pragma unroll
            for (int b = 0; b < MB; ++b) {
                f32x4v& sum = acc[b][i / Kind::each < NA ? i / Kind::each : NA - 1][d];
                sum = mfma16<VT>(vf, part[b][i], sum);
            }
    }
    if constexpr (FOLD) __builtin_amdgcn_s_setprio(0);
    v_read();
}

// DT: type of q and out, and of a 16-bit cache; I8: int8 cache.
template <int DT, bool I8, int D>
__global__ __launch_bounds__(64 * (AttnShape<D * (I8 ? 1 : 2)>::waves)) void paged_attention_kernel(AttnArgs a)
{
    constexpr int RB = D * (I8 ? 1 : 2);
    using Sh = AttnShape<RB>;
    constexpr int NW = Sh::waves, NL = Sh::loads, KK = D / 32, DB = D / 16;
    constexpr int WP = I8 || DT != CK_DT_FP16 ? 3 : 4;       // 16-bit parts of a weight
    constexpr int NA = AttnKind<DT, I8, WP>::NA;
    __shared__ __attribute__((aligned(1024))) uint8_t ring[NW * 2 * Sh::tile];
    __shared__ __attribute__((aligned(16))) uint32_t offs[kAttnChunk];
    __shared__ __attribute__((aligned(16))) float kscale[I8 ? kAttnChunk : 4], vscale[I8 ? kAttnChunk : 4];
    __shared__ float wave_m[NW][16], wave_l[NW][16], wave_v[NW];
    __shared__ int bad_page;

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int G = lane >> 4, i16 = lane & 15;
    // chunk fastest: a sequence's blocks run side by side (4 x 131072 bf16 tokens
    // 394 us, 48 ragged int8 sequences 53 us; chunk slowest 400 and 57 us)
    const int split = blockIdx.x % a.splits;
    const int64_t rest = blockIdx.x / a.splits;
    const int rb = (int)(rest % a.row_blocks);
    const int64_t bk = rest / a.row_blocks;
    const int kvh = (int)(bk % a.hk);
    const int64_t b = bk / a.hk;
    const int heads = min(16, a.group - 16 * rb);            // query heads of this block
    const int h0 = kvh * a.group + 16 * rb;
    const Visible vis = visible(a, a.lens[b]);
    const int64_t first = (int64_t)split * a.chunk;
    const int n = (int)min<int64_t>(a.chunk, vis.count - first);
    if (n <= 0) {
        if (split == 0)                                      // nothing is visible at all
            for (int e = tid; e < heads * D; e += 64 * NW) a.out[b * a.o_bs + (h0 + e / D) * a.o_hs + e % D] = 0;
        return;
    }
    const int tiles = (n + kAttnTile - 1) / kAttnTile;

    // Queries: lane 16 G + i holds elements 32 kk + 8 G + 0 .. 7 of head i.
    v4i qf[1][KK];
    const uint16_t* qp = a.q + b * a.q_bs + (h0 + min(i16, heads - 1)) * a.q_hs + 8 * G;
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) qf[0][kk] = *reinterpret_cast<const v4i*>(qp + 32 * kk);

    // Row offsets of the chunk's tokens, in 16-byte units; the last token's
    // again up to the end of the last tile, so that masked places hold
    // values of a visible row.  A thread's loads go out together, the pages
    // of all its tokens and then the scales.
    if (tid == 0) bad_page = 0;
    constexpr int PT = kAttnChunk / (64 * NW);               // tokens per thread
    int32_t pages[PT], ats[PT];
#pragma unroll
    for (int j = 0; j < PT; ++j) {
        const int i = tid + j * 64 * NW;
        if (i < tiles * kAttnTile) {
            const int64_t tok = vis.token(first + min(i, n - 1));
            pages[j] = a.table[b * a.table_stride + (tok >> a.page_shift)];
            ats[j] = (int32_t)(tok & ((1 << a.page_shift) - 1));
        }
    }
    __syncthreads();
    float vmax = 0.0f;
    if (a.pages > 0) {
        float ks[PT], vs[PT];
#pragma unroll
        for (int j = 0; j < PT; ++j) {
            const int i = tid + j * 64 * NW;
            if (i < tiles * kAttnTile) {
                int64_t page = pages[j];
                if (page < 0 || page >= a.pages) {
                    bad_page = 1;
                    page = 0;
                }
                offs[i] = (uint32_t)((page * a.c_ps + kvh * a.c_hs + ats[j] * a.c_ts) * (I8 ? 1 : 2) / 16);
                if constexpr (I8) {
                    const int64_t so = page * a.s_ps + kvh * a.s_hs + ats[j] * a.s_ts;
                    ks[j] = a.cks[so];
                    vs[j] = a.cvs[so];
                }
            }
        }
        if constexpr (I8) {
#pragma unroll
            for (int j = 0; j < PT; ++j) {
                const int i = tid + j * 64 * NW;
                if (i < tiles * kAttnTile) {
                    kscale[i] = ks[j] * a.scale * 1.44269504f;
                    vscale[i] = vs[j];
                    vmax = fmaxf(vmax, __builtin_fabsf(vs[j]));
                }
            }
        }
    }
    if constexpr (I8) {
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) vmax = fmaxf(vmax, __shfl_xor(vmax, off));
        if (lane == 0) wave_v[wave] = vmax;
    }
    float qscale = 1.0f;
    if constexpr (!I8) {
        // Take q now: a wait for it inside the main loop would also wait for
        // the direct-to-LDS loads, which the compiler does not count.
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) asm volatile("" : "+v"(qf[0][kk]));
    } else {
        // to fp16, the largest element in [2^13, 2^14)
        float f[KK][8], m = 0.0f;
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
            widen8<DT>(qf[0][kk], f[kk]);
#pragma unroll
            for (int e = 0; e < 8; ++e) m = fmaxf(m, __builtin_fabsf(f[kk][e]));
        }
        m = fmaxf(m, __shfl_xor(m, 16));
        m = fmaxf(m, __shfl_xor(m, 32));
        const int e = m > 0.0f ? 14 - __builtin_amdgcn_frexp_expf(m) : 0;
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
#pragma unroll
            for (int w = 0; w < 4; ++w)
                qf[0][kk][w] = (int)f16x2_rne_bits(__builtin_amdgcn_ldexpf(f[kk][2 * w], e), __builtin_amdgcn_ldexpf(f[kk][2 * w + 1], e));
        qscale = __builtin_amdgcn_ldexpf(1.0f, -e);
    }
    __syncthreads();
    if (bad_page || a.pages == 0) {                          // an error of this sequence
        if (a.splits == 1 || vis.count <= a.chunk) {
            for (int e = tid; e < heads * D; e += 64 * NW)
                a.out[b * a.o_bs + (h0 + e / D) * a.o_hs + e % D] = (uint16_t)(kNan2<DT> & 0xffffu);
        } else if (tid < heads) {
            a.part_ml[(b * a.hq + h0 + tid) * a.splits + split] = make_float2(0.0f, NAN);
        }
        return;
    }
    // Value scales are taken relative to 2^ve, which the largest of the chunk is
    // just below: exact, and right for subnormal scales too, whose reciprocal
    // would be infinite.
    int ve = 0;
    if constexpr (I8) {
        vmax = wave_v[0];
#pragma unroll
        for (int w = 1; w < NW; ++w) vmax = fmaxf(vmax, wave_v[w]);
        ve = vmax > 0.0f ? __builtin_amdgcn_frexp_expf(vmax) : 0;
    }

    uint8_t* const kring = ring + wave * (2 * Sh::tile);
    uint8_t* const vring = kring + Sh::tile;
    const uint32_t klds = lds_addr(kring), vlds = klds + Sh::tile;
    // Load j copies pieces 64 j .. 64 j + 63 of a tile, one per lane.
    uint32_t off[NL];
    auto read_offs = [&](int t) {
#pragma unroll
        for (int j = 0; j < NL; ++j) off[j] = offs[t * kAttnTile + (64 * j + lane) / Sh::chunks];
    };
    auto issue_k = [&]() {
#pragma unroll
        for (int j = 0; j < NL; ++j) {
            const int row = (64 * j + lane) / Sh::chunks, pc = (64 * j + lane) % Sh::chunks;
            dma16_at(a.ck + (uint64_t)(off[j] + (uint32_t)(pc ^ Sh::swz(row))) * 16, klds + j * 1024);
        }
    };
    auto issue_v = [&]() {
#pragma unroll
        for (int j = 0; j < NL; ++j) {
            const int row = (64 * j + lane) / Sh::chunks, pc = (64 * j + lane) % Sh::chunks;
            dma16_at(a.cv + (uint64_t)(off[j] + (uint32_t)(pc ^ (I8 ? Sh::swz(row) : Sh::swz2(row)))) * 16, vlds + j * 1024);
        }
    };

    f32x4v acc[1][NA][DB];
#pragma unroll
    for (int i = 0; i < NA; ++i)
#pragma unroll
        for (int d = 0; d < DB; ++d) acc[0][i][d] = f32x4v{0.0f, 0.0f, 0.0f, 0.0f};
    float Ms[1] = {kAttnLow}, Ls[1] = {0.0f};
    const float sc[1] = {I8 ? qscale : a.scale * 1.44269504f};

    if (wave < tiles) {
        read_offs(wave);
        issue_k();
        issue_v();
    }
    const AttnLane<I8, D> at(kring, vring, lane);
    for (int t = wave; t < tiles; t += NW) {
        const bool more = t + NW < tiles;
        wait_vmcnt<NL>();                                    // K of this tile; V came after it
        attn_tile<DT, I8, D, 1, WP, false>(
            at, 0, qf, sc, &kscale[I8 ? t * kAttnTile : 0], &vscale[I8 ? t * kAttnTile : 0], ve,
            n - t * kAttnTile, t == wave, Ms, Ls, acc,
            [&] {
                asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory"); // K is read: its place is free
                if (more) {
                    read_offs(t + NW);
                    issue_k();
                }
            },
            [&] {
                if (more) wait_vmcnt<NL>();                  // V of this tile; the next K came after it
                else wait_vmcnt<0>();
            },
            [&] {
                asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory"); // V is read
                if (more) issue_v();
            });
    }
    const float M = Ms[0];
    float L = Ls[0];

    // The waves' sums meet in LDS: each in its own ring, [head][d], 16-byte
    // pieces exchanged by xor.
    L += __shfl_xor(L, 16);
    L += __shfl_xor(L, 32);
    float* const own = reinterpret_cast<float*>(kring);
#pragma unroll
    for (int d = 0; d < DB; ++d) {
        f32x4v sum = acc[0][0][d];
        if constexpr (NA == 2) sum = sum + acc[0][1][d] * (1.0f / AttnKind<DT, I8, WP>::fine);
        *reinterpret_cast<f32x4v*>(own + i16 * D + (((4 * d + G) ^ (i16 & 7)) << 2)) = sum;
    }
    if (lane < 16) {
        wave_m[wave][lane] = M;
        wave_l[wave][lane] = L;
    }
    __syncthreads();
    const bool last = vis.count <= a.chunk;                  // the only chunk: write the output
    for (int e = tid; e < heads * (D / 4); e += 64 * NW) {
        const int h = e / (D / 4), c = e % (D / 4);
        float m = wave_m[0][h];
#pragma unroll
        for (int w = 1; w < NW; ++w) m = fmaxf(m, wave_m[w][h]);
        float l = 0.0f;
        f32x4v o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float f = __builtin_amdgcn_exp2f(wave_m[w][h] - m);   // a wave without tiles: 0
            l = __builtin_fmaf(f, wave_l[w][h], l);
            const f32x4v v = *reinterpret_cast<const f32x4v*>(reinterpret_cast<const float*>(ring + w * (2 * Sh::tile)) + h * D + ((c ^ (h & 7)) << 2));
#pragma unroll
            for (int r = 0; r < 4; ++r) o[r] = __builtin_fmaf(f, v[r], o[r]);
        }
        if constexpr (I8) {
#pragma unroll
            for (int r = 0; r < 4; ++r) o[r] = __builtin_amdgcn_ldexpf(o[r], ve);
        }
        if (last) {
            const float inv = 1.0f / l;
            uint2 w;
            w.x = narrow2<DT>(o[0] * inv, o[1] * inv);
            w.y = narrow2<DT>(o[2] * inv, o[3] * inv);
            *reinterpret_cast<uint2*>(a.out + b * a.o_bs + (h0 + h) * a.o_hs + 4 * c) = w;
        } else {
            const int64_t at = (b * a.hq + h0 + h) * a.splits + split;
            *reinterpret_cast<f32x4v*>(a.part + at * D + 4 * c) = o;
            if (c == 0) a.part_ml[at] = make_float2(m, l);
        }
    }
}

// Joins the chunks of one sequence and head: a lane has four elements of the
// values, P groups of lanes each add every P-th chunk (four at a time, under
// a running M as above), and their sums are added in LDS, all in an order that
// the sizes fix.  Bound by latency: the first loads go out before the length
// is known, within the workspace whatever it is.
template <int DT, int D>
__global__ __launch_bounds__(256) void attention_join_kernel(AttnArgs a)
{
    constexpr int C = D / 4;                                 // lanes that hold the values, four each
    constexpr int P = 256 / C;                               // chunks added side by side
    constexpr int U = 4;
    __shared__ f32x4v sums[P][C];
    __shared__ float ms[P], ls[P];
    const int tid = threadIdx.x, c = tid % C, g = tid / C;
    const int64_t bh = blockIdx.x;
    const int h = (int)(bh % a.hq);
    const int64_t b = bh / a.hq;
    const float2* const ml = a.part_ml + bh * a.splits;
    const float* const part = a.part + bh * a.splits * D + 4 * c;
    float2 x[U];
    f32x4v v[U];
    auto load = [&](int s0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int s = s0 + P * u;
            if (g < P && s < a.splits) {
                x[u] = ml[s];
                v[u] = *reinterpret_cast<const f32x4v*>(part + (int64_t)s * D);
            }
        }
    };
    load(g);
    const Visible vis = visible(a, a.lens[b]);
    if (vis.count <= a.chunk) return;                        // written by its only block
    const int splits = (int)((vis.count + a.chunk - 1) / a.chunk);
    float m = kAttnLow, l = 0.0f;
    f32x4v o = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int s0 = g; g < P && s0 < splits; s0 += P * U) {
        if (s0 != g) load(s0);
        float top = m;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (s0 + P * u < splits) top = fmaxf(top, x[u].x);
        const float old = __builtin_amdgcn_exp2f(m - top);
        m = top;
        l *= old;
        o = o * old;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s0 + P * u < splits) {
                const float f = __builtin_amdgcn_exp2f(x[u].x - m);
                l = __builtin_fmaf(f, x[u].y, l);
#pragma unroll
                for (int r = 0; r < 4; ++r) o[r] = __builtin_fmaf(f, v[u][r], o[r]);
            }
        }
    }
    if (g < P) {
        sums[g][c] = o;
        if (c == 0) {
            ms[g] = m;
            ls[g] = l;
        }
    }
    __syncthreads();
    if (tid < C) {
        m = ms[0];
#pragma unroll
        for (int p = 1; p < P; ++p) m = fmaxf(m, ms[p]);
        o = f32x4v{0.0f, 0.0f, 0.0f, 0.0f};
        l = 0.0f;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const float f = __builtin_amdgcn_exp2f(ms[p] - m);   // a group without chunks: 0
            l = __builtin_fmaf(f, ls[p], l);
            const f32x4v q = sums[p][tid];
#pragma unroll
            for (int r = 0; r < 4; ++r) o[r] = __builtin_fmaf(f, q[r], o[r]);
        }
        const float inv = 1.0f / l;
        uint2 w;
        w.x = narrow2<DT>(o[0] * inv, o[1] * inv);
        w.y = narrow2<DT>(o[2] * inv, o[3] * inv);
        *reinterpret_cast<uint2*>(a.out + b * a.o_bs + h * a.o_hs + 4 * tid) = w;
    }
}

namespace {

bool attention_dim_ok(int64_t d) { return d == 64 || d == 96 || d == 128 || d == 192 || d == 256; }

// The most tokens that can be visible to any sequence.
int64_t most_visible(int64_t table_width, int64_t page_size, int64_t window, int64_t sinks)
{
    const int64_t cap = table_width * page_size;
    if (window <= 0 || window >= cap) return cap;
    return window + std::min(sinks, cap - window);
}

int attn_waves(int64_t row_bytes)
{
    const int64_t fit = 65536 / (2 * kAttnTile * row_bytes);
    return fit >= 8 ? 8 : fit >= 4 ? 4 : 2;
}

// Tokens per block: as many as give every CU two blocks, if all sequences
// were as long as they can be, but a tile per wave at least and kAttnChunk
// at most: short sequences are spread over the chip, and long ones in parts
// small enough to even out sequences of different lengths.  A part's sums,
// (d + 2) * 4 bytes a head, are written and read: for a group of 8 heads of 128
// 1.6 % of the traffic of its rows with 1024 bf16 tokens, 3.1 % with int8 ones,
// and more in smaller chunks (1 x 1000 bf16 tokens in groups of 4, 128 a
// block: 6.3 %; one sequence of 4096 with 16 / 2 heads of 256, 64 a block: 25 %),
// which are taken where the chip would stand idle otherwise.  Measured, 4
// sequences of 131072 bf16 tokens / 48 of up to 9001 int8 ones: 512 a block 420
// us / 54 us, 768 - / 67, 1024 394 / 54, 2048 380 / 61.
//
// The rule goes by what a row of the table can name, not by the lengths, which
// the host does not know: a table wider than its sequences costs empty blocks
// and smaller shares (one of 1000 tokens in a table for 131072 17 us, 64 of
// them 579 us in place of 48).
int64_t attn_chunk(int64_t batch, int64_t hq, int64_t hk, int64_t row_bytes, int64_t most)
{
    const int64_t pairs = batch * hk * cdiv(hq / hk, 16);
    const int64_t tiles = std::min<int64_t>(cdiv(most, kAttnTile), 1 << 20);   // past the cap below, far from 64 bits
    const int64_t waves = attn_waves(row_bytes);
    const int64_t want = cdiv(cdiv(tiles * pairs, 2 * kNumCUs), waves) * waves;
    return std::min<int64_t>(std::max(want, waves) * kAttnTile, kAttnChunk);
}

bool attention_sizes_ok(int64_t batch, int64_t hq, int64_t hk, int64_t table_width, int64_t page_size)
{
    return batch <= (1 << 20) && hq <= 65536 && hk <= 65536 && table_width <= (int64_t(1) << 31) - 1 &&
           table_width * page_size <= (int64_t(1) << 40);
}

struct AttnPlan {
    int64_t chunk, splits, blocks, bytes;                    // tokens a block, blocks a row block, the grid, the workspace
};

// False for more blocks, or rows of the output, than a launch takes.
bool attn_plan(AttnPlan& p, int64_t batch, int64_t hq, int64_t hk, int64_t head_dim, int64_t row_bytes, int64_t most)
{
    const int64_t limit = 0x7fffffff, pairs = batch * hk * cdiv(hq / hk, 16);
    p.chunk = attn_chunk(batch, hq, hk, row_bytes, most);
    p.splits = std::max<int64_t>(1, cdiv(most, p.chunk));
    if (batch * hq > limit || pairs > limit / p.splits) return false;
    p.blocks = pairs * p.splits;
    if (!grid_ok(p.blocks, 64 * attn_waves(row_bytes)) || (p.splits > 1 && !grid_ok(batch * hq, 256))) return false;
    p.bytes = p.splits > 1 ? batch * hq * p.splits * (head_dim + 2) * 4 : 0;
    return true;
}

template <int DT, bool I8>
const void* attention_fn(int64_t d)
{
    switch (d) {
    case 64: return reinterpret_cast<const void*>(&paged_attention_kernel<DT, I8, 64>);
    case 96: return reinterpret_cast<const void*>(&paged_attention_kernel<DT, I8, 96>);
    case 128: return reinterpret_cast<const void*>(&paged_attention_kernel<DT, I8, 128>);
    case 192: return reinterpret_cast<const void*>(&paged_attention_kernel<DT, I8, 192>);
    default: return reinterpret_cast<const void*>(&paged_attention_kernel<DT, I8, 256>);
    }
}

template <int DT>
const void* attention_join_fn(int64_t d)
{
    switch (d) {
    case 64: return reinterpret_cast<const void*>(&attention_join_kernel<DT, 64>);
    case 96: return reinterpret_cast<const void*>(&attention_join_kernel<DT, 96>);
    case 128: return reinterpret_cast<const void*>(&attention_join_kernel<DT, 128>);
    case 192: return reinterpret_cast<const void*>(&attention_join_kernel<DT, 192>);
    default: return reinterpret_cast<const void*>(&attention_join_kernel<DT, 256>);
    }
}

}  // namespace

// The layout does not tell the element type of the cache, so the size is the
// larger of the two chunk rules', of those that a launch takes.
extern "C" int64_t ck_paged_attention_workspace(int64_t batch, int64_t hq, int64_t hk, int64_t head_dim,
                                                int64_t table_width, int64_t page_size, int64_t window,
                                                int64_t sinks)
{
    if (batch < 0 || hq < 0 || hk < 1 || hq % hk != 0 || !attention_dim_ok(head_dim) || table_width < 0 ||
        !is_pow2(page_size) || page_size > 32768 || window < 0 || sinks < 0 ||
        !attention_sizes_ok(batch, hq, hk, table_width, page_size))
        return -1;
    const int64_t most = most_visible(table_width, page_size, window, sinks);
    int64_t bytes = -1;
    for (int esz = 1; esz <= 2; ++esz) {
        AttnPlan plan;
        if (attn_plan(plan, batch, hq, hk, head_dim, esz * head_dim, most)) bytes = std::max(bytes, plan.bytes);
    }
    return bytes;
}

extern "C" ck_status ck_paged_attention(const ck_attention_args* args, const ck_kv_cache* cache,
                                        hipStream_t stream)
{
    if (!args || !cache) return fail(CK_ERR_INVALID_ARG, "NULL args or cache");
    const ck_attention_args& p = *args;
    if (p.dtype != CK_DT_BF16 && p.dtype != CK_DT_FP16) return fail(CK_ERR_INVALID_ARG, "bad dtype");
    if (p.batch < 0 || p.hq < 0 || p.table_width < 0 || p.window < 0 || p.sinks < 0)
        return fail(CK_ERR_INVALID_ARG, "negative size");
    if (!attention_dim_ok(cache->head_dim)) return fail(CK_ERR_UNSUPPORTED, "head_dim must be 64, 96, 128, 192 or 256");
    ck_status s = check_cache(cache, p.dtype, cache->head_dim, 16);
    if (s != CK_OK) return s;
    if (p.hq % cache->heads != 0) return fail(CK_ERR_INVALID_ARG, "query heads are not a multiple of the cache's");
    if (p.batch == 0 || p.hq == 0) return ok();
    if (!attention_sizes_ok(p.batch, p.hq, cache->heads, p.table_width, cache->page_size))
        return fail(CK_ERR_UNSUPPORTED, "too large a batch, table or number of heads");
    if (!p.q || !p.out || !p.lens || (!p.table && p.table_width > 0))
        return fail(CK_ERR_INVALID_ARG, "NULL q, out, table or lens");
    if (!rows16(p.q, p.batch, p.q_batch_stride, p.hq, p.q_head_stride) ||
        !rows16(p.out, p.batch, p.out_batch_stride, p.hq, p.out_head_stride))
        return fail(CK_ERR_UNSUPPORTED, "q and out rows must start 16 bytes apart");
    if (!aligned(p.table, 4) || !aligned(p.lens, 4)) return fail(CK_ERR_UNSUPPORTED, "misaligned table or lens");
    if (p.table_stride < p.table_width && p.batch > 1) return fail(CK_ERR_INVALID_ARG, "table_stride smaller than table_width");
    if (!(p.scale == p.scale)) return fail(CK_ERR_INVALID_ARG, "scale is NaN");
    const bool i8 = cache->dtype == CK_DT_INT8, f16 = p.dtype == CK_DT_FP16;
    const int64_t d = cache->head_dim, row_bytes = d * (i8 ? 1 : 2);
    // row offsets are 32 bits of 16-byte units
    if (cache_reach(cache, cache->page_stride, cache->head_stride, cache->token_stride, d) * (row_bytes / d) > 0x1p36)
        return fail(CK_ERR_UNSUPPORTED, "the cache spans more than 64 GiB");
    AttnArgs a{};
    const int64_t most = most_visible(p.table_width, cache->page_size, p.window, p.sinks);
    AttnPlan plan;
    if (!attn_plan(plan, p.batch, p.hq, cache->heads, d, row_bytes, most)) return fail(CK_ERR_UNSUPPORTED, "too many blocks");
    if (plan.bytes > 0 && (!p.workspace || p.workspace_bytes < plan.bytes))
        return fail(CK_ERR_INVALID_ARG, "the workspace needs %lld bytes", (long long)plan.bytes);
    if (!rows_apart(d, {p.batch, p.out_batch_stride}, {p.hq, p.out_head_stride}))
        return fail(CK_ERR_INVALID_ARG, "rows of out overlap");
    if (!aligned(p.workspace, 256)) return fail(CK_ERR_UNSUPPORTED, "misaligned workspace");
    a.hq = (int)p.hq; a.hk = (int)cache->heads; a.group = (int)(p.hq / cache->heads);
    a.row_blocks = (int)cdiv(a.group, 16);
    a.chunk = (int)plan.chunk;
    a.splits = (int)plan.splits;
    if ((s = check_device()) != CK_OK) return s;
    a.q = (const uint16_t*)p.q; a.out = (uint16_t*)p.out; a.table = p.table; a.lens = p.lens;
    a.part = (float*)p.workspace;
    a.part_ml = (float2*)(a.part + p.batch * p.hq * plan.splits * d);
    a.ck = (const uint8_t*)cache->k; a.cv = (const uint8_t*)cache->v; a.cks = cache->k_scale; a.cvs = cache->v_scale;
    a.q_bs = p.q_batch_stride; a.q_hs = p.q_head_stride; a.o_bs = p.out_batch_stride; a.o_hs = p.out_head_stride;
    a.table_stride = p.table_stride;
    a.c_ps = cache->page_stride; a.c_hs = cache->head_stride; a.c_ts = cache->token_stride;
    a.s_ps = cache->scale_page_stride; a.s_hs = cache->scale_head_stride; a.s_ts = cache->scale_token_stride;
    a.pages = cache->pages; a.capacity = p.table_width * cache->page_size;
    a.window = p.window; a.sinks = p.sinks; a.scale = p.scale;
    a.page_shift = ilog2(cache->page_size);
    const void* fn = f16 ? (i8 ? attention_fn<CK_DT_FP16, true>(d) : attention_fn<CK_DT_FP16, false>(d))
                         : (i8 ? attention_fn<CK_DT_BF16, true>(d) : attention_fn<CK_DT_BF16, false>(d));
    void* kargs[] = {&a};
    if ((s = launch(fn, (unsigned)plan.blocks, 64u * attn_waves(row_bytes), kargs, stream, "paged_attention")) != CK_OK) return s;
    if (plan.splits > 1) {
        const void* join = f16 ? attention_join_fn<CK_DT_FP16>(d) : attention_join_fn<CK_DT_BF16>(d);
        if ((s = launch(join, (unsigned)(p.batch * p.hq), 256, kargs, stream, "paged_attention_join")) != CK_OK) return s;
    }
    return ok();
}
