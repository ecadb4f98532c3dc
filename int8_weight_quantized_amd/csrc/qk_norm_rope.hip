// qk_norm_rope.hip -- norm and rotation of query and key heads, and the
// write of keys and values into a paged cache, in one pass.
//
// Mathematics, per token and head (x: head_dim values widened to fp32):
//   y = x * (1 / sqrt(mean(x^2) + eps)) * w, then each pair (a, b) of the
//   first `rot` elements turned by the position's angle,
//   (a c - b s, b c + a s); one rounding, to 16 bits or to an int8 code.
// Squares, sums, the rotation and the int8 row's amax are fp32.
//
// Bound: HBM (each value is read and written once: 2 + 2 bytes, or 2 + 1):
// 8192 tokens of 32 / 8 / 8 heads of 128, 201 MB, 48.2 us or 4.2 TB/s.  Into an
// int8 cache they take 65 us (2.9 TB/s): normed heads, queries too, pay for the
// ordered sum and the 64-bit root and division below, and with rotated halves
// for a second load of the row.  515 tokens of 24 / 8 / 8 heads of 96 take 5.2
// us, into an int8 cache 7.0; a decode call of one token is a launch, 3.2 us.
// One group of L lanes (a power of two, 8 values a lane) holds a head, so the
// norm is a reduction over the group and nothing passes through LDS.  With halves rotated, a lane has four
// elements of the first half and their four partners of the second, so the
// rotation stays inside the lane.  A group takes several heads of one token,
// HB at a time: the angles and weights are read once for all of them, and HB
// loads are on their way together.

struct QkArgs {
    const uint16_t* q;
    const uint16_t* k;
    const uint16_t* v;
    const int64_t* positions;
    const float* cos_sin;
    const float* qw;
    const float* kw;
    uint16_t* qo;
    uint16_t* ko;
    const int64_t* slots;
    int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, qo_ts, qo_hs, ko_ts, ko_hs;
    int64_t units;                       // tokens * slices
    int64_t table_rows;
    int64_t cells;                       // slots of the cache
    uint8_t* ck;
    uint8_t* cv;
    float* cks;
    float* cvs;
    int64_t c_ps, c_hs, c_ts, s_ps, s_hs, s_ts;
    int hq, hk, heads;                   // heads: of a token, values included when there is a cache
    int slices;                          // groups that share a token's heads
    int d, rot, page_shift;
    float eps, inv_d;
};

template <int L>
__device__ __forceinline__ float group_sum(float v)
{
#pragma unroll
    for (int off = L / 2; off > 0; off >>= 1) v += __shfl_xor(v, off);
    return v;
}

// The sum of a row's d terms, eight a lane, in one particular order.  Below
// 128 terms: those 64 apart, then neighbours, pairs of neighbours and so on.
// From 128 on: those 128 (256 from d = 256 on) apart, then each four in
// sequence, then neighbouring fours and so on.  Any order is as right; this is
// the one in which the torch this was compared with (2.10) sums such rows on
// this device.  With the root rounded from 64 bits, as torch's is, the key
// codes of an int8 cache, which jump where a value lies between two of them,
// are then those of the same formula in torch operations (tested at widths of
// 64, 96, 128, 192 and 256; another torch may sum in another order).
template <int L>
__device__ __forceinline__ float group_sum_ordered(const float (&x)[8], int d)
{
    const bool fours = L >= 16 && d >= 128;
    const int fold = L == 16 ? (fours ? 0 : 8) : L == 32 ? (d >= 256 ? 0 : 16) : L == 64 ? 32 : 0;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = fold ? x[i] + __shfl_xor(x[i], fold) : x[i];
    float sum = fours ? (((v[0] + v[1]) + v[2]) + v[3]) + (((v[4] + v[5]) + v[6]) + v[7])
                      : ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
#pragma unroll
    for (int off = 1; off < L; off *= 2)
        if (fold == 0 || off < fold) sum = sum + __shfl_xor(sum, off);
    return sum;
}

template <int L>
__device__ __forceinline__ float group_max(float v)
{
#pragma unroll
    for (int off = L / 2; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor(v, off));
    return v;
}

template <int DT>
__device__ __forceinline__ void widen8(const v4i w, float (&f)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 p = widen2<DT>((uint32_t)w[i]);
        f[2 * i] = p.x;
        f[2 * i + 1] = p.y;
    }
}

__device__ __forceinline__ void load8(const float* p, float (&f)[8])
{
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

// Four 16-bit values from each of two places.
template <int DT>
__device__ __forceinline__ void widen44(uint2 a, uint2 b, float (&f)[8])
{
    widen8<DT>(v4i{(int)a.x, (int)a.y, (int)b.x, (int)b.y}, f);
}

// DT: the activations' type; L: lanes per head; I8: int8 cache; PAIRS:
// neighbouring elements are rotated together, else halves.
template <int DT, int L, bool I8, bool PAIRS, int HB>
__global__ __launch_bounds__(256) void qk_norm_rope_kernel(QkArgs a)
{
    const int64_t unit = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L;
    if (unit >= a.units) return;         // whole groups: the shuffles stay inside one
    const int64_t t = unit / a.slices;
    const int first = (int)(unit - t * a.slices);        // heads first, first + slices, ...
    const int lane = threadIdx.x % L;
    const bool in = lane * 8 < a.d, turn = lane * 8 < a.rot;
    const int half = a.rot >> 1;
    // this lane's elements of a head: four from e0, four from e1
    const int e0 = !PAIRS && turn ? lane * 4 : lane * 8;
    const int e1 = !PAIRS && turn ? half + lane * 4 : lane * 8 + 4;

    bool lost = false;                   // the position is outside the table
    float4 c = {1.0f, 1.0f, 1.0f, 1.0f}, s = {0.0f, 0.0f, 0.0f, 0.0f};
    if (a.rot > 0) {
        const int64_t pos = a.positions[t];
        lost = pos < 0 || pos >= a.table_rows;
        if (turn) {
            const float* const row = a.cos_sin + (lost ? 0 : pos) * a.rot + lane * 4;
            c = *reinterpret_cast<const float4*>(row);
            s = *reinterpret_cast<const float4*>(row + half);
        }
    }
    // the row of the cache, if the token has one
    bool kept = false;
    int64_t cell = 0, scell = 0;
    if (a.ck) {
        const int64_t slot = a.slots[t];
        kept = slot >= 0 && slot < a.cells && !lost;     // a value goes with its key: both or neither
        const int64_t page = slot >> a.page_shift, at = slot & ((1 << a.page_shift) - 1);
        cell = page * a.c_ps + at * a.c_ts;
        scell = page * a.s_ps + at * a.s_ts;
    }
    // weights at e0 and e1
    float4 wq0 = {1.0f, 1.0f, 1.0f, 1.0f}, wq1 = wq0, wk0 = wq0, wk1 = wq0;
    if (in && a.qw) {
        wq0 = *reinterpret_cast<const float4*>(a.qw + e0);
        wq1 = *reinterpret_cast<const float4*>(a.qw + e1);
    }
    if (in && a.kw) {
        wk0 = *reinterpret_cast<const float4*>(a.kw + e0);
        wk1 = *reinterpret_cast<const float4*>(a.kw + e1);
    }

    for (int h0 = first; h0 < a.heads; h0 += HB * a.slices) {
        uint2 x0[HB], x1[HB];
        v4i flat[HB];                    // the same head's eight elements from 8 * lane on, for the ordered sum
#pragma unroll
        for (int i = 0; i < HB; ++i) {
            const int h = h0 + i * a.slices;
            x0[i] = x1[i] = make_uint2(0u, 0u);
            flat[i] = v4i{0, 0, 0, 0};
            if (h < a.heads && in) {
                const uint16_t* const src = h < a.hq          ? a.q + t * a.q_ts + h * a.q_hs
                                            : h < a.hq + a.hk ? a.k + t * a.k_ts + (h - a.hq) * a.k_hs
                                                              : a.v + t * a.v_ts + (h - a.hq - a.hk) * a.v_hs;
                x0[i] = *reinterpret_cast<const uint2*>(src + e0);
                x1[i] = *reinterpret_cast<const uint2*>(src + e1);
                if (I8 && !PAIRS) flat[i] = *reinterpret_cast<const v4i*>(src + lane * 8);
            }
        }
        auto one = [&](int h, const uint2& p0, const uint2& p1, const v4i& natural) {
            const bool is_q = h < a.hq, is_v = h >= a.hq + a.hk;
            const int hh = is_q ? h : is_v ? h - a.hq - a.hk : h - a.hq;
            float y[8];
            widen44<DT>(p0, p1, y);
            if (!is_v) {
                if (is_q ? a.qw != nullptr : a.kw != nullptr) {
                    float r;
                    if constexpr (I8) {
                        float sq[8];
                        if constexpr (PAIRS) widen44<DT>(p0, p1, sq);
                        else widen8<DT>(natural, sq);
#pragma unroll
                        for (int e = 0; e < 8; ++e) sq[e] = sq[e] * sq[e];
                        const float mean = group_sum_ordered<L>(sq, a.d) * a.inv_d + a.eps;
                        r = (float)(1.0 / __builtin_sqrt((double)mean));
                    } else {
                        float sum = 0.0f;
#pragma unroll
                        for (int e = 0; e < 8; ++e) sum = __builtin_fmaf(y[e], y[e], sum);
                        r = rsqrtf(group_sum<L>(sum) * a.inv_d + a.eps);
                    }
                    float4 w0, w1;
                    w0.x = is_q ? wq0.x : wk0.x; w0.y = is_q ? wq0.y : wk0.y; w0.z = is_q ? wq0.z : wk0.z; w0.w = is_q ? wq0.w : wk0.w;
                    w1.x = is_q ? wq1.x : wk1.x; w1.y = is_q ? wq1.y : wk1.y; w1.z = is_q ? wq1.z : wk1.z; w1.w = is_q ? wq1.w : wk1.w;
                    y[0] = y[0] * r * w0.x; y[1] = y[1] * r * w0.y; y[2] = y[2] * r * w0.z; y[3] = y[3] * r * w0.w;
                    y[4] = y[4] * r * w1.x; y[5] = y[5] * r * w1.y; y[6] = y[6] * r * w1.z; y[7] = y[7] * r * w1.w;
                }
                if (turn) {
                    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        const int u = PAIRS ? 2 * p : p, v = PAIRS ? 2 * p + 1 : p + 4;
                        const float yu = y[u], yv = y[v];
                        y[u] = yu * cc[p] - yv * ss[p];
                        y[v] = yv * cc[p] + yu * ss[p];
                    }
                }
            }
            uint2 o0, o1;
            if (lost && !is_v) {
                o0 = o1 = make_uint2(kNan2<DT>, kNan2<DT>);
            } else {
                o0 = make_uint2(narrow2<DT>(y[0], y[1]), narrow2<DT>(y[2], y[3]));
                o1 = make_uint2(narrow2<DT>(y[4], y[5]), narrow2<DT>(y[6], y[7]));
            }
            if (!is_v && in) {
                uint16_t* const dst = is_q ? a.qo + t * a.qo_ts + hh * a.qo_hs : a.ko ? a.ko + t * a.ko_ts + hh * a.ko_hs : nullptr;
                if (dst) {
                    *reinterpret_cast<uint2*>(dst + e0) = o0;
                    *reinterpret_cast<uint2*>(dst + e1) = o1;
                }
            }
            if (is_q || !kept) return;
            const int64_t row = cell + hh * a.c_hs;
            uint8_t* const cache = is_v ? a.cv : a.ck;
            if constexpr (I8) {
                float m = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) m = fmaxf(m, __builtin_fabsf(y[e]));
                const float scale = group_max<L>(in ? m : 0.0f) * (1.0f / 127.0f);
                // codes8_pk's argument holds for |y / scale| up to 127 (1 + 2^-22)
                const float inv = 1.0f / scale;
                uint2 code = make_uint2(0u, 0u);
                if (!(__builtin_fabsf(inv) >= 0x1p-126f && inv <= 0x1.fffffep127f && codes8_pk(y, inv, code))) {
                    code = make_uint2(0u, 0u);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint32_t byte = (uint32_t)(quant_code(y[e], scale) & 0xff) << (8 * (e & 3));
                        if (e < 4) code.x |= byte;
                        else code.y |= byte;
                    }
                }
                if (in) {
                    *reinterpret_cast<uint32_t*>(cache + row + e0) = code.x;
                    *reinterpret_cast<uint32_t*>(cache + row + e1) = code.y;
                }
                if (lane == 0) (is_v ? a.cvs : a.cks)[scell + hh * a.s_hs] = scale;
            } else if (in) {
                *reinterpret_cast<uint2*>(cache + 2 * (row + e0)) = o0;
                *reinterpret_cast<uint2*>(cache + 2 * (row + e1)) = o1;
            }
        };
#pragma unroll
        for (int i = 0; i < HB; ++i)
            if (h0 + i * a.slices < a.heads) one(h0 + i * a.slices, x0[i], x1[i], flat[i]);
    }
}

namespace {

template <int DT, bool I8, bool PAIRS, int HB>
const void* qk_fn_lanes(int lanes)
{
    switch (lanes) {
    case 8: return reinterpret_cast<const void*>(&qk_norm_rope_kernel<DT, 8, I8, PAIRS, HB>);
    case 16: return reinterpret_cast<const void*>(&qk_norm_rope_kernel<DT, 16, I8, PAIRS, HB>);
    case 32: return reinterpret_cast<const void*>(&qk_norm_rope_kernel<DT, 32, I8, PAIRS, HB>);
    default: return reinterpret_cast<const void*>(&qk_norm_rope_kernel<DT, 64, I8, PAIRS, HB>);
    }
}

template <int DT, int HB>
const void* qk_fn(int lanes, bool i8, bool pairs)
{
    if (i8) return pairs ? qk_fn_lanes<DT, true, true, HB>(lanes) : qk_fn_lanes<DT, true, false, HB>(lanes);
    return pairs ? qk_fn_lanes<DT, false, true, HB>(lanes) : qk_fn_lanes<DT, false, false, HB>(lanes);
}

}  // namespace

extern "C" ck_status ck_qk_norm_rope(const ck_qk_args* args, const ck_kv_cache* cache, hipStream_t stream)
{
    if (!args) return fail(CK_ERR_INVALID_ARG, "NULL args");
    const ck_qk_args& p = *args;
    if (p.dtype != CK_DT_BF16 && p.dtype != CK_DT_FP16) return fail(CK_ERR_INVALID_ARG, "bad dtype");
    if (p.tokens < 0 || p.hq < 0 || p.hk < 0 || p.rot < 0 || p.table_rows < 0)
        return fail(CK_ERR_INVALID_ARG, "negative size");
    if (p.head_dim < 8 || p.head_dim > 512 || p.head_dim % 8 != 0)
        return fail(CK_ERR_UNSUPPORTED, "head_dim must be a multiple of 8 from 8 to 512");
    if (p.rot > p.head_dim) return fail(CK_ERR_INVALID_ARG, "rot larger than head_dim");
    if (p.rot % 16 != 0) return fail(CK_ERR_UNSUPPORTED, "rot must be a multiple of 16");
    if (p.hq > 65536 || p.hk > 65536) return fail(CK_ERR_UNSUPPORTED, "too many heads");
    if (!(p.eps >= 0.0f)) return fail(CK_ERR_INVALID_ARG, "eps must not be negative");
    ck_status s;
    if (cache) {
        if (p.hk != cache->heads) return fail(CK_ERR_INVALID_ARG, "keys and cache disagree on the heads");
        if ((s = check_cache(cache, p.dtype, p.head_dim, cache->dtype == CK_DT_INT8 ? 8 : 16)) != CK_OK) return s;
    }
    const int64_t heads = p.hq + p.hk + (cache ? p.hk : 0);
    if (p.tokens == 0 || heads == 0) return ok();
    if (p.hq > 0 && (!p.q || !p.q_out)) return fail(CK_ERR_INVALID_ARG, "NULL q or q_out");
    if (p.hk > 0 && (!p.k || (!p.k_out && !cache))) return fail(CK_ERR_INVALID_ARG, "NULL k, or no place for the keys");
    if (cache && (!p.v || !p.slots)) return fail(CK_ERR_INVALID_ARG, "a cache needs v and slots");
    if (p.rot > 0 && (!p.positions || (!p.cos_sin && p.table_rows > 0)))
        return fail(CK_ERR_INVALID_ARG, "NULL positions or cos_sin");
    if (p.rot > 0 && p.table_rows == 0) return fail(CK_ERR_INVALID_ARG, "empty cos_sin");
    if ((p.hq > 0 && (!rows16(p.q, p.tokens, p.q_token_stride, p.hq, p.q_head_stride) ||
                      !rows16(p.q_out, p.tokens, p.q_out_token_stride, p.hq, p.q_out_head_stride))) ||
        (p.hk > 0 && (!rows16(p.k, p.tokens, p.k_token_stride, p.hk, p.k_head_stride) ||
                      (p.k_out && !rows16(p.k_out, p.tokens, p.k_out_token_stride, p.hk, p.k_out_head_stride)))) ||
        (cache && !rows16(p.v, p.tokens, p.v_token_stride, p.hk, p.v_head_stride)))
        return fail(CK_ERR_UNSUPPORTED, "q, k, v and out rows must start 16 bytes apart");
    if ((p.hq > 0 && !rows_apart(p.head_dim, {p.tokens, p.q_out_token_stride}, {p.hq, p.q_out_head_stride})) ||
        (p.hk > 0 && p.k_out && !rows_apart(p.head_dim, {p.tokens, p.k_out_token_stride}, {p.hk, p.k_out_head_stride})))
        return fail(CK_ERR_INVALID_ARG, "rows of q_out or k_out overlap");
    if (cache && !rows_apart(p.head_dim, {cache->pages, cache->page_stride}, {cache->heads, cache->head_stride},
                             {cache->page_size, cache->token_stride}))
        return fail(CK_ERR_INVALID_ARG, "rows of the cache overlap");
    if (!aligned(p.cos_sin, 16) || !aligned(p.q_weight, 16) || !aligned(p.k_weight, 16) ||
        !aligned(p.positions, 8) || !aligned(p.slots, 8))
        return fail(CK_ERR_UNSUPPORTED, "misaligned positions, slots, cos_sin or weight");
    int lanes = 8;
    while (lanes * 8 < p.head_dim) lanes *= 2;
    if (p.tokens > (int64_t(1) << 40)) return fail(CK_ERR_UNSUPPORTED, "too many tokens");
    // A group per head while that leaves the chip short of waves (32 a CU),
    // else up to eight heads a group, two at a time (8192 tokens of 32 + 8 + 8
    // heads of 128: 50 us, 4.1 TB/s, against 60 us with a group per head; four
    // at a time 52 us, six or twelve heads a group 53 and 52 us, loads and
    // stores past the caches 48 us here and 20 % slower at other sizes).
    const int64_t slices = std::min(heads, std::max(cdiv(heads, 8), cdiv(32 * kNumCUs * 64, lanes * p.tokens)));
    const bool many = slices < heads;
    const int64_t blocks = cdiv(p.tokens * slices, 256 / lanes);
    if (!grid_ok(blocks, 256)) return fail(CK_ERR_UNSUPPORTED, "too many heads in all");
    if ((s = check_device()) != CK_OK) return s;

    QkArgs a{};
    a.q = (const uint16_t*)p.q; a.k = (const uint16_t*)p.k; a.v = (const uint16_t*)p.v;
    a.positions = p.positions; a.cos_sin = p.cos_sin; a.qw = p.q_weight; a.kw = p.k_weight;
    a.qo = (uint16_t*)p.q_out; a.ko = (uint16_t*)p.k_out; a.slots = p.slots;
    a.q_ts = p.q_token_stride; a.q_hs = p.q_head_stride; a.k_ts = p.k_token_stride; a.k_hs = p.k_head_stride;
    a.v_ts = p.v_token_stride; a.v_hs = p.v_head_stride;
    a.qo_ts = p.q_out_token_stride; a.qo_hs = p.q_out_head_stride;
    a.ko_ts = p.k_out_token_stride; a.ko_hs = p.k_out_head_stride;
    a.units = p.tokens * slices; a.slices = (int)slices; a.table_rows = p.table_rows;
    a.hq = (int)p.hq; a.hk = (int)p.hk; a.heads = (int)heads;
    a.d = (int)p.head_dim; a.rot = (int)p.rot; a.eps = p.eps; a.inv_d = 1.0f / (float)p.head_dim;
    if (cache && cache->pages > 0) {
        a.ck = (uint8_t*)cache->k; a.cv = (uint8_t*)cache->v; a.cks = cache->k_scale; a.cvs = cache->v_scale;
        a.c_ps = cache->page_stride; a.c_hs = cache->head_stride; a.c_ts = cache->token_stride;
        a.s_ps = cache->scale_page_stride; a.s_hs = cache->scale_head_stride; a.s_ts = cache->scale_token_stride;
        a.cells = cache->pages * cache->page_size;
        a.page_shift = ilog2(cache->page_size);
    }
    const bool i8 = cache && cache->dtype == CK_DT_INT8, pairs = p.interleaved != 0;
    const bool f16 = p.dtype == CK_DT_FP16;
    const void* fn = many ? (f16 ? qk_fn<CK_DT_FP16, 2>(lanes, i8, pairs) : qk_fn<CK_DT_BF16, 2>(lanes, i8, pairs))
                          : (f16 ? qk_fn<CK_DT_FP16, 1>(lanes, i8, pairs) : qk_fn<CK_DT_BF16, 1>(lanes, i8, pairs));
    void* kargs[] = {&a};
    s = launch(fn, (unsigned)blocks, 256, kargs, stream, "qk_norm_rope");
    return s == CK_OK ? ok() : s;
}
