// qk_norm_rope.hip -- norm and rotation of query and key heads, and the
// write of keys and values into a paged cache, in one pass.
//
// Mathematics, per token and head (x: head_dim values widened to fp32):
//   y = x * (1 / sqrt(mean(x^2) + eps)) * w, then each pair (a, b) of the
//   first `rot` elements turned by the position's angle,
//   (a c - b s, b c + a s); one rounding, to 16 bits or to an int8 code.
// Squares, sums, the rotation and the int8 row's amax are fp32.
//
// Bound: HBM (each value is read and written once: 2 + 2 bytes, or 2 + 1);
// a decode call is bound by the launch.  One group of L lanes (a power of
// two, 8 values a lane) holds a head, so the norm is a reduction over the
// group and nothing passes through LDS.  With halves rotated, a lane's
// partner values are another lane's own: it loads them a second time (the
// line is in L1) instead of exchanging eight values, and the norm's factor,
// the same for the whole head, is applied to both.

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
    int64_t items;                       // tokens * heads of a token
    int64_t table_rows;
    int64_t cells;                       // slots of the cache
    uint8_t* ck;
    uint8_t* cv;
    float* cks;
    float* cvs;
    int64_t c_ps, c_hs, c_ts, s_ps, s_hs, s_ts;
    int hq, hk, heads;                   // heads: of a token, values included when there is a cache
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
// sequence, then neighbouring fours and so on.  It is the order in which
// torch sums such rows on this device; with the root rounded from 64 bits, as
// torch's is, the key codes of an int8 cache, which jump where a value lies
// between two of them, are those of the same formula in torch operations.
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

// DT: the activations' type; L: lanes per head; I8: int8 cache; PAIRS:
// neighbouring elements are rotated together, else halves.
template <int DT, int L, bool I8, bool PAIRS>
__global__ __launch_bounds__(256) void qk_norm_rope_kernel(QkArgs a)
{
    const int64_t item = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L;
    if (item >= a.items) return;         // whole groups: the shuffles stay inside one
    const int64_t t = item / a.heads;
    const int h = (int)(item - t * a.heads);
    const bool is_q = h < a.hq, is_v = h >= a.hq + a.hk;
    const int hh = is_q ? h : is_v ? h - a.hq - a.hk : h - a.hq;
    const int e0 = (threadIdx.x % L) * 8;               // this lane's elements of the head
    const bool in = e0 < a.d;
    const uint16_t* src = is_q   ? a.q + t * a.q_ts + hh * a.q_hs
                          : is_v ? a.v + t * a.v_ts + hh * a.v_hs
                                 : a.k + t * a.k_ts + hh * a.k_hs;
    const v4i zero = {0, 0, 0, 0};
    const v4i raw = in ? *reinterpret_cast<const v4i*>(src + e0) : zero;
    float y[8];
    widen8<DT>(raw, y);

    const float* w = is_v ? nullptr : is_q ? a.qw : a.kw;
    const bool turn = !is_v && e0 < a.rot;
    int64_t pos = 0;
    bool lost = false;                   // the position is outside the table
    if (a.rot > 0) {
        pos = a.positions[t];
        lost = pos < 0 || pos >= a.table_rows;
    }
    float other[8], c[8], s[8];
    const int half = a.rot >> 1;
    const bool second = e0 >= half;
    int partner = e0;
    if (turn) {
        const float* row = a.cos_sin + (lost ? 0 : pos) * a.rot;
        if constexpr (PAIRS) {
            const float4 cc = *reinterpret_cast<const float4*>(row + (e0 >> 1));
            const float4 ss = *reinterpret_cast<const float4*>(row + half + (e0 >> 1));
            c[0] = cc.x; c[2] = cc.y; c[4] = cc.z; c[6] = cc.w;
            s[0] = ss.x; s[2] = ss.y; s[4] = ss.z; s[6] = ss.w;
        } else {
            partner = second ? e0 - half : e0 + half;
            widen8<DT>(*reinterpret_cast<const v4i*>(src + partner), other);
            const int p = second ? partner : e0;
            load8(row + p, c);
            load8(row + half + p, s);
        }
    }
    if (w) {
        float sum = 0.0f;
        if constexpr (I8) {
            float sq[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) sq[i] = y[i] * y[i];
            sum = group_sum_ordered<L>(sq, a.d);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = __builtin_fmaf(y[i], y[i], sum);
            sum = group_sum<L>(sum);
        }
        const float mean = sum * a.inv_d + a.eps;
        const float r = I8 ? (float)(1.0 / __builtin_sqrt((double)mean)) : rsqrtf(mean);
        float f[8];
        if (in) {
            load8(w + e0, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = y[i] * r * f[i];
        }
        if (!PAIRS && turn) {
            load8(w + partner, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) other[i] = other[i] * r * f[i];
        }
    }
    if (turn) {
        if constexpr (PAIRS) {
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const float u = y[i], v = y[i + 1];
                y[i] = u * c[i] - v * s[i];
                y[i + 1] = v * c[i] + u * s[i];
            }
        } else {
            // first half: y c - other s; second half: y c + other s
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = y[i] * c[i] + (second ? other[i] * s[i] : -(other[i] * s[i]));
        }
    }

    v4i out;
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = lost && !is_v ? (int)kNan2<DT> : (int)narrow2<DT>(y[2 * i], y[2 * i + 1]);
    if (!is_v && in) {
        uint16_t* dst = is_q ? a.qo + t * a.qo_ts + hh * a.qo_hs : a.ko ? a.ko + t * a.ko_ts + hh * a.ko_hs : nullptr;
        if (dst) *reinterpret_cast<v4i*>(dst + e0) = out;
    }
    if (is_q || !a.ck || lost) return;   // a value goes with its key: both or neither
    const int64_t slot = a.slots[t];
    if (slot < 0 || slot >= a.cells) return;
    const int64_t page = slot >> a.page_shift, at = slot & ((1 << a.page_shift) - 1);
    const int64_t row = page * a.c_ps + hh * a.c_hs + at * a.c_ts;
    uint8_t* cache = is_v ? a.cv : a.ck;
    if constexpr (I8) {
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, __builtin_fabsf(y[i]));
        const float scale = group_max<L>(in ? m : 0.0f) * (1.0f / 127.0f);
        uint32_t word[2] = {0u, 0u};
#pragma unroll
        for (int i = 0; i < 8; ++i) word[i >> 2] |= (uint32_t)(quant_code(y[i], scale) & 0xff) << (8 * (i & 3));
        if (in) *reinterpret_cast<uint2*>(cache + row + e0) = make_uint2(word[0], word[1]);
        if (threadIdx.x % L == 0) (is_v ? a.cvs : a.cks)[page * a.s_ps + hh * a.s_hs + at * a.s_ts] = scale;
    } else {
        if (in) *reinterpret_cast<v4i*>(cache + 2 * (row + e0)) = out;
    }
}

namespace {

template <int DT, bool I8, bool PAIRS>
const void* qk_fn_lanes(int lanes)
{
    switch (lanes) {
    case 8: return reinterpret_cast<const void*>(&qk_norm_rope_kernel<DT, 8, I8, PAIRS>);
    case 16: return reinterpret_cast<const void*>(&qk_norm_rope_kernel<DT, 16, I8, PAIRS>);
    case 32: return reinterpret_cast<const void*>(&qk_norm_rope_kernel<DT, 32, I8, PAIRS>);
    default: return reinterpret_cast<const void*>(&qk_norm_rope_kernel<DT, 64, I8, PAIRS>);
    }
}

template <int DT>
const void* qk_fn(int lanes, bool i8, bool pairs)
{
    if (i8) return pairs ? qk_fn_lanes<DT, true, true>(lanes) : qk_fn_lanes<DT, true, false>(lanes);
    return pairs ? qk_fn_lanes<DT, false, true>(lanes) : qk_fn_lanes<DT, false, false>(lanes);
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
    if (!aligned(p.cos_sin, 16) || !aligned(p.q_weight, 16) || !aligned(p.k_weight, 16) ||
        !aligned(p.positions, 8) || !aligned(p.slots, 8))
        return fail(CK_ERR_UNSUPPORTED, "misaligned positions, slots, cos_sin or weight");
    int lanes = 8;
    while (lanes * 8 < p.head_dim) lanes *= 2;
    if (p.tokens > (int64_t(1) << 40)) return fail(CK_ERR_UNSUPPORTED, "too many tokens");
    const int64_t blocks = cdiv(p.tokens * heads, 256 / lanes);
    if (blocks > 0x7fffffffLL) return fail(CK_ERR_UNSUPPORTED, "too many heads in all");
    if ((s = check_device()) != CK_OK) return s;

    QkArgs a{};
    a.q = (const uint16_t*)p.q; a.k = (const uint16_t*)p.k; a.v = (const uint16_t*)p.v;
    a.positions = p.positions; a.cos_sin = p.cos_sin; a.qw = p.q_weight; a.kw = p.k_weight;
    a.qo = (uint16_t*)p.q_out; a.ko = (uint16_t*)p.k_out; a.slots = p.slots;
    a.q_ts = p.q_token_stride; a.q_hs = p.q_head_stride; a.k_ts = p.k_token_stride; a.k_hs = p.k_head_stride;
    a.v_ts = p.v_token_stride; a.v_hs = p.v_head_stride;
    a.qo_ts = p.q_out_token_stride; a.qo_hs = p.q_out_head_stride;
    a.ko_ts = p.k_out_token_stride; a.ko_hs = p.k_out_head_stride;
    a.items = p.tokens * heads; a.table_rows = p.table_rows;
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
    const void* fn = p.dtype == CK_DT_FP16 ? qk_fn<CK_DT_FP16>(lanes, i8, pairs) : qk_fn<CK_DT_BF16>(lanes, i8, pairs);
    void* kargs[] = {&a};
    s = launch(fn, (unsigned)blocks, 256, kargs, stream, "qk_norm_rope");
    return s == CK_OK ? ok() : s;
}
