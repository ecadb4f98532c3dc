// lora_add.hip -- y + s (x A^T) B^T with a low-rank adapter for every row.
//
// Mathematics.  For a row i with adapter t: v = x[i] A_t^T (rank sums over k),
// then out[i] = y[i] + (s_t v) B_t^T.  Both products run on the matrix cores
// (16 x 16 x 32) with fp32 sums.  v stays 32 bits: it enters the second product
// in 16-bit parts, three of bf16 (2^-24 of it), or two of fp16 after a power of
// two that brings the row's largest to [2^13, 2^14) (2^-22 of it, or 2^-39 of the
// largest).
//
// Bound: HBM, by the adapters that a decode batch asks for or by y of a
// prompt, and the launches of small calls.  Rows are taken 64 at a time, those
// with the same adapter together whatever their order, so an adapter is read
// once for its rows; a row without one is copied.
//   - Up to kLoraRows rows, a block has one adapter of one group of 64 rows and a
//     slice of the columns.  Where A is small every block makes v by itself, in
//     the same launch: A comes from L2 then, once for each slice.
//   - Otherwise a first launch makes v, with k split over blocks where there
//     are few of them (their parts are added in order by the second).
//   - More rows are those of prompts: a block goes through the adapters of its
//     rows in turn, mostly one, and holds a piece of B for 64 rows.

struct LoraArgs {
    const uint16_t* x;
    const uint16_t* a;
    const uint16_t* b;
    const float* scale;
    const int32_t* ids;
    const void* y;
    void* out;
    float* v;                            // [ksplits][m][vstride], of the first launch
    int64_t ldx, ldy, ldo, a_stride, b_stride, m;
    int n, k, rank, adapters, out_dtype;
    int vstride, ksplits, slices;
    int copy, wide;                      // rows without an adapter are copied; 16-byte accesses of y and out
};

constexpr int kLoraRows = 512;           // rows up to which every adapter of 64 rows has its own blocks
constexpr int kLoraWaves = 8;

// The next adapter among up to 64 rows, each lane with its row's id, and the
// rows that have it; `left`: those still to come.
__device__ __forceinline__ uint64_t lora_members(uint64_t& left, int ids, int& id)
{
    id = __builtin_amdgcn_readlane(ids, __builtin_ctzll(left));
    const uint64_t members = __ballot(ids == id) & left;
    left &= ~members;
    return members;
}

// The members in order: lane p gets the p-th one's row.
__device__ __forceinline__ int lora_places(uint64_t members)
{
    const int lane = threadIdx.x & 63, before = __popcll(members & ((1ull << lane) - 1));
    return __builtin_amdgcn_ds_permute((members >> lane & 1 ? before : __popcll(members) + lane - before) * 4, lane);
}

// v^T of 16 rows over the columns k0 .. k1 - 1 of this wave: lane 16 G + i gets
// ranks 16 f + 4 G + r of the row that its xp points at.
template <int DT, int RF>
__device__ __forceinline__ void lora_shrink(const LoraArgs& a, const uint16_t* xp, const uint16_t* ap, int k0, int k1,
                                            f32x4v (&acc)[RF])
{
    constexpr int U = RF == 1 ? 8 : RF == 2 ? 6 : RF == 4 ? 4 : RF == 8 ? 2 : 1;     // steps whose loads go out together
    const int lane = threadIdx.x & 63, G = lane >> 4, i16 = lane & 15;
    const uint16_t* rows[RF];
#pragma unroll
    for (int f = 0; f < RF; ++f) {
        acc[f] = f32x4v{0.0f, 0.0f, 0.0f, 0.0f};
        rows[f] = ap + (int64_t)min(16 * f + i16, a.rank - 1) * a.k;
    }
    for (int k = k0; k < k1; k += 32 * U) {
        v4i x[U], w[U][RF];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = k + 32 * u + 8 * G;
            const bool in = at < k1;
            x[u] = in ? *reinterpret_cast<const v4i*>(xp + at) : v4i{0, 0, 0, 0};
#pragma unroll
            for (int f = 0; f < RF; ++f) w[u][f] = in ? *reinterpret_cast<const v4i*>(rows[f] + at) : v4i{0, 0, 0, 0};
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int f = 0; f < RF; ++f) acc[f] = mfma16<DT>(w[u][f], x[u], acc[f]);
    }
}

// The first launch: v of a group of rows, over one part of k.
template <int DT, int RF>
__global__ __launch_bounds__(64 * kLoraWaves) void lora_shrink_kernel(LoraArgs a, int group, int each)
{
    __shared__ f32x4v red[kLoraWaves][RF][64];
    const int tid = threadIdx.x, lane = tid & 63, i16 = lane & 15, G = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int split = blockIdx.x % a.ksplits;
    const int64_t unit = blockIdx.x / a.ksplits;
    // `each`: a block for every row, which works if it is the first of its
    // adapter among its group; otherwise one for every group.
    const int64_t r0 = each ? unit / group * group : unit * group;
    const int count = (int)min<int64_t>(group, a.m - r0);
    const int ids = lane < count ? a.ids[r0 + lane] : -1;
    uint64_t left = __ballot(ids >= 0 && ids < a.adapters);
    if (each) {
        const int u = (int)(unit - r0);
        if (!(left >> u & 1)) return;
        left &= __ballot(ids == __builtin_amdgcn_readlane(ids, u));
        if (__builtin_ctzll(left) != u) return;
    }
    const int steps = (a.k + 31) / 32;
    const int part = split * kLoraWaves + wave, parts = a.ksplits * kLoraWaves;
    const int k0 = (int)((int64_t)steps * part / parts) * 32, k1 = min(a.k, (int)((int64_t)steps * (part + 1) / parts) * 32);
    while (left) {
        int id;
        const uint64_t members = lora_members(left, ids, id);
        const int rows = __popcll(members), places = lora_places(members);
        for (int t = 0; t < rows; t += 16) {
            const int64_t row = r0 + __shfl(places, min(t + i16, rows - 1));
            f32x4v acc[RF];
            lora_shrink<DT, RF>(a, a.x + row * a.ldx, a.a + id * a.a_stride, k0, k1, acc);
#pragma unroll
            for (int f = 0; f < RF; ++f) red[wave][f][lane] = acc[f];
            __syncthreads();
            for (int f = wave; f < RF; f += kLoraWaves) {
                f32x4v sum = red[0][f][lane];
#pragma unroll
                for (int w = 1; w < kLoraWaves; ++w) sum = sum + red[w][f][lane];
                if (t + i16 < rows) *reinterpret_cast<f32x4v*>(a.v + ((int64_t)split * a.m + row) * a.vstride + 16 * f + 4 * G) = sum;
            }
            __syncthreads();
        }
    }
}

// 16 columns of a row, from c on: out = y + d.
template <int OUT>
__device__ __forceinline__ void lora_store(const LoraArgs& a, int64_t row, int c, const float (&d)[16])
{
    constexpr int E = OUT == CK_OUT_FP32 ? 4 : 8;
    constexpr int T = OUT == CK_OUT_FP16 ? CK_DT_FP16 : CK_DT_BF16;
    if (a.wide && c + 16 <= a.n) {
        const v4i* const yp = reinterpret_cast<const v4i*>(static_cast<const char*>(a.y) + (row * a.ldy + c) * (16 / E));
        v4i* const op = reinterpret_cast<v4i*>(static_cast<char*>(a.out) + (row * a.ldo + c) * (16 / E));
        v4i y[16 / E];
#pragma unroll
        for (int j = 0; j < 16 / E; ++j) y[j] = yp[j];
#pragma unroll
        for (int j = 0; j < 16 / E; ++j) {
            v4i o;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (OUT == CK_OUT_FP32) {
                    o[i] = __float_as_int(__int_as_float(y[j][i]) + d[4 * j + i]);
                } else {
                    const float2 f = widen2<T>((uint32_t)y[j][i]);
                    o[i] = (int)narrow2<T>(f.x + d[8 * j + 2 * i], f.y + d[8 * j + 2 * i + 1]);
                }
            }
            op[j] = o;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        if (c + i >= a.n) break;
        const int64_t yi = row * a.ldy + c + i, oi = row * a.ldo + c + i;
        if constexpr (OUT == CK_OUT_FP32)
            static_cast<float*>(a.out)[oi] = static_cast<const float*>(a.y)[yi] + d[i];
        else
            static_cast<uint16_t*>(a.out)[oi] =
                (uint16_t)narrow2<T>(widen2<T>((uint32_t) static_cast<const uint16_t*>(a.y)[yi]).x + d[i], 0.0f);
    }
}

// The second product for MB blocks of 16 rows, or all of it (RF > 0: v is made
// here).  A wave has 64 columns at a time, as four tiles: tile t's operand row
// p is column 16 (p / 4) + 4 t + p % 4, so that lane 16 G + i ends up with 16
// columns in a row, 16 G and on, of row i.
template <int DT, int MB, int RF>
__global__ __launch_bounds__(64 * kLoraWaves) void lora_expand_kernel(LoraArgs a, int each)
{
    constexpr int PARTS = DT == CK_DT_FP16 ? 2 : 3;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int tid = threadIdx.x, lane = tid & 63, i16 = lane & 15, G = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int slice = blockIdx.x % a.slices;
    const int64_t unit = blockIdx.x / a.slices, r0 = each ? unit / 64 * 64 : unit * 64;
    const int count = (int)min<int64_t>(64, a.m - r0);
    const int chunks = (a.n + 63) / 64;
    const int c0 = (int)((int64_t)chunks * slice / a.slices), c1 = (int)((int64_t)chunks * (slice + 1) / a.slices);
    const int ids = lane < count ? a.ids[r0 + lane] : -1;
    const uint64_t having = __ballot(ids >= 0 && ids < a.adapters);
    uint64_t left = having, without = (count == 64 ? ~0ull : (1ull << count) - 1) & ~having;
    if (each) {
        const int u = (int)(unit - r0);
        without &= 1ull << u;
        left &= __ballot(ids == __builtin_amdgcn_readlane(ids, u));
        if (left && __builtin_ctzll(left) != u) left = 0;
    }
    if (a.copy) {                                            // rows without an adapter, as they are
        const int esz = a.out_dtype == CK_OUT_FP32 ? 4 : 2;
        for (; without; without &= without - 1) {
            const int64_t row = r0 + __builtin_ctzll(without);
            const char* const yp = static_cast<const char*>(a.y) + row * a.ldy * esz;
            char* const op = static_cast<char*>(a.out) + row * a.ldo * esz;
            const int end = min(a.n, c1 * 64);
            for (int c = c0 * 64 + tid; c < end; c += 64 * kLoraWaves) {
                if (esz == 4) reinterpret_cast<uint32_t*>(op)[c] = reinterpret_cast<const uint32_t*>(yp)[c];
                else reinterpret_cast<uint16_t*>(op)[c] = reinterpret_cast<const uint16_t*>(yp)[c];
            }
        }
    }
    const int steps = (a.rank + 31) / 32, vs = 32 * steps + 4;       // of the second product's sum; floats of a row of v
    v4i* const frags = reinterpret_cast<v4i*>(lds);                  // [MB][PARTS][steps][64]
    float* const v = reinterpret_cast<float*>(frags + MB * PARTS * steps * 64);   // [16 MB][vs]
    float* const back = v + 16 * MB * vs;                            // [16 MB] powers of two that v was divided by
    while (left) {
        int id;
        const uint64_t members = lora_members(left, ids, id);
        const int rows = __popcll(members), places = lora_places(members);
        const float scale = a.scale ? a.scale[id] : 1.0f;
        const uint16_t* const bp = a.b + id * a.b_stride;
        for (int t0 = 0; t0 < rows; t0 += 16 * MB) {
            const int here = min(16 * MB, rows - t0);
            int64_t row[MB];                                 // this lane's of each block; the last one again past the end
#pragma unroll
            for (int b = 0; b < MB; ++b) row[b] = r0 + __shfl(places, min(t0 + 16 * b + i16, rows - 1));
            // v, fp32, with the adapter's scale; ranks past the last are zero
            if constexpr (RF > 0) {
                f32x4v* const red = reinterpret_cast<f32x4v*>(back + 16 * MB);   // [waves][RF][64]
                const int part = wave, all = (a.k + 31) / 32;
                const int k0 = all * part / kLoraWaves * 32, k1 = min(a.k, all * (part + 1) / kLoraWaves * 32);
                f32x4v acc[RF];
                lora_shrink<DT, RF>(a, a.x + row[0] * a.ldx, a.a + id * a.a_stride, k0, k1, acc);
#pragma unroll
                for (int f = 0; f < RF; ++f) red[(wave * RF + f) * 64 + lane] = acc[f];
                for (int i = tid; i < 16 * vs; i += 64 * kLoraWaves) v[i] = 0.0f;
                __syncthreads();
                if (wave < RF) {
                    f32x4v sum = red[wave * 64 + lane];
#pragma unroll
                    for (int w = 1; w < kLoraWaves; ++w) sum = sum + red[(w * RF + wave) * 64 + lane];
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (i16 < here && 16 * wave + 4 * G + r < a.rank) v[i16 * vs + 16 * wave + 4 * G + r] = sum[r] * scale;
                }
            } else {
                for (int e = tid; e < 16 * MB * 32 * steps; e += 64 * kLoraWaves) {
                    const int i = e / (32 * steps), r = e % (32 * steps);
                    const int64_t at = r0 + __shfl(places, min(t0 + i, rows - 1));
                    float sum = 0.0f;
                    if (i < here && r < a.rank) {
                        sum = a.v[at * a.vstride + r];
                        for (int s = 1; s < a.ksplits; ++s) sum = sum + a.v[(s * a.m + at) * a.vstride + r];
                        sum *= scale;
                    }
                    v[i * vs + r] = sum;
                }
            }
            __syncthreads();
            // and its 16-bit parts, as the second product's second operand
            for (int i = wave; i < 16 * MB; i += kLoraWaves) {
                float top = 0.0f;
                if constexpr (DT == CK_DT_FP16) {
                    for (int r = lane; r < 32 * steps; r += 64) top = fmaxf(top, __builtin_fabsf(v[i * vs + r]));
#pragma unroll
                    for (int off = 32; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off));
                }
                const int e = top > 0.0f && top < INFINITY ? 14 - __builtin_amdgcn_frexp_expf(top) : 0;
                if (lane == 0) back[i] = __builtin_amdgcn_ldexpf(1.0f, -e);
                for (int r = 2 * lane; r < 32 * steps; r += 128) {
                    float x = __builtin_amdgcn_ldexpf(v[i * vs + r], e), z = __builtin_amdgcn_ldexpf(v[i * vs + r + 1], e);
                    uint32_t* const to = reinterpret_cast<uint32_t*>(frags + (i / 16 * PARTS * steps + r / 32) * 64 + r / 8 % 4 * 16 + i % 16) + r % 8 / 2;
#pragma unroll
                    for (int p = 0; p < PARTS; ++p) {
                        const uint32_t h = narrow2<DT>(x, z);
                        const float2 f = widen2<DT>(h);
                        to[p * steps * 256] = h;
                        x -= f.x;
                        z -= f.y;
                    }
                }
            }
            __syncthreads();
            for (int c = (c0 + wave) * 64; c < c1 * 64; c += 64 * kLoraWaves) {
                f32x4v acc[MB][4];
#pragma unroll
                for (int b = 0; b < MB; ++b)
#pragma unroll
                    for (int t = 0; t < 4; ++t) acc[b][t] = f32x4v{0.0f, 0.0f, 0.0f, 0.0f};
                for (int s = 0; s < steps; ++s) {
                    v4i w[4];
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        const int col = min(c + 16 * (i16 >> 2) + 4 * t + (i16 & 3), a.n - 1);
                        w[t] = 32 * s + 8 * G < a.rank ? *reinterpret_cast<const v4i*>(bp + (int64_t)col * a.rank + 32 * s + 8 * G)
                                                       : v4i{0, 0, 0, 0};
                    }
#pragma unroll
                    for (int b = 0; b < MB; ++b)
#pragma unroll
                        for (int p = 0; p < PARTS; ++p) {
                            const v4i f = frags[((b * PARTS + p) * steps + s) * 64 + lane];
#pragma unroll
                            for (int t = 0; t < 4; ++t) acc[b][t] = mfma16<DT>(w[t], f, acc[b][t]);
                        }
                }
#pragma unroll
                for (int b = 0; b < MB; ++b) {
                    if (16 * b + i16 >= here) continue;
                    const float up = DT == CK_DT_FP16 ? back[16 * b + i16] : 1.0f;
                    float d[16];
#pragma unroll
                    for (int t = 0; t < 4; ++t)
#pragma unroll
                        for (int r = 0; r < 4; ++r) d[4 * t + r] = acc[b][t][r] * up;
                    if (a.out_dtype == CK_OUT_FP32) lora_store<CK_OUT_FP32>(a, row[b], c + 16 * G, d);
                    else if (a.out_dtype == CK_OUT_FP16) lora_store<CK_OUT_FP16>(a, row[b], c + 16 * G, d);
                    else lora_store<CK_OUT_BF16>(a, row[b], c + 16 * G, d);
                }
            }
            __syncthreads();
        }
    }
}

namespace {

bool lora_sizes_ok(int64_t m, int64_t n, int64_t k, int64_t rank)
{
    return m >= 0 && n >= 0 && k >= 0 && m <= (1 << 24) && n <= (1 << 24) && k <= (1 << 24) && k % 8 == 0 && rank >= 8 &&
           rank <= 256 && rank % 8 == 0;
}

struct LoraPlan {
    bool each, fused;
    int mb;                                                  // row blocks of the second product
    int64_t group, ksplits, vstride, bytes;                  // of the first launch: rows of a block, parts of k
};

LoraPlan lora_plan(int64_t m, int64_t n, int64_t k, int64_t rank)
{
    LoraPlan p{};
    p.each = m <= kLoraRows;
    p.fused = p.each && rank <= 32 && rank * k <= 131072;
    p.mb = p.each || rank > 64 ? 1 : 4;                      // within 64 KiB of LDS
    p.vstride = rank <= 16 ? 16 : rank <= 32 ? 32 : rank <= 64 ? 64 : rank <= 128 ? 128 : 256;   // 16 RF of the first launch
    p.group = p.each ? 64 : 16;
    const int64_t units = p.each ? std::min<int64_t>(m, 16) : cdiv(m, p.group);
    p.ksplits = std::max<int64_t>(1, std::min<int64_t>(cdiv(kNumCUs, std::max<int64_t>(units, 1)), k / (64 * kLoraWaves)));
    if (!p.fused) p.bytes = p.ksplits * m * p.vstride * 4;
    return p;
}

template <int DT>
const void* lora_shrink_fn(int64_t rank)
{
    return rank <= 16   ? reinterpret_cast<const void*>(&lora_shrink_kernel<DT, 1>)
           : rank <= 32 ? reinterpret_cast<const void*>(&lora_shrink_kernel<DT, 2>)
           : rank <= 64 ? reinterpret_cast<const void*>(&lora_shrink_kernel<DT, 4>)
           : rank <= 128 ? reinterpret_cast<const void*>(&lora_shrink_kernel<DT, 8>)
                         : reinterpret_cast<const void*>(&lora_shrink_kernel<DT, 16>);
}

template <int DT>
const void* lora_expand_fn(const LoraPlan& p, int64_t rank)
{
    if (p.fused)
        return rank <= 16 ? reinterpret_cast<const void*>(&lora_expand_kernel<DT, 1, 1>)
                          : reinterpret_cast<const void*>(&lora_expand_kernel<DT, 1, 2>);
    return p.mb == 1 ? reinterpret_cast<const void*>(&lora_expand_kernel<DT, 1, 0>)
                  : reinterpret_cast<const void*>(&lora_expand_kernel<DT, 4, 0>);
}

}  // namespace

extern "C" int64_t ck_lora_add_workspace(int64_t m, int64_t n, int64_t k, int64_t rank)
{
    return lora_sizes_ok(m, n, k, rank) ? lora_plan(m, n, k, rank).bytes : -1;
}

extern "C" ck_status ck_lora_add(const ck_lora_args* args, hipStream_t stream)
{
    if (!args) return fail(CK_ERR_INVALID_ARG, "NULL args");
    const ck_lora_args& p = *args;
    if (p.dtype != CK_DT_BF16 && p.dtype != CK_DT_FP16) return fail(CK_ERR_INVALID_ARG, "bad dtype");
    if (p.out_dtype != CK_OUT_BF16 && p.out_dtype != CK_OUT_FP16 && p.out_dtype != CK_OUT_FP32)
        return fail(CK_ERR_INVALID_ARG, "bad out_dtype");
    if (p.m < 0 || p.n < 0 || p.k < 0 || p.rank < 0 || p.adapters < 0) return fail(CK_ERR_INVALID_ARG, "negative size");
    if (p.rank < 8 || p.rank > 256 || p.rank % 8 != 0) return fail(CK_ERR_UNSUPPORTED, "rank must be a multiple of 8 from 8 to 256");
    if (p.k % 8 != 0) return fail(CK_ERR_UNSUPPORTED, "k must be a multiple of 8");
    if (!lora_sizes_ok(p.m, p.n, p.k, p.rank) || p.adapters > (1 << 24)) return fail(CK_ERR_UNSUPPORTED, "m, n, k or adapters past 2^24");
    if (p.m == 0 || p.n == 0) return ok();
    if (!p.y || !p.out || !p.ids) return fail(CK_ERR_INVALID_ARG, "NULL y, out or ids");
    if (p.m > 1 && (p.ldy < p.n || p.ldo < p.n)) return fail(CK_ERR_INVALID_ARG, "ldy or ldo smaller than n");
    if (p.m > 1 && p.out == p.y && p.ldo != p.ldy) return fail(CK_ERR_INVALID_ARG, "out is y with another ld");
    if (p.adapters > 0) {
        if (!p.b || (p.k > 0 && (!p.x || !p.a))) return fail(CK_ERR_INVALID_ARG, "NULL x, a or b");
        if (p.k > 0 && p.m > 1 && p.ldx < p.k) return fail(CK_ERR_INVALID_ARG, "ldx smaller than k");
        if (p.adapters > 1 && (p.a_stride < p.rank * p.k || p.b_stride < p.rank * p.n))
            return fail(CK_ERR_INVALID_ARG, "a_stride or b_stride smaller than an adapter");
        if ((p.k > 0 && p.m > 1 && p.ldx % 8 != 0) || (p.adapters > 1 && (p.a_stride % 8 != 0 || p.b_stride % 8 != 0)) ||
            !aligned(p.x, 16) || !aligned(p.a, 16) || !aligned(p.b, 16))
            return fail(CK_ERR_UNSUPPORTED, "rows of x and adapters must start 16 bytes apart");
    }
    const int esz = p.out_dtype == CK_OUT_FP32 ? 4 : 2;
    if (!aligned(p.y, esz) || !aligned(p.out, esz) || !aligned(p.ids, 4) || !aligned(p.scale, 4))
        return fail(CK_ERR_UNSUPPORTED, "misaligned y, out, ids or scale");
    const LoraPlan plan = lora_plan(p.m, p.n, p.k, p.rank);
    if (plan.bytes > 0 && (!p.workspace || p.workspace_bytes < plan.bytes))
        return fail(CK_ERR_INVALID_ARG, "the workspace needs %lld bytes", (long long)plan.bytes);
    if (!aligned(p.workspace, 256)) return fail(CK_ERR_UNSUPPORTED, "misaligned workspace");
    ck_status s = check_device();
    if (s != CK_OK) return s;
    LoraArgs a{(const uint16_t*)p.x, (const uint16_t*)p.a, (const uint16_t*)p.b, p.scale, p.ids, p.y, p.out, (float*)p.workspace,
               p.ldx, p.ldy, p.ldo, p.a_stride, p.b_stride, p.m, (int)p.n, (int)p.k, (int)p.rank,
               (int)(p.k > 0 ? p.adapters : 0), p.out_dtype, (int)plan.vstride, (int)plan.ksplits, 1, p.out != p.y, 0};
    a.wide = aligned(p.y, 16) && aligned(p.out, 16) && p.ldy * esz % 16 == 0 && p.ldo * esz % 16 == 0;
    const bool f16 = p.dtype == CK_DT_FP16;
    int group = (int)plan.group, each = plan.each;
    if (!plan.fused && a.adapters > 0) {
        void* kargs[] = {&a, &group, &each};
        const int64_t blocks = (plan.each ? p.m : cdiv(p.m, plan.group)) * plan.ksplits;
        const void* fn = f16 ? lora_shrink_fn<CK_DT_FP16>(p.rank) : lora_shrink_fn<CK_DT_BF16>(p.rank);
        if ((s = launch(fn, (unsigned)blocks, 64 * kLoraWaves, kargs, stream, "lora_shrink")) != CK_OK) return s;
    }
    // Column slices: as many blocks as give every CU two, of 512 columns at least.
    const int64_t units = plan.each ? std::min(p.m, std::max<int64_t>(p.adapters, 1)) : cdiv(p.m, 64);
    a.slices = (int)std::max<int64_t>(1, std::min(cdiv(2 * kNumCUs, units), cdiv(p.n, 64 * kLoraWaves)));
    const int mb = plan.mb, parts = f16 ? 2 : 3;
    const int64_t steps = cdiv(p.rank, 32), rf = plan.fused ? cdiv(p.rank, 16) : 0;
    const size_t lds = mb * parts * steps * 1024 + 16 * mb * (32 * steps + 4) * 4 + 64 * mb + kLoraWaves * rf * 1024;
    const void* fn = f16 ? lora_expand_fn<CK_DT_FP16>(plan, p.rank) : lora_expand_fn<CK_DT_BF16>(plan, p.rank);
    void* kargs[] = {&a, &each};
    const int64_t blocks = (plan.each ? p.m : cdiv(p.m, 64)) * a.slices;
    hipError_t e = hipLaunchKernel(fn, dim3((unsigned)blocks), dim3(64 * kLoraWaves), kargs, lds, stream);
    if (e != hipSuccess) return fail(CK_ERR_HIP, "lora_add launch: %s", hipGetErrorString(e));
    return ok();
}
