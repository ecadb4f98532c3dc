// int4_linear.hip -- x W^T with 4-bit weights and a scale (and zero point)
// per group of weights along K, for 16-bit x, and the layout of the weights.

struct Int4PackArgs {
    const uint8_t* codes;
    const uint16_t* scales;
    const uint8_t* zeros;
    uint32_t* w;
    uint16_t* ws;
    uint8_t* wz;
    int64_t ldc, lds, ldz, n, k, chunks, groups;
};

// One thread per packed word: columns k0 .. k0 + 7 of a row, the even ones in
// the lower half, so that column pairs (2 i, 2 i + 1) sit 16 bits apart.
__global__ __launch_bounds__(256) void int4_pack_kernel(Int4PackArgs a)
{
    const int64_t word = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t tiles = (a.n + 15) / 16;
    if (word < tiles * a.chunks * 256) {
        const int i = word & 3, lane = (int)(word >> 2) & 63;
        const int64_t block = word >> 8, tile = block / a.chunks, chunk = block - tile * a.chunks;
        const int64_t row = tile * 16 + (lane & 15), k0 = chunk * 128 + 32 * i + 8 * (lane >> 4);
        uint32_t v = 0;
        if (row < a.n && k0 < a.k) {         // k % 8 == 0: all eight columns or none
            const uint8_t* p = a.codes + row * a.ldc + k0 / 2;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t byte = p[j];
                v |= (byte & 15u) << (4 * j) | (byte >> 4) << (16 + 4 * j);
            }
        }
        a.w[word] = v;
    }
    if (word < tiles * a.groups * 16) {
        const int64_t tile = word / (a.groups * 16), g = word / 16 % a.groups, row = tile * 16 + (word & 15);
        a.ws[word] = row < a.n ? a.scales[row * a.lds + g] : 0;
        if (a.wz) a.wz[word] = row < a.n ? a.zeros[row * a.ldz + g] : 0;
    }
}

struct Int4Args {
    const uint16_t* x;
    const uint8_t* w;
    const uint16_t* ws;
    const uint8_t* wz;
    const void* bias;
    void* out;
    int64_t ldx, ldo, m, n, k, chunks, groups;
    int out_dtype;
};

// One output: the bias, then one rounding to out's type.
__device__ __forceinline__ void store_int4(const Int4Args& a, int64_t row, int64_t col, float v)
{
    if (a.out_dtype == CK_OUT_FP32) {
        if (a.bias) v = v + bias_at<EPI_F32>(a.bias, col);
        static_cast<float*>(a.out)[row * a.ldo + col] = v;
        return;
    }
    uint16_t* const out = static_cast<uint16_t*>(a.out) + row * a.ldo + col;
    if (a.out_dtype == CK_OUT_FP16) {
        if (a.bias) v = v + bias_at<EPI_F16>(a.bias, col);
        *out = (uint16_t)(pack2<EPI_F16>(v, 0.0f) & 0xffffu);
    } else {
        if (a.bias) v = v + bias_at<EPI_BF16>(a.bias, col);
        *out = (uint16_t)(pack2<EPI_BF16>(v, 0.0f) & 0xffffu);
    }
}

// Few rows of x (up to 32).  Mathematics: for each group g of columns,
//   out[i, j] += s[j, g] (sum_t x[i, t] (16 + c[j, t]) - (16 + z[j, g]) X[i, g]),
//   X[i, g] = sum_t x[i, t],
// because 16 + c is one bit operation away from a code: the code's four bits
// are the upper mantissa bits of 16 in bf16 and in fp16 alike.  The products
// are exact in fp32, X comes from the same matrix cores (a product with
// ones), and the group's sum keeps about 3 bits less than one of c - z would,
// far below the output's rounding.
//
// Bound: HBM; the weights are read once, 1 KiB at a time, in the order that
// ck_int4_pack laid them out in.  Each wave streams its part of K for NT row
// tiles of W through a ring of its own in LDS, filled by direct-to-LDS loads
// (W, scales and zeros, and x), so that no barrier and no register waits for
// them; the waves' sums meet in LDS at the end, in a fixed order.
//
// Products (16 x 16 x 32): x rows are the first operand and W rows the second,
// so lane 16 G + i holds column i.  Row j of a 16-row block of x sits at
// operand row 4 (j % 4) + j / 4, which puts it into register j / 4 of lanes
// G = j % 4: with up to 4 (8) rows only one (two) of the four accumulator
// registers are in use, and only those get the scales (MR).
template <int DT>
__device__ __forceinline__ v4i codes16(uint32_t w)
{
    constexpr uint32_t mask = DT == CK_DT_FP16 ? 0x03c003c0u : 0x00780078u;
    constexpr uint32_t base = DT == CK_DT_FP16 ? 0x4c004c00u : 0x41804180u;       // 16, twice
    constexpr int up = DT == CK_DT_FP16 ? 6 : 3;                                  // bit of the code's place
    v4i r;
#pragma unroll
    for (int p = 0; p < 4; ++p)
        r[p] = (int)(((4 * p <= up ? w << (up - 4 * p) : w >> (4 * p - up)) & mask) | base);
    return r;
}

template <int DT>
__device__ __forceinline__ float widen1(uint32_t bits16)
{
    return widen2<DT>(bits16).x;
}

template <int GS, int MR, int MB, int NT, int KW>
struct Int4Few {
    static constexpr int xl = MB * MR;                       // 1 KiB loads of x: four rows of 128
    static constexpr int slot = (NT + xl + 1) * 1024;        // W, x, then scales and zeros
    static constexpr int loads = NT + xl + 1;
    static constexpr int lds = 80 * 1024;                    // two blocks a CU
    static constexpr int fit = lds / (KW * slot);
    static constexpr int ahead = fit >= 6 ? 6 : fit >= 2 ? fit : 2;
    static constexpr int ring = KW * ahead * slot;
    static constexpr int regs = NT * MB * MR;
    static constexpr int sums = KW * regs * 256;
    static_assert(sums <= ring && ring <= 163840 && (ahead - 1) * loads < 64, "the ring, then the sums");
};

template <int DT, int GS, int MR, int MB, int NT, int KW>
__global__ __launch_bounds__(64 * KW) void int4_few_kernel(Int4Args a)
{
    using S = Int4Few<GS, MR, MB, NT, KW>;
    constexpr int AH = S::ahead, XL = S::xl, L = S::loads;
    __shared__ __attribute__((aligned(1024))) uint8_t ring[S::ring];
    const int lane = threadIdx.x & 63, G = lane >> 4, i16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t tiles = (a.n + 15) / 16, tile0 = (int64_t)blockIdx.x * NT;
    const int64_t m0 = (int64_t)blockIdx.y * (16 * MB);
    const int rows = (int)min<int64_t>(a.m - m0, 16 * MB);
    const int cb = (int)(a.chunks * wave / KW), ce = (int)(a.chunks * (wave + 1) / KW), nc = ce - cb;

    const uint8_t* const xb = reinterpret_cast<const uint8_t*>(a.x + m0 * a.ldx);
    uint32_t x_off[XL], x_at[XL];                            // row, and byte of the chunk's 256
#pragma unroll
    for (int j = 0; j < XL; ++j) {
        const int row = 4 * j + G;
        x_off[j] = (uint32_t)(min(row, rows - 1) * a.ldx * 2);
        x_at[j] = (uint32_t)((i16 ^ (row & 15)) * 16);
    }
    // Scales: two lanes a tile and group; zeros from lane 32 on, one lane.
    const bool zl = a.wz != nullptr && lane >= 32;
    const int su = zl ? lane - 32 : lane, per = zl ? 1 : 2;
    const int st = min(su / (GS * per), NT - 1), sg = su / per % GS;
    const int64_t stile = min(tile0 + st, tiles - 1);
    const uint8_t* const s_base = zl ? a.wz + stile * a.groups * 16
                                     : reinterpret_cast<const uint8_t*>(a.ws) + stile * a.groups * 32 + (su & 1) * 16;
    const uint32_t s_step = zl ? 16 : 32;
    const uint8_t* w_base[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) w_base[t] = a.w + min(tile0 + t, tiles - 1) * a.chunks * 1024;

    uint8_t* const my = ring + wave * (AH * S::slot);
    const uint32_t my_lds = lds_addr(my);
    auto issue = [&](int slot, int c) {
        const uint32_t dst = my_lds + slot * S::slot;
        const int64_t kc = cb + c;
#pragma unroll
        for (int t = 0; t < NT; ++t) dma16(reinterpret_cast<const int8_t*>(w_base[t] + kc * 1024), lane * 16, dst + t * 1024);
        const uint32_t left = (uint32_t)min<int64_t>(256, (a.k - kc * 128) * 2) - 16;   // past k: the last piece again
#pragma unroll
        for (int j = 0; j < XL; ++j)
            dma16(reinterpret_cast<const int8_t*>(xb + kc * 256), x_off[j] + min(x_at[j], left), dst + (NT + j) * 1024);
        const uint32_t g = (uint32_t)min<int64_t>(kc * GS + sg, a.groups - 1);
        dma16_at(s_base + (uint64_t)g * s_step, dst + (NT + XL) * 1024);
    };

    // x: operand row i of a 16-row block is row 4 (i % 4) + i / 4
    int x_rd[MB], x_sw[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b) {
        const int row = 16 * b + 4 * min(i16 & 3, MR - 1) + (i16 >> 2);
        x_rd[b] = NT * 1024 + row * 256;
        x_sw[b] = row & 15;
    }
    const uint32_t one2 = DT == CK_DT_FP16 ? 0x3c003c00u : 0x3f803f80u;
    const v4i one = {(int)one2, (int)one2, (int)one2, (int)one2};
    const f32x4v zero4 = {0.0f, 0.0f, 0.0f, 0.0f};
    float tot[NT][MB][MR];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
            for (int r = 0; r < MR; ++r) tot[t][b][r] = 0.0f;

    if (nc > 0) {
#pragma unroll
        for (int i = 0; i < AH; ++i)
            if (i < nc) issue(i, i);
    }
    int slot = 0;
    for (int c = 0; c < nc; ++c) {
        // the loads of up to AH - 1 later chunks may still be on their way
        const int later = min(AH - 1, nc - 1 - c);
        if (later >= AH - 1) wait_vmcnt<(AH - 1) * L>();
        else if (AH > 5 && later == 4) wait_vmcnt<4 * L < 64 ? 4 * L : 63>();
        else if (AH > 4 && later == 3) wait_vmcnt<3 * L < 64 ? 3 * L : 63>();
        else if (AH > 3 && later == 2) wait_vmcnt<2 * L < 64 ? 2 * L : 63>();
        else if (AH > 2 && later == 1) wait_vmcnt<L>();
        else wait_vmcnt<0>();
        const uint8_t* const base = my + slot * S::slot;
        v4i w[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) w[t] = *reinterpret_cast<const v4i*>(base + t * 1024 + lane * 16);
        const int kleft = (int)min<int64_t>(128, a.k - (int64_t)(cb + c) * 128);
#pragma unroll
        for (int g = 0; g < GS; ++g) {
            f32x4v acc[NT][MB], xs[MB];
#pragma unroll
            for (int b = 0; b < MB; ++b) {
                xs[b] = zero4;
#pragma unroll
                for (int t = 0; t < NT; ++t) acc[t][b] = zero4;
            }
#pragma unroll
            for (int s = g * (4 / GS); s < (g + 1) * (4 / GS); ++s) {
                v4i x[MB];
#pragma unroll
                for (int b = 0; b < MB; ++b) {
                    x[b] = *reinterpret_cast<const v4i*>(base + x_rd[b] + (((4 * s + G) ^ x_sw[b]) << 4));
                    if (kleft < 128 && 32 * s + 8 * G >= kleft) x[b] = v4i{0, 0, 0, 0};
                    xs[b] = mfma16<DT>(x[b], one, xs[b]);
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const v4i wf = codes16<DT>((uint32_t)w[t][s]);
#pragma unroll
                    for (int b = 0; b < MB; ++b) acc[t][b] = mfma16<DT>(x[b], wf, acc[t][b]);
                }
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const uint8_t* const sp = base + (NT + XL) * 1024;
                const float sc = widen1<DT>(*reinterpret_cast<const uint16_t*>(sp + (t * GS + g) * 32 + i16 * 2));
                const float z = a.wz ? 16.0f + (float)sp[512 + (t * GS + g) * 16 + i16] : 24.0f;
#pragma unroll
                for (int b = 0; b < MB; ++b)
#pragma unroll
                    for (int r = 0; r < MR; ++r)
                        tot[t][b][r] = __builtin_fmaf(sc, __builtin_fmaf(-z, xs[b][r], acc[t][b][r]), tot[t][b][r]);
            }
        }
        asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory"); // the slot is read
        if (c + AH < nc) issue(slot, c + AH);
        slot = slot + 1 == AH ? 0 : slot + 1;
    }

    // The waves' sums, over the rings, then in their order.
    __syncthreads();
    float* const red = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int b = 0; b < MB; ++b)
#pragma unroll
            for (int r = 0; r < MR; ++r) red[((wave * NT + t) * MB * MR + b * MR + r) * 64 + lane] = tot[t][b][r];
    __syncthreads();
    for (int o = threadIdx.x; o < S::regs * 64; o += 64 * KW) {
        const int l = o & 63, q = o >> 6, r = q % MR, b = q / MR % MB, t = q / (MR * MB);
        const int64_t col = (tile0 + t) * 16 + (l & 15);
        const int row = 16 * b + 4 * r + (l >> 4);
        if (col >= a.n || row >= rows) continue;
        float v = red[o];
#pragma unroll
        for (int w = 1; w < KW; ++w) v = v + red[w * S::regs * 64 + o];
        store_int4(a, m0 + row, col, v);
    }
}

namespace {

ck_status check_int4_sizes(int64_t n, int64_t k, int64_t group)
{
    if (n < 0 || k < 0) return fail(CK_ERR_INVALID_ARG, "negative size");
    if (group != 32 && group != 64 && group != 128) return fail(CK_ERR_UNSUPPORTED, "group must be 32, 64 or 128");
    if (k % 8 != 0) return fail(CK_ERR_UNSUPPORTED, "k must be a multiple of 8");
    if (n > (int64_t(1) << 31) - 1 || k > (int64_t(1) << 31) - 1) return fail(CK_ERR_UNSUPPORTED, "n or k too large");
    return CK_OK;
}

// The kernel for a call, and what a block of it covers.
struct Int4Plan {
    const void* fn;
    int tiles, rows, waves;
};

template <int DT, int GS>
Int4Plan int4_plan_gs(int64_t m, int64_t n)
{
#define CK_INT4_FEW(MR, MB, NT, KW) \
    Int4Plan{reinterpret_cast<const void*>(&int4_few_kernel<DT, GS, MR, MB, NT, KW>), NT, 16 * MB, KW}
    const bool wide = n > 16 * 2 * kNumCUs;
    if (m <= 4) return wide ? CK_INT4_FEW(1, 1, 2, 4) : CK_INT4_FEW(1, 1, 1, 8);
    if (m <= 8) return wide ? CK_INT4_FEW(2, 1, 2, 4) : CK_INT4_FEW(2, 1, 1, 8);
    if (m <= 16) return wide ? CK_INT4_FEW(4, 1, 2, 4) : CK_INT4_FEW(4, 1, 1, 8);
    return wide ? CK_INT4_FEW(4, 2, 4, 4) : CK_INT4_FEW(4, 2, 2, 4);
#undef CK_INT4_FEW
}

Int4Plan int4_plan(int dtype, int64_t m, int64_t n, int64_t group)
{
    if (dtype == CK_DT_FP16)
        return group == 32 ? int4_plan_gs<CK_DT_FP16, 4>(m, n) : group == 64 ? int4_plan_gs<CK_DT_FP16, 2>(m, n)
                                                                            : int4_plan_gs<CK_DT_FP16, 1>(m, n);
    return group == 32 ? int4_plan_gs<CK_DT_BF16, 4>(m, n) : group == 64 ? int4_plan_gs<CK_DT_BF16, 2>(m, n)
                                                                        : int4_plan_gs<CK_DT_BF16, 1>(m, n);
}

}  // namespace

extern "C" ck_status ck_int4_pack(const uint8_t* codes, int64_t ldc, const uint16_t* scales, int64_t lds,
                                  const uint8_t* zeros, int64_t ldz, uint8_t* w, uint16_t* w_scale,
                                  uint8_t* w_zero, int64_t n, int64_t k, int64_t group, hipStream_t stream)
{
    ck_status s = check_int4_sizes(n, k, group);
    if (s != CK_OK) return s;
    if (n == 0 || k == 0) return ok();
    if (!codes || !scales || !w || !w_scale) return fail(CK_ERR_INVALID_ARG, "NULL codes, scales, w or w_scale");
    if (!zeros != !w_zero) return fail(CK_ERR_INVALID_ARG, "zeros and w_zero go together");
    const int64_t groups = cdiv(k, group);
    if (ldc < k / 2 || lds < groups || (zeros && ldz < groups))
        return fail(CK_ERR_INVALID_ARG, "ldc, lds or ldz smaller than a row");
    if (!aligned(scales, 2) || !aligned(w, 16) || !aligned(w_scale, 16) || !aligned(w_zero, 16))
        return fail(CK_ERR_UNSUPPORTED, "misaligned scales, w, w_scale or w_zero");
    Int4PackArgs a{codes, scales, zeros, (uint32_t*)w, w_scale, w_zero, ldc, lds, ldz, n, k, cdiv(k, 128), groups};
    const int64_t blocks = cdiv(n, 16) * a.chunks;           // 256 words a block; 16 scales a group fit
    if (blocks > 0x7fffffffLL) return fail(CK_ERR_UNSUPPORTED, "too many blocks");
    if ((s = check_device()) != CK_OK) return s;
    void* kargs[] = {&a};
    s = launch(reinterpret_cast<const void*>(&int4_pack_kernel), (unsigned)blocks, 256, kargs, stream, "int4_pack");
    return s == CK_OK ? ok() : s;
}

extern "C" ck_status ck_int4_linear(const ck_int4_args* args, hipStream_t stream)
{
    if (!args) return fail(CK_ERR_INVALID_ARG, "NULL args");
    const ck_int4_args& p = *args;
    if (p.dtype != CK_DT_BF16 && p.dtype != CK_DT_FP16) return fail(CK_ERR_INVALID_ARG, "bad dtype");
    if (p.out_dtype != CK_OUT_BF16 && p.out_dtype != CK_OUT_FP16 && p.out_dtype != CK_OUT_FP32)
        return fail(CK_ERR_INVALID_ARG, "bad out_dtype");
    if (p.m < 0) return fail(CK_ERR_INVALID_ARG, "negative size");
    ck_status s = check_int4_sizes(p.n, p.k, p.group);
    if (s != CK_OK) return s;
    if (p.m == 0 || p.n == 0) return ok();
    if (!p.out) return fail(CK_ERR_INVALID_ARG, "NULL out");
    if (p.m > 1 && p.ldo < p.n) return fail(CK_ERR_INVALID_ARG, "ldo smaller than n");
    if (p.k > 0) {
        if (!p.x || !p.w || !p.w_scale) return fail(CK_ERR_INVALID_ARG, "NULL x, w or w_scale");
        if (p.m > 1 && p.ldx < p.k) return fail(CK_ERR_INVALID_ARG, "ldx smaller than k");
        if ((p.m > 1 && p.ldx % 8 != 0) || !aligned(p.x, 16))
            return fail(CK_ERR_UNSUPPORTED, "x rows must start 16 bytes apart (ldx %% 8 == 0)");
    }
    const int esz = p.out_dtype == CK_OUT_FP32 ? 4 : 2;
    if (!aligned(p.w, 16) || !aligned(p.w_scale, 16) || !aligned(p.w_zero, 16) || !aligned(p.out, esz) ||
        (p.bias && !aligned(p.bias, esz)))
        return fail(CK_ERR_UNSUPPORTED, "misaligned w, w_scale, w_zero, bias or out");
    // 32-bit offsets of a block's rows of x
    if (p.m > 1 && 64 * p.ldx >= (int64_t(1) << 31))
        return fail(CK_ERR_UNSUPPORTED, "rows of x too long for 32-bit offsets");
    const Int4Plan plan = int4_plan(p.dtype, p.m, p.n, p.group);
    const int64_t bx = cdiv(cdiv(p.n, 16), plan.tiles), by = cdiv(p.m, plan.rows);
    if (by > 65535) return fail(CK_ERR_UNSUPPORTED, "too many rows");
    if ((s = check_device()) != CK_OK) return s;
    Int4Args a{(const uint16_t*)p.x, p.w, p.w_scale, p.w_zero, p.bias, p.out, p.ldx, p.ldo, p.m, p.n, p.k,
               cdiv(p.k, 128), cdiv(p.k, p.group), p.out_dtype};
    void* kargs[] = {&a};
    hipError_t e = hipLaunchKernel(plan.fn, dim3((unsigned)bx, (unsigned)by), dim3(64 * plan.waves), kargs, 0, stream);
    if (e != hipSuccess) return fail(CK_ERR_HIP, "int4_linear launch: %s", hipGetErrorString(e));
    return ok();
}
