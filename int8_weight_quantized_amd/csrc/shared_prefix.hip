// shared_prefix.hip -- attention of one new token per sequence over a paged
// cache, where the sequences of a group begin with the same tokens.
//
// Mathematics: that of paged_attention.hip.  The tokens that a sequence sees
// are those of its prefix and its own; both are cut into chunks, each chunk's
// sums kept relative to a reference of their own, and joined.
//
// A chunk of a prefix is read once for all query rows of its group: sequence
// by sequence the heads of one key head, R = members x (hq / hk) rows.  Per
// byte of a 16-bit cache there are R multiply-adds, so HBM bounds a small group
// and the matrix cores a large one.  Two forms of a block:
//   - up to 16 rows (a small group, or a sequence's own tokens): the waves
//     split the tokens, each with tiles of its own, as in paged_attention.hip;
//   - more rows: the waves split the rows, up to MB blocks of 16 each, and
//     share tiles of K and V in LDS, one in use and one on its way, one barrier
//     a tile.
// A weight enters the value product in 16-bit parts: three of bf16 (a bf16 or
// int8 cache), which hold it to fp32's own 2^-24, or two of fp16, the second the
// rest that the first left, 2^11 times finer, in sums of its own: 2^-23 of a
// weight or 2^-42 of the largest (2^-25 of 2^11 times what is left, beside weights of
// which the largest is 2^6 at least).

struct PrefixArgs {
    const uint16_t* q;
    uint16_t* out;
    const int32_t* ptable;
    const int32_t* plens;
    const int32_t* starts;
    const int32_t* table;
    const int32_t* lens;
    float* part;                         // [batch * hq][slots][d] weighted values
    float2* part_ml;                     // [batch * hq][slots] (M, sum)
    const uint8_t* ck;
    const uint8_t* cv;
    const float* cks;
    const float* cvs;
    int64_t q_bs, q_hs, o_bs, o_hs, pt_stride, table_stride, c_ps, c_hs, c_ts, s_ps, s_hs, s_ts;
    int64_t pages, pcap, cap;            // pcap, cap: tokens that a row of ptable, table can name
    int64_t pblocks;                     // blocks of prefixes; those of sequences follow
    float scale;
    int batch, hq, hk, group, prefixes, page_shift;
    int prows, psplits, pshare;          // of prefixes: row blocks, places for chunks, blocks that share a list
    int row_blocks, splits, share;       // and of sequences
    int few;                             // prefixes have up to 16 rows on average
};

// 16-bit parts of a weight.  With two of bf16, 2^-17 of it, more outputs are not the
// value nearest to the 64-bit result than of plain fp32 arithmetic, with three fewer
// (0.25 %, 0.21 % and 0.11 % of 128 sequences behind 65536 bf16 tokens, 0.22 %, 0.11 %
// and 0.04 % of 48 behind three int8 prefixes), in 400 and 477 us, 48 and 51 us.  Of fp16
// two do (0.37 % of 24 behind 20000, 0.39 % with four, 1.25 % of fp32; 39 and 47 us).
template <int DT, bool I8>
constexpr int kPrefixParts = I8 || DT != CK_DT_FP16 ? 3 : 2;
constexpr int kPrefixMost = 1 << 30;     // a prefix's tokens
constexpr int kPrefixOwn = 512;          // a sequence's own tokens in a chunk, at most
constexpr int kPrefixSeg = 512;          // tokens whose row offsets are made at a time

// Sizes for rows of RB bytes: four waves, 64 KiB of K and V in LDS, so that two
// blocks share a CU.
template <int RB>
struct PrefixShape {
    static constexpr int tile = RB <= 256 ? 64 : 32;         // tokens of a shared tile
    static constexpr int walkers = RB <= 256 ? 4 : 2;        // waves with tiles of their own
    static constexpr int shared = 4 * tile * RB, walked = walkers * 2 * kAttnTile * RB;
    static constexpr int ring = shared > walked ? shared : walked;
};

__host__ __device__ constexpr int prefix_rows(int d) { return d <= 128 ? 128 : 64; }

// What a block works on: rows row0 .. row0 + rows - 1 of the group that begins
// at sequence seq0 (row r: sequence seq0 + r / group, head r % group of the key
// head), and chunks split, split + share and so on of the `len` tokens that
// `table` names: now tokens first .. first + n - 1, whose sums go to place slot.
struct PrefixWork {
    const int32_t* table;
    uint32_t len, chunk;
    int split, share, place, rows, row0, seq0, kvh;
    int64_t first;
    int n, slot;

    __device__ __forceinline__ bool next()
    {
        first = (int64_t)split * chunk;
        if (first >= len) return false;
        n = (int)min<int64_t>(chunk, len - first);
        slot = place + split;
        split += share;
        return true;
    }
};

// The tokens of a list, at most as many as its table can name; 0 for any
// negative length.
__device__ __forceinline__ uint32_t prefix_tokens(int32_t len, int64_t cap) { return (uint32_t)min<int64_t>(max(len, 0), cap); }

// The length of its chunks: `share` blocks have one each, unless that would be
// less than 128 tokens, or more than `most` for the form that takes few rows.
__device__ __forceinline__ uint32_t prefix_chunk(uint32_t len, int share, int most)
{
    const uint32_t all = 128u * share;
    return min((uint32_t)most, max((len + all - 1) / all, 1u) * 128);
}

// Of the chunks of a prefix that has so many sequences: 1024 tokens where all
// their rows are few and it was planned so, else any number.
__device__ __forceinline__ int prefix_most(const PrefixArgs& a, int members)
{
    return a.few && members <= 16 / a.group ? kAttnChunk : kPrefixMost;
}

// False if there is nothing to do.
template <int ROWS>
__device__ __forceinline__ bool prefix_work(const PrefixArgs& a, PrefixWork& w)
{
    const int lane = threadIdx.x & 63;
    if ((int64_t)blockIdx.x >= a.pblocks) {                  // a sequence's own tokens
        const int64_t id = (int64_t)blockIdx.x - a.pblocks, rest = id / a.row_blocks, bk = rest % ((int64_t)a.batch * a.hk);
        const int rb = (int)(id % a.row_blocks);
        w.split = (int)(rest / ((int64_t)a.batch * a.hk));
        w.kvh = (int)(bk % a.hk);
        w.seq0 = (int)(bk / a.hk);
        w.row0 = 16 * rb;
        w.rows = min(16, a.group - w.row0);
        w.table = a.table + w.seq0 * a.table_stride;
        w.len = prefix_tokens(a.lens[w.seq0], a.cap);
        w.chunk = prefix_chunk(w.len, a.share, kPrefixOwn);
        w.share = a.share;
        w.place = a.psplits;
        return w.next();
    }
    // The row blocks of a chunk and key head, which read the same rows, follow
    // each other on one XCD (blocks go to the eight in turn).
    const int64_t per = 8 * (int64_t)a.prows, unit = blockIdx.x / per * 8 + blockIdx.x % 8;
    int slot = (int)(blockIdx.x % per / 8);
    if (unit >= (int64_t)a.hk * a.pshare) return false;
    w.split = (int)(unit / a.hk);
    w.kvh = (int)(unit % a.hk);
    constexpr int most = 1 << 29;
    int p = -1, members = 0;                                 // the prefix, and its sequences
    for (int base = 0; base < a.prefixes; base += 64) {      // whose row block it is: a sum over the prefixes before
        int s0 = 0, blocks = 0;
        members = 0;
        if (base + lane < a.prefixes) {
            s0 = min(max(a.starts[base + lane], 0), a.batch);
            members = min(max(a.starts[base + lane + 1], s0), a.batch) - s0;
            blocks = (int)min<int64_t>(((int64_t)members * a.group + ROWS - 1) / ROWS, most);
        }
        int sum = blocks;                                    // at most `most`, whatever starts holds
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int o = __shfl_up(sum, off);
            if (lane >= off) sum = min(sum + o, most);
        }
        const int prev = __shfl_up(sum, 1);
        const unsigned long long past = __ballot(sum > slot);
        if (past) {
            const int at = __builtin_ctzll(past);
            p = base + at;
            if (at > 0) slot -= __shfl(prev, at);
            w.seq0 = __shfl(s0, at);
            w.row0 = slot * ROWS;
            members = __shfl(members, at);
            w.rows = min(ROWS, members * a.group - w.row0);
            break;
        }
        slot -= __shfl(sum, 63);
    }
    if (p < 0) return false;
    members = __builtin_amdgcn_readfirstlane(members);
    p = __builtin_amdgcn_readfirstlane(p);
    w.seq0 = __builtin_amdgcn_readfirstlane(w.seq0);
    w.row0 = __builtin_amdgcn_readfirstlane(w.row0);
    w.rows = __builtin_amdgcn_readfirstlane(w.rows);
    w.table = a.ptable + p * a.pt_stride;
    w.len = prefix_tokens(a.plens[p], a.pcap);
    w.chunk = prefix_chunk(w.len, a.pshare, prefix_most(a, members));
    w.share = a.pshare;
    w.place = 0;
    return w.next();
}

// The queries of 16 rows: lane 16 G + i holds elements 32 kk + 8 G + 0 .. 7 of
// row i; for an int8 cache as fp16, its largest element in [2^13, 2^14).
// -> what a score is to be multiplied by.
template <int DT, bool I8, int D>
__device__ __forceinline__ float prefix_queries(const PrefixArgs& a, const PrefixWork& w, int row, v4i (&qf)[D / 32])
{
    constexpr int KK = D / 32;
    const int G = (threadIdx.x & 63) >> 4;
    const int r = w.row0 + min(row, w.rows - 1), seq = r / a.group, head = w.kvh * a.group + r - seq * a.group;
    const uint16_t* const qp = a.q + (int64_t)(w.seq0 + seq) * a.q_bs + head * a.q_hs + 8 * G;
#pragma unroll
    for (int kk = 0; kk < KK; ++kk) qf[kk] = *reinterpret_cast<const v4i*>(qp + 32 * kk);
    if constexpr (!I8) {
        // Take them now: a later wait would also wait for the direct-to-LDS
        // loads, which the compiler does not count.
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) asm volatile("" : "+v"(qf[kk]));
        return a.scale * 1.44269504f;
    } else {
        float f[KK][8], m = 0.0f;
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
            widen8<DT>(qf[kk], f[kk]);
#pragma unroll
            for (int e = 0; e < 8; ++e) m = fmaxf(m, __builtin_fabsf(f[kk][e]));
        }
        m = fmaxf(m, __shfl_xor(m, 16));
        m = fmaxf(m, __shfl_xor(m, 32));
        const int e = m > 0.0f ? 14 - __builtin_amdgcn_frexp_expf(m) : 0;
#pragma unroll
        for (int kk = 0; kk < KK; ++kk)
#pragma unroll
            for (int x = 0; x < 4; ++x)
                qf[kk][x] = (int)f16x2_rne_bits(__builtin_amdgcn_ldexpf(f[kk][2 * x], e), __builtin_amdgcn_ldexpf(f[kk][2 * x + 1], e));
        return __builtin_amdgcn_ldexpf(1.0f, -e);
    }
}

// Where the sums of row `row` go.
__device__ __forceinline__ int64_t prefix_part(const PrefixArgs& a, const PrefixWork& w, int row)
{
    const int r = w.row0 + row, seq = r / a.group, head = w.kvh * a.group + r - seq * a.group;
    return ((int64_t)(w.seq0 + seq) * a.hq + head) * (a.psplits + a.splits) + w.slot;
}

template <int RB, bool I8>
struct PrefixShared {
    __attribute__((aligned(1024))) uint8_t ring[PrefixShape<RB>::ring];
    __attribute__((aligned(16))) uint32_t offs[kAttnChunk];
    __attribute__((aligned(16))) float kscale[I8 ? kAttnChunk : 4], vscale[I8 ? kAttnChunk : 4];
    float wave_m[4][16], wave_l[4][16], wave_v[2][4];
    int bad_page;
};

// Row offsets (in 16-byte units) and scales of the chunk's tokens from ..
// from + 256 PT - 1 into places dst and on; the last token's again up to
// `end`, so that masked places hold values of a visible row.  A thread's loads
// go out together, the pages of all its tokens and then the scales.
// -> the largest value scale of the wave's tokens.
template <int RB, bool I8, int PT>
__device__ __forceinline__ float prefix_fill(const PrefixArgs& a, const PrefixWork& w, PrefixShared<RB, I8>& sh, int from,
                                             int dst, int end)
{
    const int tid = threadIdx.x;
    int32_t pages[PT], ats[PT];
    float ks[PT], vs[PT], vmax = 0.0f;
#pragma unroll
    for (int j = 0; j < PT; ++j) {
        const int i = from + tid + j * 256;
        if (i < end) {
            const int64_t tok = w.first + min(i, w.n - 1);
            pages[j] = w.table[tok >> a.page_shift];
            ats[j] = (int32_t)(tok & ((1 << a.page_shift) - 1));
        }
    }
#pragma unroll
    for (int j = 0; j < PT; ++j) {
        if (from + tid + j * 256 < end) {
            int64_t page = pages[j];
            if (page < 0 || page >= a.pages) {
                sh.bad_page = 1;
                page = 0;
            }
            sh.offs[dst + tid + j * 256] = (uint32_t)((page * a.c_ps + w.kvh * a.c_hs + ats[j] * a.c_ts) * (I8 ? 1 : 2) / 16);
            if constexpr (I8) {
                const int64_t so = page * a.s_ps + w.kvh * a.s_hs + ats[j] * a.s_ts;
                ks[j] = a.cks[so];
                vs[j] = a.cvs[so];
            }
        }
    }
    if constexpr (I8) {
#pragma unroll
        for (int j = 0; j < PT; ++j) {
            if (from + tid + j * 256 < end) {
                sh.kscale[dst + tid + j * 256] = ks[j] * a.scale * 1.44269504f;
                sh.vscale[dst + tid + j * 256] = vs[j];
                vmax = fmaxf(vmax, __builtin_fabsf(vs[j]));
            }
        }
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) vmax = fmaxf(vmax, __shfl_xor(vmax, off));
    }
    return vmax;
}

// Up to 16 rows: the waves split the tokens (at most kAttnChunk of them).
template <int DT, bool I8, int D>
__device__ __forceinline__ void prefix_walk(const PrefixArgs& a, const PrefixWork& w, PrefixShared<D * (I8 ? 1 : 2), I8>& sh)
{
    constexpr int RB = D * (I8 ? 1 : 2);
    using Sh = AttnShape<RB>;
    using Kind = AttnKind<DT, I8, kPrefixParts<DT, I8>>;
    constexpr int NW = PrefixShape<RB>::walkers, NL = Sh::loads, DB = D / 16, NA = Kind::NA;
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));                            // nothing that follows from it is kept from chunk to chunk: registers are short
    const int lane = tid & 63, G = lane >> 4, i16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int tiles = (w.n + kAttnTile - 1) / kAttnTile;
    v4i qf[1][D / 32];
    float sc[1];
    const float vwave = prefix_fill<RB, I8, 4>(a, w, sh, 0, 0, tiles * kAttnTile);
    if (I8 && lane == 0) sh.wave_v[0][wave] = vwave;
    sc[0] = prefix_queries<DT, I8, D>(a, w, i16, qf[0]);
    __syncthreads();
    int ve = 0;                                              // value scales are taken relative to 2^ve
    if constexpr (I8) {
        const float vmax = fmaxf(fmaxf(sh.wave_v[0][0], sh.wave_v[0][1]), fmaxf(sh.wave_v[0][2], sh.wave_v[0][3]));
        ve = vmax > 0.0f ? __builtin_amdgcn_frexp_expf(vmax) : 0;
    }
    float M[1] = {kAttnLow}, L[1] = {0.0f};
    f32x4v acc[1][NA][DB];
#pragma unroll
    for (int i = 0; i < NA; ++i)
#pragma unroll
        for (int d = 0; d < DB; ++d) acc[0][i][d] = f32x4v{0.0f, 0.0f, 0.0f, 0.0f};
    uint8_t* const kring = sh.ring + (wave < NW ? wave : 0) * (2 * Sh::tile);
    uint8_t* const vring = kring + Sh::tile;
    const uint32_t klds = lds_addr(kring), vlds = klds + Sh::tile;
    uint32_t off[NL];
    auto read_offs = [&](int t) {
#pragma unroll
        for (int j = 0; j < NL; ++j) off[j] = sh.offs[t * kAttnTile + (64 * j + lane) / Sh::chunks];
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
    if (wave < NW) {
        if (wave < tiles) {
            read_offs(wave);
            issue_k();
            issue_v();
        }
        const AttnLane<I8, D> at(kring, vring, lane);
        for (int t = wave; t < tiles; t += NW) {
            const bool more = t + NW < tiles;
            wait_vmcnt<NL>();                                // K of this tile; V came after it
            attn_tile<DT, I8, D, 1, kPrefixParts<DT, I8>, false>(
                at, 0, qf, sc, &sh.kscale[I8 ? t * kAttnTile : 0], &sh.vscale[I8 ? t * kAttnTile : 0], ve,
                w.n - t * kAttnTile, t == wave, M, L, acc,
                [&] {
                    asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory"); // K is read: its place is free
                    if (more) {
                        read_offs(t + NW);
                        issue_k();
                    }
                },
                [&] {
                    if (more) wait_vmcnt<NL>();              // V of this tile; the next K came after it
                    else wait_vmcnt<0>();
                },
                [&] {
                    asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory"); // V is read
                    if (more) issue_v();
                });
        }
        // The waves' sums meet in LDS: each in its own ring, [row][d], 16-byte
        // pieces exchanged by xor.
        L[0] += __shfl_xor(L[0], 16);
        L[0] += __shfl_xor(L[0], 32);
        float* const own = reinterpret_cast<float*>(kring);
#pragma unroll
        for (int d = 0; d < DB; ++d) {
            f32x4v sum = acc[0][0][d];
            if constexpr (NA == 2) sum = sum + acc[0][1][d] * (1.0f / Kind::fine);
            *reinterpret_cast<f32x4v*>(own + i16 * D + (((4 * d + G) ^ (i16 & 7)) << 2)) = sum;
        }
        if (lane < 16) {
            sh.wave_m[wave][lane] = M[0];
            sh.wave_l[wave][lane] = L[0];
        }
    }
    __syncthreads();
    for (int e = tid; e < w.rows * (D / 4); e += 256) {
        const int h = e / (D / 4), c = e % (D / 4);
        float m = sh.wave_m[0][h];
#pragma unroll
        for (int x = 1; x < NW; ++x) m = fmaxf(m, sh.wave_m[x][h]);
        float l = 0.0f;
        f32x4v o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int x = 0; x < NW; ++x) {
            const float f = __builtin_amdgcn_exp2f(sh.wave_m[x][h] - m);   // a wave without tiles: 0
            l = __builtin_fmaf(f, sh.wave_l[x][h], l);
            const f32x4v v = *reinterpret_cast<const f32x4v*>(reinterpret_cast<const float*>(sh.ring + x * (2 * Sh::tile)) + h * D + ((c ^ (h & 7)) << 2));
#pragma unroll
            for (int r = 0; r < 4; ++r) o[r] = __builtin_fmaf(f, v[r], o[r]);
        }
        if constexpr (I8) {
#pragma unroll
            for (int r = 0; r < 4; ++r) o[r] = __builtin_amdgcn_ldexpf(o[r], ve);
        }
        const int64_t at = prefix_part(a, w, h);
        *reinterpret_cast<f32x4v*>(a.part + at * D + 4 * c) = o;
        if (c == 0) a.part_ml[at] = sh.bad_page ? make_float2(0.0f, NAN) : make_float2(m, l);
    }
}

// More rows: row block b of wave x is the group's b * 4 + x th of 16, and all
// waves go through the same tiles.
template <int DT, bool I8, int D, int MB>
__device__ __forceinline__ void prefix_share(const PrefixArgs& a, const PrefixWork& w, PrefixShared<D * (I8 ? 1 : 2), I8>& sh)
{
    constexpr int RB = D * (I8 ? 1 : 2), T = PrefixShape<RB>::tile;
    using Sh = AttnShape<RB>;
    using Kind = AttnKind<DT, I8, kPrefixParts<DT, I8>>;
    constexpr int DB = D / 16, NA = Kind::NA, LT = T * RB / 1024;    // 1 KiB loads of a tile's K
    constexpr int NL = (LT + 3) / 4;                         // and of those a wave's
    constexpr int TS = kPrefixSeg / T;                       // tiles of a segment
    const int lane = threadIdx.x & 63, G = lane >> 4, i16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tiles = (w.n + T - 1) / T, end = tiles * T;
    v4i qf[MB][D / 32];
    float sc[MB], M[MB], L[MB];
    f32x4v acc[MB][NA][DB];
    auto fill = [&](int seg) {
        const float v = prefix_fill<RB, I8, kPrefixSeg / 256>(a, w, sh, seg * kPrefixSeg, (seg & 1) * kPrefixSeg, end);
        if (I8 && lane == 0) sh.wave_v[seg & 1][wave] = v;
    };
    fill(0);
    if (end > kPrefixSeg) fill(1);
#pragma unroll
    for (int b = 0; b < MB; ++b) {
        sc[b] = prefix_queries<DT, I8, D>(a, w, (b * 4 + wave) * 16 + i16, qf[b]);
        M[b] = kAttnLow;
        L[b] = 0.0f;
#pragma unroll
        for (int i = 0; i < NA; ++i)
#pragma unroll
            for (int d = 0; d < DB; ++d) acc[b][i][d] = f32x4v{0.0f, 0.0f, 0.0f, 0.0f};
    }
    const uint32_t lds0 = lds_addr(sh.ring);
    // A wave copies every fourth KiB of a tile.
    auto issue = [&](int t) {
        const uint32_t dst = lds0 + (t & 1) * (2 * T * RB);
        uint32_t off[NL];
#pragma unroll
        for (int j = 0; j < NL; ++j)
            if (4 * j + wave < LT) off[j] = sh.offs[t % (2 * TS) * T + (64 * (4 * j + wave) + lane) / Sh::chunks];
#pragma unroll
        for (int j = 0; j < NL; ++j) {
            if (4 * j + wave >= LT) break;
            const int at = 64 * (4 * j + wave) + lane, row = at / Sh::chunks, pc = at % Sh::chunks;
            dma16_at(a.ck + (uint64_t)(off[j] + (uint32_t)(pc ^ Sh::swz(row))) * 16, dst + (4 * j + wave) * 1024);
        }
#pragma unroll
        for (int j = 0; j < NL; ++j) {
            if (4 * j + wave >= LT) break;
            const int at = 64 * (4 * j + wave) + lane, row = at / Sh::chunks, pc = at % Sh::chunks;
            dma16_at(a.cv + (uint64_t)(off[j] + (uint32_t)(pc ^ (I8 ? Sh::swz(row) : Sh::swz2(row)))) * 16,
                     dst + T * RB + (4 * j + wave) * 1024);
        }
    };
    const bool busy = wave * 16 < w.rows;
    int ve = -300;                                           // value scales are taken relative to 2^ve: none yet
    __syncthreads();
    issue(0);
    const AttnLane<I8, D> at(sh.ring, sh.ring + T * RB, lane);
    auto tile = [&](int t, auto odd) {
        constexpr int place = decltype(odd)::value ? 2 * T * RB : 0;
        wait_vmcnt<0>();
        __syncthreads();                                     // the tile has landed, the one before it is read
        if (t % TS == 0 && t > 0 && (t / TS + 1) * kPrefixSeg < end) fill(t / TS + 1);
        if (t + 1 < tiles) issue(t + 1);
        if constexpr (I8) {
            if (t % TS == 0) {                               // raised where a segment's scales are far above it
                const float* const v = sh.wave_v[t / TS & 1];
                const float vmax = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
                const int e = vmax > 0.0f ? __builtin_amdgcn_frexp_expf(vmax) : -300;
                if (e > (ve == -300 ? -300 : ve + 8)) {
#pragma unroll
                    for (int b = 0; b < MB; ++b)
#pragma unroll
                        for (int i = 0; i < NA; ++i)
#pragma unroll
                            for (int d = 0; d < DB; ++d)
#pragma unroll
                                for (int r = 0; r < 4; ++r) acc[b][i][d][r] = __builtin_amdgcn_ldexpf(acc[b][i][d][r], ve - e);
                    ve = e;
                }
            }
        }
        if (!busy) return;
#pragma unroll
        for (int u = 0; u < T / kAttnTile; ++u) {
            const int limit = w.n - t * T - u * kAttnTile, from = t % (2 * TS) * T + u * kAttnTile;
            if (limit <= 0) break;
            attn_tile<DT, I8, D, MB, kPrefixParts<DT, I8>, true>(at, place + u * (kAttnTile * RB), qf, sc,
                                                                 &sh.kscale[I8 ? from : 0], &sh.vscale[I8 ? from : 0], ve,
                                                                 limit, t + u == 0, M, L, acc, [] {}, [] {}, [] {});
        }
        asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
    };
    for (int t = 0; t < tiles; t += 2) {
        tile(t, BoolTag<false>{});
        if (t + 1 < tiles) tile(t + 1, BoolTag<true>{});
    }
#pragma unroll
    for (int b = 0; b < MB; ++b) {
        L[b] += __shfl_xor(L[b], 16);
        L[b] += __shfl_xor(L[b], 32);
        const int row = (b * 4 + wave) * 16 + i16;
        if (row < w.rows) {
            const int64_t at = prefix_part(a, w, row);
#pragma unroll
            for (int d = 0; d < DB; ++d) {
                f32x4v sum = acc[b][0][d];
                if constexpr (NA == 2) sum = sum + acc[b][1][d] * (1.0f / Kind::fine);
                if constexpr (I8) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) sum[r] = __builtin_amdgcn_ldexpf(sum[r], ve);
                }
                *reinterpret_cast<f32x4v*>(a.part + at * D + 16 * d + 4 * G) = sum;
            }
            if (G == 0) a.part_ml[at] = sh.bad_page ? make_float2(0.0f, NAN) : make_float2(M[b], L[b]);
        }
    }
}

template <int DT, bool I8, int D>
__global__ __launch_bounds__(256, 2) void shared_prefix_kernel(PrefixArgs a)
{
    constexpr int RB = D * (I8 ? 1 : 2);
    __shared__ PrefixShared<RB, I8> sh;
    PrefixWork w;
    if (!prefix_work<prefix_rows(D)>(a, w)) return;
    if (a.pages == 0) {                                      // no page is inside the cache
        do {
            for (int r = threadIdx.x; r < w.rows; r += 256) a.part_ml[prefix_part(a, w, r)] = make_float2(0.0f, NAN);
        } while (w.next());
        return;
    }
    if (threadIdx.x == 0) sh.bad_page = 0;
    __syncthreads();
    if (w.rows <= 16 && w.chunk <= kAttnChunk) {
        for (;;) {
            prefix_walk<DT, I8, D>(a, w, sh);
            if (!w.next()) break;
            __syncthreads();                                 // the chunk has been read
            if (threadIdx.x == 0) sh.bad_page = 0;
            __syncthreads();
        }
    } else if (D > 128 || w.rows <= 64) {
        prefix_share<DT, I8, D, 1>(a, w, sh);
    } else {
        if constexpr (D <= 128) prefix_share<DT, I8, D, 2>(a, w, sh);
    }
}

// Joins the chunks of a sequence and head, those of its prefix and its own, one
// wave for each: a lane has four elements of the values, P groups of lanes
// each add every P-th chunk (eight at a time, under a running M), and then theirs,
// all in an order that the sizes fix.  Each wave looks through starts itself.
template <int DT, int D>
__global__ __launch_bounds__(256) void shared_prefix_join_kernel(PrefixArgs a)
{
    constexpr int C = D <= 128 ? D / 4 : D / 8, V = D / 4 / C;       // lanes that hold the values, 16-byte pieces of each
    constexpr int P = 64 / C;                                // chunks added side by side
    constexpr int U = 8;
    const int lane = threadIdx.x & 63, c = lane % C, g = lane / C;
    const int64_t bh = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (bh >= (int64_t)a.batch * a.hq) return;
    const int h = (int)(bh % a.hq);
    const int64_t b = bh / a.hq;
    // Its prefix: as many entries of starts as are not past b, less one.
    int before = 0;
    bool wrong = false;
    for (int base = 0; base <= a.prefixes && a.prefixes > 0; base += 64) {
        const int i = base + lane;
        const bool in = i <= a.prefixes;
        const int s = in ? a.starts[i] : 0;
        before += __popcll(__ballot(in && s <= b));
        wrong |= __any(in && (s < 0 || s > a.batch || (i > 0 && s < a.starts[i - 1])));
    }
    const int p = before - 1;
    const uint32_t np = p < 0 || p >= a.prefixes ? 0 : prefix_tokens(a.plens[p], a.pcap), no = prefix_tokens(a.lens[b], a.cap);
    const int members = np > 0 ? a.starts[p + 1] - a.starts[p] : 0;
    const uint32_t pchunk = prefix_chunk(np, a.pshare, prefix_most(a, members)), chunk = prefix_chunk(no, a.share, kPrefixOwn);
    const int shared = (int)((np + pchunk - 1) / pchunk), count = wrong ? 0 : shared + (int)((no + chunk - 1) / chunk);
    const int64_t slots = a.psplits + a.splits;
    const float2* const ml = a.part_ml + bh * slots;
    const float* const part = a.part + bh * slots * D + 4 * c;
    float m = kAttnLow, l = 0.0f;
    f32x4v o[V];
#pragma unroll
    for (int v = 0; v < V; ++v) o[v] = f32x4v{0.0f, 0.0f, 0.0f, 0.0f};
    for (int s0 = g; g < P && s0 < count; s0 += P * U) {
        float2 x[U];
        f32x4v f[U][V];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int s = s0 + P * u;
            if (s < count) {
                const int64_t slot = s < shared ? s : a.psplits + (s - shared);
                x[u] = ml[slot];
#pragma unroll
                for (int v = 0; v < V; ++v) f[u][v] = *reinterpret_cast<const f32x4v*>(part + slot * D + 4 * C * v);
            }
        }
        float top = m;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (s0 + P * u < count) top = fmaxf(top, x[u].x);
        const float old = __builtin_amdgcn_exp2f(m - top);
        m = top;
        l *= old;
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = o[v] * old;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (s0 + P * u < count) {
                const float w = __builtin_amdgcn_exp2f(x[u].x - m);
                l = __builtin_fmaf(w, x[u].y, l);
#pragma unroll
                for (int v = 0; v < V; ++v)
#pragma unroll
                    for (int r = 0; r < 4; ++r) o[v][r] = __builtin_fmaf(w, f[u][v][r], o[v][r]);
            }
        }
    }
    // the groups' sums, in their order, in every group
    float high = m;
#pragma unroll
    for (int i = 0; i < P; ++i) high = fmaxf(high, __shfl(m, i * C));
    const float w = __builtin_amdgcn_exp2f(m - high);        // a group without chunks: 0
    float sum = 0.0f;
    f32x4v t[V];
#pragma unroll
    for (int v = 0; v < V; ++v) t[v] = f32x4v{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < P; ++i) {
        sum += __shfl(l * w, i * C);
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int r = 0; r < 4; ++r) t[v][r] += __shfl(o[v][r] * w, i * C + c);
    }
    if (g != 0) return;
    uint16_t* const out = a.out + b * a.o_bs + h * a.o_hs + 4 * c;
    const float inv = 1.0f / sum;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        uint2 y;
        y.x = narrow2<DT>(t[v][0] * inv, t[v][1] * inv);
        y.y = narrow2<DT>(t[v][2] * inv, t[v][3] * inv);
        if (wrong) y = make_uint2(kNan2<DT>, kNan2<DT>);
        else if (count == 0) y = make_uint2(0, 0);
        *reinterpret_cast<uint2*>(out + 4 * C * v) = y;
    }
}

namespace {

struct PrefixPlan {
    int64_t prows, psplits, pshare, pblocks;                 // of prefixes
    int64_t row_blocks, splits, share, blocks;               // of sequences; blocks: the whole grid
    int64_t bytes;
    bool few;
};

// Chunks.  The host knows how many tokens the tables can name, the kernel how
// many there are, and a table may be far wider than any length.  So the host
// chooses how many blocks share the tokens of a list, and they divide those that
// there are, 128 at least each (48 sequences of 600 tokens behind prefixes of
// 1000, in tables for 1024 tokens 30 us, for 131072 31 us, where chunks that
// follow from the tables took 28 and 154, with two parts of a weight).
//
// A prefix's blocks are so many that all take the least time, if the table is
// full, where a round of up to two blocks a CU takes as long as its chunk, a fixed
// part and its rows' sums, which are written and read; up to one block a CU run
// half as fast again.  (128 sequences behind 65536 tokens: 512 blocks 471 us, 256
// blocks 670; 48 behind three int8 prefixes: 512 blocks 57 us, 256 blocks 51; 24
// behind 20000 tokens at head_dim 256: 41.5 and 38.7.)  Where groups have up to 16
// rows on average, those that have no more get chunks of 1024 tokens at most, which
// the form for few rows takes, and a block goes through several.
//
// Uneven groups: the average decides, and a group's last row block may hold one
// row, for which three of four waves stand by and the prefix is read once more.
// (32/8 heads of 128, groups of 100, 2, 2 and 2 sequences behind 6000 tokens each 54
// us, the first alone 47, the others alone 21, 26 or 27 each 58; 8/8 heads, one group
// behind 20000: 128 rows 45 us, 129 rows 59, 192 rows 65.)
//
// All sequences have two blocks a CU, and their chunks 512 tokens at most (the
// 48 sequences: 1024 and 512 tokens 51 us, 256 56): they run beside the prefixes'
// long ones.  The first chunks of all come first, as they are the likeliest to
// have tokens.  From 512 pairs of a sequence and a key head on each pair has one
// block, which goes through a long sequence's chunks one after the other, whatever
// the others' lengths: one of 60000 tokens among 127 of 100, 32/8 heads, 812 us
// (among 31 567), where paged_attention takes 122 (61).
bool prefix_plan(PrefixPlan& p, int64_t batch, int64_t hq, int64_t hk, int64_t head_dim, int64_t prefixes,
                 int64_t pcap, int64_t cap)
{
    const int64_t limit = 0x7fffffff, group = hq / hk, round = 2 * kNumCUs;
    if (batch * hq > limit || pcap > kPrefixMost) return false;
    p = PrefixPlan{};
    cap = std::min(cap, limit);                              // no length is larger
    const int64_t used = std::min(prefixes, batch);          // prefixes with a sequence, at most
    p.pshare = 1;
    p.few = batch * group <= 16 * used;
    if (used > 0 && pcap > 0 && hq > 0) {
        p.prows = cdiv(batch * group, prefix_rows((int)head_dim)) + used - 1;
        const int64_t pairs = p.prows * hk;
        int64_t least = INT64_MAX;
        for (int64_t r = 1; r <= 16; r += r < 2 ? 1 : 2) {   // half a round, and whole ones
            const int64_t share = std::min(std::max<int64_t>(1, r * kNumCUs / pairs), cdiv(pcap, 128));
            const int64_t chunk = cdiv(cdiv(pcap, share), 128) * 128;
            const int64_t n = pairs * share, rest = n % round;
            const int64_t each = chunk + 128 + 2 * prefix_rows((int)head_dim);
            const int64_t time = n / round * each + (rest > kNumCUs ? each : rest > 0 ? each * 2 / 3 : 0);
            if (time < least) least = time, p.pshare = share;
        }
        p.psplits = p.few ? std::max(p.pshare, cdiv(pcap, kAttnChunk)) : p.pshare;
        if (pairs > limit / (p.pshare + 8)) return false;
        p.pblocks = cdiv(hk * p.pshare, 8) * 8 * p.prows;
    }
    p.row_blocks = cdiv(group, 16);
    const int64_t pairs = std::max<int64_t>(batch * hk * p.row_blocks, 1);
    p.share = std::max<int64_t>(std::min(cdiv(round, pairs), cdiv(cap, 128)), 1);
    p.splits = std::max(p.share, cdiv(cap, kPrefixOwn));
    if (pairs > limit / p.share || pairs * p.share + p.pblocks > limit) return false;
    p.blocks = p.pblocks + pairs * p.share;
    if (!grid_ok(p.blocks, 256) || !grid_ok(cdiv(batch * hq, 4), 256)) return false;
    if ((double)batch * hq * (p.psplits + p.splits) * (head_dim + 2) > 0x1p60) return false;
    p.bytes = batch * hq * (p.psplits + p.splits) * (head_dim + 2) * 4;
    return true;
}

template <int DT, bool I8>
const void* prefix_fn(int64_t d)
{
    switch (d) {
    case 64: return reinterpret_cast<const void*>(&shared_prefix_kernel<DT, I8, 64>);
    case 96: return reinterpret_cast<const void*>(&shared_prefix_kernel<DT, I8, 96>);
    case 128: return reinterpret_cast<const void*>(&shared_prefix_kernel<DT, I8, 128>);
    case 192: return reinterpret_cast<const void*>(&shared_prefix_kernel<DT, I8, 192>);
    default: return reinterpret_cast<const void*>(&shared_prefix_kernel<DT, I8, 256>);
    }
}

template <int DT>
const void* prefix_join_fn(int64_t d)
{
    switch (d) {
    case 64: return reinterpret_cast<const void*>(&shared_prefix_join_kernel<DT, 64>);
    case 96: return reinterpret_cast<const void*>(&shared_prefix_join_kernel<DT, 96>);
    case 128: return reinterpret_cast<const void*>(&shared_prefix_join_kernel<DT, 128>);
    case 192: return reinterpret_cast<const void*>(&shared_prefix_join_kernel<DT, 192>);
    default: return reinterpret_cast<const void*>(&shared_prefix_join_kernel<DT, 256>);
    }
}

}  // namespace

extern "C" int64_t ck_shared_prefix_attention_workspace(int64_t batch, int64_t hq, int64_t hk, int64_t head_dim,
                                                        int64_t prefixes, int64_t prefix_width, int64_t table_width,
                                                        int64_t page_size)
{
    if (batch < 0 || hq < 0 || hk < 1 || hq % hk != 0 || !attention_dim_ok(head_dim) || prefixes < 0 || prefix_width < 0 ||
        table_width < 0 || !is_pow2(page_size) || page_size > 32768 || prefixes > (1 << 20) ||
        !attention_sizes_ok(batch, hq, hk, table_width, page_size) || !attention_sizes_ok(batch, hq, hk, prefix_width, page_size))
        return -1;
    PrefixPlan plan;
    return prefix_plan(plan, batch, hq, hk, head_dim, prefixes, prefix_width * page_size, table_width * page_size) ? plan.bytes : -1;
}

extern "C" ck_status ck_shared_prefix_attention(const ck_prefix_args* args, const ck_kv_cache* cache, hipStream_t stream)
{
    if (!args || !cache) return fail(CK_ERR_INVALID_ARG, "NULL args or cache");
    const ck_prefix_args& p = *args;
    if (p.dtype != CK_DT_BF16 && p.dtype != CK_DT_FP16) return fail(CK_ERR_INVALID_ARG, "bad dtype");
    if (p.batch < 0 || p.hq < 0 || p.table_width < 0 || p.prefixes < 0 || p.prefix_width < 0)
        return fail(CK_ERR_INVALID_ARG, "negative size");
    if (!attention_dim_ok(cache->head_dim)) return fail(CK_ERR_UNSUPPORTED, "head_dim must be 64, 96, 128, 192 or 256");
    ck_status s = check_cache(cache, p.dtype, cache->head_dim, 16);
    if (s != CK_OK) return s;
    if (p.hq % cache->heads != 0) return fail(CK_ERR_INVALID_ARG, "query heads are not a multiple of the cache's");
    if (p.batch == 0 || p.hq == 0) return ok();
    if (!attention_sizes_ok(p.batch, p.hq, cache->heads, p.table_width, cache->page_size) ||
        !attention_sizes_ok(p.batch, p.hq, cache->heads, p.prefix_width, cache->page_size) || p.prefixes > (1 << 20))
        return fail(CK_ERR_UNSUPPORTED, "too large a batch, table or number of heads or prefixes");
    if (!p.q || !p.out || !p.lens || (!p.table && p.table_width > 0))
        return fail(CK_ERR_INVALID_ARG, "NULL q, out, table or lens");
    if (p.prefixes > 0 && (!p.starts || !p.prefix_lens || (!p.prefix_table && p.prefix_width > 0)))
        return fail(CK_ERR_INVALID_ARG, "NULL starts, prefix_lens or prefix_table");
    if (!rows16(p.q, p.batch, p.q_batch_stride, p.hq, p.q_head_stride) ||
        !rows16(p.out, p.batch, p.out_batch_stride, p.hq, p.out_head_stride))
        return fail(CK_ERR_UNSUPPORTED, "q and out rows must start 16 bytes apart");
    if (!aligned(p.table, 4) || !aligned(p.lens, 4) || !aligned(p.prefix_table, 4) || !aligned(p.prefix_lens, 4) || !aligned(p.starts, 4))
        return fail(CK_ERR_UNSUPPORTED, "misaligned table, lens or starts");
    if ((p.table_stride < p.table_width && p.batch > 1) || (p.prefix_table_stride < p.prefix_width && p.prefixes > 1))
        return fail(CK_ERR_INVALID_ARG, "table_stride smaller than table_width");
    if (!(p.scale == p.scale)) return fail(CK_ERR_INVALID_ARG, "scale is NaN");
    const bool i8 = cache->dtype == CK_DT_INT8, f16 = p.dtype == CK_DT_FP16;
    const int64_t d = cache->head_dim, row_bytes = d * (i8 ? 1 : 2);
    if (cache_reach(cache, cache->page_stride, cache->head_stride, cache->token_stride, d) * (row_bytes / d) > 0x1p36)
        return fail(CK_ERR_UNSUPPORTED, "the cache spans more than 64 GiB");
    if (!rows_apart(d, {p.batch, p.out_batch_stride}, {p.hq, p.out_head_stride}))
        return fail(CK_ERR_INVALID_ARG, "rows of out overlap");
    PrefixPlan plan;
    if (!prefix_plan(plan, p.batch, p.hq, cache->heads, d, p.prefixes, p.prefix_width * cache->page_size, p.table_width * cache->page_size))
        return fail(CK_ERR_UNSUPPORTED, "too many blocks");
    if (!p.workspace || p.workspace_bytes < plan.bytes)
        return fail(CK_ERR_INVALID_ARG, "the workspace needs %lld bytes", (long long)plan.bytes);
    if (!aligned(p.workspace, 256)) return fail(CK_ERR_UNSUPPORTED, "misaligned workspace");
    if ((s = check_device()) != CK_OK) return s;
    PrefixArgs a{};
    a.q = (const uint16_t*)p.q; a.out = (uint16_t*)p.out; a.ptable = p.prefix_table; a.plens = p.prefix_lens; a.starts = p.starts;
    a.table = p.table; a.lens = p.lens;
    a.ck = (const uint8_t*)cache->k; a.cv = (const uint8_t*)cache->v; a.cks = cache->k_scale; a.cvs = cache->v_scale;
    a.q_bs = p.q_batch_stride; a.q_hs = p.q_head_stride; a.o_bs = p.out_batch_stride; a.o_hs = p.out_head_stride;
    a.pt_stride = p.prefix_table_stride; a.table_stride = p.table_stride;
    a.c_ps = cache->page_stride; a.c_hs = cache->head_stride; a.c_ts = cache->token_stride;
    a.s_ps = cache->scale_page_stride; a.s_hs = cache->scale_head_stride; a.s_ts = cache->scale_token_stride;
    a.pages = cache->pages; a.pcap = p.prefix_width * cache->page_size; a.cap = p.table_width * cache->page_size;
    a.scale = p.scale; a.batch = (int)p.batch; a.hq = (int)p.hq; a.hk = (int)cache->heads; a.prefixes = (int)p.prefixes;
    a.page_shift = ilog2(cache->page_size); a.group = (int)(p.hq / cache->heads);
    a.part = (float*)p.workspace;
    a.part_ml = (float2*)(a.part + p.batch * p.hq * (plan.psplits + plan.splits) * d);
    a.prows = (int)plan.prows; a.psplits = (int)plan.psplits; a.pshare = (int)plan.pshare; a.pblocks = plan.pblocks; a.few = plan.few;
    a.row_blocks = (int)plan.row_blocks; a.splits = (int)plan.splits; a.share = (int)plan.share;
    const void* fn = f16 ? (i8 ? prefix_fn<CK_DT_FP16, true>(d) : prefix_fn<CK_DT_FP16, false>(d))
                         : (i8 ? prefix_fn<CK_DT_BF16, true>(d) : prefix_fn<CK_DT_BF16, false>(d));
    const void* join = f16 ? prefix_join_fn<CK_DT_FP16>(d) : prefix_join_fn<CK_DT_BF16>(d);
    void* kargs[] = {&a};
    if ((s = launch(fn, (unsigned)plan.blocks, 256, kargs, stream, "shared_prefix_attention")) != CK_OK) return s;
    if ((s = launch(join, (unsigned)cdiv(p.batch * p.hq, 4), 256, kargs, stream, "shared_prefix_join")) != CK_OK) return s;
    return ok();
}
