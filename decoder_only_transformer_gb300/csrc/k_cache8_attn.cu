// k_cache8_attn.cu - attention of the newest tokens of every sequence over its 8-bit cache.
//
// Row (sequence b, new token t of n, head h), at position p = len - n + t:
//   o = sum_j w_j s_v(j) c_v(j) / sum_j w_j,  w_j = exp(scale s_k(j) q . c_k(j) - max)
// over the positions max(0, p - window + 1) <= j <= p of kv head h / (H / Hkv); s_k, s_v are
// the scales of j's block.  A row that sees nothing is zero.
//
// Bound by reading the codes: two bytes a position, kv head and coordinate, for up to 128 rows
// (n H / Hkv).  An SM's share of HBM bandwidth is ~23 codes a clock, and what has to be kept
// below that is the work per code:
//   - products by mma.sync m16n8k16 in fp16 with fp32 sums.  It takes its operands from
//     registers, where the codes have just been converted; tcgen05 reads them from shared
//     memory, so every converted code (two bytes) would be written there and read again, for
//     tiles of 128 rows of which a decode step fills 1 to 16.  int8 codes and e4m3 codes are
//     fp16 numbers, so the products are exact; so is a row of q after division by a power of two (but
//     for elements below 2^-14 of its largest).
//   - the scales are not multiplied into the codes: s_k is one factor of the 16 scores of a
//     warp's step, which lies in one block; s_v multiplies the step's 16-key sum of P V as it
//     is added to the fp32 output.
//   - a code costs 1.25 to 1.5 instructions: for int8, bytes to the low halves of fp16 numbers
//     1024 + (c + 128) by masks, less 1152; for e4m3 the conversion of two at a time.
//   - the order of the coordinates inside a product of 16, and of the keys inside a step, is
//     free.  They are taken as 16-byte loads from shared memory bring them (see kappa below):
//     no transposition, no bank conflicts.
//   - the running maximum of a row moves only when a score exceeds it by 2^8: weights are
//     2^(x - m + 7), below 2^15 and so fp16 numbers; what is flushed to zero is below 2^-31
//     of the largest weight.
//
// Tiles of 64 keys (K and V, by TMA, a ring of them filled by a warp of its own); the four
// warps of a row group take 16 keys each and hold all of d_head.  All tiles of all
// (sequence, kv head, row block) jobs lie end to end and are cut into equal runs, one per
// resident CTA, whatever the lengths are; a run's first and last job may be pieces, whose
// (max, sum, unnormalised o) a second kernel joins exactly, in a fixed order.
#include "cache8.cuh"

namespace tfm {

namespace {

constexpr int kTileKeys = 64;
constexpr int kMaxRuns = 152 * 3 * 2;             // CTAs at most, and places for them in the workspace

template <int DH, bool HALF, int RG>
struct Ax {
    static constexpr int kTile = kTileKeys * DH;                       // bytes of K or V
    static constexpr int kStages = (HALF ? 3 : 4) * (128 / DH);
    static constexpr int kCtas = HALF ? 3 : RG == 1 ? 2 : 1;           // per SM
    static constexpr int kRows = HALF ? 8 : 16;                        // of a warp
    static constexpr int kThreads = 128 * RG + 32;
    static constexpr int kBuf = 4 * RG * kRows * DH * 4;               // the warps' o, to be added up
    static constexpr int kBufOff = kStages * 2 * kTile;
    static constexpr int kMlOff = kBufOff + kBuf;                      // float2 [RG][4][rows]
    static constexpr int kBarOff = kMlOff + RG * 4 * kRows * 8;
    static constexpr int kCumOff = kBarOff + 16 * kStages + 16;
    static constexpr int kBase = kCumOff + 1024;                       // + 4 (B + 1); the ring on a multiple of 1024
    static constexpr uint32_t kSwzMask = DH == 128 ? 7 : DH == 64 ? 3 : 0;
    static constexpr int kSwzShift = DH == 128 ? 0 : 1;
};

struct Geom {
    int B, T, H, Hkv, G, max_new, max_seq, nblk, shift;
    int per;                  // rows per sequence without offsets
    int window;
    int block_rows;           // rows of a job: 8, 16 or 32
    int row_blocks;           // of max_new tokens
    float scale_log2;
    int64_t sq_t, sq_h, so_t, so_h;
};

// A piece of a run that a join has to look at: the job's tiles [start, end) among all, and
// where its rows go.
struct PieceHead {
    int start, end, job_row;      // job_row: (b * Hkv + g) * row_blocks + row block
    int total;                    // tiles of all jobs
};

struct Seq {
    int row0, n, len;
    int tile0, tiles, blocks;     // key tiles of a job, row blocks
};

__device__ __forceinline__ Seq get_seq(const int32_t* __restrict__ cu, const int32_t* __restrict__ lens, const Geom& gm,
                                       int b, bool& bad) {
    const SeqRows r = seq_rows(cu, lens, b, gm.per, gm.T, gm.max_seq);
    Seq s;
    bad = !r.ok || r.n > gm.max_new;
    s.row0 = r.row0;
    s.n = r.n > gm.max_new ? 0 : r.n;
    s.len = r.len < 0 || r.len > gm.max_seq ? 0 : r.len;
    const int first = gm.window > 0 ? max(0, s.len - s.n - gm.window + 1) : 0;
    s.tile0 = first / kTileKeys;
    s.tiles = max(1, (s.len + kTileKeys - 1) / kTileKeys - s.tile0);
    s.blocks = (s.n * gm.G + gm.block_rows - 1) / gm.block_rows;
    return s;
}

__device__ __forceinline__ int run_start(int i, int total, int runs) {
    const int q = total / runs, r = total - q * runs;
    return i * q + min(i, r);
}
// Runs of at least kLeast tiles.
constexpr int kLeast = 2;
__device__ __forceinline__ int run_count(int total, int ctas) { return max(1, min(ctas, total / kLeast)); }

// The run's place among the jobs: sequence b, job j of it (kv head j / blocks, row block
// j % blocks), tile t of the job.
struct Walk {
    int b, j, t, left;
    Seq s;
};
// Tiles [t0, t1) of job j of sequence b.
struct Seg {
    int b, j, t0, t1;
    Seq s;
};
__device__ __forceinline__ bool next_seg(Walk& w, Seg& g, const Geom& gm, const int* cum,
                                         const int32_t* __restrict__ cu, const int32_t* __restrict__ lens) {
    if (w.left <= 0) return false;
    bool bad;
    if (w.t >= w.s.tiles) {                                // the next job
        w.t = 0;
        if (++w.j >= w.s.blocks * gm.Hkv) {
            w.j = 0;
            do ++w.b;
            while (cum[w.b + 1] == cum[w.b]);              // a run ends before the jobs do
            w.s = get_seq(cu, lens, gm, w.b, bad);
        }
    }
    g.b = w.b;
    g.j = w.j;
    g.s = w.s;
    g.t0 = w.t;
    g.t1 = min(w.s.tiles, w.t + w.left);
    w.left -= g.t1 - g.t0;
    w.t = g.t1;
    return true;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1, float c0, float c1, float c2, float c3) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

__device__ __forceinline__ uint32_t half2_sub(uint32_t a) {          // less 1152 in both halves, exact
    const __half2 v = __hsub2(*reinterpret_cast<__half2*>(&a), __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t e4m3x2(uint32_t w) {             // the low two bytes as fp16
    uint32_t r;
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(r) : "r"(w));
    return r;
}

// Four codes of one key, as the two fp16 pairs of a product's operand: (0, 2) and (1, 3)
// for int8, (0, 1) and (2, 3) for e4m3.
template <bool E4M3>
__device__ __forceinline__ void key_halves(uint32_t w, uint32_t& lo, uint32_t& hi) {
    if constexpr (E4M3) {
        lo = e4m3x2(w);
        hi = e4m3x2(w >> 16);
    } else {
        lo = half2_sub((w & 0x00FF00FFu) ^ 0x64806480u);
        hi = half2_sub(((w >> 8) & 0x00FF00FFu) ^ 0x64806480u);
    }
}
// Four codes of two keys, a and b: pair i is (a's code i, b's code i).
template <bool E4M3>
__device__ __forceinline__ void value_halves(uint32_t a, uint32_t b, uint32_t (&v)[4]) {
    if constexpr (E4M3) {
        const uint32_t x = __byte_perm(a, b, 0x5140), y = __byte_perm(a, b, 0x7362);
        v[0] = e4m3x2(x);
        v[1] = e4m3x2(x >> 16);
        v[2] = e4m3x2(y);
        v[3] = e4m3x2(y >> 16);
    } else {
        const uint32_t x = __byte_perm(a, b, 0x5410), y = __byte_perm(a, b, 0x7632);
        v[0] = half2_sub((x & 0x00FF00FFu) ^ 0x64806480u);
        v[1] = half2_sub(((x >> 8) & 0x00FF00FFu) ^ 0x64806480u);
        v[2] = half2_sub((y & 0x00FF00FFu) ^ 0x64806480u);
        v[3] = half2_sub(((y >> 8) & 0x00FF00FFu) ^ 0x64806480u);
    }
}

// Key of column c (0..7) of a step's scores.  Lane (g, t) reads K of key kappa(g) and V of
// keys kappa(2t), kappa(2t + 1); with the tile's swizzle these orders spread every
// load over all banks.
template <int DH>
__device__ __forceinline__ int kappa(int c) {
    if constexpr (DH == 128) return c & 1 ? c ^ 4 : c;                 // 0 5 2 7 4 1 6 3
    else if constexpr (DH == 64) return (0x65742130u >> (4 * c)) & 7;  // 0 3 1 2 4 7 5 6
    else return (0x67453210u >> (4 * c)) & 7;                          // 0 1 2 3 5 4 7 6
}

__device__ __forceinline__ void lds(uint32_t addr, uint32_t (&w)[4]) {
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr));
}
__device__ __forceinline__ void lds(uint32_t addr, uint32_t (&w)[2]) {
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
}
__device__ __forceinline__ void lds(uint32_t addr, uint32_t (&w)[1]) {
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(addr));
}

template <int DH, bool HALF, int RG>
__device__ __forceinline__ int buf_at(int row, int f) {      // place of float4 f of a row, spread over the banks
    constexpr int VPT = DH / 16;                             // float4s of a lane
    const int t = f / VPT;
    if constexpr (DH == 128) return row * 32 + (f ^ (2 * t + (row & 1)));
    else if constexpr (DH == 64) return row * 16 + (f ^ ((t >> 1) | (row & 1) << 1));
    else return row * 8 + (f ^ (row & 1));
}

template <bool E4M3, int DH, bool HALF, int RG>
__global__ void __launch_bounds__(Ax<DH, HALF, RG>::kThreads, Ax<DH, HALF, RG>::kCtas)
    k_cache8_part(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                  const __nv_bfloat16* __restrict__ q, const float* __restrict__ ks, const float* __restrict__ vs,
                  __nv_bfloat16* __restrict__ o, const int32_t* __restrict__ cu, const int32_t* __restrict__ lens,
                  PieceHead* __restrict__ heads, float2* __restrict__ part_ml, float4* __restrict__ part_o, const Geom gm,
                  int* err) {
    using X = Ax<DH, HALF, RG>;
    constexpr int KW = DH >= 64 ? 4 : 2;                     // words of a load of K
    constexpr int KL = DH == 128 ? 2 : 1;                    // loads of K per key
    constexpr int VW = DH / 32;                              // words of a load of V
    constexpr int VPT = DH / 16;                             // float4s of o that a lane holds per row
    constexpr int R = X::kRows;
    extern __shared__ uint8_t smem_raw[];
    __shared__ int abort_flag, place;
    const uint32_t raw_base = smem_u32(smem_raw);
    const uint32_t sbase = (raw_base + 1023u) & ~1023u;
    uint8_t* sm = smem_raw + (sbase - raw_base);
    const uint32_t full = sbase + X::kBarOff, empty = full + 8 * X::kStages;
    int* cum = reinterpret_cast<int*>(sm + X::kCumOff);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        abort_flag = 0;
        for (int i = 0; i < X::kStages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 4 * RG);
        }
        fence_mbar_init();
        tma_prefetch_desc(&kmap);
        tma_prefetch_desc(&vmap);
    }
    pdl_wait();
    pdl_trigger();
    // tiles of the sequences, added up
    for (int b = tid; b < gm.B; b += X::kThreads) {
        bool bad;
        const Seq s = get_seq(cu, lens, gm, b, bad);
        if (bad && blockIdx.x == 0) raise_error(err, TFM_EINVAL);
        cum[b + 1] = s.tiles * s.blocks * gm.Hkv;
    }
    if (tid == 0) cum[0] = 0;
    __syncthreads();
    if (warp == 0) {
        int carry = 0;
        for (int b0 = 0; b0 < gm.B; b0 += 32) {
            int x = b0 + lane < gm.B ? cum[b0 + lane + 1] : 0;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, d);
                if (lane >= d) x += y;
            }
            x += carry;
            if (b0 + lane < gm.B) cum[b0 + lane + 1] = x;
            carry = __shfl_sync(0xffffffffu, x, 31);
        }
    }
    __syncthreads();
    const int total = cum[gm.B];
    const int runs = run_count(total, gridDim.x);
    if ((int)blockIdx.x >= runs || total == 0) {
        if (tid == 0) heads[blockIdx.x] = PieceHead{0, 0, -1, total};
        return;
    }
    const int u0 = run_start(blockIdx.x, total, runs), u1 = run_start(blockIdx.x + 1, total, runs);
    for (int b = tid; b < gm.B; b += X::kThreads)
        if (cum[b] <= u0 && u0 < cum[b + 1]) place = b;
    __syncthreads();
    Walk w;
    {
        bool bad;
        w.b = place;
        w.s = get_seq(cu, lens, gm, w.b, bad);
        w.j = (u0 - cum[w.b]) / w.s.tiles;
        w.t = (u0 - cum[w.b]) % w.s.tiles;
        w.left = u1 - u0;
        if (tid == 0) {
            const int start = u0 - w.t;
            heads[blockIdx.x] = PieceHead{start, start + w.s.tiles,
                                          (w.b * gm.Hkv + w.j / w.s.blocks) * gm.row_blocks + w.j % w.s.blocks, total};
        }
    }
    Seg seg;
    int st = 0;                                              // stage of the ring, and its phase
    uint32_t phase = 0;
    if (warp == 4 * RG) {
        // ---------------------------------------------------------------- loads
        if (lane != 0) return;
        bool filled = false;                                 // every stage once
        while (next_seg(w, seg, gm, cum, cu, lens)) {
            const int row = (seg.b * gm.Hkv + seg.j / seg.s.blocks) * gm.max_seq + seg.s.tile0 * kTileKeys;
            for (int t = seg.t0; t < seg.t1; ++t) {
                if (filled && !mbar_wait(empty + 8 * st, phase ^ 1, err, &abort_flag)) return;
                mbar_arrive_expect_tx(full + 8 * st, 2 * X::kTile);
                tma_load_2d(sbase + st * 2 * X::kTile, &kmap, 0, row + t * kTileKeys, full + 8 * st);
                tma_load_2d(sbase + st * 2 * X::kTile + X::kTile, &vmap, 0, row + t * kTileKeys, full + 8 * st);
                if (++st == X::kStages) st = 0, phase ^= 1, filled = true;
            }
        }
        return;
    }
    // -------------------------------------------------------------------- rows
    const int kw = warp & 3, rg = warp >> 2, g = lane >> 2, t = lane & 3;
    // where this lane reads, inside a tile
    uint32_t koff[2][KL], voff[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = kw * 16 + i * 8 + kappa<DH>(g);
#pragma unroll
        for (int p = 0; p < KL; ++p)
            koff[i][p] = r * DH + (DH >= 64 ? ((t + 4 * p) ^ ((r >> X::kSwzShift) & X::kSwzMask)) * 16 : t * 8);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = kw * 16 + (i >> 1) * 8 + kappa<DH>(2 * t + (i & 1));
        voff[i] = r * DH + (DH == 128 ? (g ^ (r & 7)) * 16 : DH == 64 ? ((g >> 1) ^ ((r >> 1) & 3)) * 16 + (g & 1) * 8 : g * 4);
    }
    float4* buf = reinterpret_cast<float4*>(sm + X::kBufOff) + rg * 4 * R * (DH / 4);
    float2* ml = reinterpret_cast<float2*>(sm + X::kMlOff) + rg * 4 * R;
    bool dead = false;
    bool first_seg = true;
    while (next_seg(w, seg, gm, cum, cu, lens)) {
        const Seq& s = seg.s;
        const int kvh = seg.j / s.blocks, rb = seg.j % s.blocks;
        const int64_t bh = (int64_t)seg.b * gm.Hkv + kvh;
        const int nrows = min(s.n * gm.G - rb * gm.block_rows, gm.block_rows) - rg * R;     // of this row group
        // q: row r of the group is token r / G, head r % G
        uint32_t qa[HALF ? 1 : 2][KL * KW][2];
        float qinv[2];
        int seen_hi[2], seen_lo[2];                          // a row sees the positions [lo, hi]
#pragma unroll
        for (int i = 0; i < (HALF ? 1 : 2); ++i) {
            const int r = g + 8 * i;
            const int rr = rb * gm.block_rows + rg * R + r;
            const int tok = rr / gm.G;
            seen_hi[i] = r < nrows ? s.len - s.n + tok : s.len - 1;
            seen_lo[i] = gm.window > 0 ? seen_hi[i] - gm.window + 1 : 0;
            uint2 raw[KL * KW];
            float top = 0.0f;
            if (r < nrows) {
                const __nv_bfloat16* at = q + ((int64_t)s.row0 + tok) * gm.sq_t + (int64_t)(kvh * gm.G + rr % gm.G) * gm.sq_h;
#pragma unroll
                for (int p = 0; p < KL; ++p) {
                    const uint4* a4 = reinterpret_cast<const uint4*>(at + p * 64 + t * (DH >= 64 ? 16 : 8));
#pragma unroll
                    for (int x = 0; x < KW / 2; ++x) {
                        const uint4 y = __ldg(a4 + x);
                        raw[p * KW + 2 * x] = make_uint2(y.x, y.y);
                        raw[p * KW + 2 * x + 1] = make_uint2(y.z, y.w);
                    }
                }
            } else {
#pragma unroll
                for (int x = 0; x < KL * KW; ++x) raw[x] = make_uint2(0, 0);
            }
#pragma unroll
            for (int x = 0; x < KL * KW; ++x)
                top = fmaxf(top, fmaxf(fmaxf(fabsf(bf16_lo(raw[x].x)), fabsf(bf16_hi(raw[x].x))),
                                       fmaxf(fabsf(bf16_lo(raw[x].y)), fabsf(bf16_hi(raw[x].y)))));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // the row divided by the power of two of its largest element
            int e = (int)(__float_as_uint(top) >> 23);
            e = e == 0 || e == 255 ? 127 : min(e, 253);
            const float mul = __uint_as_float((uint32_t)(254 - e) << 23);
            qinv[i] = __uint_as_float((uint32_t)e << 23);
#pragma unroll
            for (int x = 0; x < KL * KW; ++x) {
                const float y0 = bf16_lo(raw[x].x) * mul, y1 = bf16_hi(raw[x].x) * mul;
                const float y2 = bf16_lo(raw[x].y) * mul, y3 = bf16_hi(raw[x].y) * mul;
                const __half2 a = E4M3 ? __floats2half2_rn(y0, y1) : __floats2half2_rn(y0, y2);
                const __half2 b = E4M3 ? __floats2half2_rn(y2, y3) : __floats2half2_rn(y1, y3);
                qa[i][x][0] = *reinterpret_cast<const uint32_t*>(&a);
                qa[i][x][1] = *reinterpret_cast<const uint32_t*>(&b);
            }
        }
        float acc[VW * 4][HALF ? 2 : 4];
#pragma unroll
        for (int i = 0; i < VW * 4; ++i)
#pragma unroll
            for (int j = 0; j < (HALF ? 2 : 4); ++j) acc[i][j] = 0.0f;
        float m[2] = {-3.402823466e38f, -3.402823466e38f}, l[2] = {0.0f, 0.0f};
        // positions that some row sees, that every row sees
        const int any_lo = gm.window > 0 ? max(0, s.len - s.n - gm.window + 1) : 0;
        const int all_lo = gm.window > 0 ? s.len - gm.window : 0, all_hi = s.len - s.n;
        const float* ksp = ks + bh * gm.nblk;
        const float* vsp = vs + bh * gm.nblk;
        int key = (s.tile0 + seg.t0) * kTileKeys + kw * 16;
        const int last_blk = s.len > 0 ? (s.len - 1) >> gm.shift : 0;
        float ksc = __ldg(ksp + min(key >> gm.shift, last_blk)), vsc = __ldg(vsp + min(key >> gm.shift, last_blk));
        for (int tile = seg.t0; tile < seg.t1; ++tile, key += kTileKeys) {
            const int nb = min((key + kTileKeys) >> gm.shift, last_blk);       // the next step's block
            const float ksn = __ldg(ksp + nb), vsn = __ldg(vsp + nb);
            if (!dead) dead = !warp_wait(full + 8 * st, phase, err, &abort_flag);
            if (key < s.len && key + 16 > any_lo) {
                const uint32_t kt = sbase + st * 2 * X::kTile, vt = kt + X::kTile;
                float c[2][4];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t kwd[KL][KW];
#pragma unroll
                    for (int p = 0; p < KL; ++p) lds(kt + koff[i][p], kwd[p]);
                    c[i][0] = c[i][1] = c[i][2] = c[i][3] = 0.0f;
#pragma unroll
                    for (int p = 0; p < KL; ++p)
#pragma unroll
                        for (int x = 0; x < KW; ++x) {
                            uint32_t b0, b1;
                            key_halves<E4M3>(kwd[p][x], b0, b1);
                            const int y = p * KW + x;
                            mma16816(c[i], qa[0][y][0], HALF ? 0u : qa[HALF ? 0 : 1][y][0], qa[0][y][1],
                                     HALF ? 0u : qa[HALF ? 0 : 1][y][1], b0, b1, c[i][0], c[i][1], c[i][2], c[i][3]);
                        }
                }
                const bool inside = key >= all_lo && key + 15 <= all_hi;
                float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int r = 0; r < (HALF ? 1 : 2); ++r) {
                    const float f = qinv[r] * ksc * gm.scale_log2;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float& y = c[i >> 1][2 * r + (i & 1)];
                        y *= f;
                        if (!inside) {
                            const int p = key + (i >> 1) * 8 + kappa<DH>(2 * t + (i & 1));
                            if (p > seen_hi[r] || p < seen_lo[r]) y = -INFINITY;
                        }
                        top[r] = fmaxf(top[r], y);
                    }
                }
                const bool up = top[0] > m[0] + 8.0f || (!HALF && top[1] > m[1] + 8.0f);
                if (__any_sync(0xffffffffu, up)) {
#pragma unroll
                    for (int r = 0; r < (HALF ? 1 : 2); ++r) {
                        float y = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
                        y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 2));
                        y = fmaxf(y, m[r]);
                        const float keep = ex2(m[r] - y);
                        m[r] = y;
                        l[r] *= keep;
#pragma unroll
                        for (int i = 0; i < VW * 4; ++i) {
                            acc[i][2 * r] *= keep;
                            acc[i][2 * r + 1] *= keep;
                        }
                    }
                }
                uint32_t pa[2][2];                            // [8 keys][row]
#pragma unroll
                for (int r = 0; r < (HALF ? 1 : 2); ++r) {
                    const float base = m[r] - 7.0f;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float p0 = ex2(c[i][2 * r] - base), p1 = ex2(c[i][2 * r + 1] - base);
                        l[r] += p0 + p1;
                        const __half2 h = __floats2half2_rn(p0, p1);
                        pa[i][r] = *reinterpret_cast<const uint32_t*>(&h);
                    }
                }
                uint32_t vw[4][VW];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    lds(vt + voff[i], vw[i]);
                    if (E4M3 && !inside) {                    // a code that nothing sees may be a NaN
                        const int p = key + (i >> 1) * 8 + kappa<DH>(2 * t + (i & 1));
                        if (p >= s.len || p < any_lo)
#pragma unroll
                            for (int x = 0; x < VW; ++x) vw[i][x] = 0;
                    }
                }
#pragma unroll
                for (int x = 0; x < VW; ++x) {
                    uint32_t b0[4], b1[4];
                    value_halves<E4M3>(vw[0][x], vw[1][x], b0);
                    value_halves<E4M3>(vw[2][x], vw[3][x], b1);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float d[4];
                        mma16816(d, pa[0][0], HALF ? 0u : pa[0][1], pa[1][0], HALF ? 0u : pa[1][1], b0[i], b1[i], 0.0f, 0.0f,
                                 0.0f, 0.0f);
#pragma unroll
                        for (int j = 0; j < (HALF ? 2 : 4); ++j) acc[4 * x + i][j] = fmaf(vsc, d[j], acc[4 * x + i][j]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty + 8 * st);
            if (++st == X::kStages) st = 0, phase ^= 1;
            ksc = ksn;
            vsc = vsn;
        }
        // The four warps' parts, added up.  Lane (g, t) holds coordinates [t DH / 4, (t + 1) DH / 4) of its rows:
        // column n = 2 t + j of product (x, i) is coordinate n DH / 8 + 4 x + i.
#pragma unroll
        for (int r = 0; r < (HALF ? 1 : 2); ++r) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
        }
        asm volatile("bar.sync %0, 128;" ::"r"(1 + rg) : "memory");           // the last segment's have been read
#pragma unroll
        for (int r = 0; r < (HALF ? 1 : 2); ++r) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int x = 0; x < VW; ++x)
                    buf[kw * R * (DH / 4) + buf_at<DH, HALF, RG>(g + 8 * r, t * VPT + j * VW + x)] =
                        make_float4(acc[4 * x][2 * r + j], acc[4 * x + 1][2 * r + j], acc[4 * x + 2][2 * r + j],
                                    acc[4 * x + 3][2 * r + j]);
            if (t == 0) ml[kw * R + g + 8 * r] = make_float2(m[r], l[r]);
        }
        asm volatile("bar.sync %0, 128;" ::"r"(1 + rg) : "memory");
        const bool whole = seg.t0 == 0 && seg.t1 == s.tiles;
        const int slot = (int)blockIdx.x * 2 + (first_seg ? 0 : 1);
        first_seg = false;
        const int lt = tid & 127;
        for (int e = lt; e < R * (DH / 4); e += 128) {
            const int r = e / (DH / 4), f = e % (DH / 4);
            if (r >= nrows) break;
            float2 x[4];
            float top = -3.402823466e38f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = ml[i * R + r];
                top = fmaxf(top, x[i].x);
            }
            float sum = 0.0f;
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float k = ex2(x[i].x - top);
                const float4 y = buf[i * R * (DH / 4) + buf_at<DH, HALF, RG>(r, f)];
                sum = fmaf(k, x[i].y, sum);
                v.x = fmaf(k, y.x, v.x);
                v.y = fmaf(k, y.y, v.y);
                v.z = fmaf(k, y.z, v.z);
                v.w = fmaf(k, y.w, v.w);
            }
            const int rr = rb * gm.block_rows + rg * R + r;
            if (whole) {
                const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                __nv_bfloat16* at = o + ((int64_t)s.row0 + rr / gm.G) * gm.so_t + (int64_t)(kvh * gm.G + rr % gm.G) * gm.so_h + f * 4;
                *reinterpret_cast<uint2*>(at) = make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
            } else {
                const int64_t pr = (int64_t)slot * gm.block_rows + rg * R + r;
                part_o[pr * (DH / 4) + f] = v;
                if (f == 0) part_ml[pr] = make_float2(top, sum);
            }
        }
    }
}

// Joins the pieces of the jobs that runs cut: CTA i looks at the boundary before run i + 1, and
// takes the job if that is the first boundary inside it.  Row by row; a row's float4s by
// DH / 4 threads, the pieces by the groups of threads in turn.
template <int DH>
__global__ void __launch_bounds__(256)
    k_cache8_join(const PieceHead* __restrict__ heads, const float2* __restrict__ part_ml, const float4* __restrict__ part_o,
                  __nv_bfloat16* __restrict__ o, const int32_t* __restrict__ cu, const int32_t* __restrict__ lens,
                  const Geom gm, int ctas) {
    constexpr int F = DH / 4, GR = 256 / F;
    __shared__ float4 sum_o[GR][F];
    __shared__ float2 sum_ml[GR];
    pdl_wait();
    pdl_trigger();
    const int i = (int)blockIdx.x + 1;
    const PieceHead h = heads[i];
    if (h.job_row < 0) return;
    const int runs = run_count(h.total, ctas);
    const int u = run_start(i, h.total, runs), before = run_start(i - 1, h.total, runs);
    if (u == h.start || before > h.start) return;
    // pieces: run i - 1's last segment, then the first of the runs from i on, as far as the job goes
    const int first_slot = before == h.start ? 2 * (i - 1) : 2 * (i - 1) + 1;
    int pieces = 1;
    {
        // runs from i on that begin before the job's end
        int lo = i, hi = runs;                               // run_start(lo) < end; first that does not, at most runs
        while (lo + 1 < hi) {
            const int mid = (lo + hi) >> 1;
            if (run_start(mid, h.total, runs) < h.end) lo = mid;
            else hi = mid;
        }
        pieces += lo - i + 1;
    }
    const int rb = h.job_row % gm.row_blocks, bh = h.job_row / gm.row_blocks, b = bh / gm.Hkv, kvh = bh % gm.Hkv;
    bool bad;
    const Seq s = get_seq(cu, lens, gm, b, bad);
    const int rows = min(s.n * gm.G - rb * gm.block_rows, gm.block_rows);
    const int f = threadIdx.x % F, gr = threadIdx.x / F;
    for (int r = blockIdx.y; r < rows; r += gridDim.y) {
        float top = -3.402823466e38f, sum = 0.0f;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int p = gr; p < pieces; p += GR) {
            const int64_t pr = (int64_t)(p == 0 ? first_slot : 2 * (i - 1 + p)) * gm.block_rows + r;
            const float2 x = part_ml[pr];
            const float4 y = part_o[pr * F + f];
            const float nt = fmaxf(top, x.x), k0 = ex2(top - nt), k1 = ex2(x.x - nt);
            sum = sum * k0 + x.y * k1;
            v = make_float4(v.x * k0 + y.x * k1, v.y * k0 + y.y * k1, v.z * k0 + y.z * k1, v.w * k0 + y.w * k1);
            top = nt;
        }
        sum_o[gr][f] = v;
        if (f == 0) sum_ml[gr] = make_float2(top, sum);
        __syncthreads();
        if (gr == 0) {
            float all = -3.402823466e38f;
            for (int k = 0; k < GR; ++k) all = fmaxf(all, sum_ml[k].x);
            float den = 0.0f;
            float4 z = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int k = 0; k < GR; ++k) {
                const float w = ex2(sum_ml[k].x - all);
                const float4 y = sum_o[k][f];
                den = fmaf(w, sum_ml[k].y, den);
                z = make_float4(fmaf(w, y.x, z.x), fmaf(w, y.y, z.y), fmaf(w, y.z, z.z), fmaf(w, y.w, z.w));
            }
            const float inv = den == 0.0f ? 0.0f : 1.0f / den;
            const int rr = rb * gm.block_rows + r;
            __nv_bfloat16* at = o + ((int64_t)s.row0 + rr / gm.G) * gm.so_t + (int64_t)(kvh * gm.G + rr % gm.G) * gm.so_h + f * 4;
            *reinterpret_cast<uint2*>(at) = make_uint2(pack_bf16x2(z.x * inv, z.y * inv), pack_bf16x2(z.z * inv, z.w * inv));
        }
        __syncthreads();
    }
}

// Rows of a job by the rows that max_new tokens of a kv head have: 8 in one warp's tile half,
// 16 in one, 32 in two row groups; more are blocks of 32, each of which reads the tiles.
int job_rows(int group, int max_new) {
    const int rows = group * max_new;
    return rows <= 8 ? 8 : rows <= 16 ? 16 : 32;
}

struct Space {
    size_t heads, ml, o, bytes;
};
Space space(int rows, int dh) {
    Space s;
    const size_t runs = kMaxRuns;
    s.heads = 0;
    s.ml = s.heads + runs * sizeof(PieceHead);
    s.o = s.ml + 2 * runs * rows * sizeof(float2);
    s.bytes = s.o + 2 * runs * rows * dh * sizeof(float);
    return s;
}

template <bool E4M3, int DH, bool HALF, int RG>
cudaError_t launch_part(const Cache8AttnArgs& a, const CUtensorMap& km, const CUtensorMap& vm, const Geom& gm, cudaStream_t st) {
    using X = Ax<DH, HALF, RG>;
    static std::atomic<uint64_t> done{0};
    const int smem = X::kBase + 4 * (a.B + 1);
    // sequences beyond those that leave room for kCtas have fewer CTAs per SM; 4096 still fit
    cudaError_t e = allow_smem(done, k_cache8_part<E4M3, DH, HALF, RG>, X::kBase + 4 * 4097);
    if (e != cudaSuccess) return e;
    const int ctas = sm_count() * X::kCtas < kMaxRuns ? sm_count() * X::kCtas : kMaxRuns;
    char* ws = static_cast<char*>(a.ws);
    const Space sp = space(gm.block_rows, DH);
    PieceHead* heads = reinterpret_cast<PieceHead*>(ws + sp.heads);
    float2* ml = reinterpret_cast<float2*>(ws + sp.ml);
    float4* po = reinterpret_cast<float4*>(ws + sp.o);
    e = launch_pdl(k_cache8_part<E4M3, DH, HALF, RG>, dim3(ctas), dim3(X::kThreads), smem, st, km, vm,
                   static_cast<const __nv_bfloat16*>(a.q), a.ks, a.vs, static_cast<__nv_bfloat16*>(a.o), a.cu, a.lens, heads,
                   ml, po, gm, device_error_word());
    if (e != cudaSuccess) return e;
    return launch_pdl(k_cache8_join<DH>, dim3(ctas - 1, gm.block_rows < 8 ? gm.block_rows : 8), dim3(256), 0, st,
                      static_cast<const PieceHead*>(heads), static_cast<const float2*>(ml), static_cast<const float4*>(po),
                      static_cast<__nv_bfloat16*>(a.o), a.cu, a.lens, gm, ctas);
}

template <bool E4M3, int DH>
cudaError_t by_rows(const Cache8AttnArgs& a, const CUtensorMap& km, const CUtensorMap& vm, const Geom& gm, cudaStream_t st) {
    if (gm.block_rows == 8) return launch_part<E4M3, DH, true, 1>(a, km, vm, gm, st);
    if (gm.block_rows == 16) return launch_part<E4M3, DH, false, 1>(a, km, vm, gm, st);
    return launch_part<E4M3, DH, false, 2>(a, km, vm, gm, st);
}

template <bool E4M3>
cudaError_t by_dh(const Cache8AttnArgs& a, const CUtensorMap& km, const CUtensorMap& vm, const Geom& gm, cudaStream_t st) {
    switch (a.dh) {
        case 32: return by_rows<E4M3, 32>(a, km, vm, gm, st);
        case 64: return by_rows<E4M3, 64>(a, km, vm, gm, st);
        default: return by_rows<E4M3, 128>(a, km, vm, gm, st);
    }
}

}  // namespace

size_t cache8_attention_workspace_bytes(int B, int H, int Hkv, int max_new, int dh) {
    (void)B;
    return space(job_rows(H / Hkv, max_new), dh).bytes;
}

tfm_status launch_cache8_attention(const Cache8AttnArgs& a, cudaStream_t st, cudaError_t* e) {
    CUtensorMap km, vm;
    if (!byte_rows_map(&km, a.kc, (int64_t)a.B * a.Hkv * a.max_seq, a.dh, kTileKeys) ||
        !byte_rows_map(&vm, a.vc, (int64_t)a.B * a.Hkv * a.max_seq, a.dh, kTileKeys))
        return TFM_ECUDA;
    Geom gm{};
    gm.B = a.B;
    gm.T = a.T;
    gm.H = a.H;
    gm.Hkv = a.Hkv;
    gm.G = a.H / a.Hkv;
    gm.max_new = a.max_new;
    gm.max_seq = a.max_seq;
    gm.shift = __builtin_ctz(a.block);
    gm.nblk = (a.max_seq + a.block - 1) >> gm.shift;
    gm.per = a.cu ? 0 : a.T / a.B;
    gm.window = a.window;
    gm.block_rows = job_rows(gm.G, a.max_new);
    gm.row_blocks = (gm.G * a.max_new + gm.block_rows - 1) / gm.block_rows;
    gm.scale_log2 = a.scale * 1.4426950408889634f;
    gm.sq_t = a.strides[0];
    gm.sq_h = a.strides[1];
    gm.so_t = a.strides[2];
    gm.so_h = a.strides[3];
    *e = a.e4m3 ? by_dh<true>(a, km, vm, gm, st) : by_dh<false>(a, km, vm, gm, st);
    return TFM_OK;
}

}  // namespace tfm
