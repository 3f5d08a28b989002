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
//     fp16 numbers, so the products are exact; so is a row of q times a power of two (but
//     for elements below 2^-24 of its largest).
//   - the scales are not multiplied into the codes: s_k is one factor of the 16 scores of a
//     warp's step, which lies in one block; s_v multiplies the step's 16-key sum of P V as it
//     is added to the fp32 output, whose unit is 2^64 from the first s_v above 2^64 on (sums over 2^31 keys of values
//     near the largest would leave fp32).
//   - a code costs 0.75 to 1 instruction: an int8 byte with its sign bit turned over is the fp16
//     subnormal (c + 128) 2^-24, and 128 times the sum of q, or of the step's weights (one product more), is
//     taken off inside each product, whose fp32 sums round to 2^-16 or so of a step of the code; what is summed over the
//     steps has no bias (with the bias left in until the end, the loss grew with the length: 2^-13 of a step after
//     256 steps of a warp, 2^-11 after 2048); e4m3 codes are converted two at a time.
//   - the order of the coordinates inside a product of 16, and of the keys inside a step, is
//     free.  They are taken as 16-byte loads from shared memory bring them (see kappa below):
//     no transposition, no bank conflicts.
//   - the running maximum of a row moves only when a score exceeds it by 2^8: weights are
//     2^(x - m + 7), below 2^15 and so fp16 numbers; what is flushed to zero is below 2^-32
//     of the largest weight.
//
// Tiles of 64 keys (K and V, by TMA, a ring of them filled by a warp of its own, which also hands over
// the jobs and their rows of q); the four computing warps take 16 keys each and hold all of
// d_head for up to 32 rows.  All tiles of all (sequence, kv head, row block) jobs lie end to end and are cut
// into equal runs, one per resident CTA, whatever the lengths are; a run's first and last job may
// be pieces, whose (max, sum, unnormalised o) a second kernel joins exactly, in a fixed
// order.  Short caches are not cut, and need no second kernel.
//
// Measured (graph replays; GB/s of the bytes that count): 64 chats of up to 4096 positions, 16/4 x 128,
// int8: 30.3 us, 4.4 TB/s; 131072 positions of one, e4m3: 28.0 us, 4.8 TB/s; 32 x 16 caches of 64
// with a window of 1024: 20.5 us; up to 5 new tokens of 16 over up to 8192: 22.4 us (int8: 23.9); 8 of them, 32 rows:
// 31.8 (int8: 35.1, whose kernel spills); 4 chats under 511: 6.9 us (8.9 where the cache has room for 8192: what is cut
// is decided by the capacity).  Of each but the last ~2 us pass until the first tile is asked for (lengths, runs, q),
// ~2 until it is there, ~1.5 with the last sums, ~3 with the second kernel; in between memory is
// nearly full for up to 8 rows, and a step's latency (~1500 cycles at 24 rows, two warps a
// scheduler) counts for more.  Tried and slower: the values' scales in the weights' exponents (P V without
// the fp32 additions: +1 to 2 us), the next step's scores ahead of this one's softmax (no
// change), three row groups of warps with 8 rows each for 24 (24.6 for 23.9), two scaled additions in
// one instruction (no change), runs and zeroed counters from a kernel ahead, the last writer adding the
// pieces up (+3 to 6 us), deeper rings (+1), the second kernel launched early with its CTAs spread by
// shared memory (no change).
#include <cmath>
#include <type_traits>

#include "cache8.cuh"

namespace tfm {

namespace {

constexpr int kTileKeys = 64;
constexpr int kMaxRuns = 152 * 3;                 // CTAs at most; the workspace has places for them

// NT: groups of 8 rows that a warp holds.  From two on, registers are what is short: the four
// computing warps are a warpgroup that takes over most of the registers of a second one, of
// which one warp loads (128 a thread at launch, 200 and 56 after).
template <int DH, int NT>
struct Ax {
    static constexpr int kTile = kTileKeys * DH;                       // bytes of K or V
    static constexpr bool kSplit = NT > 1;
    static constexpr int kComputeRegs = NT == 4 ? 208 : 200, kLoadRegs = 256 - kComputeRegs;   // kSplit: of 2 x 128 at launch
    static constexpr bool kSharedQ = NT > 2;                           // q's operands in shared memory
    static constexpr int kCtas = NT > 1 || DH == 128 ? 2 : 3;          // per SM
    static constexpr int kStages = (NT > 1 ? 3 : DH == 128 ? 4 : 2) * (DH == 128 ? 1 : DH == 64 ? 2 : 4);
    static constexpr int kRows = 8 * NT;                               // of a job
    static constexpr int kThreads = kSplit ? 256 : 160;
    static constexpr int kBuf = 4 * 8 * DH * 4;                        // the warps' o of 8 rows, to be added up
    static constexpr int kBufOff = kStages * 2 * kTile;
    static constexpr int kMlOff = kBufOff + kBuf;                      // float2 [4][8]
    static constexpr int kQ = kRows * DH * 2;                          // the job's rows of q, as they are
    static constexpr int kQOff = kMlOff + 4 * 8 * 8;                   // two places
    static constexpr int kFragOff = kQOff + 2 * kQ;                    // q's operands
    static constexpr int kRowOff = kFragOff + (kSharedQ ? kQ : 0);     // float4 [rows]: what belongs to a row
    static constexpr int kBarOff = kRowOff + (kSharedQ ? 16 * kRows : 0);    // of the ring, the places for q, the buffer, the operands
    static constexpr int kCumOff = kBarOff + 16 * kStages + 32 + 16 + 8;
    static constexpr int kBase = kCumOff + 1024;                       // + 4 (B + 1); the ring on a multiple of 1024
    // What a segment costs beside its tiles, in tiles: q, the first scores, the sum over the warps.
    static constexpr int kPiece = DH == 32 ? 5 : 3;
    static constexpr uint32_t kSwzMask = DH == 128 ? 7 : DH == 64 ? 3 : 0;
    static constexpr int kSwzShift = DH == 128 ? 0 : 1;
};

struct Geom {
    int B, T, H, Hkv, G, max_new, max_seq, nblk, shift;
    int per;                  // rows per sequence without offsets
    int window;
    int block_rows;           // rows of a job: 8, 16, 24 or 32
    int row_blocks;           // of max_new tokens
    int whole;                // no job is cut; 2: each of max_new tokens has a CTA of its own
    float scale_m;            // scale * log2(e) = scale_m 2^scale_e, scale_m in [0.5, 1)
    int scale_e;
    int64_t sq_t, sq_h, so_t, so_h;
};

// What the join has to know of the boundary before a run: the pieces of the job that it cuts (0:
// none), and where that job's rows go.
struct __align__(16) Cut {
    int pieces, share;            // which of the pieces - 1 boundaries this is
    int run0, place0;             // the run of the first piece, and the place of its part
    int row0, rb, kvh, nrows;
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
    s.blocks = 0;
    for (int r = s.n * gm.G; r > 0; r -= gm.block_rows) ++s.blocks;    // (no division: 128 / 8 at most)
    return s;
}

__device__ __forceinline__ int run_start(int i, int total, int runs) {
    const int q = total / runs, r = total - q * runs;
    return i * q + min(i, r);
}
__device__ __forceinline__ int run_of(int u, int total, int runs) {      // the run that tile u is in
    const int q = total / runs, r = total - q * runs;
    return u < r * (q + 1) ? u / (q + 1) : r + (u - r * (q + 1)) / q;
}
// Runs of at least kLeast units.  A job has kPiece units (what it costs beside its tiles), then one
// for each tile; a run that ends among the first ones has none of the job's tiles.
constexpr int kLeast = 3;
// Units of a job that is not worth cutting.  A CTA for each job against cut jobs and their join (us), caches of 12 to 13 units /
// 15 / 17 / 20 / 23: 4 x 12 of 64 6.8 for 8.3 / 7.6 for 8.9 / 8.2 for 8.9 / 9.6 for 8.9 / 10.3 for 8.9; 16 x 4 of 128 7.6 for 9.6 /
// 8.9 for 9.6 / 9.6 for 9.6 / 11.3 for 9.6; one sequence of 4 x 128 7.5 for 8.9 / 8.9 for 8.9 / 9.6 for 8.9; 188 x 12 of 64 26.6 for
// 28.0 / 32.5 for 32.8 / 36.2 for 35.7.  Never slower up to 15, and 14 is below that: capacities are longer than their sequences.
constexpr int kWhole = 14;
__device__ __forceinline__ int run_count(int total, int ctas) { return max(1, min(ctas, total / kLeast)); }

// The run's place among the jobs: sequence b, job j of it (kv head j / blocks, row block
// j % blocks), unit t of the job.
struct Walk {
    int b, j, t, left;
};
// A segment: tiles of one job, as the warps that load tell those that compute.
struct Seg {
    int tiles;                // none: the run is over
    int key;                  // first key
    int len, n;
    int bh;                   // sequence and kv head
    int nrows;
    int piece;                // -1: the whole job; else where its part goes
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {     // without an arrival
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float c0, float c1,
                                         float c2, float c3) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
// An 8 x 8 block of fp16: lane (g, t) gives row g, columns 2 t and 2 t + 1, and gets rows 2 t
// and 2 t + 1 of column g.
__device__ __forceinline__ uint32_t transposed(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

__device__ __forceinline__ uint32_t and_xor(uint32_t a, uint32_t mask, uint32_t x) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(r) : "r"(a), "r"(mask), "r"(x));
    return r;
}
// int8 codes in bytes 0 and 2 of a word as a pair of fp16 numbers (c + 128) 2^-24, which are
// subnormals: the byte itself, the sign bit turned over.
__device__ __forceinline__ uint32_t biased(uint32_t w) { return and_xor(w, 0x00FF00FFu, 0x00800080u); }
__device__ __forceinline__ uint32_t e4m3x2(uint32_t w) {             // the low two bytes as fp16
    uint32_t r;
    asm("{\n\t.reg .b16 t, u;\n\tmov.b32 {t, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(r) : "r"(w));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x2_hi(uint32_t w) {          // the high two
    uint32_t r;
    asm("{\n\t.reg .b16 t, u;\n\tmov.b32 {t, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, u;\n\t}" : "=r"(r) : "r"(w));
    return r;
}

// Four codes of one key, as the two fp16 pairs of a product's operand: (0, 2) and (1, 3)
// for int8, (0, 1) and (2, 3) for e4m3.
template <bool E4M3>
__device__ __forceinline__ void key_halves(uint32_t w, uint32_t& lo, uint32_t& hi) {
    if constexpr (E4M3) {
        lo = e4m3x2(w);
        hi = e4m3x2_hi(w);
    } else {
        lo = biased(w);
        hi = biased(w >> 8);
    }
}
// Four codes of two keys, a and b: pair i is (a's code i, b's code i).
template <bool E4M3>
__device__ __forceinline__ void value_halves(uint32_t a, uint32_t b, uint32_t (&v)[4]) {
    if constexpr (E4M3) {
        const uint32_t x = __byte_perm(a, b, 0x5140), y = __byte_perm(a, b, 0x7362);
        v[0] = e4m3x2(x);
        v[1] = e4m3x2_hi(x);
        v[2] = e4m3x2(y);
        v[3] = e4m3x2_hi(y);
    } else {
        const uint32_t x = __byte_perm(a, b, 0x5410), y = __byte_perm(a, b, 0x7632);
        v[0] = biased(x);
        v[1] = biased(x >> 8);
        v[2] = biased(y);
        v[3] = biased(y >> 8);
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

// W words of a tile.
template <int W>
__device__ __forceinline__ void words(const uint8_t* at, uint32_t (&w)[W]) {
    if constexpr (W == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(at);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if constexpr (W == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(at);
        w[0] = v.x, w[1] = v.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t*>(at);
    }
}

// Place of float4 f of a row in the buffer where warps add up, spread over the banks.
template <int DH>
__device__ __forceinline__ int buf_at(int row, int f) {
    const int t = (row >> 1) & 3;
    return row * (DH / 4) + (f ^ (DH == 128 ? t : DH == 64 ? (t & 1) | (t >> 1) << 2 : t << 1));
}

template <bool E4M3, int DH, int NT>
__global__ void __launch_bounds__(Ax<DH, NT>::kThreads, Ax<DH, NT>::kCtas)
    k_cache8_part(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                  const __nv_bfloat16* __restrict__ q, const float* __restrict__ ks, const float* __restrict__ vs,
                  __nv_bfloat16* __restrict__ o, const int32_t* __restrict__ cu, const int32_t* __restrict__ lens,
                  Cut* __restrict__ cuts, float2* __restrict__ part_ml, float4* __restrict__ part_o, const Geom gm,
                  int* err) {
    using X = Ax<DH, NT>;
    constexpr int KW = DH >= 64 ? 4 : 2;                     // words of a load of K
    constexpr int KL = DH == 128 ? 2 : 1;                    // loads of K per key
    constexpr int VW = DH / 32;                              // words of a load of V, float4s of o of a lane and row
    extern __shared__ uint8_t smem_raw[];
    __shared__ int abort_flag;
    __shared__ Seg segs[2];
    __shared__ int64_t orow[2][8 * NT];                      // where a row of o lies,
    __shared__ int seen[2][8 * NT];                          // and the last position that it sees
    const uint32_t raw_base = smem_u32(smem_raw);
    const uint32_t sbase = (raw_base + 1023u) & ~1023u;
    uint8_t* sm = smem_raw + (sbase - raw_base);
    const uint32_t full = sbase + X::kBarOff, empty = full + 8 * X::kStages;
    const uint32_t qfull = empty + 8 * X::kStages, qempty = qfull + 16, bfull = qempty + 16, bempty = bfull + 8, ffull = bempty + 8;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 128) {
        abort_flag = 0;
        for (int i = 0; i < X::kStages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(qfull + 8 * i, 1);
            mbar_init(qempty + 8 * i, 4);
        }
        mbar_init(bfull, 4);
        mbar_init(bempty, 4);
        mbar_init(ffull, 4);
        fence_mbar_init();
        tma_prefetch_desc(&kmap);
        tma_prefetch_desc(&vmap);
    }
    __syncthreads();
    int st = 0;                                              // stage of the ring, and its phase
    uint32_t phase = 0;
    int sn = 0;                                              // segments so far
    pdl_wait();
    // (a join that is launched early sits on the SMs that are free first, many CTAs on few: 2 to 10 % slower)
    if (gm.whole) pdl_trigger();
    if (warp >= 4) {
        // ---------------------------------------------------------------- loads
        if (X::kSplit) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(X::kLoadRegs));
        if (warp > 4) return;
        // (the join has a record to read even if a wait gives up)
        if (lane == 0 && !gm.whole) cuts[blockIdx.x].pieces = 0;
        Walk w{0, 0, 0, 0};
        Seq s;
        int total = 0, runs = 0, u = 0;                      // units of all jobs; this run's next one
        bool bad = false;
        if (gm.whole == 2) {
            const int per = gm.Hkv * gm.row_blocks, kvh = (int)blockIdx.x % per / gm.row_blocks, rb = (int)blockIdx.x % gm.row_blocks;
            w.b = (int)blockIdx.x / per;
            s = get_seq(cu, lens, gm, w.b, bad);
            if (bad && lane == 0) raise_error(err, TFM_EINVAL);
            w.j = kvh * s.blocks + rb;
            if (rb < s.blocks) w.left = s.tiles + X::kPiece;
        } else {
            // Units of the sequences, added up (by this warp alone; the others wait for its first segment).
            int* cum = reinterpret_cast<int*>(sm + X::kCumOff);
            if (lane == 0) cum[0] = 0;
            for (int b0 = 0; b0 < gm.B; b0 += 128) {
                int x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {                // the loads of 128 sequences together
                    const int b = b0 + 32 * i + lane;
                    x[i] = 0;
                    if (b < gm.B) {
                        const Seq y = get_seq(cu, lens, gm, b, bad);
                        if (bad && blockIdx.x == 0) raise_error(err, TFM_EINVAL);
                        x[i] = (y.tiles + X::kPiece) * y.blocks * gm.Hkv;
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (b0 + 32 * i >= gm.B) break;
#pragma unroll
                    for (int d = 1; d < 32; d <<= 1) {
                        const int y = __shfl_up_sync(0xffffffffu, x[i], d);
                        if (lane >= d) x[i] += y;
                    }
                    x[i] += total;
                    if (b0 + 32 * i + lane < gm.B) cum[b0 + 32 * i + lane + 1] = x[i];
                    total = __shfl_sync(0xffffffffu, x[i], 31);
                }
            }
            __syncwarp();
            runs = run_count(total, gridDim.x);
            if ((int)blockIdx.x < runs && total > 0) {
                const int q = total / runs, r = total - q * runs;
                u = (int)blockIdx.x * q + min((int)blockIdx.x, r);
                w.left = q + ((int)blockIdx.x < r);
                int lo = 0, hi = gm.B;                       // cum[lo] <= u < cum[hi]
                while (hi - lo > 1) {
                    const int step = (hi - lo + 31) / 32;
                    const int b = lo + lane * step;
                    const int last = 31 - __clz(__ballot_sync(0xffffffffu, b < hi && cum[b] <= u) | 1u);
                    lo += last * step;
                    hi = min(hi, lo + step);
                }
                w.b = lo;
                s = get_seq(cu, lens, gm, lo, bad);
                w.j = (u - cum[lo]) / (s.tiles + X::kPiece);
                w.t = u - cum[lo] - w.j * (s.tiles + X::kPiece);
                if (gm.whole && w.t > 0) {                   // a job belongs to the run that it begins in
                    const int rest = s.tiles + X::kPiece - w.t;
                    w.left -= rest;
                    u += rest;
                    w.t = 0;
                    ++w.j;
                }
            }
        }
        const int* cum = reinterpret_cast<const int*>(sm + X::kCumOff);
        bool filled = false;                                 // every stage of the ring once
        const int cut_units = w.t;                           // of the job that the run begins in: units before the run
        for (;; ++sn) {
            const int place = sn & 1;
            // the next segment with tiles
            int t0 = 0, tiles = 0, j = 0, b = 0, first = 0;
            while (tiles <= 0 && w.left > 0) {
                if (w.j >= s.blocks * gm.Hkv) {
                    do ++w.b;
                    while (w.b < gm.B && cum[w.b + 1] == cum[w.b]);
                    if (w.b >= gm.B) break;                  // (a run ends before the jobs do, while the lengths stay)
                    s = get_seq(cu, lens, gm, w.b, bad);
                    w.j = 0;
                    if (s.blocks == 0) break;
                }
                const int units = gm.whole ? s.tiles + X::kPiece : min(s.tiles + X::kPiece - w.t, w.left);
                t0 = max(w.t - X::kPiece, 0);
                tiles = w.t + units - X::kPiece - t0;
                first = u - w.t + X::kPiece;                 // the unit of the job's first tile
                j = w.j;
                b = w.b;
                w.left -= units;
                u += units;
                w.t = 0;                                     // whatever comes next is another job
                ++w.j;
            }
            if (sn >= 2 && !warp_wait(qempty + 8 * place, (sn >> 1) + 1 & 1, err, &abort_flag)) return;
            if (tiles <= 0) {
                if (lane == 0) {
                    segs[place].tiles = 0;
                    mbar_arrive(qfull + 8 * place);
                }
                return;
            }
            const int kvh = s.blocks == 1 ? j : j / s.blocks, rb = j - kvh * s.blocks, bh = b * gm.Hkv + kvh;
            const int nrows = min(s.n * gm.G - rb * gm.block_rows, gm.block_rows);
            int row = bh * gm.max_seq + (s.tile0 + t0) * kTileKeys;
            // q first: it is needed first, and the first tiles are as much as memory gives in some microseconds
            const int rr = rb * gm.block_rows + lane, tok = gm.G == 1 ? rr : rr / gm.G, head = kvh * gm.G + rr - tok * gm.G;
            if (lane == 0) mbar_expect_tx(qfull + 8 * place, nrows * DH * 2);
            __syncwarp();
            if (lane < nrows)
                bulk_load(sbase + X::kQOff + place * X::kQ + lane * DH * 2,
                          q + ((int64_t)s.row0 + tok) * gm.sq_t + (int64_t)head * gm.sq_h, DH * 2, qfull + 8 * place);
            int done = 0;
            if (sn == 0 && lane == 0) {                      // the ring is empty: no waits
                for (; done < min(tiles, 2); ++done, row += kTileKeys) {
                    mbar_arrive_expect_tx(full + 8 * done, 2 * X::kTile);
                    tma_load_2d(sbase + done * 2 * X::kTile, &kmap, 0, row, full + 8 * done);
                    tma_load_2d(sbase + done * 2 * X::kTile + X::kTile, &vmap, 0, row, full + 8 * done);
                }
                st = done;
                if (st == X::kStages) st = 0, phase = 1, filled = true;
            }
            if (lane < X::kRows) {
                orow[place][lane] = ((int64_t)s.row0 + tok) * gm.so_t + (int64_t)head * gm.so_h;
                seen[place][lane] = lane < nrows ? s.len - s.n + tok : s.len - 1;
            }
            if (lane == 0)
                segs[place] = Seg{tiles, (s.tile0 + t0) * kTileKeys, s.len, s.n, bh, nrows,
                                  tiles == s.tiles ? -1 : (int)blockIdx.x * 2 + (sn > 0)};
            __syncwarp();
            if (lane == 0) mbar_arrive(qfull + 8 * place);
            if (sn == 0 && lane == 0 && !gm.whole) {
                // the boundary before this run cuts the job if some of its tiles lie before it
                Cut c{0, 0, 0, 0, s.row0, rb, kvh, nrows};
                if (cut_units > X::kPiece) {
                    const int end = min(first + s.tiles, total);
                    c.run0 = run_of(first, total, runs);
                    c.pieces = run_of(end - 1, total, runs) - c.run0 + 1;
                    if (c.pieces < 2) c.pieces = 0;
                    c.share = (int)blockIdx.x - c.run0 - 1;
                    c.place0 = 2 * c.run0 + (run_start(c.run0, total, runs) < first - X::kPiece);
                }
                cuts[blockIdx.x] = c;
            }
            bool ok = true;
            // (the first tile before a third is asked for: all CTAs ask at once, and memory serves the last ones too)
            if (lane == 0 && sn == 0) ok = mbar_wait(full, 0, err, &abort_flag);
            if (lane == 0 && ok)
                for (; done < tiles; ++done, row += kTileKeys) {
                    if (filled && !mbar_wait(empty + 8 * st, phase ^ 1, err, &abort_flag)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(full + 8 * st, 2 * X::kTile);
                    tma_load_2d(sbase + st * 2 * X::kTile, &kmap, 0, row, full + 8 * st);
                    tma_load_2d(sbase + st * 2 * X::kTile + X::kTile, &vmap, 0, row, full + 8 * st);
                    if (++st == X::kStages) st = 0, phase ^= 1, filled = true;
                }
            if (!__shfl_sync(0xffffffffu, (int)ok, 0)) return;
        }
    }
    // -------------------------------------------------------------------- rows
    // (no function is called behind the split, not by a wait either: it would not know of the registers it has)
    if (X::kSplit) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(X::kComputeRegs));
    const int kw = warp, g = lane >> 2, t = lane & 3;
    // where this lane reads, inside a tile: keys of the step's second half are 8 rows further, the
    // second half of a K row of 128 bytes is 64 bytes away (both keep the swizzle)
    const int kr = kw * 16 + kappa<DH>(g);
    const uint32_t koff = kr * DH + (DH >= 64 ? (t ^ ((kr >> X::kSwzShift) & X::kSwzMask)) * 16 : t * 8);
    uint32_t voff[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = kw * 16 + kappa<DH>(2 * t + i);
        voff[i] = X::kTile + r * DH + (DH == 128 ? (g ^ (r & 7)) * 16 : DH == 64 ? ((g >> 1) ^ ((r >> 1) & 3)) * 16 + (g & 1) * 8 : g * 4);
    }
    float4* buf = reinterpret_cast<float4*>(sm + X::kBufOff);
    float2* ml = reinterpret_cast<float2*>(sm + X::kMlOff);
    uint4* frag = reinterpret_cast<uint4*>(sm + X::kFragOff) + lane;          // [n][pair of words][lane]
    float4* rowf = reinterpret_cast<float4*>(sm + X::kRowOff);
    for (;; ++sn) {
        if (!warp_wait(qfull + 8 * (sn & 1), sn >> 1 & 1, err, &abort_flag)) return;
        const Seg& s = segs[sn & 1];
        const int tiles = s.tiles, len = s.len, news = s.n;
        if (tiles == 0) return;
        const int nrows = s.nrows;
        const float* ksp = ks + (int64_t)s.bh * gm.nblk;
        const float* vsp = vs + (int64_t)s.bh * gm.nblk;
        int key = s.key + kw * 16;
        const int last_blk = len > 0 ? (len - 1) >> gm.shift : 0;
        // The scales of 32 blocks, one in each lane, and of the next 32 (read past L1: as in k_cache8.cu).
        int blk0 = s.key >> gm.shift;
        // positions that some row sees, that every row sees
        const int any_lo = gm.window > 0 ? max(0, len - news - gm.window + 1) : 0;
        const int all_lo = gm.window > 0 ? len - gm.window : 0, all_hi = len - news;
        const int first_blk = any_lo >> gm.shift;
        const auto scales32 = [&](const float* at, int first) { return __ldcg(at + min(max(first + lane, first_blk), last_blk)); };
        float k32 = scales32(ksp, blk0), v32 = scales32(vsp, blk0);
        float k64 = scales32(ksp, blk0 + 32), v64 = scales32(vsp, blk0 + 32);
        // q: row r of the job is token r / G, head r % G.  Lane (g, t) holds row 8 n + g, for the products, of
        // what belongs to the rows 8 n + 2 t and + 1, whose scores it gets, in the arrays [n][2].
        // (kSharedQ: warp n prepares rows 8 n .. 8 n + 7 for all, in shared memory.)
        constexpr int NQ = X::kSharedQ ? 1 : NT;
        uint32_t qb[NQ][KL * KW][2];
        float qinv[NQ][2], qbias[NQ][2];
        int seen_hi[NQ][2];                                  // the last position that a row sees
        const auto prepare = [&](int nn, uint32_t (&qb)[KL * KW][2], float (&qinv)[2], float (&qbias)[2], int (&seen_hi)[2]) {
            const int r = 8 * nn + g;
            uint2 raw[KL * KW];
            if (r < nrows) {
                const uint8_t* at = sm + X::kQOff + (sn & 1) * X::kQ + r * DH * 2;
#pragma unroll
                for (int p = 0; p < KL; ++p) {
                    const uint4* a4 = reinterpret_cast<const uint4*>(at + p * 128 + t * (DH >= 64 ? 32 : 16));
#pragma unroll
                    for (int x = 0; x < KW / 2; ++x) {
                        const uint4 y = a4[x];
                        raw[p * KW + 2 * x] = make_uint2(y.x, y.y);
                        raw[p * KW + 2 * x + 1] = make_uint2(y.z, y.w);
                    }
                }
            } else {
#pragma unroll
                for (int x = 0; x < KL * KW; ++x) raw[x] = make_uint2(0, 0);
            }
            float top = 0.0f;
#pragma unroll
            for (int x = 0; x < KL * KW; ++x)
                top = fmaxf(top, fmaxf(fmaxf(fabsf(bf16_lo(raw[x].x)), fabsf(bf16_hi(raw[x].x))),
                                       fmaxf(fabsf(bf16_lo(raw[x].y)), fabsf(bf16_hi(raw[x].y)))));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // The row times the power of two that brings its largest element to [2^10, 2^12), of two such the one
            // that leaves an even power 2^r for the scores: f = k's scale scale_m 2^r takes them from the products' units.
            // 2^(r/2) is multiplied twice, so that on the way from the scale to f nothing is larger or smaller than both:
            // f is right wherever fp32 holds it (it stays below 2^107, as the header limits scale, q and k's scales).
            int e = (int)(__float_as_uint(top) >> 23);
            const bool infinite = e == 255;
            e = max(e, 11);
            int r2 = e - 127 + gm.scale_e + (E4M3 ? -10 : 14);
            e -= r2 & 1;
            r2 = min(max(r2 >> 1, -126), 127);
            // (of a row with an infinity every score is NaN: scores of minus infinity alone would be a row that sees nothing)
            const float mul = infinite ? __uint_as_float(0x7FFFFFFFu) : __uint_as_float((uint32_t)(264 - e) << 23);
            float sum = 0.0f;
#pragma unroll
            for (int x = 0; x < KL * KW; ++x) {
                const float y0 = bf16_lo(raw[x].x) * mul, y1 = bf16_hi(raw[x].x) * mul;
                const float y2 = bf16_lo(raw[x].y) * mul, y3 = bf16_hi(raw[x].y) * mul;
                const __half2 a = E4M3 ? __floats2half2_rn(y0, y1) : __floats2half2_rn(y0, y2);
                const __half2 b = E4M3 ? __floats2half2_rn(y2, y3) : __floats2half2_rn(y1, y3);
                qb[x][0] = *reinterpret_cast<const uint32_t*>(&a);
                qb[x][1] = *reinterpret_cast<const uint32_t*>(&b);
                const float2 fa = __half22float2(a), fb = __half22float2(b);
                sum += (fa.x + fa.y) + (fb.x + fb.y);
            }
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int from = (2 * t + j) * 4;            // a lane of that row
                qinv[j] = __uint_as_float((uint32_t)(__shfl_sync(0xffffffffu, r2, from) + 127) << 23);
                qbias[j] = E4M3 ? 0.0f : __shfl_sync(0xffffffffu, sum, from) * -0x1p-17f;      // 128 of the codes' 2^-24
                seen_hi[j] = seen[sn & 1][8 * nn + 2 * t + j];
            }
        };
        if constexpr (X::kSharedQ) {
            if (kw < NT) {
                prepare(kw, qb[0], qinv[0], qbias[0], seen_hi[0]);
#pragma unroll
                for (int y = 0; y < KL * KW; y += 2)
                    frag[(kw * KL * KW + y) * 16] = make_uint4(qb[0][y][0], qb[0][y][1], qb[0][y + 1][0], qb[0][y + 1][1]);
                if (g == 0)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        rowf[8 * kw + 2 * t + j] = make_float4(qinv[0][j], qbias[0][j], __int_as_float(seen_hi[0][j]), 0.0f);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(ffull);
            if (!warp_wait(ffull, sn & 1, err, &abort_flag)) return;
        } else {
#pragma unroll
            for (int n = 0; n < NT; ++n) prepare(n, qb[n], qinv[n], qbias[n], seen_hi[n]);
        }
        // acc[n][2 x + h]: rows 8 n + 2 t (elements 0, 2) and + 1 (1, 3), coordinates g DH / 8 + 4 x + 2 h (0, 1) and + 1
        float acc[NT][2 * VW][4];
        float m[NT][2], l[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int i = 0; i < 2 * VW; ++i) acc[n][i][0] = acc[n][i][1] = acc[n][i][2] = acc[n][i][3] = 0.0f;
            m[n][0] = m[n][1] = -3.402823466e38f;
            l[n][0] = l[n][1] = 0.0f;
        }
        // Weights times values are summed as they are (int8 products are in 2^-24), up to scales of kLarge: weights of up to 2^15
        // and 2^31 keys then stay within fp32.  From the first larger scale on they are summed in units of 2^64.  (32 blocks are
        // looked at together, outside the loop over their tiles: looked at inside, drafted tokens took 23.3 us for 22.2.)
        constexpr float kUnit = E4M3 ? 1.0f : 0x1p24f, kLarge = 0x1p64f, kDown = 0x1p-64f;
        bool large = false;
        const auto step = [&](auto edge, float ksc, float vsc) {
            constexpr bool EDGE = decltype(edge)::value;
            const uint8_t* kt = sm + st * 2 * X::kTile;
            float c[NT][4];
            {
                uint32_t kd[2][KL][KW];
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int p = 0; p < KL; ++p) words<KW>(kt + (koff ^ (p * 64)) + i * 8 * DH, kd[i][p]);
                float c2[4] = {0.0f, 0.0f, 0.0f, 0.0f};   // a second chain of sums: half the latency
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float b0 = 0.0f, b1 = 0.0f;
                    if constexpr (!E4M3) {
                        if constexpr (X::kSharedQ) b0 = rowf[8 * n + 2 * t].y, b1 = rowf[8 * n + 2 * t + 1].y;
                        else b0 = qbias[n][0], b1 = qbias[n][1];
                    }
                    c[n][0] = c[n][2] = b0;
                    c[n][1] = c[n][3] = b1;
                }
#pragma unroll
                for (int p = 0; p < KL; ++p)
#pragma unroll
                    for (int x = 0; x < KW; x += 2) {
                        uint32_t a[2][4];                 // keys g, g + 8
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            key_halves<E4M3>(kd[0][p][x + z], a[z][0], a[z][2]);
                            key_halves<E4M3>(kd[1][p][x + z], a[z][1], a[z][3]);
                        }
                        const int y = p * KW + x;
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            uint4 b;
                            if constexpr (X::kSharedQ) b = frag[(n * KL * KW + y) * 16];
                            else b = make_uint4(qb[n][y][0], qb[n][y][1], qb[n][y + 1][0], qb[n][y + 1][1]);
                            float(&d)[4] = NT == 1 ? c2 : c[n];
                            mma16816(c[n], a[0], b.x, b.y, c[n][0], c[n][1], c[n][2], c[n][3]);
                            mma16816(d, a[1], b.z, b.w, d[0], d[1], d[2], d[3]);
                        }
                    }
                if (NT == 1)
#pragma unroll
                    for (int i = 0; i < 4; ++i) c[0][i] += c2[i];
            }
            const int p0 = key + kappa<DH>(g);
            bool up = false;
            float top[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float inv;
                    int hi = 0;
                    if constexpr (X::kSharedQ) {
                        const float4 w = rowf[8 * n + 2 * t + j];
                        inv = w.x;
                        hi = __float_as_int(w.z);
                    } else {
                        inv = qinv[n][j];
                        hi = seen_hi[n][j];
                    }
                    const float f = ksc * inv * inv;                       // (ksc: times scale_m)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float& y = c[n][2 * i + j];
                        y *= f;
                        if (EDGE && (p0 + 8 * i > hi || (gm.window > 0 && p0 + 8 * i <= hi - gm.window)))
                            y = -INFINITY;
                    }
                    top[n][j] = fmaxf(c[n][j], c[n][2 + j]);
                    up = up || top[n][j] > m[n][j] + 8.0f;
                }
            if (__any_sync(0xffffffffu, up)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float y = top[n][j];
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, d));
                        y = fmaxf(y, m[n][j]);
                        const float keep = ex2(m[n][j] - y);
                        m[n][j] = y;
                        l[n][j] *= keep;
#pragma unroll
                        for (int i = 0; i < 2 * VW; ++i) {
                            acc[n][i][j] *= keep;
                            acc[n][i][2 + j] *= keep;
                        }
                    }
            }
            uint32_t pb[NT][2];                           // weights of keys 2 t, 2 t + 1 (+ 8) for row g
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float b0 = m[n][0] - 7.0f, b1 = m[n][1] - 7.0f;
                float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const __half2 h = __floats2half2_rn(ex2(c[n][2 * i] - b0), ex2(c[n][2 * i + 1] - b1));
                    const float2 p = __half22float2(h);   // summed as they are multiplied
                    s0 += p.x;
                    s1 += p.y;
                    pb[n][i] = transposed(*reinterpret_cast<const uint32_t*>(&h));
                }
                l[n][0] += s0;
                l[n][1] += s1;
            }
            // What the codes' bias of 128 adds to the products below, taken off inside them, so that what is summed over the
            // steps has none: -2^-17 (in fp16, as the codes) times the sum of the weights, in the lanes that need it.
            float z[NT][4] = {};
            if constexpr (!E4M3) {
                const uint32_t bias[4] = {0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u};
#pragma unroll
                for (int n = 0; n < NT; ++n) mma16816(z[n], bias, pb[n][0], pb[n][1], 0.0f, 0.0f, 0.0f, 0.0f);
            }
            uint32_t vw[4][VW];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                words<VW>(kt + voff[i & 1] + (i >> 1) * 8 * DH, vw[i]);
                if (E4M3 && EDGE) {                    // a code that nothing sees may be a NaN
                    const int p = key + (i >> 1) * 8 + kappa<DH>(2 * t + (i & 1));
                    if (p >= len || p < any_lo)
#pragma unroll
                        for (int x = 0; x < VW; ++x) vw[i][x] = 0;
                }
            }
#pragma unroll
            for (int x = 0; x < VW; ++x) {
                uint32_t v0[4], v1[4];                    // keys 2 t, 2 t + 1; 8 further
                value_halves<E4M3>(vw[0][x], vw[1][x], v0);
                value_halves<E4M3>(vw[2][x], vw[3][x], v1);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t a[4] = {v0[2 * h], v0[2 * h + 1], v1[2 * h], v1[2 * h + 1]};
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float d[4];
                        mma16816(d, a, pb[n][0], pb[n][1], z[n][0], z[n][1], z[n][2], z[n][3]);
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[n][2 * x + h][j] = fmaf(vsc, d[j], acc[n][2 * x + h][j]);
                    }
                }
            }
        };
        // 32 blocks at a time, of which a tile has at most 4
        int end = min(tiles, ((32 << gm.shift) - (s.key - (blk0 << gm.shift))) / kTileKeys);
        for (int tile = 0;;) {
            if (!large && __any_sync(0xffffffffu, fabsf(v32) > kLarge)) {
                large = true;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 2 * VW; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) acc[n][i][j] *= kDown;
            }
            v32 *= large ? kUnit * kDown : kUnit;
            for (; tile < end; ++tile, key += kTileKeys) {
                const int blk = min(key >> gm.shift, last_blk) - blk0;
                const float ksc = __shfl_sync(0xffffffffu, k32, blk) * gm.scale_m, vsc = __shfl_sync(0xffffffffu, v32, blk);
                if (!warp_wait(full + 8 * st, phase, err, &abort_flag)) return;
                // a step whose keys every row sees needs no masks
                if (key >= all_lo && key + 15 <= all_hi) step(std::false_type{}, ksc, vsc);
                else if (key < len && key + 16 > any_lo) step(std::true_type{}, ksc, vsc);
                __syncwarp();
                if (lane == 0) mbar_arrive(empty + 8 * st);
                if (++st == X::kStages) st = 0, phase ^= 1;
            }
            if (tile == tiles) break;
            end = min(tiles, tile + (32 << gm.shift) / kTileKeys);
            blk0 += 32;
            k32 = k64;
            v32 = v64;
            k64 = scales32(ksp, blk0 + 32);
            v64 = scales32(vsp, blk0 + 32);
        }
        // The four warps' parts, added up, 8 rows at a time.
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int pass = sn * NT + n;
            if (pass > 0 && !warp_wait(bempty, pass + 1 & 1, err, &abort_flag)) return;      // the last ones have been read
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) {
                    l[n][j] += __shfl_xor_sync(0xffffffffu, l[n][j], d);
                }
                const int r = 2 * t + j;
#pragma unroll
                for (int x = 0; x < VW; ++x) {
                    const float4 v = make_float4(acc[n][2 * x][j], acc[n][2 * x][2 + j], acc[n][2 * x + 1][j], acc[n][2 * x + 1][2 + j]);
                    buf[kw * 8 * (DH / 4) + buf_at<DH>(r, g * VW + x)] = v;
                }
                // (a part in units of 2^64 has a negative sum)
                if (g == 0) ml[kw * 8 + r] = make_float2(m[n][j], large ? -l[n][j] : l[n][j]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bfull);
            if (!warp_wait(bfull, pass & 1, err, &abort_flag)) return;
            for (int e = tid; e < 8 * (DH / 4); e += 128) {
                const int r = e / (DH / 4), f = e % (DH / 4);
                if (8 * n + r >= nrows) break;
                float2 x[4];
                float top = -3.402823466e38f, least = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[i] = ml[i * 8 + r];
                    top = fmaxf(top, x[i].x);
                    least = fminf(least, x[i].y);
                }
                float sum = 0.0f;
                float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float k = ex2(x[i].x - top);
                    const float4 y = buf[i * 8 * (DH / 4) + buf_at<DH>(r, f)];
                    sum = fmaf(k, fabsf(x[i].y), sum);
                    if (least < 0.0f && x[i].y >= 0.0f) k *= kDown;
                    v.x = fmaf(k, y.x, v.x);
                    v.y = fmaf(k, y.y, v.y);
                    v.z = fmaf(k, y.z, v.z);
                    v.w = fmaf(k, y.w, v.w);
                }
                if (s.piece < 0) {
                    float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                    if (least < 0.0f) inv *= 1.0f / kDown;
                    __nv_bfloat16* at = o + orow[sn & 1][8 * n + r] + f * 4;
                    *reinterpret_cast<uint2*>(at) = make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
                } else {
                    const int64_t pr = (int64_t)s.piece * gm.block_rows + 8 * n + r;
                    part_o[pr * (DH / 4) + f] = v;
                    if (f == 0) part_ml[pr] = make_float2(top, least < 0.0f ? -sum : sum);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bempty);
        }
        if (lane == 0) mbar_arrive(qempty + 8 * (sn & 1));
    }
}

// Joins the pieces of the jobs that runs cut.  A job of P pieces has P - 1 boundaries of runs inside
// it; CTA i takes that before run i + 1 and with it a share of the job's rows, in
// float4s, kJoin of them at least.  The pieces are taken by the groups of threads in turn and
// added in an order that depends on their number alone.  Pieces in units of 2^64 (their sums are negative) bring the others to
// these units.  (256 threads: drafted tokens 23.4 for 21.9 us, windowed 20.5 for 20.0;
// 64: 64 chats 32.0 for 30.6; eight entries at least: 131072 positions 28.6 for 28.1.)
constexpr int kJoin = 4, kJoinThreads = 128;
template <int DH>
__global__ void __launch_bounds__(kJoinThreads)
    k_cache8_join(const Cut* __restrict__ cuts, const float2* __restrict__ part_ml, const float4* __restrict__ part_o,
                  __nv_bfloat16* __restrict__ o, const Geom gm) {
    constexpr int F = DH / 4;
    constexpr float kDown = 0x1p-64f;
    __shared__ float4 sum_o[kJoinThreads];
    __shared__ float2 sum_ml[kJoinThreads];
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x;
    const int4* at4 = reinterpret_cast<const int4*>(cuts + blockIdx.x + 1);
    const int4 c0 = __ldcg(at4), c1 = __ldcg(at4 + 1);
    const Cut h{c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
    if (h.pieces == 0) return;
    const int pieces = h.pieces, all = h.nrows * F;
    const int shares = (pieces - 1) * (int)gridDim.y;
    const int share = max(kJoin, shares == 1 ? all : (all + shares - 1) / shares);
    const int e0 = (h.share * (int)gridDim.y + (int)blockIdx.y) * share, e1 = min(all, e0 + share);
    // entries side by side, a power of two of them; the other threads share the pieces
    int width = kJoin;
    while (width < share && width < kJoinThreads) width <<= 1;
    const int groups = kJoinThreads / width, gr = tid / width;
    for (int at = e0; at < e1; at += width) {
        const int e = at + tid % width;
        const int r = e / F, f = e % F;
        float top = -3.402823466e38f, sum = 0.0f;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        bool large = false;
        for (int p0 = gr; p0 < pieces && e < e1; p0 += 4 * groups) {         // four at a time: their loads together
            float2 x[4];
            float4 y[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int p = p0 + k * groups;
                x[k] = make_float2(-3.402823466e38f, 0.0f);
                y[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (p < pieces) {
                    const int64_t pr = (int64_t)(p == 0 ? h.place0 : 2 * (h.run0 + p)) * gm.block_rows + r;
                    x[k] = part_ml[pr];
                    y[k] = part_o[pr * F + f];
                }
            }
            const float nt = fmaxf(fmaxf(fmaxf(x[0].x, x[1].x), fmaxf(x[2].x, x[3].x)), top), k0 = ex2(top - nt);
            sum *= k0;
            v = make_float4(v.x * k0, v.y * k0, v.z * k0, v.w * k0);
            if (large || fminf(fminf(x[0].y, x[1].y), fminf(x[2].y, x[3].y)) < 0.0f) {
                if (!large) v = make_float4(v.x * kDown, v.y * kDown, v.z * kDown, v.w * kDown);
                large = true;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (x[k].y >= 0.0f) y[k] = make_float4(y[k].x * kDown, y[k].y * kDown, y[k].z * kDown, y[k].w * kDown);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float w = ex2(x[k].x - nt);
                sum = fmaf(w, fabsf(x[k].y), sum);
                v = make_float4(fmaf(w, y[k].x, v.x), fmaf(w, y[k].y, v.y), fmaf(w, y[k].z, v.z), fmaf(w, y[k].w, v.w));
            }
            top = nt;
        }
        // a warp's groups, then the warps, whose units are one if any is large
        const bool was = large;
        large = __syncthreads_or(large);
        if (large && !was) v = make_float4(v.x * kDown, v.y * kDown, v.z * kDown, v.w * kDown);
        for (int d = width; d < 32; d <<= 1) {
            const float t1 = __shfl_xor_sync(0xffffffffu, top, d), s1 = __shfl_xor_sync(0xffffffffu, sum, d);
            const float4 y = make_float4(__shfl_xor_sync(0xffffffffu, v.x, d), __shfl_xor_sync(0xffffffffu, v.y, d),
                                         __shfl_xor_sync(0xffffffffu, v.z, d), __shfl_xor_sync(0xffffffffu, v.w, d));
            const float nt = fmaxf(top, t1), k0 = ex2(top - nt), k1 = ex2(t1 - nt);
            sum = sum * k0 + s1 * k1;
            v = make_float4(v.x * k0 + y.x * k1, v.y * k0 + y.y * k1, v.z * k0 + y.z * k1, v.w * k0 + y.w * k1);
            top = nt;
        }
        sum_o[tid] = v;
        sum_ml[tid] = make_float2(top, sum);
        __syncthreads();
        if (gr == 0 && e < e1) {
            const int step = width < 32 ? 32 : width;
#pragma unroll 4
            for (int k = step; k < kJoinThreads; k += step) top = fmaxf(top, sum_ml[k + tid].x);
            float den = 0.0f;
            v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
            for (int k = 0; k < kJoinThreads; k += step) {
                const float2 x = sum_ml[k + tid];
                const float w = ex2(x.x - top);
                const float4 y = sum_o[k + tid];
                den = fmaf(w, x.y, den);
                v = make_float4(fmaf(w, y.x, v.x), fmaf(w, y.y, v.y), fmaf(w, y.z, v.z), fmaf(w, y.w, v.w));
            }
            float inv = den == 0.0f ? 0.0f : 1.0f / den;
            if (large) inv *= 1.0f / kDown;
            const int rr = h.rb * gm.block_rows + r;
            __nv_bfloat16* to = o + ((int64_t)h.row0 + rr / gm.G) * gm.so_t + (int64_t)(h.kvh * gm.G + rr % gm.G) * gm.so_h + f * 4;
            *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
        }
        __syncthreads();
    }
}

// Rows of a job by the rows that max_new tokens of a kv head have: all of up to 32; more are blocks
// of 32, each of which reads the tiles.  (Blocks of 8 where the caches are small: launch_cache8_attention.)
int job_rows(int group, int max_new) {
    const int rows = group * max_new;
    return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 24 ? 24 : 32;
}

// Units that a job has at most.
int job_units(const Cache8AttnArgs& a, int piece) {
    const int keys = a.window > 0 && a.window + a.max_new < a.max_seq ? a.window + a.max_new : a.max_seq;
    return (keys + kTileKeys - 2) / kTileKeys + 1 + piece;
}

struct Space {
    size_t cuts, ml, o, bytes;
};
Space space(int rows, int dh) {
    Space s;
    const size_t runs = kMaxRuns;
    s.cuts = 0;
    s.ml = s.cuts + runs * sizeof(Cut);
    s.o = s.ml + 2 * runs * rows * sizeof(float2);
    s.bytes = s.o + 2 * runs * rows * dh * sizeof(float);
    return s;
}

template <bool E4M3, int DH, int NT>
cudaError_t launch_part(const Cache8AttnArgs& a, const CUtensorMap& km, const CUtensorMap& vm, Geom gm, cudaStream_t st) {
    using X = Ax<DH, NT>;
    static std::atomic<uint64_t> done{0};
    const int smem = X::kBase + 4 * (a.B + 1);
    // sequences beyond those that leave room for kCtas have fewer CTAs per SM; 4096 still fit
    cudaError_t e = allow_smem(done, k_cache8_part<E4M3, DH, NT>, X::kBase + 4 * 4097);
    if (e != cudaSuccess) return e;
    if (X::kSplit) {
        // the warps that take registers over would wait for ever if the launch had fewer than they count on
        static std::atomic<int> regs{0};
        if (regs.load(std::memory_order_relaxed) == 0) {
            cudaFuncAttributes f;
            e = cudaFuncGetAttributes(&f, k_cache8_part<E4M3, DH, NT>);
            if (e != cudaSuccess) return e;
            regs.store(f.numRegs, std::memory_order_relaxed);
        }
        if (regs.load(std::memory_order_relaxed) * 2 < X::kComputeRegs + X::kLoadRegs) return cudaErrorInvalidDeviceFunction;
    }
    const int ctas = sm_count() * X::kCtas < kMaxRuns ? sm_count() * X::kCtas : kMaxRuns;
    char* ws = static_cast<char*>(a.ws);
    const Space sp = space(gm.block_rows, DH);
    Cut* cuts = reinterpret_cast<Cut*>(ws + sp.cuts);
    float2* ml = reinterpret_cast<float2*>(ws + sp.ml);
    float4* po = reinterpret_cast<float4*>(ws + sp.o);
    // A few tiles more in a row are faster than a second kernel: where no job can have more than kWhole
    // units, none is cut.
    const int64_t jobs = (int64_t)a.B * a.Hkv * gm.row_blocks;
    gm.whole = job_units(a, X::kPiece) > kWhole ? 0 : jobs > ctas ? 1 : 2;
    e = launch_pdl(k_cache8_part<E4M3, DH, NT>, dim3(gm.whole == 2 ? (unsigned)jobs : ctas), dim3(X::kThreads), smem, st, km, vm,
                   static_cast<const __nv_bfloat16*>(a.q), a.ks, a.vs, static_cast<__nv_bfloat16*>(a.o), a.cu, a.lens, cuts,
                   ml, po, gm, device_error_word());
    if (e != cudaSuccess || gm.whole) return e;
    return launch_pdl(k_cache8_join<DH>, dim3(ctas - 1, gm.block_rows / 8), dim3(kJoinThreads), 0, st,
                      static_cast<const Cut*>(cuts), static_cast<const float2*>(ml), static_cast<const float4*>(po),
                      static_cast<__nv_bfloat16*>(a.o), gm);
}

template <bool E4M3, int DH>
cudaError_t by_rows(const Cache8AttnArgs& a, const CUtensorMap& km, const CUtensorMap& vm, const Geom& gm, cudaStream_t st) {
    switch (gm.block_rows) {
        case 8: return launch_part<E4M3, DH, 1>(a, km, vm, gm, st);
        case 16: return launch_part<E4M3, DH, 2>(a, km, vm, gm, st);
        case 24: return launch_part<E4M3, DH, 3>(a, km, vm, gm, st);
        default: return launch_part<E4M3, DH, 4>(a, km, vm, gm, st);
    }
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
    // Where even full caches are no more than 16 units for each CTA, rows on more CTAs are faster than tiles read once: 5
    // tokens of 16/4 x 128 over 300 positions 10.7 -> 6.9 us, of 4 sequences over 4000 13.9 -> 12.4 (10 units), over 8192
    // 15.9 -> 16.3 (21).  (Full caches: in one of 8192 positions 5 tokens over 300 take 9.6 us, in one of 131072 13.7.)
    const int64_t jobs8 = (int64_t)a.B * a.Hkv * ((gm.G * a.max_new + 7) / 8);
    const int piece = a.dh == 32 ? Ax<32, 1>::kPiece : Ax<64, 1>::kPiece, ctas8 = a.dh == 128 ? Ax<128, 1>::kCtas : Ax<64, 1>::kCtas;
    if (jobs8 * job_units(a, piece) <= (int64_t)16 * ctas8 * sm_count()) gm.block_rows = 8;
    gm.row_blocks = (gm.G * a.max_new + gm.block_rows - 1) / gm.block_rows;
    gm.scale_m = (float)std::frexp((double)a.scale * 1.4426950408889634, &gm.scale_e);
    gm.sq_t = a.strides[0];
    gm.sq_h = a.strides[1];
    gm.so_t = a.strides[2];
    gm.so_h = a.strides[3];
    *e = a.e4m3 ? by_dh<true>(a, km, vm, gm, st) : by_dh<false>(a, km, vm, gm, st);
    return TFM_OK;
}

}  // namespace tfm
