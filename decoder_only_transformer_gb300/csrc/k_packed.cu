// k_packed.cu - causal attention over packed sequences of different lengths.
//
// o_i = sum_j p_ij v_j with p_i = softmax_j(scale q_i . k_j) over the keys of
// row i's own sequence, max(start, i - window + 1) <= j <= i (window 0: from the
// sequence's start); query head h reads kv head h / (H / Hkv).
#include <climits>

#include "common.cuh"
#include "internal.h"

namespace tfm {

namespace {

// Rows [start, start + len) of sequence b, or an empty range for offsets that
// decrease or leave [0, T].
struct SeqRange {
    int start, len;
};
__device__ __forceinline__ SeqRange seq_range(int s, int e, int T) {
    const bool ok = s >= 0 && s <= e && e <= T;
    return SeqRange{ok ? s : 0, ok ? e - s : 0};
}

struct PackedStrides {
    int64_t qt, qh, kt, kh, vt, vh, ot, oh;
};

// Block t of sequence b has the slot cu[b] / rows + b + t, so that blocks are found
// without a scan: slots of different sequences never meet (a sequence of L rows from
// row c on has at most (c + L) / rows - c / rows + 1 blocks), and the sequence of a
// slot is the last b with cu[b] / rows + b <= slot, which grows with b.  By a warp,
// 32 probes at a time; -1: none.
__device__ __forceinline__ int sequence_of(const int32_t* __restrict__ cu, int n_seq, int rows, int slot) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = n_seq;                             // the answer + 1 lies in [lo, lo + n]
    while (n > 0) {
        const int step = (n + 31) / 32, b = lo + lane * step;
        const bool in = lane * step < n && __ldg(cu + b) / rows + b <= slot;
        const int k = __popc(__ballot_sync(0xffffffffu, in));
        if (k == 0) break;
        const int from = (k - 1) * step;               // probe k - 1 holds, probe k does not
        lo += from + 1;
        n = min(n - from, step) - 1;
    }
    return lo - 1;
}

// ------------------------------------------------------------------ fp32
// CUDA cores: tf32 keeps 10 mantissa bits and fp32 mode is there for fp32 results.
// A CTA takes 32 query rows of a head against key tiles of 64, 128 threads with 4 x 4
// scores and 4 rows x 4 or more columns of the output each (below d_head 64 the
// threads that this leaves share the keys out and add up at the end: with one or two
// columns each the loads of P and V bound it), K and V tiles copied asynchronously one ahead.
// Per 16-byte step of the products a warp reads 12 shared-memory wavefronts for
// 2048 FMAs (16 cycles), so the FMA pipe is what bounds a long sequence at a large d_head.
// At d_head 16 the instructions beside the products do, ~600 of ~800 a warp and tile, at
// half of the issue slots: 19 us for 64 lines of up to 300 tokens at 4 x 16.  (A division
// per copy, the accurate exponential and the scale as a product of its own: 24 us; one
// warp per row 291; blocks of 64 rows 30, as more of them lies above the diagonal and the
// last ones end later.)
constexpr int kF32Rows = 32, kF32Keys = 64, kF32Threads = 128;

__device__ __forceinline__ void cp_async16(float* dst, const float* src, bool in) {
    const int bytes = in ? 16 : 0;                     // 0: zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(bytes)
                 : "memory");
}

template <int DP>
struct F32Smem {
    static constexpr int kPitch = DP + 4;              // floats; rows four banks apart
    static constexpr int kQ = 0, kK = kF32Rows * kPitch, kV = kK + 2 * kF32Keys * kPitch;
    static constexpr int kP = kV + 2 * kF32Keys * kPitch;             // [key][row]
    static constexpr int kBytes = (kP + kF32Keys * (kF32Rows + 4)) * 4;
};

template <int DP>
__global__ void __launch_bounds__(kF32Threads, DP <= 64 ? 4 : 1) k_packed_f32(const float* __restrict__ q, const float* __restrict__ k,
                                                    const float* __restrict__ v, float* __restrict__ o,
                                                    const int32_t* __restrict__ cu, int n_seq, int T, int slots,
                                                    int H, int group, int dh, PackedStrides sd,
                                                    float scale_log2, int window, int* err) {
    using Sm = F32Smem<DP>;
    constexpr int NC = DP < 64 ? 4 : DP / 16;          // output columns per thread
    constexpr int KG = DP < 64 ? 64 / DP : 1;          // threads that share a column group's keys
    extern __shared__ __align__(16) float sm[];
    pdl_wait();
    pdl_trigger();
    if (blockIdx.x == 0)
        for (int b = threadIdx.x; b < n_seq; b += kF32Threads) {
            const int s = cu[b], e = cu[b + 1];
            if (s < 0 || s > e || e > T) raise_error(err, TFM_EINVAL);
        }
    // the last blocks of a sequence, which see the most keys, first
    const int slot = slots - 1 - (int)(blockIdx.x / (unsigned)H), h = (int)(blockIdx.x % (unsigned)H), g = h / group;
    const int b = sequence_of(cu, n_seq, kF32Rows, slot);
    if (b < 0) return;
    const SeqRange sr = seq_range(__ldg(cu + b), __ldg(cu + b + 1), T);
    const int row0 = (slot - (sr.start / kF32Rows + b)) * kF32Rows;
    if (row0 < 0 || row0 >= sr.len) return;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int cg = tx % (16 / KG), kg = tx / (16 / KG);
    const int d4 = dh / 4;
    const float* kb = k + sr.start * sd.kt + g * sd.kh;
    const float* vb = v + sr.start * sd.vt + g * sd.vh;
    const int j0 = (window > 0 && row0 - window + 1 > 0) ? (row0 - window + 1) / kF32Keys : 0;
    const int j1 = (row0 + kF32Rows - 1) / kF32Keys;                 // key tiles j0..j1
    const int first_r = tid / d4, first_c = tid - first_r * d4;
    const int step_r = kF32Threads / d4, step_c = kF32Threads - step_r * d4;
    auto load_kv = [&](int j) {
        float* ks = sm + Sm::kK + (j & 1) * kF32Keys * Sm::kPitch;
        float* vs = sm + Sm::kV + (j & 1) * kF32Keys * Sm::kPitch;
        int r = first_r, c = first_c;
        while (r < kF32Keys) {
            const int key = j * kF32Keys + r;
            const bool in = key < sr.len;
            const int64_t at = in ? key : 0;
            cp_async16(ks + r * Sm::kPitch + 4 * c, kb + at * sd.kt + 4 * c, in);
            cp_async16(vs + r * Sm::kPitch + 4 * c, vb + at * sd.vt + 4 * c, in);
            r += step_r;
            c += step_c;
            if (c >= d4) {
                c -= d4;
                ++r;
            }
        }
    };
    const float* qb = q + (int64_t)(sr.start + row0) * sd.qt + h * sd.qh;
    for (int i = tid; i < kF32Rows * d4; i += kF32Threads) {
        const int r = i / d4, c = (i - r * d4) * 4;
        const bool in = row0 + r < sr.len;
        cp_async16(sm + Sm::kQ + r * Sm::kPitch + c, qb + (in ? r : 0) * sd.qt + c, in);
    }
    load_kv(j0);
    asm volatile("cp.async.commit_group;" ::: "memory");
    float m[4], l[4];
    uint64_t acc[4][NC / 2];                           // column pairs
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < NC / 2; ++c) acc[i][c] = 0ull;
    }
    float* ps = sm + Sm::kP;                           // [key][row]
    for (int j = j0; j <= j1; ++j) {
        if (j < j1) load_kv(j + 1);
        asm volatile("cp.async.commit_group;" ::: "memory");
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncthreads();
        const float* qs = sm + Sm::kQ + ty * 4 * Sm::kPitch;
        const float* ks = sm + Sm::kK + (j & 1) * kF32Keys * Sm::kPitch + tx * Sm::kPitch;
        const float* vs = sm + Sm::kV + (j & 1) * kF32Keys * Sm::kPitch + cg * 4;
        // Packed pairs: even and odd coordinates of a score side by side, added at the end.
        uint64_t s2[4][4];                             // rows 4 ty + i, keys tx + 16 e
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) s2[i][e] = 0ull;
#pragma unroll 2
        for (int c = 0; c < d4; ++c) {
            ulonglong2 qa[4], ka[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) qa[i] = *reinterpret_cast<const ulonglong2*>(qs + i * Sm::kPitch + 4 * c);
#pragma unroll
            for (int e = 0; e < 4; ++e) ka[e] = *reinterpret_cast<const ulonglong2*>(ks + 16 * e * Sm::kPitch + 4 * c);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) s2[i][e] = f2_fma(qa[i].y, ka[e].y, f2_fma(qa[i].x, ka[e].x, s2[i][e]));
        }
        float s[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float even, odd;
                f2_unpack(s2[i][e], even, odd);
                s[i][e] = even + odd;
            }
        // keys of this tile that row i sees: [lo, hi]
        const int k0 = j * kF32Keys;
        const bool masked = k0 + kF32Keys - 1 > row0 || (window > 0 && k0 < row0 + kF32Rows - window);
        if (masked)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int hi = row0 + ty * 4 + i - k0 - tx, lo = window > 0 ? hi - window + 1 : INT_MIN;
#pragma unroll
                for (int e = 0; e < 4; ++e) s[i][e] = 16 * e > hi || 16 * e < lo ? -INFINITY : s[i][e];
            }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float mx = fmaxf(fmaxf(s[i][0], s[i][1]), fmaxf(s[i][2], s[i][3]));
#pragma unroll
            for (int w = 8; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
            const float mn = fmaxf(m[i], mx * scale_log2), ref = mn == -INFINITY ? 0.f : -mn;
            const float corr = fast_exp2(m[i] + ref);  // m = -inf: 0
            m[i] = mn;
            l[i] *= corr;
            const uint64_t corr2 = f2_pack(corr, corr);
#pragma unroll
            for (int c = 0; c < NC / 2; ++c) acc[i][c] = f2_fma(acc[i][c], corr2, 0ull);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[i][e] = fast_exp2(fmaf(s[i][e], scale_log2, ref));
                l[i] += s[i][e];
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            *reinterpret_cast<float4*>(ps + (tx + 16 * e) * (kF32Rows + 4) + ty * 4) =
                make_float4(s[0][e], s[1][e], s[2][e], s[3][e]);
        __syncthreads();
        auto add = [&](int key, bool check) {
            const float4 p4 = *reinterpret_cast<const float4*>(ps + key * (kF32Rows + 4) + ty * 4);
            const float p[4] = {p4.x, p4.y, p4.z, p4.w};
            uint64_t x[NC / 2];
#pragma unroll
            for (int c = 0; c < NC; c += 4) {
                const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(vs + key * Sm::kPitch + 16 * c);
                x[c / 2] = w.x;
                x[c / 2 + 1] = w.y;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                // a weight of zero does not make a product zero if the value is not finite
                const int hi = row0 + ty * 4 + i - k0;
                if (check && (key > hi || (window > 0 && key < hi - window + 1))) continue;
                const uint64_t p2 = f2_pack(p[i], p[i]);
#pragma unroll
                for (int c = 0; c < NC / 2; ++c) acc[i][c] = f2_fma(p2, x[c], acc[i][c]);
            }
        };
        if (masked) {
#pragma unroll 2
            for (int key = kg; key < kF32Keys; key += KG) add(key, true);
        } else {
#pragma unroll 4
            for (int key = kg; key < kF32Keys; key += KG) add(key, false);
        }
        __syncthreads();                               // this tile's buffers are free
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float sum = l[i];
#pragma unroll
        for (int w = 8; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
        float out[NC];
#pragma unroll
        for (int c = 0; c < NC / 2; ++c) f2_unpack(acc[i][c], out[2 * c], out[2 * c + 1]);
#pragma unroll
        for (int w = 8; w > 16 / KG / 2; w >>= 1)
#pragma unroll
            for (int c = 0; c < NC; ++c) out[c] += __shfl_xor_sync(0xffffffffu, out[c], w);
        const int qi = row0 + ty * 4 + i;
        if (qi >= sr.len || kg) continue;
        const float inv = 1.0f / sum;
        float* orow = o + (int64_t)(sr.start + qi) * sd.ot + h * sd.oh + cg * 4;
#pragma unroll
        for (int c = 0; c < NC; c += 4)
            if (cg * 4 + 16 * c < dh)
                *reinterpret_cast<float4*>(orow + 16 * c) =
                    make_float4(out[c] * inv, out[c + 1] * inv, out[c + 2] * inv, out[c + 3] * inv);
    }
}

template <int DP>
cudaError_t launch_f32_dp(const PackedArgs& a, int slots, const PackedStrides& sd, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(done, k_packed_f32<DP>, F32Smem<DP>::kBytes);
    if (e != cudaSuccess) return e;
    return launch_pdl(k_packed_f32<DP>, dim3((unsigned)slots * a.H), dim3(kF32Threads), F32Smem<DP>::kBytes, st,
                      static_cast<const float*>(a.q), static_cast<const float*>(a.k),
                      static_cast<const float*>(a.v), static_cast<float*>(a.o), a.cu, a.n_seq, a.T, slots, a.H,
                      a.H / a.Hkv, a.dh, sd, a.scale * 1.4426950408889634f, a.window, device_error_word());
}

cudaError_t launch_f32(const PackedArgs& a, cudaStream_t st) {
    const int slots = a.T / kF32Rows + a.n_seq;
    const PackedStrides sd{a.strides[0], a.strides[1], a.strides[2], a.strides[3],
                           a.strides[4], a.strides[5], a.strides[6], a.strides[7]};
    return a.dh <= 16   ? launch_f32_dp<16>(a, slots, sd, st)
           : a.dh <= 32 ? launch_f32_dp<32>(a, slots, sd, st)
           : a.dh <= 64 ? launch_f32_dp<64>(a, slots, sd, st)
                        : launch_f32_dp<128>(a, slots, sd, st);
}

// ------------------------------------------------------------------ work list
// A work item is two query tiles of 128 rows that read the same keys: with an
// even group two neighbouring query heads on the same rows (equal lengths, no
// half-empty pair in short sequences), otherwise two neighbouring tiles of one
// head.  The list holds one entry per block of kRows rows (128 or 256) of a
// sequence, the longest key ranges first, from which the persistent kernel's CTAs take
// their items.
//
// Blocks are found without a scan, by their slots (sequence_of; here a slot a thread).  A
// counting sort over at most 256 length classes then orders them (by 256 threads: 1024 took
// 0.5 us more, and most batches have fewer blocks).
constexpr int kPlanThreads = 256;
constexpr int kBins = 256;
constexpr int kPlanCache = 4096;        // offsets kept in shared memory

struct __align__(16) Block {
    int start, len;    // rows of the sequence
    int row;           // the block's first row in it
    int j0;            // first key tile
    int n0, n1, lo1;   // key tiles of the two query tiles (struct Item)
    int pad;
};

// The block of `rows` rows (128: one query tile, 256: two) at a slot of sequence b;
// false: there is none.
__device__ __forceinline__ bool make_block(Block& blk, const SeqRange r, int b, int slot, int rows, int window) {
    const int t = slot - (r.start / rows + b);
    if (t < 0 || (int64_t)t * rows >= r.len) return false;
    const int rowA = t * rows, rowB = rows == 128 ? rowA : rowA + 128;
    const int jA = window > 0 && rowA >= window ? (rowA - window + 1) / 128 : 0;
    const int jB = window > 0 && rowB >= window ? (rowB - window + 1) / 128 : 0;
    const bool two = rowB < r.len;
    blk = Block{r.start, r.len, rowA, jA, rowA / 128 + 1 - jA, two ? rowB / 128 + 1 - jA : 0, two ? jB - jA : 0, 0};
    return true;
}

template <int kRows>
__global__ void __launch_bounds__(kPlanThreads) k_packed_plan(const int32_t* __restrict__ cu, int n_seq,
                                                              int T, int slots, int shift, int window,
                                                              int* __restrict__ count,
                                                              Block* __restrict__ list, int* err) {
    __shared__ int bins[kBins];
    __shared__ int warp_sum[kPlanThreads / 32];
    __shared__ int cached[kPlanCache];
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    bins[tid] = 0;
    // the searches read shared memory, if the offsets fit: a trip to L2 per probe made
    // most of this kernel
    const bool in_smem = n_seq < kPlanCache;
    if (in_smem)
        for (int b = tid; b <= n_seq; b += kPlanThreads) cached[b] = __ldg(cu + b);
    __syncthreads();
    auto offset = [&](int b) { return in_smem ? cached[b] : __ldg(cu + b); };
    for (int b = tid; b < n_seq; b += kPlanThreads) {
        const int s = offset(b), e = offset(b + 1);
        if (s < 0 || s > e || e > T) raise_error(err, TFM_EINVAL);
    }
    // block of slot s, and its length class; false: the slot is empty
    auto find = [&](int s, Block& blk, int& bin) -> bool {
        int lo = 0, hi = n_seq;                       // the last b with cu[b] / kRows + b <= s
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (offset(mid) / kRows + mid <= s) lo = mid + 1; else hi = mid;
        }
        if (lo == 0) return false;
        const int b = lo - 1;
        if (!make_block(blk, seq_range(offset(b), offset(b + 1), T), b, s, kRows, window)) return false;
        bin = kBins - 1 - ((max(blk.n0, blk.n1) - 1) >> shift);
        return true;
    };
    // Counted, then placed; what a thread finds last it keeps, which is all there is to
    // find up to 256 slots.
    Block blk;
    int bin;
    bool found = false;
    for (int s = tid; s < slots; s += kPlanThreads) {
        found = find(s, blk, bin);
        if (found) atomicAdd(&bins[bin], 1);
    }
    __syncthreads();
    // exclusive sums of the classes' counts
    const int n = bins[tid];
    int sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
    }
    if (lane == 31) warp_sum[warp] = sum;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < warp; ++w) before += warp_sum[w];
    bins[tid] = before + sum - n;
    if (tid == kPlanThreads - 1) {
        count[0] = before + sum;
        count[1] = 0;                                  // items taken beyond the CTAs' first
    }
    __syncthreads();
    if (found) list[atomicAdd(&bins[bin], 1)] = blk;
    for (int s = tid; s + kPlanThreads < slots; s += kPlanThreads)
        if (find(s, blk, bin)) list[atomicAdd(&bins[bin], 1)] = blk;
}

// ------------------------------------------------------------------ tensor cores
// A persistent CTA per SM: a TMA warp, an MMA warp per query tile, a warp that checks V, and
// four softmax warps per query tile, a row a thread.  S = Q K^T and O += P V on tcgen05, S, P
// and O in tensor memory.  Key tiles of 64 with two places for S per query tile, P in the place
// of S: the softmax of one tile runs beside the products of the next, and a diagonal tile
// is half as wide.  (Tiles of 128 with one place: 12 prompts of up to 2048 at 16/4 x 128 90 us
// instead of 77, 24 of up to 1024 at 12 x 64 35.5 instead of 32.5; 3 of up to 8192 at
// 16 x 64 the same 168.)  What bounds it is latency, of softmax and MMA warps alike: at
// d_head 64 a pair of tiles takes ~1260 cycles, of them ~510 the exponentials of both on
// the MUFU, ~550 the tensor pipe; of 1210 (before the row maxima were taken from the scores)
// 960 were left without exponentials, 860 without any arithmetic of the softmax, and 690 with a
// quarter of the MMAs besides.  (Two CTAs per
// SM, one place for S each and 96 registers a softmax thread: 173 us instead of 168.)
constexpr int kQ = 128;
constexpr int kThreadsP = 384;          // control, softmax of tile A, softmax of tile B
constexpr int kKV = 64;                 // keys per tile
constexpr float kRescale = 8.0f;        // log2 units: P entries stay below 2^8
constexpr int kItems = 8;               // entries of work items in shared memory
// Items whose V held values that are not finite.  A softmax warp in the epilogue of item i
// has released the entries up to i's, so item i + kItems can be on its way while the other
// tile's warps run ahead: its mark must not take the place of item i's.
constexpr int kPoison = 16;
static_assert(kPoison > kItems, "a mark lives until the item's last epilogue");

template <int DH>
struct Pk {
    static constexpr int kRowBytes = DH >= 64 ? 128 : 64;   // of a shared-memory tile
    static constexpr int kSub = DH / 64 > 1 ? DH / 64 : 1;  // 64-column sub-tiles
    static constexpr int kQTile = kQ * DH * 2;              // bytes of a Q tile
    static constexpr int kTile = kKV * DH * 2;              // of a K or V tile
    static constexpr int kSubQ = kQ * 128, kSubKV = kKV * 128;      // of their sub-tiles
    static constexpr int kNQ = DH == 128 ? 2 : 4;
    static constexpr int kRing = DH == 128 ? 4 : 8;         // slots of a K and a V tile
    static constexpr int kKOff = kNQ * kQTile;
    static constexpr int kVOff = kKOff + kRing * kTile;
    // output rows of a softmax warp, 64 columns at a time
    static constexpr int kStageRow = DH >= 64 ? 128 : 64;
    static constexpr int kStage = 32 * kStageRow;
    static constexpr int kStageOff = kVOff + kRing * kTile;
    static constexpr int kBarOff = kStageOff + 8 * kStage;
    static constexpr int kNumBars = 2 * kNQ + 3 * kRing + 2 * kItems + 13;
    static constexpr int kMiscOff = kBarOff + 8 * kNumBars;
    static constexpr int kItemOff = kMiscOff + 16 + 4 * kPoison;
    static constexpr int kBytes = kItemOff + 32 * kItems + 16 + 1024;
    // tensor-memory columns: S (2 x 2 x 64, P in its place), O (2 x DH)
    static constexpr int kOCol = 4 * kKV;
    static constexpr uint32_t kSwz = DH == 32 ? 4u : 2u;
    static constexpr uint32_t kGroup = 8 * kRowBytes;
    static_assert(kBytes <= 232448, "shared memory budget");
    static_assert(kOCol + 2 * DH <= 512, "tensor memory budget");
};

// Both tiles of an item read key tiles j0 + j, j in [0, nmax); tile x those with
// lo[x] <= j < n[x] (n[1] = 0: there is no tile B).
struct Item {
    int start, len, row[2], h[2], g, j0, lo[2], n[2], nmax;
};

struct PackedGeom {
    int group, subs;       // subs: items per block (H / 2 pairs of heads, or H heads)
    int by_heads;          // 1: two heads of one tile, 0: two tiles of one head
    int window;
    uint32_t subs_inv, group_inv;
    // the offsets, if every slot has a CTA of its own for each sub-item: no list then
    const int32_t* cu;
    int n_seq, T;
};

// x / d with inv = floor(2^32 / d) (2^32 - 1 for d = 1): the estimate is at most one
// too small.
__device__ __forceinline__ int div_by(int x, int d, uint32_t inv) {
    const int q = (int)__umulhi((uint32_t)x, inv);
    return x - q * d >= d ? q + 1 : q;
}

__device__ __forceinline__ void make_item(Item& it, const int4 a, const int4 b, const PackedGeom& gm) {
    const int sub = b.w;
    constexpr int kPer = 128 / kKV;                    // a block's entry counts in 128 keys
    it.start = a.x;
    it.len = a.y;
    it.row[0] = a.z;
    it.row[1] = gm.by_heads ? a.z : a.z + kQ;
    it.h[0] = gm.by_heads ? 2 * sub : sub;
    it.h[1] = gm.by_heads ? it.h[0] + 1 : sub;
    it.g = div_by(it.h[0], gm.group, gm.group_inv);
    it.j0 = a.w * kPer;
    it.lo[0] = 0;
    it.lo[1] = b.z * kPer;
    it.n[0] = b.x * kPer;
    it.n[1] = b.y * kPer;
    it.nmax = it.n[1] > it.n[0] ? it.n[1] : it.n[0];
}

// Whether key tile j of the item holds a key that some row of it does not see:
// the diagonals, and with a window the tiles that start before some row's window.
template <bool kWin>
__device__ __forceinline__ bool masked_tile(const Item& it, int j, int window) {
    const int k0 = (it.j0 + j) * kKV;
    auto diagonal = [&](int row) { return k0 >= row && k0 < row + kQ; };
    return diagonal(it.row[0]) || (it.n[1] && diagonal(it.row[1])) ||
           (kWin && k0 < (it.n[1] ? it.row[1] : it.row[0]) + kQ - window);
}

// Adds the values of n keys that are not finite to an output row.
__device__ __noinline__ void put_back(__nv_bfloat16* orow, const __nv_bfloat16* __restrict__ v, int64_t vt, int dh,
                                      int n) {
    for (int k = 0; k < n; ++k)
        for (int c = 0; c < dh; ++c) {
            const float w = __bfloat162float(v[k * vt + c]);
            if (!(fabsf(w) < INFINITY)) orow[c] = __float2bfloat16_rn(__bfloat162float(orow[c]) + w);
        }
}

template <int DH, bool kWin>
__global__ void __launch_bounds__(kThreadsP, 1)
    k_packed_tc(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                const __grid_constant__ CUtensorMap vmap, const __nv_bfloat16* __restrict__ v,
                __nv_bfloat16* __restrict__ o, int* __restrict__ count,
                const Block* __restrict__ list, PackedGeom gm, int64_t vt, int64_t vh, int64_t ot,
                int64_t oh, float scale_log2, int* err) {
    using L = Pk<DH>;
    constexpr int NQ = L::kNQ, R = L::kRing;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    const uint32_t sQ = base, sK = base + L::kKOff, sV = base + L::kVOff, bars = base + L::kBarOff;
    auto q_full = [&](int s) { return bars + 8u * s; };
    auto q_empty = [&](int s) { return bars + 8u * (NQ + s); };
    // A slot of the ring takes, in step u, K of round u and V of round u - 1, which are
    // multiplied in the same step: loaded, V checked, both multiplied.
    constexpr int B0 = 2 * NQ;
    auto full = [&](int s) { return bars + 8u * (B0 + s); };
    auto clean = [&](int s) { return bars + 8u * (B0 + R + s); };
    auto empty = [&](int s) { return bars + 8u * (B0 + 2 * R + s); };
    // of tile x's n-th S, in buffer n & 1: S is complete, P is written, P.V is complete
    constexpr int B1 = B0 + 3 * R;
    auto s_full = [&](int x, int n) { return bars + 8u * (B1 + 2 * x + (n & 1)); };
    auto p_full = [&](int x, int n) { return bars + 8u * (B1 + 4 + 2 * x + (n & 1)); };
    auto o_done = [&](int x, int n) { return bars + 8u * (B1 + 8 + 2 * x + (n & 1)); };
    auto phase = [&](int n) { return (uint32_t)(n >> 1) & 1u; };
    const uint32_t done_bar = bars + 8u * (B1 + 12);
    auto item_full = [&](int i) { return bars + 8u * (B1 + 13 + i); };
    auto item_empty = [&](int i) { return bars + 8u * (B1 + 13 + kItems + i); };
    const uint32_t item_at = base + (L::kItemOff + 15 & ~15);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(gbase + L::kMiscOff);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + L::kMiscOff + 4);
    volatile int* poison = reinterpret_cast<volatile int*>(gbase + L::kMiscOff + 16);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == 0 && lane == 0) {
        for (int s = 0; s < NQ; ++s) {
            mbar_init(q_full(s), 1);
            mbar_init(q_empty(s), 1);
        }
        for (int s = 0; s < R; ++s) {
            mbar_init(full(s), 1);
            mbar_init(clean(s), 1);
            mbar_init(empty(s), 2);                    // both MMA warps are done with the slot
        }
        for (int x = 0; x < 2; ++x)
            for (int i = 0; i < 2; ++i) {
                mbar_init(s_full(x, i), 1);
                mbar_init(p_full(x, i), 4);
                mbar_init(o_done(x, i), 1);
            }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(item_full(i), 1);
            mbar_init(item_empty(i), kThreadsP / 32 - 1);
        }
        mbar_init(done_bar, 2);
        abort_flag[0] = abort_flag[1] = 0;
        for (int i = 0; i < kPoison; ++i) poison[i] = 0;
        fence_mbar_init();
        tma_prefetch_desc(&qmap);
        tma_prefetch_desc(&kmap);
        tma_prefetch_desc(&vmap);
    }
    if (warp == 1) tmem_alloc(smem_u32(tmem_holder), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;
    pdl_wait();
    pdl_trigger();

    // A CTA's first item is its own number, each further one the next in the list that no CTA
    // has taken yet: the longest come first, so that all end together (dealt in a fixed order,
    // to and fro: 77 us instead of 73 for 12 prompts at 16/4 x 128, 167 instead of 163 for 3
    // of up to 8192 at 16 x 64).  The TMA warp takes it and leaves its entry for the others.
    int n_item = 0;
    auto take_item = [&](Item& it) -> bool {
        const int slot = n_item % kItems, c = (int)blockIdx.x;
        if (n_item >= kItems && !warp_wait(item_empty(slot), ((uint32_t)(n_item / kItems) & 1u) ^ 1u, err, abort_flag))
            return false;
        int4 ea = make_int4(0, 0, 0, 0), eb = ea;      // none: no key tiles
        if (gm.cu) {
            if (n_item == 0) {
                const int k = c / gm.subs, rows = gm.by_heads ? 128 : 256, b = sequence_of(gm.cu, gm.n_seq, rows, k);
                Block blk;
                if (b >= 0 && make_block(blk, seq_range(__ldg(gm.cu + b), __ldg(gm.cu + b + 1), gm.T), b, k, rows, gm.window)) {
                    ea = make_int4(blk.start, blk.len, blk.row, blk.j0);
                    eb = make_int4(blk.n0, blk.n1, blk.lo1, c - k * gm.subs);
                }
            }
        } else {
            int idx = c;
            if (n_item > 0) {
                if (lane == 0) idx = (int)gridDim.x + atomicAdd(count + 1, 1);
                idx = __shfl_sync(0xffffffffu, idx, 0);
            }
            if (idx < __ldg(count) * gm.subs) {
                const int k = div_by(idx, gm.subs, gm.subs_inv);
                const int4* e = reinterpret_cast<const int4*>(list + k);
                ea = __ldg(e);
                eb = __ldg(e + 1);
                eb.w = idx - k * gm.subs;
            }
        }
        if (lane == 0) {
            st_shared_v4(item_at + slot * 32, ea.x, ea.y, ea.z, ea.w);
            st_shared_v4(item_at + slot * 32 + 16, eb.x, eb.y, eb.z, eb.w);
            mbar_arrive(item_full(slot));
        }
        __syncwarp();
        ++n_item;
        if (eb.x == 0) return false;
        make_item(it, ea, eb, gm);
        return true;
    };
    // The next item, for the other warps; false when there is none.
    auto next_item = [&](Item& it) -> bool {
        const int slot = n_item % kItems;
        if (!warp_wait(item_full(slot), (uint32_t)(n_item / kItems) & 1u, err, abort_flag)) return false;
        const uint4 a = ld_shared_v4(item_at + slot * 32), b = ld_shared_v4(item_at + slot * 32 + 16);
        __syncwarp();
        if (lane == 0) mbar_arrive(item_empty(slot));
        ++n_item;
        if (b.x == 0) return false;
        make_item(it, make_int4(a.x, a.y, a.z, a.w), make_int4(b.x, b.y, b.z, b.w), gm);
        return true;
    };
    if (gm.cu && blockIdx.x == 0)
        for (int k = threadIdx.x; k < gm.n_seq; k += kThreadsP) {
            const int from = __ldg(gm.cu + k), to = __ldg(gm.cu + k + 1);
            if (from < 0 || from > to || to > gm.T) raise_error(err, TFM_EINVAL);
        }

    constexpr uint32_t idesc_s = umma_idesc_bf16(kQ, kKV);
    constexpr uint32_t idesc_o = umma_idesc_bf16(kQ, DH, true);
    // Q, K: K-major tiles in 64-column sub-tiles of 16 KB; V: MN-major
    const uint64_t dq = sdesc(sQ, L::kSwz, 16, L::kGroup), dk = sdesc(sK, L::kSwz, 16, L::kGroup);
    const uint64_t dv = sdesc(sV, L::kSwz, DH > 64 ? L::kSubKV : 0, L::kGroup);
    const uint32_t tm = uniform(tmem_base);

    if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
    if (warp == 0) {
        // ---------------------------------------------------------- TMA producer
        // Per step K of a round and V of the round before; Q_A and Q_B behind the first K of
        // an item, as their slots may still be read and the last V of the item before is
        // waited for.  The next item is taken before the last round is loaded: two trips to L2
        // that are over when its first K is due.
        int qn = 0, u = 0, vy = 0, vg = 0;             // Q tiles, steps; place of the V to be loaded
        bool ok = true;
        auto load_v = [&](int s) {
#pragma unroll
            for (int c2 = 0; c2 < L::kSub; ++c2)
                tma_load_3d_e(sV + s * L::kTile + c2 * L::kSubKV, &vmap, 64 * c2, vy, vg, full(s));
        };
        auto slot_free = [&]() -> bool {
            return u < R || (ok = warp_wait(empty(u % R), ((uint32_t)(u / R) & 1u) ^ 1u, err, abort_flag));
        };
        Item it, next;
        bool has = take_item(it);
        while (has && ok) {
            const int nmax = (int)uniform(it.nmax), two = (int)uniform(it.n[1]);
            int y = it.start + it.j0 * kKV;            // the next K tile's first row
            for (int j = 0; j < nmax && ok; ++j, ++u, y += kKV) {
                const int s = u % R;
                if (j == nmax - 1) has = take_item(next);
                if (!slot_free()) break;
                mbar_arrive_expect_tx_e(full(s), u > 0 ? 2 * L::kTile : L::kTile);
#pragma unroll
                for (int c2 = 0; c2 < L::kSub; ++c2)
                    tma_load_3d_e(sK + s * L::kTile + c2 * L::kSubKV, &kmap, 64 * c2, y, it.g, full(s));
                if (u > 0) load_v(s);
                vy = y;
                vg = it.g;
                if (j > 0) continue;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    if (!ok || (x && !two)) continue;
                    const int q = qn % NQ;
                    if (qn >= NQ) ok = warp_wait(q_empty(q), ((uint32_t)(qn / NQ) & 1u) ^ 1u, err, abort_flag);
                    if (!ok) continue;
                    mbar_arrive_expect_tx_e(q_full(q), L::kQTile);
#pragma unroll
                    for (int c2 = 0; c2 < L::kSub; ++c2)
                        tma_load_3d_e(sQ + q * L::kQTile + c2 * L::kSubQ, &qmap, 64 * c2, it.start + it.row[x], it.h[x], q_full(q));
                    ++qn;
                }
            }
            it = next;
        }
        if (ok && u > 0 && slot_free()) {              // the last V
            mbar_arrive_expect_tx_e(full(u % R), L::kTile);
            load_v(u % R);
            ++u;
        }
        // The other warps wait for every load; after a wait that gave up, the last
        // ones still have to land before the CTA ends.
        if (!ok && lane == 0) {
            volatile int* never = abort_flag + 1;       // stays 0: these waits run to their own limit
            for (int k = qn < NQ ? 0 : qn - NQ; k < qn; ++k) mbar_wait(q_full(k % NQ), (uint32_t)(k / NQ) & 1u, nullptr, never);
            for (int k = u < R ? 0 : u - R; k < u; ++k) mbar_wait(full(k % R), (uint32_t)(k / R) & 1u, nullptr, never);
        }
    } else if (warp == 3) {
        // ---------------------------------------------------------- V check
        // In a tile that some row does not see whole, P is zero where the row
        // does not look, but zero times infinity is not: such values are taken
        // out here (and added back for the rows that see them, in the epilogue).
        // Every step passes through here, so that no barrier runs past a phase that this
        // warp has not seen.
        int u = 0, items = 0, v_item = 0;              // steps, items; item of V
        bool ok = true, has = true, masked = false;    // some row does not see all of V
        Item it;
        while (has && ok) {
            has = next_item(it);
            if (!has && u == 0) break;
            const int nmax = has ? it.nmax : 1;
            for (int j = 0; j < nmax; ++j, ++u) {
                const int s = u % R;
                if (!(ok = warp_wait(full(s), (uint32_t)(u / R) & 1u, err, abort_flag))) break;
                const bool check = masked;
                const int at_item = v_item;
                masked = has && masked_tile<kWin>(it, j, gm.window);
                v_item = items;
                if (!check) {
                    if (lane == 0) mbar_arrive(clean(s));
                    continue;
                }
                // An exponent of all ones carries into the bit above it when one is
                // added; eight vectors are looked at together.
                const uint32_t at = sV + s * L::kTile + lane * 16;
                bool found = false;
#pragma unroll 1
                for (int i = 0; i < L::kTile; i += 8 * 512) {
                    uint4 w[8];
#pragma unroll
                    for (int u = 0; u < 8; ++u) w[u] = ld_shared_v4(at + i + u * 512);
                    auto carry = [](uint32_t v) { return (v & 0x7F807F80u) + 0x00800080u; };
                    uint32_t any = 0;
#pragma unroll
                    for (int u = 0; u < 8; ++u) any |= carry(w[u].x) | carry(w[u].y) | carry(w[u].z) | carry(w[u].w);
                    if (any & 0x80008000u) {
                        found = true;
                        auto keep = [&](uint32_t v) {  // 0 in place of each that is not finite
                            const uint32_t bad = (carry(v) & 0x80008000u) >> 15;
                            return v & ~(bad * 0xFFFFu);
                        };
#pragma unroll
                        for (int u = 0; u < 8; ++u)
                            st_shared_v4(at + i + u * 512, keep(w[u].x), keep(w[u].y), keep(w[u].z), keep(w[u].w));
                    }
                }
                if (__any_sync(0xffffffffu, found)) {
                    if (lane == 0) poison[at_item % kPoison] = at_item + 1;
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(clean(s));
            }
            ++items;
        }
    } else {
        // ---------------------------------------------------------- MMAs (warp 1: tile A, warp 2: tile B)
        // A warp per tile: each runs at the pace of its own softmax, and the two
        // pipelines drift into the phase in which one's exponentials run beside the
        // other's products (issued by one warp in the order A, B, A, ..., each waited for
        // the other: 46 us instead of 40 for 24 prompts of up to 1024 tokens at 12 x 64).
        // Step u: S of round u, then P.V of round u - 1, each if its key tile is one that
        // this tile's queries see.  The two places of S let the softmax of round u - 1
        // run beside S of round u, and S of an item's first round beside the last softmax
        // of the item before.  MMAs of one thread complete in the order they are issued:
        // S of round u, in the place of P of round u - 2, lies behind its P.V.
        const int x = (int)uniform((uint32_t)(warp - 1));
        // This loop is what a short tile waits for: the warp waits out the latency of each of
        // its instructions (~10 cycles, two busy warps beside it), so its own rounds, an even
        // number in every item, go in pairs with the places of S and P fixed.
        const uint32_t t_s = tm + 2 * x * kKV, t_o = tm + L::kOCol + x * DH;
        const uint32_t hi_k = (uint32_t)(dq >> 32), hi_v = (uint32_t)(dv >> 32);
        const uint32_t s_bar = uniform(s_full(x, 0)), p_bar = uniform(p_full(x, 0)), o_bar = uniform(o_done(x, 0));
        bool ok = true, pv = false;                     // P.V of an odd round is to come
        uint32_t slot = 0, par = 0, pair = 0;           // ring slot and its phase's parity; parity of own pairs
        int qn = 0;                                     // Q tiles so far
        auto ready = [&]() -> bool { return ok = warp_wait_short(clean(slot), par, err, abort_flag); };
        auto scores = [&](uint32_t q_lo, int b) {
            tc_fence_after();
            umma_scores<DH>(t_s + b * kKV, q_lo, q_lo + (L::kSubQ >> 4), (uint32_t)dk + slot * (L::kTile >> 4), hi_k, idesc_s, s_bar + 8 * b);
        };
        auto values = [&](int b, uint32_t parity, uint32_t acc) -> bool {
            if (!(ok = warp_wait_short(p_bar + 8 * b, parity, err, abort_flag))) return false;
            tc_fence_after();
            umma_values<DH>(t_o, t_s + b * kKV, (uint32_t)dv + slot * (L::kTile >> 4), hi_v, idesc_o, acc, o_bar + 8 * b);
            return true;
        };
        auto release = [&]() {
            umma_commit_e(empty(slot));
            if (++slot == R) {
                slot = 0;
                par ^= 1u;
            }
        };
        // a round that this tile does not see, or the step behind the last round
        auto pass = [&]() {
            if (!ready() || (pv && !values(1, pair ^ 1u, 1u))) return;
            pv = false;
            release();
        };
        // all rounds of the next item (0: none), those of this tile, its Q tile
        int t_max, t_lo, t_n, t_q;
        auto fetch = [&]() {
            Item it;
            it.nmax = it.n[1] = 0;
            const bool has = next_item(it);
            t_max = has ? (int)uniform(it.nmax) : 0;
            t_lo = (int)uniform(x ? it.lo[1] : 0);
            t_n = (int)uniform(x ? it.n[1] : it.n[0]);
            t_q = qn + x;
            qn += uniform(it.n[1]) ? 2 : 1;
        };
        fetch();
        const bool any = t_max > 0;
        while (ok && t_max > 0) {
            const int nmax = t_max, lo = t_lo, n = t_n, qs = t_q;
            int j = 0;
            for (; j < lo && ok; ++j) pass();
            const uint32_t q_lo = (uint32_t)dq + (qs % NQ) * (L::kQTile >> 4);
            for (; j < n && ok; j += 2) {
                if (!ready()) break;
                if (j == lo) {
                    // the last P.V of the item before is waited for, Q may still be on its way
                    if (pv && !values(1, pair ^ 1u, 1u)) break;
                    if (!(ok = warp_wait_short(q_full(qs % NQ), (uint32_t)(qs / NQ) & 1u, err, abort_flag))) break;
                    scores(q_lo, 0);
                } else {
                    scores(q_lo, 0);
                    if (!values(1, pair ^ 1u, 1u)) break;
                }
                release();
                if (!ready()) break;
                scores(q_lo, 1);
                if (j == n - 2) umma_commit_e(q_empty(qs % NQ));
                if (!values(0, pair, j > lo ? 1u : 0u)) break;
                release();
                pv = true;
                pair ^= 1u;
                // (before the next item's first S is due; its entry waits for none of this
                // warp's rounds: all their tiles are on their way)
                if (j == n - 2) fetch();
            }
            for (; j < nmax && ok; ++j) pass();
            if (n == 0 && ok) fetch();
        }
        if (any && ok) pass();
        umma_commit_e(done_bar);
        warp_wait(done_bar, 0, err, abort_flag);
    }
    } else {
        // ---------------------------------------------------------- softmax (warps 4..11)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        const int x = (warp >> 2) - 1;                 // 0: tile A, 1: tile B
        const int q4 = warp & 3;
        const int r = q4 * 32 + lane;
        const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
        const uint32_t t_s = tmem_base + 2 * x * kKV + lane_off;
        const uint32_t t_o = tmem_base + L::kOCol + x * DH + lane_off;
        int cnt = 0, items = 0;                        // own tiles, items
        bool ok = true;
        Item it;
        for (; ok && next_item(it); ++items) {
            const int n = x ? it.n[1] : it.n[0], lo = x ? it.lo[1] : 0;
            if (n == 0) continue;
            const int row0 = x ? it.row[1] : it.row[0], qi = row0 + r;
            const int kmin = kWin ? qi - gm.window + 1 : 0;
            const int win_lo = kWin ? row0 + kQ - gm.window : INT_MIN;
            float m = -INFINITY, l = 0.f;
            for (int j = lo; j < n; ++j, ++cnt) {
                if (!(ok = warp_wait(s_full(x, cnt), phase(cnt), err, abort_flag))) break;
                tc_fence_after();
                uint32_t sr[kKV / 32][32];
#pragma unroll
                for (int cc = 0; cc < kKV / 32; ++cc) tmem_ld32_issue(t_s + (cnt & 1) * kKV + cc * 32, sr[cc]);
                tmem_ld_wait();
                float s[kKV];
#pragma unroll
                for (int cc = 0; cc < kKV / 32; ++cc) {
                    reg_fence32(sr[cc]);
#pragma unroll
                    for (int e = 0; e < 32; ++e) s[cc * 32 + e] = __uint_as_float(sr[cc][e]);
                }
                const int k0 = (it.j0 + j) * kKV;
                // A row of the sequence sees keys up to itself, which lie in the
                // sequence: the diagonal masks the next sequence's keys too.
                if (k0 >= row0) {
                    const int to = r - (k0 - row0);
#pragma unroll
                    for (int cc = 0; cc < kKV; ++cc) s[cc] = cc > to ? -INFINITY : s[cc];
                }
                if (kWin && k0 < win_lo) {
                    const int from = kmin - k0;
#pragma unroll
                    for (int cc = 0; cc < kKV; ++cc) s[cc] = cc < from ? -INFINITY : s[cc];
                }
                // row maximum: four independent chains of three-input maxima
                float mx4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                for (int cc = 4; cc + 8 <= kKV; cc += 8)
#pragma unroll
                    for (int e = 0; e < 4; ++e) mx4[e] = fmax3(mx4[e], s[cc + 2 * e], s[cc + 2 * e + 1]);
#pragma unroll
                for (int e = 0; e < 4; ++e) mx4[e] = fmaxf(mx4[e], s[kKV - 4 + e]);
                const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * scale_log2;
                float corr = 1.f;
                if (mx > m + kRescale) {
                    corr = fast_exp2(m - mx);
                    m = mx;
                }
                const bool rescale = __any_sync(0xffffffffu, corr != 1.f && j > lo && qi < it.len);
                const uint64_t scale2 = f2_pack(scale_log2, scale_log2);
                const float negm = m == -INFINITY ? 0.f : -m;      // a row that has seen no key yet
                const uint64_t negm2 = f2_pack(negm, negm);
                uint64_t sum2[4] = {0ull, 0ull, 0ull, 0ull};
                // P in bf16, as the MMA that sums in fp32 takes it with V in bf16: up to 2^-8 off each, at
                // random, which the average over the keys keeps below the output's own rounding; the
                // row sum adds the weights before it (rounded ones would be unpacked again for it).
                uint32_t pw[32];
#pragma unroll
                for (int e = 0; e < kKV; e += 2) {
                    float t0, t1;
                    f2_unpack(f2_fma(f2_pack(s[e], s[e + 1]), scale2, negm2), t0, t1);
                    const float p0 = fast_exp2(t0), p1 = fast_exp2(t1);
                    sum2[(e >> 1) & 3] = f2_add(sum2[(e >> 1) & 3], f2_pack(p0, p1));
                    pw[e >> 1] = pack_bf16x2(p0, p1);
                }
                tmem_st32_async(t_s + (cnt & 1) * kKV, pw);
                tmem_st_wait();
                float sa[4], sb[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) f2_unpack(sum2[e], sa[e], sb[e]);
                const float sum = ((sa[0] + sb[0]) + (sa[1] + sb[1])) + ((sa[2] + sb[2]) + (sa[3] + sb[3]));
                l = l * corr + sum;
                if (rescale) {
                    // O must hold what the tile before adds to it
                    if (!(ok = warp_wait(o_done(x, cnt - 1), phase(cnt - 1), err, abort_flag))) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int cc = 0; cc < DH / 32; ++cc) {
                        float ov[32];
                        tmem_ld32(t_o + cc * 32, ov);
#pragma unroll
                        for (int e = 0; e < 32; ++e) ov[e] *= corr;
                        tmem_st32(t_o + cc * 32, ov);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full(x, cnt));
            }
            if (!ok) break;
            ok = warp_wait(o_done(x, cnt - 1), phase(cnt - 1), err, abort_flag);
            if (!ok) break;
            tc_fence_after();
            const float inv = 1.0f / l;
            // Rows go out through shared memory, 64 columns (32 at d_head 32) at a time,
            // so that a store writes whole lines: 16 bytes of 32 rows per store kept the
            // warp for 5000 to 10000 cycles at d_head 128.
            __nv_bfloat16* obase = o + (int64_t)(it.start + row0 + q4 * 32) * ot + (int64_t)(x ? it.h[1] : it.h[0]) * oh;
            const int rows = it.len - row0 - q4 * 32;  // of this warp's 32, those of the sequence
            const uint32_t stage = base + L::kStageOff + (warp - 4) * L::kStage;
            constexpr int kChunks = L::kStageRow / 16, kRowsPer = 32 / kChunks;
            uint32_t ov[DH / 32][32];
#pragma unroll
            for (int cc = 0; cc < DH / 32; ++cc) tmem_ld32_issue(t_o + cc * 32, ov[cc]);
            tmem_ld_wait();
#pragma unroll
            for (int cc = 0; cc < DH / 32; ++cc) reg_fence32(ov[cc]);
#pragma unroll
            for (int c0 = 0; c0 < DH / 32; c0 += L::kStageRow / 64) {
#pragma unroll
                for (int cc = 0; cc < L::kStageRow / 64; ++cc) {
                    auto two = [&](int e) {
                        return pack_bf16x2(__uint_as_float(ov[c0 + cc][e]) * inv, __uint_as_float(ov[c0 + cc][e + 1]) * inv);
                    };
#pragma unroll
                    for (int e = 0; e < 32; e += 8)
                        st_shared_v4(stage + lane * L::kStageRow + (((cc * 4 + e / 8) ^ (lane & (kChunks - 1))) * 16),
                                     two(e), two(e + 2), two(e + 4), two(e + 6));
                }
                __syncwarp();
                const int ch = lane % kChunks;
#pragma unroll
                for (int i = 0; i < 32; i += kRowsPer) {
                    const int rr = i + lane / kChunks;
                    const uint4 w = ld_shared_v4(stage + rr * L::kStageRow + ((ch ^ (rr & (kChunks - 1))) * 16));
                    if (rr < rows) *reinterpret_cast<uint4*>(obase + rr * ot + c0 * 32 + ch * 8) = w;
                }
                __syncwarp();
            }
            if (poison[items % kPoison] == items + 1 && qi < it.len) {
                // what the V check took out, for the keys this row sees
#pragma unroll 1
                for (int j = lo; j < n; ++j)
                    if (masked_tile<kWin>(it, j, gm.window)) {
                        const int k0 = (it.j0 + j) * kKV, from = max(k0, kWin ? kmin : 0);
                        put_back(obase + lane * ot, v + (int64_t)(it.start + from) * vt + (int64_t)it.g * vh, vt, DH,
                                 min(k0 + kKV - 1, qi) - from + 1);
                    }
            }
            __syncwarp();
            // O is read out before this warp publishes the next item's first P
            tc_fence_before();
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem_base, 512);
}

template <int DH, bool kWin>
cudaError_t launch_tc(const PackedArgs& a, const CUtensorMap* maps, const PackedGeom& gm, int slots, cudaStream_t st) {
    using L = Pk<DH>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(done, k_packed_tc<DH, kWin>, L::kBytes);
    if (e != cudaSuccess) return e;
    const int64_t items = (int64_t)slots * gm.subs;
    const int grid = items < sm_count() ? (int)items : sm_count();
    return launch_pdl(k_packed_tc<DH, kWin>, dim3(grid), dim3(kThreadsP), L::kBytes, st, maps[0], maps[1], maps[2],
                      static_cast<const __nv_bfloat16*>(a.v), static_cast<__nv_bfloat16*>(a.o),
                      static_cast<int*>(a.ws),
                      reinterpret_cast<const Block*>(static_cast<const uint8_t*>(a.ws) + 256), gm,
                      a.strides[4], a.strides[5], a.strides[6], a.strides[7],
                      a.scale * 1.4426950408889634f, device_error_word());
}

template <int DH>
cudaError_t launch_tc_w(const PackedArgs& a, const CUtensorMap* maps, const PackedGeom& gm, int slots, cudaStream_t st) {
    return a.window > 0 ? launch_tc<DH, true>(a, maps, gm, slots, st) : launch_tc<DH, false>(a, maps, gm, slots, st);
}

template <int kRows>
cudaError_t launch_plan(const PackedArgs& a, int slots, cudaStream_t st) {
    // most key tiles of a block: all of T, or a window's
    const int most = a.window > 0 ? (a.window + kRows - 2) / 128 + 2 : a.T / 128 + 2;
    int shift = 0;
    while ((most >> shift) >= kBins) ++shift;
    return launch_pdl(k_packed_plan<kRows>, dim3(1), dim3(kPlanThreads), 0, st, a.cu, a.n_seq, a.T, slots, shift, a.window,
                      static_cast<int*>(a.ws), reinterpret_cast<Block*>(static_cast<uint8_t*>(a.ws) + 256),
                      device_error_word());
}

}  // namespace

// The number of blocks, then the blocks (of 128 rows, or fewer of 256).
size_t packed_workspace_bytes(int T, int n_seq) { return 256 + sizeof(Block) * ((size_t)T / 128 + n_seq); }

tfm_status launch_packed_attention(const PackedArgs& a, cudaStream_t st, cudaError_t* e) {
    if (!a.bf16) {
        *e = launch_f32(a, st);
        return TFM_OK;
    }
    CUtensorMap maps[3];
    const void* ptr[3] = {a.q, a.k, a.v};
    for (int i = 0; i < 3; ++i)
        if (!rows_heads_map(&maps[i], ptr[i], a.T, i ? a.Hkv : a.H, a.dh, a.strides[2 * i], a.strides[2 * i + 1],
                            i ? kKV : kQ))
            return TFM_ECUDA;
    PackedGeom gm;
    gm.group = a.H / a.Hkv;
    gm.by_heads = gm.group % 2 == 0;
    gm.subs = gm.by_heads ? a.H / 2 : a.H;
    gm.window = a.window;
    auto inverse = [](int d) { return d == 1 ? 0xFFFFFFFFu : (uint32_t)(((uint64_t)1 << 32) / d); };
    gm.subs_inv = inverse(gm.subs);
    gm.group_inv = inverse(gm.group);
    const int slots = a.T / (gm.by_heads ? 128 : 256) + a.n_seq;
    // Few slots: a CTA each, which finds its own sequence (6 prompts of up to 48 at 12 x 64:
    // 5.5 us instead of 7.4); more are sorted first.
    gm.cu = (int64_t)slots * gm.subs <= sm_count() ? a.cu : nullptr;
    gm.n_seq = a.n_seq;
    gm.T = a.T;
    if (!gm.cu) {
        *e = gm.by_heads ? launch_plan<128>(a, slots, st) : launch_plan<256>(a, slots, st);
        if (*e != cudaSuccess) return TFM_OK;
    }
    *e = a.dh == 32 ? launch_tc_w<32>(a, maps, gm, slots, st)
         : a.dh == 64 ? launch_tc_w<64>(a, maps, gm, slots, st)
                      : launch_tc_w<128>(a, maps, gm, slots, st);
    return TFM_OK;
}

}  // namespace tfm
