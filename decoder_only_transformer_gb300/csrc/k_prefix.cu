// k_prefix.cu - attention of the newest T tokens of every sequence over a
// prefix the whole batch shares and each sequence's own cache.
//
// Row (b, h, t): o = sum_j p_j v_j, p = softmax(scale q . k_j) over the keys
// [0, P) of the prefix and the own keys [0, lens[b] - (T - 1 - t)).
//
// The query rows that read the same keys are stacked: for the prefix all
// sequences' rows of a kv head, 128 at a time, so that its keys and values are
// read once for the batch; for an own cache the G T rows (G = H / Hkv) of its
// sequence.  Either way a job is "up to 128 rows against a range of keys", the
// tile of the tensor cores, and one kernel runs both: S = Q K^T (tcgen05, keys
// in tiles of 64), softmax with a running maximum, O += P V.  With few rows most
// of a tile's rows are padding, which costs nothing that counts: a tile of 64
// keys takes 32 KB of d_head 128 from memory, ~1500 cycles of an SM's share of
// HBM bandwidth, and its two products ~500.  (On CUDA cores G T = 4 rows would
// already need ~40 % of all FMAs to keep up with memory.)
//
// All tiles of all jobs are laid end to end and cut into runs of equal cost, one
// per CTA, whatever the lengths are (two CTAs per SM, so that one's loads run
// during the other's softmax).  The cost of a tile and of a job's beginning and end
// are measured cycles (Px below): short caches cost more per key than long ones, and
// equal numbers of tiles left the last CTAs at twice the time of the first.  A run
// crosses jobs; each piece of a job leaves (max,
// sum, unnormalised O) per row, and a second kernel joins a row's pieces of the
// prefix and its own cache exactly: with M = max m, o = sum 2^(m - M) O / sum 2^(m - M) l.
//
// Measured: own caches of 1280 positions, 192 sequences of 16 x 64, without a prefix: 152 us,
// 6.6 TB/s, as fast as a copy.  Short caches are bound by what a piece costs besides its
// tiles (2000 cycles and more of the chain S, softmax, P.V, O out; 192 over a prefix of
// 16384, up to 300 own positions: 61 us, of them ~17 pieces' ends, 20 own tiles, 18 the
// prefix), small calls by the latency of the two launches (4 chats: 8.7 us; 64 at 16/4 x 128
// under 2048: 19 us, of them ~5 until the first scores, ~3 the join).
#include "common.cuh"
#include "internal.h"

namespace tfm {

namespace {

constexpr int kRowsP = 128;
constexpr int kKeys = 64;               // keys per tile
constexpr int kThreadsX = 224;          // 4 softmax warps, TMA, MMA, V check
constexpr int kMaxCtas = 304;
constexpr float kRescaleX = 8.0f;       // log2 units: P entries stay below 2^8
constexpr int kPoisonX = 8;

template <int DH>
struct Px {
    static constexpr int kRowBytes = DH >= 64 ? 128 : 64;
    static constexpr int kSub = DH / 64 > 1 ? DH / 64 : 1;
    static constexpr int kQ = kRowsP * DH * 2;               // bytes of the Q region
    static constexpr int kTile = kKeys * DH * 2;             // of a K or V tile
    static constexpr int kSubTile = kKeys * kRowBytes;
    static constexpr int kRing = DH == 128 ? 2 : DH == 64 ? 4 : 6;
    static constexpr int kMaxQ = 8;                          // Q slots of own jobs
    // Q lies between the rings: the MMA reads 128 rows from an own piece's slot on,
    // whose last one ends with the region
    static constexpr int kQOff = kRing * kTile;
    static constexpr int kVOff = kQOff + kQ;
    static constexpr int kBarOff = kVOff + kRing * kTile;
    static constexpr int kNumBars = 2 * kMaxQ + 4 * kRing + 5;
    static constexpr int kMiscOff = kBarOff + 8 * kNumBars;
    static constexpr int kCumOff = kMiscOff + 16 + 4 * kPoisonX;
    static constexpr int kBase = kCumOff + 1024;             // + 4 (3 B + 2)
    static constexpr int kOCol = 2 * kKeys;                  // S 2 x 64 (P in its place), O
    static constexpr uint32_t kSwz = DH == 32 ? 4u : 2u;
    static constexpr uint32_t kGroup = 8 * kRowBytes;
    // Costs in ~100 cycles of a CTA: a tile of the prefix (from L2, four softmax
    // warps busy) and of an own cache (one warp; d_head 128: its share of HBM
    // bandwidth), and what a piece costs besides (Q, the last P.V, writing O out).
    static constexpr int kPreTile = DH == 128 ? 15 : 13, kPrePiece = DH == 128 ? 50 : 35;
    static constexpr int kOwnTile = DH == 128 ? 24 : 13, kOwnPiece = DH == 128 ? 24 : 32;
    static_assert(kOCol + DH <= 256, "tensor memory: two CTAs per SM");
    static_assert(kRing * kTile >= kRowsP * kRowBytes, "room around the Q slots");
};

// How the work is laid out; the same on the host and in both kernels.
struct PrefixGeom {
    int B, Hkv, GT, T, P, max_seq;
    int nb;            // sequences per row tile of the prefix: nb * GT <= 128
    int nrt;           // row tiles
    int np;            // key tiles of the prefix
    int ctas;
    int q_slots, q_pad;   // Q slots of own jobs, rows of each (GT padded)
};

// Run of CTA i of n over a cost of u: [start, end).
__device__ __forceinline__ int run_start(int i, int u, int n) {
    const int q = u / n, r = u - q * n;
    return i * q + min(i, r);
}

__device__ __forceinline__ int own_len(const int32_t* __restrict__ lens, int b, int max_seq) {
    const int n = __ldg(lens + b);
    return n < 0 || n > max_seq ? 0 : n;
}

// A piece of a job: key tiles [t0, t1) of it.
struct Seg {
    int own;           // 0: prefix
    int g, x;          // kv head; row tile, or sequence
    int t0, t1;
};
__device__ __forceinline__ int keys_of(const Seg& s, const PrefixGeom& gm, const int* slen) {
    return s.own ? slen[s.x] : gm.P;
}
__device__ __forceinline__ int rows_of(const Seg& s, const PrefixGeom& gm) {
    return s.own ? gm.GT : min(gm.nb, gm.B - s.x * gm.nb) * gm.GT;
}
__device__ __forceinline__ int job_of(const Seg& s, const PrefixGeom& gm) {    // among the jobs of its kind
    return s.own ? s.x * gm.Hkv + s.g : s.g * gm.nrt + s.x;
}

// A run's next tile: tile t of the job of kv head g and row tile x, or (own) of
// sequence x.  Jobs follow one another as prefix (g, x), then own (x, g), so the
// next piece needs no search.
struct Walk {
    int left, own, g, x, t;
};

__device__ __forceinline__ void skip_empty(Walk& w, const PrefixGeom& gm, const int* cum) {
    while (w.x < gm.B && cum[w.x + 1] == cum[w.x]) ++w.x;
}

__device__ __forceinline__ bool next_seg(Walk& w, Seg& s, const PrefixGeom& gm, const int* cum) {
    if (w.left <= 0) return false;
    s = Seg{w.own, w.g, w.x, w.t, min(w.own ? cum[w.x + 1] - cum[w.x] : gm.np, w.t + w.left)};
    w.left -= s.t1 - s.t0;
    if (w.left == 0) return true;
    w.t = 0;                                           // the run goes on with the next job
    if (w.own) {
        if (++w.g == gm.Hkv) {
            w.g = 0;
            ++w.x;
            skip_empty(w, gm, cum);
        }
    } else if (++w.x == gm.nrt) {
        w.x = 0;
        if (++w.g == gm.Hkv) {
            w.g = 0;
            w.own = 1;
            skip_empty(w, gm, cum);
        }
    }
    return true;
}

// An own tile that holds keys some row does not see: behind the length, or the
// newest tokens' own.
__device__ __forceinline__ bool check_tile(const Seg& s, int t, int keys, int T) {
    return s.own && (t + 1) * kKeys > keys - (T - 1);
}

// cum[b]: key tiles of the own caches of sequences before b; cost[b]: their cost;
// slen[b]: their lengths.  By the whole block.
template <int DH>
__device__ __forceinline__ void scan_lengths(int* cum, int* cost, int* slen, int2* warp_sum,
                                             const int32_t* __restrict__ lens, const PrefixGeom& gm) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
    int base = 0, base_c = 0;
    for (int b0 = 0; b0 < gm.B; b0 += blockDim.x) {
        const int b = b0 + tid;
        const int len = b < gm.B ? own_len(lens, b, gm.max_seq) : 0;
        if (b < gm.B) slen[b] = len;
        if (b == 0) cum[0] = cost[0] = 0;
        int sum = (len + kKeys - 1) / kKeys;
        int sum_c = sum ? Px<DH>::kOwnPiece + sum * Px<DH>::kOwnTile : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, sum, o), c = __shfl_up_sync(0xffffffffu, sum_c, o);
            if (lane >= o) {
                sum += v;
                sum_c += c;
            }
        }
        if (lane == 31) warp_sum[warp] = make_int2(sum, sum_c);
        __syncthreads();
        int before = base, before_c = base_c;
        for (int w = 0; w < nw; ++w) {
            if (w < warp) {
                before += warp_sum[w].x;
                before_c += warp_sum[w].y;
            }
            base += warp_sum[w].x;
            base_c += warp_sum[w].y;
        }
        if (b < gm.B) {
            cum[b + 1] = before + sum;
            cost[b + 1] = before_c + sum_c;
        }
        __syncthreads();
    }
}

// Cost of everything, and of a job of the prefix.
template <int DH>
__device__ __forceinline__ int prefix_job_cost(const PrefixGeom& gm) {
    return gm.np ? Px<DH>::kPrePiece + gm.np * Px<DH>::kPreTile : 0;
}

// CTAs that get a run: with runs of at least a tile's cost every run that lies
// between a job's first and last piece has a tile of it.  Runs of at least three tiles of
// the prefix: each piece of it leaves 128 rows of d_head floats for the join (16 answers of 5
// tokens over 1024 shared ones, 16/4 x 128: 10.5 us instead of 11.8 with a CTA per tile,
// over 2048 12.7 instead of 14.1).
template <int DH>
__device__ __forceinline__ int runs_of(int all, int ctas) {
    constexpr int least = 3 * Px<DH>::kPreTile > Px<DH>::kOwnTile ? 3 * Px<DH>::kPreTile : Px<DH>::kOwnTile;
    return max(1, min(ctas, all / least));
}

// The tile at cost c (a job's tiles end at its piece cost plus one tile cost each), and
// how many lie before it.
template <int DH>
__device__ __forceinline__ Walk tile_at(int c, int& before, const PrefixGeom& gm, const int* cum, const int* cost) {
    const int jc = prefix_job_cost<DH>(gm), jobs = gm.Hkv * gm.nrt;
    Walk w{0, 0, 0, 0, 0};
    if (c < jc * jobs) {
        const int job = c / jc;
        w.t = max(0, (c - job * jc - Px<DH>::kPrePiece) / Px<DH>::kPreTile);
        w.g = job / gm.nrt;
        w.x = job - w.g * gm.nrt;
        before = job * gm.np + w.t;
        return w;
    }
    const int v = c - jc * jobs, up = jobs * gm.np;
    before = up + gm.Hkv * cum[gm.B];
    if (v >= cost[gm.B] * gm.Hkv) return w;            // the end
    int lo = 0, hi = gm.B;                            // the last b with cost[b] Hkv <= v
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (cost[mid] * gm.Hkv <= v) lo = mid + 1; else hi = mid;
    }
    const int b = lo - 1, each = cost[lo] - cost[b], nt = cum[lo] - cum[b];
    const int x = v - cost[b] * gm.Hkv;
    w.own = 1;
    w.g = x / each;
    w.x = b;
    w.t = max(0, (x - w.g * each - Px<DH>::kOwnPiece) / Px<DH>::kOwnTile);
    before = up + gm.Hkv * cum[b] + w.g * nt + w.t;
    return w;
}

struct PrefixParts {
    // O column-block first, so that the rows of a warp lie side by side
    float* o_prefix;       // [jobs + ctas][dh / 4][128][4]
    float2* ml_prefix;     // [jobs + ctas][128]: max (log2), sum
    float* o_own;          // [B Hkv + ctas][dh / 4][GT][4]
    float2* ml_own;        // [B Hkv + ctas][GT]
    // per job of the prefix, and of the own caches: the CTAs of its first and last piece
    int2* range_prefix;    // [jobs]
    int2* range_own;       // [B Hkv], of caches that hold keys
};

// Adds the values of keys [k0, k1) that are not finite to a row's partial O in
// memory (column c at (c / 4) * stride + c % 4).
__device__ __noinline__ void put_back(float* orow, int stride, const __nv_bfloat16* __restrict__ v, int dh,
                                      int k0, int k1) {
    for (int key = k0; key < k1; ++key)
        for (int c = 0; c < dh; ++c) {
            const float w = __bfloat162float(v[(int64_t)key * dh + c]);
            if (!(fabsf(w) < INFINITY)) orow[(int64_t)(c >> 2) * stride + (c & 3)] += w;
        }
}

template <int DH>
__global__ void __launch_bounds__(kThreadsX, 2)
    k_prefix_part(const __grid_constant__ CUtensorMap qpmap, const __grid_constant__ CUtensorMap qomap,
                  const __grid_constant__ CUtensorMap kpmap, const __grid_constant__ CUtensorMap vpmap,
                  const __grid_constant__ CUtensorMap kcmap, const __grid_constant__ CUtensorMap vcmap,
                  const __nv_bfloat16* __restrict__ vc, const int32_t* __restrict__ lens, PrefixGeom gm,
                  PrefixParts out, float scale_log2, int* err) {
    using L = Px<DH>;
    constexpr int R = L::kRing;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    const uint32_t sK = base, sQ = base + L::kQOff, sV = base + L::kVOff, bars = base + L::kBarOff;
    auto q_full = [&](int s) { return bars + 8u * s; };
    auto q_empty = [&](int s) { return bars + 8u * (L::kMaxQ + s); };
    constexpr int B0 = 2 * L::kMaxQ;
    auto k_full = [&](int s) { return bars + 8u * (B0 + s); };
    auto v_full = [&](int s) { return bars + 8u * (B0 + R + s); };
    // S of a K slot is complete (the slot is free, S can be read); P.V of a V slot
    auto s_done = [&](int s) { return bars + 8u * (B0 + 2 * R + s); };
    auto pv_done = [&](int s) { return bars + 8u * (B0 + 3 * R + s); };
    constexpr int B1 = B0 + 4 * R;
    // Tile n can be multiplied: P is written (by the softmax warps with rows), V_n
    // is there and checked and K_{n+2} is there (the check warp), so that the MMA
    // warp, whose every wait costs ~100 cycles, waits once per tile.  The own
    // tiles have barriers of their own, as fewer softmax warps write their P.
    auto p_pre = [&](int i) { return bars + 8u * (B1 + i); };
    auto p_own = [&](int i) { return bars + 8u * (B1 + 2 + i); };
    const uint32_t done_bar = bars + 8u * (B1 + 4);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(gbase + L::kMiscOff);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + L::kMiscOff + 4);
    volatile int* poison = reinterpret_cast<volatile int*>(gbase + L::kMiscOff + 16);
    int* cum = reinterpret_cast<int*>(gbase + L::kCumOff);
    int* cost = cum + gm.B + 1;
    int* slen = cost + gm.B + 1;
    __shared__ int2 warp_sum[kThreadsX / 32];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == 4 && lane == 0) {
        for (int s = 0; s < L::kMaxQ; ++s) {
            mbar_init(q_full(s), 1);
            mbar_init(q_empty(s), 1);
        }
        for (int s = 0; s < R; ++s) {
            mbar_init(k_full(s), 1);
            mbar_init(v_full(s), 1);
            mbar_init(s_done(s), 1);
            mbar_init(pv_done(s), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(p_pre(i), (gm.nb * gm.GT + 31) / 32 + 1);    // softmax warps with rows, check warp
            mbar_init(p_own(i), (gm.GT + 31) / 32 + 1);
        }
        mbar_init(done_bar, 1);
        abort_flag[0] = abort_flag[1] = 0;
        for (int i = 0; i < kPoisonX; ++i) poison[i] = 0;
        fence_mbar_init();
        tma_prefetch_desc(&qpmap);
        tma_prefetch_desc(&qomap);
        tma_prefetch_desc(&kpmap);
        tma_prefetch_desc(&vpmap);
        tma_prefetch_desc(&kcmap);
        tma_prefetch_desc(&vcmap);
    }
    if (warp == 5) tmem_alloc(smem_u32(tmem_holder), 256);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;
    pdl_wait();
    pdl_trigger();
    scan_lengths<DH>(cum, cost, slen, warp_sum, lens, gm);
    const int cta = (int)blockIdx.x;
    if (cta == 0)
        for (int b = threadIdx.x; b < gm.B; b += kThreadsX)
            if (lens[b] < 0 || lens[b] > gm.max_seq) raise_error(err, TFM_EINVAL);
    const int up = gm.Hkv * gm.nrt * gm.np;
    const int all = prefix_job_cost<DH>(gm) * gm.Hkv * gm.nrt + cost[gm.B] * gm.Hkv;
    const int runs = runs_of<DH>(all, gm.ctas);
    // the run's ends, one in the even and one in the odd lanes
    int before = 0;
    Walk walk{0, 0, 0, 0, 0};
    if (cta < runs) walk = tile_at<DH>(run_start(cta + (lane & 1), all, runs), before, gm, cum, cost);
    const int u0 = __shfl_sync(0xffffffffu, before, 0), u1 = __shfl_sync(0xffffffffu, before, 1);
    walk.left = u1 - u0;
    walk.own = __shfl_sync(0xffffffffu, walk.own, 0);
    walk.g = __shfl_sync(0xffffffffu, walk.g, 0);
    walk.x = __shfl_sync(0xffffffffu, walk.x, 0);
    walk.t = __shfl_sync(0xffffffffu, walk.t, 0);
    const int tiles = (int)uniform(walk.left);         // of this CTA, in all its pieces
    const int own0 = max(0, min(tiles, up - u0));   // its first own tile
    auto p_full = [&](bool own, int n) { return own ? p_own(n & 1) : p_pre(n & 1); };
    auto p_phase = [&](bool own, int n) {
        return (uint32_t)((n >> 1) - (own ? (own0 + ((n ^ own0) & 1)) >> 1 : 0)) & 1u;
    };

    // Q slots: a piece of the prefix takes the whole region (slot 0's barriers),
    // own pieces take q_slots slots in turn, the first after a prefix piece slot 0
    // (a run has its pieces of the prefix first).
    if (warp == 4) {
        // ---------------------------------------------------------- TMA producer
        // Q of a piece before its first K; K_{n+1} before V_n, the order in which
        // the MMA warp takes them.
        bool ok = true;
        int slot = 0;
        uint32_t q_used = 0, q_par = 0;                 // slots used before, their parity
        Walk wk = walk;
        Seg sk{};
        int lk = 0;                                     // tiles left in the piece
        auto load_q = [&]() {
            const bool own = uniform(sk.own);
            const int s = own ? slot : 0;
            if (q_used >> s & 1u) {
                ok = warp_wait(q_empty(s), (q_par >> s) & 1u, err, abort_flag);
                q_par ^= 1u << s;
                if (!ok) return;
            }
            q_used |= 1u << s;
            const int rows = own ? gm.GT : gm.nb * gm.GT;
            const uint32_t dst = sQ + (own ? s * gm.q_pad * DH * 2 : 0);
            const uint32_t sub = (own ? gm.q_pad : kRowsP) * L::kRowBytes;
            const CUtensorMap* map = own ? &qomap : &qpmap;
            const int g = (int)uniform(sk.g), b = (int)uniform(own ? sk.x : sk.x * gm.nb);
            mbar_arrive_expect_tx_e(q_full(s), (uint32_t)rows * DH * 2);
#pragma unroll
            for (int c = 0; c < L::kSub; ++c) tma_load_4d_e(dst + c * sub, map, 64 * c, 0, g, b, q_full(s));
            slot = own ? (s + 1 == gm.q_slots ? 0 : s + 1) : 0;
        };
        int kn = 0, vn = 0;                             // K and V tiles loaded
        int ky = 0, kz = 0, vy = 0, vz = 0;             // coordinates of the next K tile, of the last one's V
        const CUtensorMap *km = &kpmap, *vm = &vpmap;
        for (int n = 0; n <= tiles && ok; ++n) {
            const int s = n % R;
            if (n < tiles) {
                if (lk == 0) {
                    next_seg(wk, sk, gm, cum);
                    lk = (int)uniform(sk.t1 - sk.t0);
                    ky = (int)uniform(sk.t0) * kKeys;
                    kz = (int)uniform(sk.own ? sk.x * gm.Hkv + sk.g : sk.g);
                    km = uniform(sk.own) ? &kcmap : &kpmap;
                    load_q();
                    if (!ok) break;
                }
                if (n >= R && !(ok = warp_wait(s_done(s), ((uint32_t)(n / R) & 1u) ^ 1u, err, abort_flag))) break;
                mbar_arrive_expect_tx_e(k_full(s), L::kTile);
#pragma unroll
                for (int c = 0; c < L::kSub; ++c)
                    tma_load_3d_e(sK + s * L::kTile + c * L::kSubTile, km, 64 * c, ky, kz, k_full(s));
                ky += kKeys;
                --lk;
                ++kn;
            }
            if (n > 0) {
                const int m = n - 1, sv_ = m % R;
                if (m >= R && !(ok = warp_wait(pv_done(sv_), ((uint32_t)(m / R) & 1u) ^ 1u, err, abort_flag))) break;
                mbar_arrive_expect_tx_e(v_full(sv_), L::kTile);
#pragma unroll
                for (int c = 0; c < L::kSub; ++c)
                    tma_load_3d_e(sV + sv_ * L::kTile + c * L::kSubTile, vm, 64 * c, vy, vz, v_full(sv_));
                ++vn;
            }
            vy = ky - kKeys;
            vz = kz;
            vm = km == &kpmap ? &vpmap : &vcmap;
        }
        // The other warps wait for every load; after a wait that gave up,
        // the last ones still have to land before the CTA ends.
        if (!ok && lane == 0) {
            volatile int* never = abort_flag + 1;       // stays 0: these waits run to their own limit
            for (int m = max(0, kn - R); m < kn; ++m) mbar_wait(k_full(m % R), (uint32_t)(m / R) & 1u, nullptr, never);
            for (int m = max(0, vn - R); m < vn; ++m) mbar_wait(v_full(m % R), (uint32_t)(m / R) & 1u, nullptr, never);
        }
    } else if (warp == 5) {
        // ---------------------------------------------------------- MMAs
        // S_0, S_1, then P_n.V_n and S_{n+2}, which takes the place of P_n: the
        // MMAs of one thread complete in the order they are issued.
        constexpr uint32_t idesc_s = umma_idesc_bf16(kRowsP, kKeys);
        constexpr uint32_t idesc_o = umma_idesc_bf16(kRowsP, DH, true);
        const uint32_t tm = uniform(tmem_base);
        const uint64_t dq = sdesc(sQ, L::kSwz, 16, L::kGroup), dk = sdesc(sK, L::kSwz, 16, L::kGroup);
        const uint64_t dv = sdesc(sV, L::kSwz, DH > 64 ? L::kSubTile : 0, L::kGroup);
        bool ok = true;
        int slot = 0, cur = 0, left = 0;                // Q slots; tiles left in the piece of S
        uint32_t q_par = 0, a0 = 0, asub = 0;
        Walk ws = walk;
        Seg ss;
        // of the tile whose S was issued last: an own tile, the first of its piece
        bool own = false, first = false;
        auto do_s = [&](int n) {
            first = left == 0;
            if (first) {
                next_seg(ws, ss, gm, cum);
                left = (int)uniform(ss.t1 - ss.t0);
                own = uniform(ss.own);
                cur = own ? slot : 0;
                slot = own ? (cur + 1 == gm.q_slots ? 0 : cur + 1) : 0;
                a0 = (uint32_t)dq + ((own ? cur * gm.q_pad * DH * 2 : 0) >> 4);
                asub = ((own ? gm.q_pad : kRowsP) * L::kRowBytes) >> 4;
                if (!(ok = warp_wait_short(q_full(cur), (q_par >> cur) & 1u, err, abort_flag))) return;
                q_par ^= 1u << cur;
            }
            const int s = n % R;
            if (n < 2 && !(ok = warp_wait_short(k_full(s), (uint32_t)(n / R) & 1u, err, abort_flag))) return;
            tc_fence_after();
            umma_scores<DH>(tm + (n & 1) * kKeys, a0, a0 + asub, (uint32_t)dk + s * (L::kTile >> 4), (uint32_t)(dq >> 32),
                            idesc_s, s_done(s));
            if (--left == 0) umma_commit_e(q_empty(cur));
        };
        if (tiles > 0) do_s(0);
        bool pv_own = own, pv_first = first;            // of tile n, and of the one behind it
        if (ok && tiles > 1) do_s(1);
        bool next_own = own, next_first = first;
        for (int n = 0; n < tiles && ok; ++n) {
            const int s = n % R;
            if (!(ok = warp_wait_short(p_full(pv_own, n), p_phase(pv_own, n), err, abort_flag))) break;
            tc_fence_after();
            umma_values<DH>(tm + L::kOCol, tm + (n & 1) * kKeys, (uint32_t)dv + s * (L::kTile >> 4), (uint32_t)(dv >> 32),
                            idesc_o, pv_first ? 0u : 1u, pv_done(s));
            pv_own = next_own;
            pv_first = next_first;
            if (n + 2 < tiles) do_s(n + 2);
            next_own = own;
            next_first = first;
        }
        umma_commit_e(done_bar);
        warp_wait(done_bar, 0, err, abort_flag);
    } else if (warp == 6) {
        // ---------------------------------------------------------- V check
        // Values that are not finite are taken out of the tiles whose keys some
        // row does not see (zero times infinity is not zero) and added back in
        // the epilogue for the rows that do.  This warp goes in step with the MMAs
        // (its arrival for tile n comes behind S_n, which comes behind P.V of tile
        // n - 2), so no barrier runs past a phase that it has not seen.
        Walk wv = walk;
        Seg sv;
        bool ok = true;
        int n = 0;
        for (int seg = 0; ok && next_seg(wv, sv, gm, cum); ++seg)
            for (int t = sv.t0; t < sv.t1; ++t, ++n) {
                const int s = n % R;
                ok = warp_wait(s_done(s), (uint32_t)(n / R) & 1u, err, abort_flag) &&
                     warp_wait(v_full(s), (uint32_t)(n / R) & 1u, err, abort_flag) &&
                     (n + 2 >= tiles || warp_wait(k_full((n + 2) % R), (uint32_t)((n + 2) / R) & 1u, err, abort_flag));
                if (!ok) break;
                if (!check_tile(sv, t, keys_of(sv, gm, slen), gm.T)) {
                    if (lane == 0) mbar_arrive(p_full(sv.own, n));
                    continue;
                }
                const uint32_t at = sV + s * L::kTile + lane * 16;
                bool found = false;
#pragma unroll 1
                for (int i = 0; i < L::kTile; i += 4 * 512) {
                    uint4 w[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) w[x] = ld_shared_v4(at + i + x * 512);
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const uint32_t bx = __vcmpeq2(w[x].x & 0x7F807F80u, 0x7F807F80u);
                        const uint32_t by = __vcmpeq2(w[x].y & 0x7F807F80u, 0x7F807F80u);
                        const uint32_t bz = __vcmpeq2(w[x].z & 0x7F807F80u, 0x7F807F80u);
                        const uint32_t bw = __vcmpeq2(w[x].w & 0x7F807F80u, 0x7F807F80u);
                        if (bx | by | bz | bw) {
                            found = true;
                            st_shared_v4(at + i + x * 512, w[x].x & ~bx, w[x].y & ~by, w[x].z & ~bz,
                                         w[x].w & ~bw);
                        }
                    }
                }
                if (__any_sync(0xffffffffu, found)) {
                    if (lane == 0) poison[seg % kPoisonX] = seg + 1;
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full(sv.own, n));
            }
    } else {
        // ---------------------------------------------------------- softmax (warps 0..3)
        const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
        Walk ww = walk;
        Seg sg;
        bool ok = true;
        int n = 0;
        for (int seg = 0; ok && next_seg(ww, sg, gm, cum); ++seg) {
            const int r0 = warp * 32, r = r0 + lane;   // this warp's first row, this lane's row
            if (r0 >= rows_of(sg, gm)) {               // this warp has no row of the piece
                if (sg.own) break;                     // nor of any later one
                if (r0 >= gm.nb * gm.GT) {             // nor of any prefix piece
                    n += sg.t1 - sg.t0;
                    continue;
                }
                // the prefix's last row tile: keep step
                for (int t = sg.t0; t < sg.t1 && ok; ++t, ++n) {
                    ok = warp_wait(s_done(n % R), (uint32_t)(n / R) & 1u, err, abort_flag);
                    if (lane == 0) mbar_arrive(p_pre(n & 1));
                }
                continue;
            }
            const uint32_t t_o = tmem_base + L::kOCol + lane_off;
            // keys this row sees: all of the prefix, or the own ones up to its token
            const int keys = keys_of(sg, gm, slen);
            const int lim = sg.own ? keys - (gm.T - 1 - r % gm.T) : keys;
            const int full = sg.own ? keys - (gm.T - 1) : keys;        // keys that all rows see
            const bool mine = r < rows_of(sg, gm);
            float m = -INFINITY, l = 0.f;
            for (int t = sg.t0; t < sg.t1; ++t, ++n) {
                const int sb = n & 1;
                if (!warp_wait(s_done(n % R), (uint32_t)(n / R) & 1u, err, abort_flag)) { ok = false; break; }
                tc_fence_after();
                {
                    const uint32_t t_s = tmem_base + sb * kKeys + lane_off;
                    uint32_t sr[2][32];
                    tmem_ld32_issue(t_s, sr[0]);
                    tmem_ld32_issue(t_s + 32, sr[1]);
                    tmem_ld_wait();
                    reg_fence32(sr[0]);
                    reg_fence32(sr[1]);
                    float s[kKeys];
#pragma unroll
                    for (int e = 0; e < kKeys; ++e) s[e] = __uint_as_float(sr[e >> 5][e & 31]);
                    const int k0 = t * kKeys;
                    if (k0 + kKeys > full) {
                        const int d = lim - k0;
#pragma unroll
                        for (int e = 0; e < kKeys; ++e) s[e] = e >= d ? -INFINITY : s[e];
                    }
                    // row maximum: four independent chains of three-input maxima
                    float mx4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                    for (int e = 4; e + 8 <= kKeys; e += 8)
#pragma unroll
                        for (int i = 0; i < 4; ++i) mx4[i] = fmax3(mx4[i], s[e + 2 * i], s[e + 2 * i + 1]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) mx4[i] = fmaxf(mx4[i], s[kKeys - 4 + i]);
                    const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * scale_log2;
                    float corr = 1.f;
                    if (mx > m + kRescaleX) {
                        corr = fast_exp2(m - mx);
                        m = mx;
                    }
                    const bool need_rescale = __any_sync(0xffffffffu, corr != 1.f && t > sg.t0 && mine);
                    const uint64_t scale2 = f2_pack(scale_log2, scale_log2);
                    const float negm = m == -INFINITY ? 0.f : -m;     // no visible key yet: every p is 0
                    const uint64_t negm2 = f2_pack(negm, negm);
                    uint64_t sum2[4] = {0ull, 0ull, 0ull, 0ull};
                    // P in bf16, the operand's type beside V in bf16; the row sum adds the weights
                    // before that rounding (up to 2^-8 each, at random)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t pw[16];
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            float t0, t1;
                            f2_unpack(f2_fma(f2_pack(s[32 * h + e], s[32 * h + e + 1]), scale2, negm2), t0, t1);
                            const float p0 = fast_exp2(t0), p1 = fast_exp2(t1);
                            sum2[(e >> 1) & 3] = f2_add(sum2[(e >> 1) & 3], f2_pack(p0, p1));
                            pw[e >> 1] = pack_bf16x2(p0, p1);
                        }
                        tmem_st16_async(t_s + 16 * h, pw);
                    }
                    tmem_st_wait();
                    float sa[4], sb4[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) f2_unpack(sum2[e], sa[e], sb4[e]);
                    l = l * corr + (((sa[0] + sb4[0]) + (sa[1] + sb4[1])) + ((sa[2] + sb4[2]) + (sa[3] + sb4[3])));
                    if (need_rescale) {
                        // O must hold P_{n-1} V_{n-1}
                        if (!warp_wait(pv_done((n - 1) % R), (uint32_t)((n - 1) / R) & 1u, err, abort_flag)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < DH / 32; ++c) {
                            float v[32];
                            tmem_ld32(t_o + c * 32, v);
#pragma unroll
                            for (int e = 0; e < 32; ++e) v[e] *= corr;
                            tmem_st32(t_o + c * 32, v);
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full(sg.own, n));
            }
            if (!ok) break;
            if (!warp_wait(pv_done((n - 1) % R), (uint32_t)((n - 1) / R) & 1u, err, abort_flag)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const int64_t piece = job_of(sg, gm) + cta;
            const int stride = sg.own ? gm.GT : kRowsP;
            const int64_t row = piece * stride + r;
            float4* orow = reinterpret_cast<float4*>((sg.own ? out.o_own : out.o_prefix) + piece * stride * DH) + r;
            if (mine) (sg.own ? out.ml_own : out.ml_prefix)[row] = make_float2(m, l);
            if (threadIdx.x == 0) {
                int2* range = (sg.own ? out.range_own : out.range_prefix) + job_of(sg, gm);
                if (sg.t0 == 0) range->x = cta;
                if (sg.t1 == (sg.own ? cum[sg.x + 1] - cum[sg.x] : gm.np)) range->y = cta;
            }
#pragma unroll 1
            for (int c = 0; c < DH / 32; ++c) {
                float v[32];
                tmem_ld32(t_o + c * 32, v);
                if (mine) {
#pragma unroll
                    for (int e = 0; e < 32; e += 4)
                        orow[(c * 8 + e / 4) * stride] = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                }
                __syncwarp();
            }
            if (poison[seg % kPoisonX] == seg + 1 && mine) {
                // what the V check took out, for the keys this row sees
                const __nv_bfloat16* vb = vc + (int64_t)job_of(sg, gm) * gm.max_seq * DH;
#pragma unroll 1
                for (int t = sg.t0; t < sg.t1; ++t)
                    if (check_tile(sg, t, keys, gm.T))
                        put_back(reinterpret_cast<float*>(orow), stride * 4, vb, DH, t * kKeys,
                                 min((t + 1) * kKeys, lim));
            }
            __syncwarp();
            // O is read out before this warp publishes the next piece's first P
            tc_fence_before();
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 5) tmem_dealloc(tmem_base, 256);
}

// A thread joins four columns of a row, its pieces of the prefix job and of the
// own job, kAtOnce at a time: their maxima, sums and values are in flight together, so
// that a row costs one trip to L2 per kAtOnce pieces.  A CTA takes the 128 rows of a row
// tile, whose prefix pieces lie side by side.  Eight at once up to a wave of CTAs (16 answers
// of 5 tokens over 8192, 16 pieces a row: 20 us in all, four at once 22); with more rows
// there are few pieces each and four at once fit more CTAs on an SM (101 sequences of 8
// tokens over 64 shared ones, 16/4 x 128: 17.0 us, eight at once 18.6).
template <int DH, int kAtOnce>
__global__ void __launch_bounds__(kRowsP, kAtOnce == 8 ? 6 : 10) k_prefix_join(PrefixParts in, PrefixGeom gm, int H,
                                                        const int32_t* __restrict__ lens,
                                                        __nv_bfloat16* __restrict__ o) {
    constexpr int S = DH / 4;
    const int c4 = (int)blockIdx.x % S, pj = (int)blockIdx.x / S;
    const int g = pj / gm.nrt, rt = pj - g * gm.nrt, r = threadIdx.x;
    const int b = rt * gm.nb + r / gm.GT, i = r % gm.GT;
    pdl_wait();
    pdl_trigger();
    if (r >= gm.nb * gm.GT || b >= gm.B) return;
    // The pieces of a job: one per CTA from that of its first tile to that of its last.
    // (In bounds even where a kernel that gave up left them unwritten.)
    int n_pre = 0, n_own = 0, first_pre = 0, first_own = 0;
    auto pieces = [&](const int2 range, int& first, int& n) {
        first = min(max(range.x, 0), gm.ctas - 1);
        n = min(max(range.y, first), gm.ctas - 1) - first + 1;
    };
    const int keys = own_len(lens, b, gm.max_seq);
    const int2 range_own = __ldcg(in.range_own + b * gm.Hkv + g);
    if (gm.np) pieces(__ldcg(in.range_prefix + pj), first_pre, n_pre);
    if (keys) pieces(range_own, first_own, n_own);
    const int64_t pre = pj + first_pre, own = (int64_t)b * gm.Hkv + g + first_own;
    const float2* ml_pre = in.ml_prefix + pre * kRowsP + r;
    const float2* ml_own = in.ml_own + own * gm.GT + i;
    const float4* o_pre = reinterpret_cast<const float4*>(in.o_prefix) + (pre * S + c4) * kRowsP + r;
    const float4* o_own = reinterpret_cast<const float4*>(in.o_own) + (own * S + c4) * gm.GT + i;
    float M = -INFINITY, L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const int n = n_pre + n_own;
    for (int k0 = 0; k0 < n; k0 += kAtOnce) {
        float2 ml[kAtOnce];
        float4 v[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const int k = k0 + j;
            ml[j] = make_float2(-INFINITY, 0.f);
            v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (k < n_pre) {
                ml[j] = ml_pre[(int64_t)k * kRowsP];
                v[j] = o_pre[(int64_t)k * S * kRowsP];
            } else if (k < n) {
                ml[j] = ml_own[(int64_t)(k - n_pre) * gm.GT];
                v[j] = o_own[(int64_t)(k - n_pre) * S * gm.GT];
            }
        }
        float Mn = M;
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) Mn = fmaxf(Mn, ml[j].x);
        const float keep = M == -INFINITY ? 0.f : exp2f(M - Mn);
        // (the sum of pieces without a maximum is 0, or NaN if the scores are: it goes on)
        L = M == -INFINITY ? L : L * keep;
        acc = make_float4(acc.x * keep, acc.y * keep, acc.z * keep, acc.w * keep);
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            // A piece in which the row sees nothing holds (-inf, 0) and no value; one of
            // NaN scores alone (-inf, NaN).
            const bool none = ml[j].x == -INFINITY;
            const float w = none ? 0.f : exp2f(ml[j].x - Mn);
            L += none ? ml[j].y : w * ml[j].y;
            if (none) continue;
            acc.x = fmaf(w, v[j].x, acc.x);
            acc.y = fmaf(w, v[j].y, acc.y);
            acc.z = fmaf(w, v[j].z, acc.z);
            acc.w = fmaf(w, v[j].w, acc.w);
        }
        M = Mn;
    }
    const float inv = L == 0.f ? 0.f : 1.0f / L;       // no key at all: zeros
    const int hh = i / gm.T, t = i - hh * gm.T, h = g * (gm.GT / gm.T) + hh;
    *reinterpret_cast<uint2*>(o + ((int64_t)(b * gm.T + t) * H + h) * DH + c4 * 4) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

PrefixGeom geom_of(int B, int H, int Hkv, int T, int P, int max_seq, int dh) {
    PrefixGeom g{};
    g.B = B;
    g.Hkv = Hkv;
    g.T = T;
    g.GT = H / Hkv * T;
    g.P = P;
    g.max_seq = max_seq;
    g.nb = kRowsP / g.GT;
    if (g.nb > B) g.nb = B > 0 ? B : 1;
    g.nrt = (B + g.nb - 1) / g.nb;
    g.np = (int)(((int64_t)P + kKeys - 1) / kKeys);
    // swizzle atoms are 8 rows of 128 bytes, or 16 of 64
    const int atom = dh == 32 ? 16 : 8;
    g.q_pad = (g.GT + atom - 1) / atom * atom;
    g.q_slots = kRowsP / g.q_pad < 8 ? kRowsP / g.q_pad : 8;
    return g;
}

struct PrefixLayout {
    size_t o_prefix, ml_prefix, o_own, ml_own, range_prefix, range_own, total;
};
PrefixLayout layout(const PrefixGeom& g, int dh) {
    PrefixLayout l{};
    const size_t np = (size_t)g.Hkv * g.nrt + kMaxCtas, no = (size_t)g.B * g.Hkv + kMaxCtas;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off += up256(bytes);
        return at;
    };
    l.o_prefix = take(np * kRowsP * dh * 4);
    l.ml_prefix = take(np * kRowsP * 8);
    l.o_own = take(no * g.GT * dh * 4);
    l.ml_own = take(no * g.GT * 8);
    l.range_prefix = take((size_t)g.Hkv * g.nrt * 8);
    l.range_own = take((size_t)g.B * g.Hkv * 8);
    l.total = off;
    return l;
}

template <int DH>
cudaError_t launch_dh(const PrefixArgs& a, PrefixGeom g, const CUtensorMap* maps, cudaStream_t st) {
    using L = Px<DH>;
    const int smem = L::kBase + 4 * (3 * a.B + 2);
    // room for the largest batch (two CTAs of the common sizes fit an SM all the same)
    static std::atomic<uint64_t> done{0};
    cudaError_t e = allow_smem(done, k_prefix_part<DH>, L::kBase + 4 * (3 * 4096 + 2));
    if (e != cudaSuccess) return e;
    const PrefixLayout l = layout(g, DH);
    uint8_t* w = static_cast<uint8_t*>(a.ws);
    PrefixParts parts;
    parts.o_prefix = reinterpret_cast<float*>(w + l.o_prefix);
    parts.ml_prefix = reinterpret_cast<float2*>(w + l.ml_prefix);
    parts.o_own = reinterpret_cast<float*>(w + l.o_own);
    parts.ml_own = reinterpret_cast<float2*>(w + l.ml_own);
    parts.range_prefix = reinterpret_cast<int2*>(w + l.range_prefix);
    parts.range_own = reinterpret_cast<int2*>(w + l.range_own);
    // two CTAs per SM; no more than there can be tiles
    const int64_t most = (int64_t)g.Hkv * g.nrt * g.np +
                         (int64_t)g.B * g.Hkv * (((int64_t)a.max_seq + kKeys - 1) / kKeys);
    g.ctas = 2 * sm_count() < kMaxCtas ? 2 * sm_count() : kMaxCtas;
    if (most < g.ctas) g.ctas = (int)most;
    e = launch_pdl(k_prefix_part<DH>, dim3((unsigned)g.ctas), dim3(kThreadsX), smem, st, maps[0], maps[1], maps[2],
                   maps[3], maps[4], maps[5], static_cast<const __nv_bfloat16*>(a.vc), a.lens, g, parts,
                   a.scale * 1.4426950408889634f, device_error_word());
    if (e != cudaSuccess) return e;
    const unsigned join = (unsigned)(g.Hkv * g.nrt * (DH / 4));
    auto* const o = static_cast<__nv_bfloat16*>(a.o);
    return join > (unsigned)(6 * sm_count()) ? launch_pdl(k_prefix_join<DH, 4>, dim3(join), dim3(kRowsP), 0, st, parts, g, a.H, a.lens, o)
                        : launch_pdl(k_prefix_join<DH, 8>, dim3(join), dim3(kRowsP), 0, st, parts, g, a.H, a.lens, o);
}

}  // namespace

size_t prefix_workspace_bytes(int B, int H, int Hkv, int T, int dh) {
    return layout(geom_of(B, H, Hkv, T, 0, 1, dh), dh).total;
}

int64_t prefix_key_tiles(int B, int H, int Hkv, int T, int P, int max_seq) {
    const PrefixGeom g = geom_of(B, H, Hkv, T, P, max_seq, 64);
    return (int64_t)g.Hkv * g.nrt * g.np + (int64_t)g.B * g.Hkv * (((int64_t)g.max_seq + kKeys - 1) / kKeys);
}

tfm_status launch_prefix_attention(const PrefixArgs& a, cudaStream_t st, cudaError_t* e) {
    const PrefixGeom g = geom_of(a.B, a.H, a.Hkv, a.T, a.P, a.max_seq, a.dh);
    CUtensorMap maps[6];
    if (!query_groups_map(&maps[0], a.q, a.B, a.Hkv, g.GT, a.dh, g.nb) ||
        !query_groups_map(&maps[1], a.q, a.B, a.Hkv, g.GT, a.dh, 1) ||
        !rows_heads_map(&maps[4], a.kc, a.max_seq, (int64_t)a.B * a.Hkv, a.dh, a.dh, (int64_t)a.max_seq * a.dh, kKeys) ||
        !rows_heads_map(&maps[5], a.vc, a.max_seq, (int64_t)a.B * a.Hkv, a.dh, a.dh, (int64_t)a.max_seq * a.dh, kKeys))
        return TFM_ECUDA;
    maps[2] = maps[4];                                 // without a prefix its maps are never used
    maps[3] = maps[5];
    if (a.P > 0 &&
        (!rows_heads_map(&maps[2], a.kp, a.P, a.Hkv, a.dh, a.dh, (int64_t)a.max_prefix * a.dh, kKeys) ||
         !rows_heads_map(&maps[3], a.vp, a.P, a.Hkv, a.dh, a.dh, (int64_t)a.max_prefix * a.dh, kKeys)))
        return TFM_ECUDA;
    *e = a.dh == 32   ? launch_dh<32>(a, g, maps, st)
         : a.dh == 64 ? launch_dh<64>(a, g, maps, st)
                      : launch_dh<128>(a, g, maps, st);
    return TFM_OK;
}

}  // namespace tfm
