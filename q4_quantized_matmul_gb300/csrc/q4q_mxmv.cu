// q4q_mxmv.cu -- products of MXFP4 weights with up to 8 tokens (dense, or per expert).
//
// The same product as q4q_mxmm.cu where all that matters is to stream the weights once at
// HBM speed and to be short around it: one launch, no workspace.  Of the 0.53 bytes a weight
// takes every byte is read once; the tensor core does the rest far below its rate.
//
// A tile is 128 weight rows; a cluster of S CTAs splits its K, and one to three CTAs share
// an SM with rings as deep as its shared memory allows (pick_spread).
//   warp 0    : TMA producer: weight codes (in the 128-byte swizzle, widened to bytes for
//               E4M3 activations) and scales, one atom of 128 shared-memory bytes a row a
//               stage.  It starts before the work queued ahead is done.
//   warp 1    : tensor memory and MMA issuer.
//   warps 2-5 : encode the activations of each atom straight into the stage (each CTA its
//               own part of K; the same arithmetic as q4q_mxfp4.cu), then the epilogue.
// The S partial tiles are joined over distributed shared memory: CTA z adds, in the order
// of K, the z-th part of the tile's values of all S CTAs and stores it.
//
// Every mbarrier wait is bounded (one that runs out records Q4Q_ERR_TIMEOUT and makes the
// CTA wind down); all threads of a cluster reach its barriers whatever happened before.
#include <algorithm>
#include <atomic>
#include <cuda.h>
#include <mutex>

#include "q4q_internal.h"
#include "q4q_mx.cuh"
#include "q4q_mx_internal.h"
#include "q4q_mx_tc.cuh"

namespace q4q {
namespace {

__device__ unsigned int g_mxmv_status = 0;

constexpr int BN = MXMV_TOKENS;
constexpr int THREADS = 192;
constexpr int ENC = 128;                      // encoder threads
constexpr int MAX_ST = 12;
constexpr int MAX_PER_SM = 3;                 // CTAs of an SM
constexpr int MAX_SPLIT = 8;                  // portable cluster size

struct MvParams {
    const void* x;
    int64_t n_src, n_rows;
    int K, M, atoms, st, nkc, n_mats, mtiles, top_k, dst_type;
    const int32_t* first;        // experts' first rows, or null (dense)
    const int32_t* slot;
    int64_t max_groups;
    const uint8_t* w_scales;
    int64_t mat_stride;
    void* dst;
    bool vec;
    uint64_t limit_ns;
    int fault;
};

template <bool E4M3>
struct Mv {
    static constexpr int ATOM_K = E4M3 ? 128 : 256;
    static constexpr int CH = ATOM_K / 128;
    static constexpr int A_BYTES = BM * 128;
    static constexpr int B_BYTES = BN * 128;
    static constexpr int CHUNK = mx_chunk_bytes(BN);
    // Weight scales come GROUP atoms at a time, in groups(st) buffers: a group's buffer is free
    // again once the atom `st` before its first has been read.  (Copying rows of 64 bytes, the
    // copy engine is the limit with E4M3 activations: an atom takes it 0.17 us, and every
    // further copy 0.045, measured on one SM.)
    static constexpr int GROUP = E4M3 ? 4 : 1;
    static constexpr int GROUP_BYTES = GROUP * CH * MX_CHUNK;
    __host__ __device__ static constexpr int groups(int st) { return (st + 2 * GROUP - 2) / GROUP; }
    static constexpr int SFB_BYTES = CH * CHUNK;
    static constexpr int STAGE = A_BYTES + B_BYTES + SFB_BYTES;
    // barriers in front (with room to align the stages: 1024 bytes, the swizzle's atoms); then
    // all stages' A tiles, their B tiles, the weight scales, the activation scales.  The last
    // chunk's copy to tensor memory reads 512 bytes from its start.
    static constexpr int FIXED = 1024 + 512 + 512;
    static constexpr int stages(int per_sm) {
        int st = MAX_ST;
        while (smem(st) + 1024 > 228 * 1024 / per_sm) --st;
        return st;
    }
    static constexpr int smem(int st) { return FIXED + st * STAGE + groups(st) * GROUP_BYTES; }
    static constexpr int TX = E4M3 ? A_BYTES / 2 : A_BYTES;     // bytes that an atom's copy reads
    static constexpr int AHEAD = 6;                              // passes of the encoders whose loads are in flight
    static constexpr int SFA_COL = BN, SFB_COL = BN + 4 * CH;
    static constexpr int COLS = 32;
    static_assert(SFB_COL + 4 * CH <= COLS && stages(MAX_PER_SM) >= 4, "three CTAs fit an SM");
};

template <typename T, bool E4M3>
__global__ void __launch_bounds__(THREADS, MAX_PER_SM) mxmv_kernel(const __grid_constant__ CUtensorMap tmap_w, const MvParams p) {
    using C = Mv<E4M3>;
    extern __shared__ uint8_t smem_raw[];
    const int ST = p.st;
    uint8_t* smem = smem_raw + 512 + ((1024u - ((smem_u32(smem_raw) + 512) & 1023u)) & 1023u);
    const uint32_t sbase = smem_u32(smem), bars = smem_u32(smem_raw);
    const uint32_t full = bars, empty = bars + 8 * MAX_ST, done = empty + 8 * MAX_ST, slot_addr = done + 8;
    volatile int* stop = reinterpret_cast<volatile int*>(smem_raw + 16 * MAX_ST + 16);
    volatile int* freed = stop + 1;
    const uint32_t b_base = sbase + ST * C::A_BYTES, sfa_base = b_base + ST * C::B_BYTES;
    const int groups = C::groups(ST), sfb_off = ST * (C::A_BYTES + C::B_BYTES) + groups * C::GROUP_BYTES;
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    uint32_t rank, ctas;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
    auto gave_up = [&]() {
        *stop = 1;
        record_error(&g_mxmv_status, DEV_TIMEOUT);
    };
    auto wait = [&](uint32_t bar, uint32_t parity) {          // the whole warp
        bool ok = mbar_try_wait(bar, parity) || mbar_wait_until(bar, parity, stop, p.limit_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok && lane == 0 && !*stop) gave_up();
        return ok;
    };

    pdl_trigger();
    if (threadIdx.x == 0) prefetch_map(&tmap_w);

    // the tile of this cluster
    int64_t tile = blockIdx.x / ctas;
    int mat = 0, m0 = 0, valid = 0;
    int64_t row0 = 0;
    if (p.first) {
        pdl_wait();                                           // the sort may still be running
        int* start = reinterpret_cast<int*>(smem);            // the segments, where the stages will be
        int* units = start + MX_MAX_EXPERTS + 1;
        mx_segments(p.first, p.n_mats, p.n_rows, BN, p.max_groups, start, units, units + MX_MAX_EXPERTS + 1);
        const int64_t groups_all = units[p.n_mats];
        if (tile < groups_all * p.mtiles) {
            // weights outermost within an expert, as its rows rarely take more than one token tile
            int lo = 0, hi = p.n_mats;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if ((int64_t)units[mid] * p.mtiles <= tile) lo = mid;
                else hi = mid;
            }
            const int groups = units[lo + 1] - units[lo];
            const int in = (int)(tile - (int64_t)units[lo] * p.mtiles);
            mat = lo;
            m0 = in / groups * BM;
            row0 = start[lo] + (int64_t)(in % groups) * BN;
            valid = (int)min((int64_t)BN, start[lo + 1] - row0);
        }
        // rows of no expert are zeros
        const int64_t from = (int64_t)start[p.n_mats] * p.M, to = p.n_rows * p.M;
        for (int64_t i = from + (int64_t)blockIdx.x * THREADS + threadIdx.x; i < to; i += (int64_t)gridDim.x * THREADS)
            mx_store(p.dst, p.dst_type, i, 0.0f);
    } else {
        m0 = (int)tile * BM;
        valid = (int)p.n_rows;
    }
    // From lane 0, so that the compiler knows these to be the same in the whole warp: a loop
    // whose bounds it does not know to be keeps the MMAs' descriptors out of uniform registers
    // (measured: 620 cycles an atom of 4 MMAs instead of 180).
    valid = __shfl_sync(0xffffffffu, valid, 0);
    m0 = __shfl_sync(0xffffffffu, m0, 0);
    mat = __shfl_sync(0xffffffffu, mat, 0);
    const int a0 = __shfl_sync(0xffffffffu, (int)((int64_t)p.atoms * rank / ctas), 0);
    const int n_atoms = __shfl_sync(0xffffffffu, valid > 0 ? (int)((int64_t)p.atoms * (rank + 1) / ctas) - a0 : 0, 0);
    if (p.first) {                                            // the segments' bytes are the stages' next
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncthreads();
    }

    const bool lead = elect_one();
    const bool skip = p.fault && blockIdx.x == 0;
    auto load = [&](int i, int s) {
        const uint32_t bar = full + 8 * s;
        const int at = a0 + i;
        int scales = 0;
        if (i % C::GROUP == 0)                                // the scales of this atom and the next GROUP - 1
            scales = min(min(C::GROUP, n_atoms - i) * C::CH, p.nkc - at * C::CH) * MX_CHUNK;
        mbar_arrive_expect_tx(bar, C::TX + scales);
        tma_load_4d(sbase + s * C::A_BYTES, &tmap_w, 0, m0, at, mat, bar);
        if (scales)
            bulk_g2s(sfa_base + i / C::GROUP % groups * C::GROUP_BYTES,
                     p.w_scales + mat * p.mat_stride + ((int64_t)(m0 / BM) * p.nkc + at * C::CH) * MX_CHUNK, scales, bar);
    };
    // The encoders take (atom, token) units in order, LANES lanes a unit: unit u is token
    // u % valid of atom u / valid, so their work goes with the tokens there are.
    constexpr int LANES = C::ATOM_K / 8, PASS = ENC / LANES;
    const int tid = (int)threadIdx.x - 64, col = (tid & (LANES - 1)) * 8;
    const int unit0 = tid / LANES, units_all = n_atoms * valid;
    MxRaw<T> v[C::AHEAD];
    // Loads without a branch around them (from row 0 where there is nothing to load), so that
    // all of them are in flight before the first is looked at.
    auto fetch = [&](int u, MxRaw<T>& x) {
        const int i = u / max(valid, 1);
        int c = (a0 + i) * C::ATOM_K + col;
        int64_t from = row0 + (u - i * valid);
        x.live = u < units_all && c < p.K;
        if (!x.live) from = row0, c = 0;
        if (p.slot && valid > 0) from = (int64_t)__ldg(p.slot + from) / p.top_k;
        x.live = x.live && from >= 0 && from < p.n_src;
        if (!x.live) from = 0, c = 0;
        x.load(static_cast<const T*>(p.x) + from * p.K + c, p.vec);
    };
    if (warp == 0) {
        if (lead) {
            for (int s = 0; s < ST; ++s) {
                mbar_init(full + 8 * s, 1 + valid);           // the copies, and each token's codes
                mbar_init(empty + 8 * s, 1);
            }
            mbar_init(done, 1);
            *stop = 0;
            *freed = ST;
            fence_mbar_init();
        }
        __syncwarp();
    } else if (warp == 1) {
        tmem_alloc(slot_addr, C::COLS);
    } else {
        pdl_wait();
#pragma unroll
        for (int h = 0; h < C::AHEAD; ++h) fetch(unit0 + h * PASS, v[h]);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    uint32_t tmem;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(slot_addr));
    tmem = __shfl_sync(0xffffffffu, tmem, 0);

    if (warp == 0) {
        // ---------------- producer: weights do not depend on the work queued ahead
        if (lead)
            for (int i = skip ? 1 : 0; i < min(n_atoms, ST); ++i) load(i, i);
        __syncwarp();
        int i = ST, s = 0;
        uint32_t parity = 0;
        for (; i < n_atoms; ++i) {
            if (!wait(empty + 8 * s, parity)) break;
            if (lead) {
                *freed = i + 1;
                load(i, s);
            }
            if (++s == ST) {
                s = 0;
                parity ^= 1;
            }
        }
        // after an abort, nothing may land in a CTA that has gone; where the encoders have given
        // up too, that means waiting out the limit (far longer than a copy takes)
        if (*stop && lead)
            for (int j = max(skip ? 1 : 0, min(i, n_atoms) - ST); j < min(i, n_atoms); ++j)
                if (!mbar_wait_bounded(full + 8 * (j % ST), (j / ST) & 1, p.limit_ns)) break;
    } else if (warp == 1) {
        // ---------------- MMA issuer
        constexpr uint32_t IDESC = ((uint32_t)(BN >> 3) << 17) | (1u << 23) | ((uint32_t)(BM >> 7) << 27) |
                                   (E4M3 ? (5u << 7) : (1u << 7) | (1u << 10));
        int s = 0, group = 0;
        uint32_t parity = 0;
        for (int i = 0; i < n_atoms; ++i) {
            if (!wait(full + 8 * s, parity)) break;
            tc_fence_after();
            if (lead) {
                const uint32_t sfa = sfa_base + group * C::GROUP_BYTES + i % C::GROUP * (C::CH * MX_CHUNK);
                const uint32_t sfb = sbase + sfb_off + s * C::SFB_BYTES;
#pragma unroll
                for (int c = 0; c < C::CH; ++c) {
                    scales_to_tmem(tmem + C::SFA_COL + 4 * c, desc_scales(sfa + c * MX_CHUNK));
                    scales_to_tmem(tmem + C::SFB_COL + 4 * c, desc_scales(sfb + c * C::CHUNK));
                }
                const uint64_t a = desc_sw128(sbase + s * C::A_BYTES), b = desc_sw128(b_base + s * C::B_BYTES);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t c = E4M3 ? 0 : j >> 1, id = E4M3 ? j : (j & 1) * 2;
                    mma_mx<E4M3>(tmem, a + (uint64_t)(j * 2), b + (uint64_t)(j * 2), IDESC | (id << 4) | (id << 29),
                                 tmem + C::SFA_COL + 4 * c, tmem + C::SFB_COL + 4 * c, i > 0 || j > 0);
                }
                mma_commit(empty + 8 * s);
            }
            __syncwarp();
            if (i % C::GROUP == C::GROUP - 1 && ++group == groups) group = 0;
            if (++s == ST) {
                s = 0;
                parity ^= 1;
            }
        }
        if (lead) mma_commit(done);
        __syncwarp();
    } else {
        // ---------------- encoders
        bool ok = true;
        auto free_through = [&](int last) {
            uint64_t t0 = 0;
            bool yes = true;
            for (uint32_t n = 1; *freed <= last; ++n) {
                if ((n & 63u) != 0u) continue;
                const uint64_t t = global_timer_ns();
                if (t0 == 0) t0 = t;
                if (*stop || t - t0 > p.limit_ns) {
                    yes = false;
                    break;
                }
            }
            yes = __all_sync(0xffffffffu, yes);
            if (!yes && lane == 0 && !*stop) gave_up();
            return yes;
        };
        // AHEAD passes are encoded from the loads in flight, then one fence and their arrivals,
        // then the next loads: a fence between would wait for loads as well as for stores.
        for (int u0 = unit0; u0 - unit0 < units_all && ok; u0 += C::AHEAD * PASS) {
            int told = 0;                                     // passes of this round handed over
            auto hand_over = [&](int upto) {
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if ((tid & (LANES - 1)) == 0)
                    for (int h = told; h < upto; ++h) {
                        const int u = u0 + h * PASS;
                        if (u < units_all) mbar_arrive(full + 8 * (u / valid % ST));
                    }
                told = upto;
            };
#pragma unroll
            for (int h = 0; h < C::AHEAD; ++h) {
                const int u = u0 + h * PASS;
                if (u - unit0 >= units_all) break;            // the same for the whole CTA
                const int i = u / valid, r = u - i * valid, s = i % ST;
                const bool mine = u < units_all;
                // Atoms are encoded by whichever warp has them, so no warp follows a slot through
                // its phases (whose parity alone would not tell them apart): the producer does,
                // and publishes the first atom whose slot it has not seen free.
                const int last = min((u0 - unit0 + h * PASS + (tid & ~31) / LANES + 32 / LANES - 1) / valid, n_atoms - 1);
                if (last >= ST && !__all_sync(0xffffffffu, *freed > last)) {
                    hand_over(h);
                    if (!free_through(last)) {
                        ok = false;
                        break;
                    }
                }
                float x[8];
                uint32_t w[2];
                v[h].values(x);
                const uint32_t byte = mx_encode8<E4M3>(x, v[h].live, w);
                if (mine) {
                    uint8_t* b = smem + ST * C::A_BYTES + s * C::B_BYTES;
                    uint8_t* sf = smem + sfb_off + s * C::SFB_BYTES;
                    // the 128-byte swizzle: 16-byte unit q of row r lies at q ^ (r % 8)
                    const int at = E4M3 ? col : col / 2;
                    uint8_t* to = b + r * 128 + (((at >> 4) ^ (r & 7)) << 4) + (at & 15);
                    if constexpr (E4M3) *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
                    else *reinterpret_cast<uint32_t*>(to) = w[0];
                    if ((tid & 3) == 0) sf[(col >> 7) * C::CHUNK + r * 16 + ((col >> 5) & 3)] = (uint8_t)byte;
                }
            }
            if (!ok) break;
            hand_over(C::AHEAD);
#pragma unroll
            for (int h = 0; h < C::AHEAD; ++h)
                if (u0 - unit0 + (h + C::AHEAD) * PASS < units_all) fetch(u0 + (h + C::AHEAD) * PASS, v[h]);
        }
    }

    // ---------------- epilogue
    __syncwarp();
    const int quad = warp & 3, row = quad * 32 + lane;
    uint32_t r[BN];
    bool good = false;
    if (warp >= 2) {
        good = wait(done, 0) && !*stop;
        tc_fence_after();
        if (good) tmem_ld<BN>(tmem + ((uint32_t)(quad * 32) << 16), r);
        tc_fence_before();
        if (ctas == 1 && good && m0 + row < p.M) {
#pragma unroll
            for (int c = 0; c < BN; ++c)
                if (c < valid) mx_store(p.dst, p.dst_type, (row0 + c) * p.M + m0 + row, __uint_as_float(r[c]));
        }
    }
    if (ctas > 1) {
        // every stage has been read: the partial tile [token][row] takes its place
        float* part = reinterpret_cast<float*>(smem);
        if (warp >= 2 && good) {
#pragma unroll
            for (int c = 0; c < BN; ++c) part[c * BM + row] = __uint_as_float(r[c]);
        }
        cluster_arrive();
        cluster_wait();
        for (int e = (int)rank * THREADS + threadIdx.x; e < valid * BM; e += (int)ctas * THREADS) {
            const int m = m0 + e % BM;
            float sum = 0.0f;
            for (uint32_t z = 0; z < ctas; ++z) {
                float f;
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(f) : "r"(mapa_shared(sbase + 4 * e, z)) : "memory");
                sum = z == 0 ? f : __fadd_rn(sum, f);
            }
            if (m < p.M) mx_store(p.dst, p.dst_type, (row0 + e / BM) * p.M + m, sum);
        }
        // no CTA leaves while another may still read its part
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    if (warp == 1) tmem_dealloc(tmem, C::COLS);
}

// How the tiles are spread: CTAs a tile's K is split over, CTAs an SM holds.
struct Spread {
    int split, per_sm;
};

// What each choice is expected to take, in ns (constants measured on the device).  A CTA
// starts up and ends in about 3600, takes 220 for an atom and 2000 to join a split tile;
// each further CTA of an SM starts 700 later; HBM gives 6500 bytes a ns.  places[s]:
// clusters of s CTAs that the device holds at one CTA an SM.
//   4096 x 14336, 1 token (112 tiles of 32 atoms): 11.7 us unsplit at 1 CTA an SM, 9.5 split
//   in 2 at 2, 10.1 in 3 at 3, 13.9 in 4 at 3; 768 x 50257, 7 tokens (393 tiles of 3 atoms):
//   18.7 unsplit at 1, 13.2 at 2, 9.6 at 3; 6 such tiles' rows of 4096 x 14336 experts: 50.7
//   at 1, 35.4 at 2, 36.0 at 3, 46.7 split in 2 at 2.
Spread pick_spread(int64_t tiles, int atoms, int atom_bytes, const int (&places)[MAX_SPLIT + 1], int sm_count) {
    Spread best{1, 1};
    double least = 1e30;
    for (int s = 1; s <= MAX_SPLIT && s <= atoms; ++s)
        for (int q = 1; q <= MAX_PER_SM; ++q) {
            const int64_t held = (int64_t)places[s] * q;
            if (held < 1) continue;
            const int64_t rounds = (tiles + held - 1) / held;
            const int64_t ctas = std::min(tiles, held) * s;
            const double of_ctas = (double)rounds * (3600 + 220 * ((atoms + s - 1) / s) + (s > 1 ? 2000 : 0));
            const double of_hbm = (double)tiles * atoms * atom_bytes / 6500 + 3600;
            const double cost = std::max(of_ctas, of_hbm) + 700.0 * ((ctas + sm_count - 1) / sm_count - 1);
            if (cost < least) {
                least = cost;
                best = Spread{s, q};
            }
        }
    return best;
}

// clusters of each size that the device holds at one CTA an SM; not known before the first call
struct Places {
    std::atomic<int> known;
    int n[MAX_SPLIT + 1];
};

template <typename T, bool E4M3>
q4q_status launch_t(const CUtensorMap& tw, MvParams p, int64_t tiles, bool pdl, cudaStream_t stream, const DeviceInfo& info) {
    using C = Mv<E4M3>;
    static Places places[64];
    static std::mutex mutex;
    auto kern = mxmv_kernel<T, E4M3>;
    if (info.device < 0 || info.device >= 64) return Q4Q_ERR_CUDA;
    constexpr int stages[MAX_PER_SM + 1] = {0, C::stages(1), C::stages(2), C::stages(3)};
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(THREADS);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    Places& here = places[info.device];
    if (!here.known.load(std::memory_order_acquire)) {
        std::lock_guard<std::mutex> lock(mutex);
        // all of the SM's memory as shared: by default it may hold one CTA's and no more
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem(stages[1])) != cudaSuccess ||
            cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) != cudaSuccess)
            return (cudaGetLastError(), Q4Q_ERR_CUDA);
        for (int s = 1; s <= MAX_SPLIT; ++s) {
            attr[0].val.clusterDim.x = (unsigned)s;
            cfg.gridDim = dim3((unsigned)s);
            cfg.dynamicSmemBytes = C::smem(stages[1]);
            if (cudaOccupancyMaxActiveClusters(&here.n[s], kern, &cfg) != cudaSuccess) return (cudaGetLastError(), Q4Q_ERR_CUDA);
        }
        here.known.store(1, std::memory_order_release);
    }
    const Spread pick = pick_spread(tiles, p.atoms, C::TX + C::CH * MX_CHUNK, here.n, info.sm_count);
    p.st = stages[pick.per_sm];
    attr[0].val.clusterDim.x = (unsigned)pick.split;
    cfg.gridDim = dim3((unsigned)(tiles * pick.split));
    cfg.dynamicSmemBytes = C::smem(p.st);
    cfg.numAttrs = pdl ? 2 : 1;
    if (cudaLaunchKernelEx(&cfg, kern, tw, p) != cudaSuccess) return (cudaGetLastError(), Q4Q_ERR_CUDA);
    return launch_status();
}

}  // namespace

unsigned int mxmv_take_device_status() {
    unsigned int v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_mxmv_status, sizeof(v)) != cudaSuccess) return Q4Q_ERR_CUDA;
    if (v) cudaMemcpyToSymbol(g_mxmv_status, &z, sizeof(z));
    return v;
}

q4q_status mxmv_run(const void* src0, int64_t ne00, int64_t ne01, int n_mats, const MxActs& m, void* dst, int dst_type,
                    bool pdl, cudaStream_t stream, const DeviceInfo& info, const KernelDebug* dbg) {
    const bool e4m3 = m.acts == Q4Q_ACTS_MXFP8;
    const int64_t kp = mx_up(ne00, MX_KP);
    CUtensorMap tw;
    if (!mx_encode_weight_map(&tw, src0, ne00, ne01, n_mats, e4m3, 1)) return Q4Q_ERR_CUDA;
    MvParams p;
    p.x = m.src;
    p.n_src = m.n_src;
    p.n_rows = m.n_rows;
    p.K = (int)ne00;
    p.M = (int)ne01;
    p.atoms = (int)((ne00 + (e4m3 ? 127 : 255)) / (e4m3 ? 128 : 256));
    p.nkc = (int)(kp / 128);
    p.n_mats = n_mats;
    p.mtiles = (int)((ne01 + BM - 1) / BM);
    p.top_k = m.top_k;
    p.dst_type = dst_type;
    p.first = m.first;
    p.slot = m.slot;
    // token tiles: every segment starts a new one
    p.max_groups = m.first ? (m.n_rows + BN - 1) / BN + std::min<int64_t>(n_mats, m.n_rows) : 1;
    p.w_scales = static_cast<const uint8_t*>(src0) + mx_code_bytes(ne00, ne01);
    p.mat_stride = mx_code_bytes(ne00, ne01) + mx_scale_bytes(ne00, ne01);
    p.dst = dst;
    p.vec = aligned(m.src, 16);
    p.limit_ns = dbg ? dbg->limit_ns : WAIT_LIMIT_NS;
    p.fault = dbg ? dbg->fault : 0;
    // with few rows no more than one token tile for each of them
    const int64_t tiles = p.mtiles * (m.first ? std::min<int64_t>(p.max_groups, m.n_rows) : 1);
    if (tiles * MAX_SPLIT >= (1ll << 31)) return Q4Q_ERR_SHAPE;
    switch (m.type) {
        case Q4Q_TYPE_F32: return e4m3 ? launch_t<float, true>(tw, p, tiles, pdl, stream, info) : launch_t<float, false>(tw, p, tiles, pdl, stream, info);
        case Q4Q_TYPE_F16: return e4m3 ? launch_t<__half, true>(tw, p, tiles, pdl, stream, info) : launch_t<__half, false>(tw, p, tiles, pdl, stream, info);
        default: return e4m3 ? launch_t<__nv_bfloat16, true>(tw, p, tiles, pdl, stream, info) : launch_t<__nv_bfloat16, false>(tw, p, tiles, pdl, stream, info);
    }
}

}  // namespace q4q
