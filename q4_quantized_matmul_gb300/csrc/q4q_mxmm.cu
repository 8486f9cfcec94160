// q4q_mxmm.cu -- products of MXFP4 weights on the block-scaled tensor cores, dense
// (q4q_mul_mat_mxfp4) and by expert (q4q_mul_mat_id_mxfp4).
//
//   dst[n][m] = sum_b 2^(ew[m][b] + ex[n][b]) * sum_{k in block b} w[m][k] * x[n][k]
//
// with w in E2M1 and x, encoded on the fly (q4q_mxfp4.cu), in E2M1 (kind::mxf4) or E4M3
// (kind::mxf8f6f4).  The tensor core takes codes and scales as they lie in memory, so
// nothing is unpacked by CUDA cores at any token count; the weight rows are the MMA's M and
// the tokens its N.  All products of two E2M1 values are multiples of 1/4 up to 36 and the
// accumulator is fp32.
//
// Roles (one CTA per SM, 384 threads):
//   warp 0    : TMA producer.  A stage is one or more atoms of 128 bytes of each smem row
//               (256 K of packed E2M1, or 128 K of E4M3 with the weights widened by the
//               tensor map to one byte each, 16U4_ALIGN16B: HBM still moves the packed
//               nibbles) and their scale chunks, in four copies.  The ring fills what
//               shared memory there is; the weights of the first stages do not wait for
//               the activation encoder, behind which the kernel is launched with
//               programmatic dependent launch.
//   warp 1    : MMA issuer: scale chunks to tensor memory (tcgen05.cp), 4 MMAs an atom.
//   warps 4-11: epilogue: accumulator (two of them while 2 BN <= 256 columns) through
//               registers to dst.
//
// Three ways to spread the tiles, picked by the expected time (pick_tile):
//   one CTA a tile of 128 rows x 8 to 64 tokens; CTA c takes tiles c, c + CTAs, ..., so that
//     neighbouring CTAs walk K together and what one reads from HBM others find in L2;
//   a pair of CTAs a tile of 256 rows x 64 to 256 tokens: each loads its 128 rows and half
//     of the tokens, the first issues the pair's MMAs (cta_group::2), which halves what the
//     token side costs in copies;
//   few tiles: a cluster of 2 to 8 CTAs shares the K of a tile of 8 to 64 tokens; each sends
//     its part of a token over distributed shared memory to the CTA that adds the token up, in
//     the order of K (fetching the parts instead: 4096 x 4096, 1 token, 7.85 us, sent 7.45).
//
// What bounds it: a CTA's copies take 1.05 ns a shared-memory row (128 bytes, two cycles),
// so an atom of 128 + 16 rows 0.165 us and of a pair's 128 + 128 rows 0.28; its MMAs 0.14 us
// up to 128 tokens, 0.27 with 256 (the tensor pipe's active time over the atoms of a launch: 12.8 us
// for 47 at 512 tokens, 25.2 for 94 at 2048).  So few tokens are bound by copies.  In the widest
// tiles an atom takes 0.27 to 0.31 us in all: MMAs and copies keep pace, and either bounds a round.
// That is why two pairs that shared their tokens by multicast, a quarter less from L2, took the same
// time (2048 tokens 14336 x 4096: 51.0 us, 51.2), as did tiles with fewer tokens than 256 and MMAs
// and copies of only so many.  The 40 to 56% of such a launch in which the tensor pipe rests are
// rounds that do not fill the device, the start, and reading a tile out: 256 columns have one
// accumulator, and the next tile's MMAs wait for it.
//
// Every mbarrier wait is bounded; one that runs out records Q4Q_ERR_TIMEOUT, raises the
// call's abort word (zeroed by the activation encoder before every launch) and the CTA
// winds down: it waits for its own copies, frees its tensor memory and returns.
#include <algorithm>
#include <atomic>
#include <cuda.h>
#include <cudaTypedefs.h>
#include <mutex>

#include "q4q_internal.h"
#include "q4q_mx.cuh"
#include "q4q_mx_tc.cuh"
#include "q4q_mx_internal.h"

namespace q4q {
namespace {

__device__ unsigned int g_mxmm_status = 0;

constexpr int EPI_WARPS = 8;
constexpr int THREADS = 128 + 32 * EPI_WARPS;
constexpr int CTRL_BYTES = 256;               // the call's control words: the abort word
constexpr int MAX_SPLIT = 8;                  // CTAs that share a tile's K: a portable cluster

// ---------------------------------------------------------------- the work --

struct MxParams {
    int M, n_mats;
    int64_t n_rows;               // rows of dst (tokens, or sorted rows)
    int64_t max_groups;           // token tiles of the activation operand
    bool wait_first;              // `first` may still be being written when the kernel starts
    int split;                    // CTAs that share a tile's K
    int mtiles, kst, nkc;         // weight row tiles, K stages, 128-column scale chunks
    const int32_t* first;         // experts' first rows, or null (dense: one segment)
    const uint8_t* w_scales;      // scale plane of matrix 0
    int64_t mat_stride;
    const uint8_t* x_scales;
    void* dst;
    int dst_type;
    unsigned int* abort_word;
    uint64_t limit_ns;
    int fault;                    // test only: CTA 0 leaves out its first stage's copies
};

// CG: CTAs of a tile.  Two of them take 256 weight rows and share the tokens: each loads its
// 128 rows and half of the token tile, and the pair's MMA reads both halves.
template <int BN, bool E4M3, int CG>
struct Cfg {
    static constexpr int ATOM_K = E4M3 ? 128 : 256;       // K of a 128-byte shared-memory row
    static constexpr int CH = ATOM_K / 128;               // scale chunks of an atom
    static constexpr int ATOMS = BN <= 64 ? 2 : 1;        // atoms of a stage
    static constexpr int NB = BN <= 128 ? 1 : BN / 128;   // 512-byte pieces of a token tile's scale chunk
    static constexpr int CHUNK = mx_chunk_bytes(BN);
    static constexpr int A_BYTES = BM * 128;              // of one atom
    static constexpr int B_ROWS = BN / CG;                // tokens that a CTA loads
    static constexpr int B_BYTES = B_ROWS * 128;
    static constexpr int OFF_B = ATOMS * A_BYTES;
    static constexpr int OFF_SFA = OFF_B + ATOMS * B_BYTES;
    static constexpr int OFF_SFB = OFF_SFA + ATOMS * CH * MX_CHUNK;
    static constexpr int STAGE = (OFF_SFB + ATOMS * CH * CHUNK + 1023) / 1024 * 1024;
    // bytes that the operand copies of a CTA's stage read (the widened weights as they lie in memory)
    static constexpr int TX = ATOMS * ((E4M3 ? A_BYTES / 2 : A_BYTES) + B_BYTES);
    static constexpr int SEG_BYTES = 2 * (MX_MAX_EXPERTS + 1) * 4 + 64;
    static constexpr int ST_ = (227 * 1024 - 2048 - SEG_BYTES) / STAGE;
    static constexpr int ST = ST_ > 12 ? 12 : ST_;
    static constexpr int OFF_BAR = ST * STAGE;
    static constexpr int OFF_SEG = OFF_BAR + 1024;
    static constexpr int SMEM = OFF_SEG + SEG_BYTES + 1024;          // + alignment slack
    static constexpr int NACC = 2 * BN <= 256 ? 2 : 1;
    static constexpr int SFA_COL = NACC * BN;
    static constexpr int SFB_COL = SFA_COL + 4 * ATOMS * CH;
    static constexpr int USED = SFB_COL + 4 * ATOMS * CH * NB;
    static constexpr int COLS = USED <= 32 ? 32 : USED <= 64 ? 64 : USED <= 128 ? 128 : USED <= 256 ? 256 : 512;
    // columns of an epilogue warp; the narrowest tile leaves half of the warps idle
    static constexpr int CW = BN <= 16 ? BN : BN / 2;
    static constexpr int EPI = BN <= 16 ? 4 : 8;          // epilogue warps at work
    static_assert(USED <= 512 && B_BYTES % 1024 == 0 && ST >= 3 && SMEM <= 227 * 1024, "fits the SM");
};

// The tiles of a CTA (or pair): pos, pos + step, ... below end; `part` of `split` parts of
// their K.
struct Walk {
    int64_t pos, end, step;
    int part, split;
};

struct Frag {
    int mat, m0, k0, k1;   // matrix, first weight row, K stages
    int x_row;             // first row of the activation operand
    int64_t dst_row;
    int valid;             // tokens of the tile
};

template <int BN, int CG>
__device__ __forceinline__ bool next_frag(Walk& w, const MxParams& p, const int* start, const int* units, Frag& f) {
    if (w.pos >= w.end) return false;
    const int64_t t = w.pos;
    w.pos += w.step;
    f.k0 = p.kst * w.part / w.split;
    f.k1 = p.kst * (w.part + 1) / w.split;
    // tiles: by segment, then weight rows, then tokens (the weights of a row tile are read
    // by consecutive tiles)
    int e = 0, g0 = 0, groups = units[1];
    if (p.first) {
        int lo = 0, hi = p.n_mats;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if ((int64_t)units[mid] * p.mtiles <= t) lo = mid;
            else hi = mid;
        }
        e = lo;
        g0 = units[e];
        groups = units[e + 1] - g0;
    }
    const int in = (int)(t - (int64_t)g0 * p.mtiles);
    const int mt = __shfl_sync(0xffffffffu, in / groups, 0), nt = __shfl_sync(0xffffffffu, in - mt * groups, 0);
    // (from lane 0, so that the compiler knows them to be the same in the whole warp: it keeps
    // the descriptors of copies and MMAs in uniform registers only then)
    f.mat = __shfl_sync(0xffffffffu, e, 0);
    f.m0 = mt * (BM * CG);
    f.x_row = (__shfl_sync(0xffffffffu, g0, 0) + nt) * BN;
    f.dst_row = (p.first ? start[e] : 0) + (int64_t)nt * BN;
    const int64_t left = (p.first ? (int64_t)start[e + 1] : p.n_rows) - f.dst_row;
    f.valid = (int)min(left, (int64_t)BN);
    return true;
}

// column c of a tile to dst[at + c * stride]
template <typename T, int N>
__device__ __forceinline__ void store_columns(void* dst, int64_t at, int64_t stride, const uint32_t (&r)[N], int valid) {
    T* p = static_cast<T*>(dst) + at;
#pragma unroll
    for (int c = 0; c < N; ++c, p += stride)
        if (c < valid) *p = mx_from_f32<T>(__uint_as_float(r[c]));
}

// whether `ok` holds in all of the n epilogue threads
__device__ __forceinline__ bool epilogue_all(bool ok, int n) {
    uint32_t all;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.and.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(all) : "r"((uint32_t)ok), "r"(n) : "memory");
    return all != 0;
}

template <int BN, bool E4M3, int CG>
__global__ void __launch_bounds__(THREADS, 1)
mxmm_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_x,
            const __grid_constant__ CUtensorMap tmap_sw, const __grid_constant__ CUtensorMap tmap_sx, const MxParams p) {
    using C = Cfg<BN, E4M3, CG>;
    constexpr int ST = C::ST;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = smem_u32(smem);
    const uint32_t full = sbase + C::OFF_BAR, empty = full + 8 * ST;
    const uint32_t acc_full = empty + 8 * ST, acc_empty = acc_full + 16;
    const uint32_t drain = acc_empty + 16, slot_addr = drain + 8;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_BAR + 16 * ST + 48);
    int* tmp = reinterpret_cast<int*>(smem + C::OFF_BAR + 512);
    int* start = reinterpret_cast<int*>(smem + C::OFF_SEG);
    int* units = start + MX_MAX_EXPERTS + 1;
    const Waiter wt{abort_flag, p.abort_word, p.limit_ns, &g_mxmm_status};
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = CG == 2 ? (int)(blockIdx.x & 1) : 0;        // in the pair; 0 issues its MMAs

    if (threadIdx.x == 0) {
        for (int s = 0; s < ST; ++s) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(acc_full + 8 * s, 1);
            mbar_init(acc_empty + 8 * s, CG * C::EPI);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        prefetch_map(&tmap_w);
        prefetch_map(&tmap_x);
    }
    if (warp == 1) tmem_alloc<CG>(slot_addr, C::COLS);
    pdl_trigger();
    // the experts' segments are known before the activations are
    Walk walk;
    if (p.first) {
        if (p.wait_first) pdl_wait();
        mx_segments(p.first, p.n_mats, p.n_rows, BN, p.max_groups, start, units, tmp);
    } else if (threadIdx.x == 0) {
        units[0] = 0;
        units[1] = (int)((p.n_rows + BN - 1) / BN);
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (CG == 2) {                                     // both CTAs' barriers and tensor memory exist
        cluster_arrive();
        cluster_wait();
    }
    tc_fence_after();
    uint32_t tmem;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(slot_addr));
    tmem = __shfl_sync(0xffffffffu, tmem, 0);

    // the same in the whole warp, and known to be (see q4q_mx_tc.cuh's elect_one)
    walk.end = (int64_t)__shfl_sync(0xffffffffu, units[p.first ? p.n_mats : 1], 0) * p.mtiles;
    walk.split = p.split;
    walk.part = p.split > 1 ? (int)(blockIdx.x % (unsigned)p.split) : 0;
    walk.pos = blockIdx.x / (unsigned)(CG * p.split);
    walk.step = gridDim.x / (unsigned)(CG * p.split);
    const Walk all = walk;
    bool pushed = false;

    if (warp == 0) {
        // ---------------- producer
        const bool lead = elect_one();
        auto load_w = [&](const Frag& g, int k, int s) {
            const uint32_t st = sbase + s * C::STAGE;
            const int kc = k * (C::ATOMS * C::CH), chunks = min(C::ATOMS * C::CH, p.nkc - kc);
            if constexpr (CG == 1) {
                const uint32_t bar = full + 8 * s;
                mbar_arrive_expect_tx(bar, C::TX + chunks * (MX_CHUNK + C::CHUNK));
                tma_load_4d(st, &tmap_w, 0, g.m0, k * C::ATOMS, g.mat, bar);
                bulk_g2s(st + C::OFF_SFA, p.w_scales + g.mat * p.mat_stride + ((int64_t)(g.m0 / BM) * p.nkc + kc) * MX_CHUNK,
                         chunks * MX_CHUNK, bar);
            } else {
                // all of the pair's bytes are counted on the first CTA's barrier
                const uint32_t bar = mapa_shared(full + 8 * s, 0);
                if (rank == 0) mbar_arrive_expect_tx(full + 8 * s, CG * (C::TX + C::ATOMS * C::CH * (MX_CHUNK + C::CHUNK)));
                // (a second half past the last row repeats the first; its rows are not stored)
                const int rows = g.m0 + rank * BM < p.M ? g.m0 + rank * BM : g.m0;
                tma_load_4d_pair(st, &tmap_w, 0, rows, k * C::ATOMS, g.mat, bar);
                tma_load_4d_pair(st + C::OFF_SFA, &tmap_sw, 0, kc, rows / BM, g.mat, bar);
            }
        };
        auto load_x = [&](const Frag& g, int k, int s) {
            const uint32_t st = sbase + s * C::STAGE;
            const int kc = k * (C::ATOMS * C::CH), chunks = min(C::ATOMS * C::CH, p.nkc - kc);
            if constexpr (CG == 1) {
                const uint32_t bar = full + 8 * s;
                tma_load_3d(st + C::OFF_B, &tmap_x, 0, g.x_row, k * C::ATOMS, bar);
                bulk_g2s(st + C::OFF_SFB, p.x_scales + ((int64_t)(g.x_row / BN) * p.nkc + kc) * C::CHUNK, chunks * C::CHUNK, bar);
            } else {
                const uint32_t bar = mapa_shared(full + 8 * s, 0);
                tma_load_3d_pair(st + C::OFF_B, &tmap_x, 0, g.x_row + rank * C::B_ROWS, k * C::ATOMS, bar);
                tma_load_3d_pair(st + C::OFF_SFB, &tmap_sx, 0, kc, g.x_row / BN, bar);
            }
        };
        // the weights of the first stages do not wait for the activation encoder
        const bool skip = p.fault && blockIdx.x == 0;
        Walk ahead = walk;
        Frag f;
        int pre = 0;
        while (pre < ST && next_frag<BN, CG>(ahead, p, start, units, f))
            for (int k = f.k0; k < f.k1 && pre < ST; ++k, ++pre)
                if (lead && !(skip && pre == 0)) load_w(f, k, pre);
        pdl_wait();
        int i = 0, s = 0;
        uint32_t parity = 1;                 // of the wait on the slot's previous use, from its second on
        bool ok = true;
        while (ok && next_frag<BN, CG>(walk, p, start, units, f))
            for (int k = f.k0; k < f.k1; ++k, ++i) {
                if (i >= pre) {
                    if (i >= ST && !warp_wait(empty + 8 * s, parity, wt)) {
                        ok = false;
                        break;
                    }
                    if (lead) load_w(f, k, s);
                }
                if (lead && !(skip && i == 0)) load_x(f, k, s);
                if (++s == ST) {
                    s = 0;
                    parity ^= 1;
                }
            }
        // every copy lands before the CTA (or the pair) can exit, also after an abort
        if (lead && rank == 0)
            for (int j = max(0, i - ST); j < i; ++j)
                if (!(skip && j == 0) && !mbar_wait_bounded(full + 8 * (j % ST), (j / ST) & 1, p.limit_ns)) break;
    } else if (warp == 1) {
        // ---------------- MMA issuer
        pdl_wait();
        // M = 128 for each CTA, N = BN, E8M0 scales, A = E2M1 (code 1 in kind::mxf4, 5 in kind::mxf8f6f4)
        constexpr uint32_t IDESC = ((uint32_t)(BN >> 3) << 17) | (1u << 23) | ((uint32_t)(CG * BM >> 7) << 27) |
                                   (E4M3 ? (5u << 7) : (1u << 7) | (1u << 10));
        if (rank == 0) {
            const bool lead = elect_one();
            const int atoms = (p.nkc + C::CH - 1) / C::CH;
            const uint32_t sfa = tmem + C::SFA_COL, sfb = tmem + C::SFB_COL;
            Frag f;
            int s = 0, n = 0;
            uint32_t parity = 0;
            bool ok = true;
            while (ok && next_frag<BN, CG>(walk, p, start, units, f)) {
                const int buf = n % C::NACC;
                if (n >= C::NACC && !warp_wait(acc_empty + 8 * buf, ((n / C::NACC) + 1) & 1, wt)) break;
                const uint32_t d = tmem + buf * BN;
                const int k0 = __shfl_sync(0xffffffffu, f.k0, 0), k1 = __shfl_sync(0xffffffffu, f.k1, 0);
                for (int k = k0; k < k1; ++k) {
                    if (!warp_wait(full + 8 * s, parity, wt)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (lead) {
                        const uint32_t st = sbase + s * C::STAGE;
                        const int n_atoms = min(C::ATOMS, atoms - k * C::ATOMS);
#pragma unroll
                        for (int q = 0; q < C::ATOMS; ++q) {
                            if (q > 0 && q >= n_atoms) break;
                            // tcgen05 operations of one thread run in order: these copies follow the
                            // MMAs that read the columns' last values, and precede the ones below
#pragma unroll
                            for (int c = 0; c < C::CH; ++c) {
                                const int h = q * C::CH + c;
                                scales_to_tmem<CG>(sfa + 4 * h, desc_scales(st + C::OFF_SFA + h * MX_CHUNK));
#pragma unroll
                                for (int b = 0; b < C::NB; ++b)
                                    scales_to_tmem<CG>(sfb + (h * C::NB + b) * 4, desc_scales(st + C::OFF_SFB + h * C::CHUNK + b * MX_CHUNK));
                            }
                            const uint64_t a = desc_sw128(st + q * C::A_BYTES), b = desc_sw128(st + C::OFF_B + q * C::B_BYTES);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                // an MMA takes 1 (E4M3) or 2 (E2M1) of a chunk's 4 scales per row
                                const uint32_t h = q * C::CH + (E4M3 ? 0 : j >> 1), id = E4M3 ? j : (j & 1) * 2;
                                mma_mx<E4M3, CG>(d, a + (uint64_t)(j * 2), b + (uint64_t)(j * 2), IDESC | (id << 4) | (id << 29),
                                                 sfa + 4 * h, sfb + 4 * C::NB * h, q > 0 || j > 0 || k > k0);
                            }
                        }
                        mma_commit<CG>(empty + 8 * s);
                        if (k == k1 - 1) mma_commit<CG>(acc_full + 8 * buf);
                    }
                    __syncwarp();
                    if (++s == ST) {
                        s = 0;
                        parity ^= 1;
                    }
                }
                ++n;
            }
            // no MMA is in flight when the CTAs free their tensor memory
            if (lead) {
                mma_commit<CG>(drain);
                mbar_wait_bounded(drain, 0, p.limit_ns);
            }
        }
        __syncwarp();
    } else if (warp >= 4 && warp < 4 + C::EPI) {
        // ---------------- epilogue: two warps to a lane quadrant, half of the columns each
        pdl_wait();
        constexpr int CW = C::CW, N_THREADS = 32 * C::EPI;
        const int quad = warp & 3, row = quad * 32 + lane, col0 = (warp - 4) / 4 * CW;
        const uint32_t tq = tmem + ((uint32_t)(quad * 32) << 16) + col0;
        const uint32_t freed = CG == 2 ? mapa_shared(acc_empty, 0) : acc_empty;
        Frag f;
        int n = 0;
        while (next_frag<BN, CG>(walk, p, start, units, f)) {
            const int buf = n % C::NACC;
            // one verdict for all warps: none of them waits below for one that gave up
            if (!epilogue_all(warp_wait(acc_full + 8 * buf, (n / C::NACC) & 1, wt), N_THREADS)) break;
            tc_fence_after();
            const int m = f.m0 + rank * BM + row;
            // the whole tile into registers, so that the next one's MMAs can start
            uint32_t r[CW];
            tmem_ld<CW>(tq + (uint32_t)(buf * BN), r);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (CG == 2) mbar_arrive_cluster(freed + 8 * buf);
                else mbar_arrive(freed + 8 * buf);
            }
            const int valid = f.valid - col0;
            if (CG == 2 || p.split == 1) {
                const int64_t at = (f.dst_row + col0) * p.M + m;
                if (m < p.M) {
                    if (p.dst_type == Q4Q_TYPE_F32) store_columns<float, CW>(p.dst, at, p.M, r, valid);
                    else if (p.dst_type == Q4Q_TYPE_F16) store_columns<__half, CW>(p.dst, at, p.M, r, valid);
                    else store_columns<__nv_bfloat16, CW>(p.dst, at, p.M, r, valid);
                }
            } else {
                // The CTA's part of its one tile goes to those that add it up: token t to CTA t % split,
                // where [part][t / split][row] takes the place of stages, once all CTAs have read theirs.
                cluster_arrive();
                cluster_wait();
                pushed = true;
                const uint32_t mask = (uint32_t)p.split - 1u, log = 31 - __clz(p.split);
                const uint32_t part = sbase + 4 * row + ((uint32_t)walk.part * (BN >> log)) * (4 * BM);
#pragma unroll
                for (int c = 0; c < CW; ++c) {
                    const uint32_t t = col0 + c;
                    if (c < valid)
                        asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(mapa_shared(part + (t >> log) * (4 * BM), t & mask)), "r"(r[c]) : "memory");
                }
            }
            ++n;
        }
        // rows of no expert are zeros
        if (p.first) {
            const int64_t from = (int64_t)start[p.n_mats] * p.M, to = p.n_rows * p.M;
            for (int64_t i = from + (int64_t)blockIdx.x * N_THREADS + (threadIdx.x - 128); i < to; i += (int64_t)gridDim.x * N_THREADS)
                mx_store(p.dst, p.dst_type, i, 0.0f);
        }
    }

    tc_fence_before();
    if (CG == 1 && p.split > 1) {
        __syncwarp();
        if (!pushed) {
            cluster_arrive();
            cluster_wait();
        }
        cluster_arrive();
        cluster_wait();
        Walk w = all;
        Frag f;
        if (next_frag<BN, CG>(w, p, start, units, f)) {
            // four rows of a token a thread, the parts in the order of K
            const int log = 31 - __clz(p.split), tokens = (f.valid - all.part + p.split - 1) >> log;
            for (int u = threadIdx.x; u < tokens * (BM / 4); u += THREADS) {
                const float4* part = reinterpret_cast<const float4*>(smem) + u;
                float4 v[MAX_SPLIT];
#pragma unroll
                for (int z = 0; z < MAX_SPLIT; ++z)
                    if (z < p.split) v[z] = part[z * (BN >> log) * (BM / 4)];
                float sum[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
                for (int z = 1; z < MAX_SPLIT; ++z)
                    if (z < p.split) {
                        sum[0] = __fadd_rn(sum[0], v[z].x);
                        sum[1] = __fadd_rn(sum[1], v[z].y);
                        sum[2] = __fadd_rn(sum[2], v[z].z);
                        sum[3] = __fadd_rn(sum[3], v[z].w);
                    }
                const int m = f.m0 + u % (BM / 4) * 4;
                const int64_t token = f.dst_row + (u / (BM / 4) << log) + all.part;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (m + k < p.M) mx_store(p.dst, p.dst_type, token * p.M + m + k, sum[k]);
            }
        }
    }
    __syncthreads();
    if constexpr (CG == 2) {                                     // neither CTA leaves while the other uses its memory
        cluster_arrive();
        cluster_wait();
    }
    tc_fence_after();
    if (warp == 1) tmem_dealloc<CG>(tmem, C::COLS);
}

// ------------------------------------------------------------------ host ----

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

bool get_encode() {
    std::call_once(g_encode_once, [] {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) ==
                cudaSuccess && q == cudaDriverEntryPointSuccess)
            g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    });
    return g_encode != nullptr;
}

// A product's tile and workspace.
struct Plan {
    int bn, cg, split;
    int64_t kp, max_groups;
    size_t scales, ctrl, total;          // offsets after the codes, and the whole size
};

// The rows of a segment that a token tile is chosen for: all of them, or twice the mean of the
// experts' shares (a larger share takes several tiles).
int64_t expected_rows(int64_t n_rows, int64_t n_tokens, int n_experts) {
    return n_experts > 0 ? std::min(n_tokens, 2 * ((n_rows + n_experts - 1) / n_experts)) : n_rows;
}

// Clusters of `split` CTAs that the device holds at one CTA an SM (152 SMs hold 76, 36, 15 of 2, 4, 8).
int64_t clusters_held(int split, int sm_count) { return split == 8 ? sm_count / 10 : split == 4 ? (sm_count - 8) / 4 : sm_count / split; }

// The form that is expected to take least.  Times in ns, fitted to 4096 x 1024, 4096 x 4096,
// 4096 x 14336 and 14336 x 4096 at 8 to 1024 tokens in every form (within a tenth): a form's start
// and end, its time for an atom of E4M3 and of E2M1 activations, 2050 (64 tokens: 2850) to join a
// tile's parts, 600 for each further round of tiles, and what HBM needs at 6500 bytes a ns behind
// a start of 4400.  For example 14336 x 4096, 8 tokens, E4M3: 20.3 us whole, 15.4 and 12.1 in 2 and
// 4 parts; 1024 x 4096, 1 token, E2M1: 6.3 whole, 5.6 in 8; 14336 x 4096, 128 tokens, E4M3:
// tiles of 64 tokens 23.5 whole, 18.6 in 2 parts, 20.5 by pairs, tiles of 128 by pairs 27.8.
void pick_tile(Plan& q, int64_t K, int64_t M, int64_t n_rows, int64_t n_tokens, int n_experts, int acts, int sm_count) {
    const int64_t expect = expected_rows(n_rows, n_tokens, n_experts);
    const int64_t segments = n_experts > 0 ? std::min<int64_t>(n_experts, n_rows) : 1, mean = (n_rows + segments - 1) / segments;
    const bool e4m3 = acts == Q4Q_ACTS_MXFP8;
    const int64_t ka = e4m3 ? 128 : 256, atoms = (K + ka - 1) / ka;
    const double hbm = (double)segments * M * K * 0.53 / 6500 + 4400;
    static const struct { int bn, cg, start, e4m3, e2m1; } forms[] = {
        {8, 1, 4700, 145, 150}, {16, 1, 4700, 155, 165}, {32, 1, 4700, 160, 170}, {64, 1, 4900, 162, 185},
        {64, 2, 6100, 122, 170}, {128, 2, 6400, 187, 220}, {256, 2, 6800, 270, 310}};
    double least = 1e300;
    for (const auto& f : forms) {
        if (f.bn < expect && f.bn < 64) continue;              // narrow tiles only where one holds the tokens
        const double atom = e4m3 ? f.e4m3 : f.e2m1;
        const int64_t tiles = segments * ((mean + f.bn - 1) / f.bn) * ((M + BM * f.cg - 1) / (BM * f.cg));
        const int64_t workers = sm_count / f.cg, rounds = (tiles + workers - 1) / workers;
        for (int split = 1; split <= (f.cg == 1 ? MAX_SPLIT : 1); split *= 2) {
            if (split > 1 && (tiles > clusters_held(split, sm_count) || atoms < 2 * split)) break;
            const double work = split > 1 ? f.start + (f.bn == 64 ? 2850 : 2050) + atom * ((atoms + split - 1) / split)
                                          : f.start + atom * rounds * atoms + 600 * (rounds - 1);
            const double cost = std::max(work, hbm) + 0.01 * f.bn;
            if (cost < least) {
                least = cost;
                q.bn = f.bn;
                q.cg = f.cg;
                q.split = split;
            }
        }
    }
}

Plan make_plan(int64_t K, int64_t M, int64_t n_rows, int64_t n_tokens, int n_experts, int acts, int sm_count) {
    Plan q{};
    pick_tile(q, K, M, n_rows, n_tokens, n_experts, acts, sm_count);
    q.kp = mx_up(K, MX_KP);
    // token tiles: each segment starts a new one, and none is without a row
    q.max_groups = (n_rows + q.bn - 1) / q.bn + (n_experts > 0 ? std::min<int64_t>(n_experts, n_rows) : 0);
    q.max_groups = std::min(q.max_groups, n_rows);
    q.scales = (size_t)mx_up(q.max_groups * q.bn * (acts == Q4Q_ACTS_MXFP8 ? q.kp : q.kp / 2), 1024);
    q.ctrl = q.scales + (size_t)mx_up(q.max_groups * (q.kp / 128) * mx_chunk_bytes(q.bn), 256);
    q.total = q.ctrl + CTRL_BYTES;
    return q;
}

int atoms_of(int bn) { return bn <= 64 ? 2 : 1; }      // of a stage (Cfg::ATOMS)

struct Maps {
    CUtensorMap w, x, sw, sx;
};

template <int BN, bool E4M3, int CG>
q4q_status launch_t(const Maps& maps, const MxParams& p, int64_t workers, cudaStream_t stream, int device) {
    const int cluster = CG * p.split;
    using C = Cfg<BN, E4M3, CG>;
    static_assert(C::ATOMS == (BN <= 64 ? 2 : 1), "the tensor maps' boxes");
    static std::atomic<int> configured[64];
    auto kern = mxmm_kernel<BN, E4M3, CG>;
    if (device < 0 || device >= 64) return Q4Q_ERR_CUDA;
    if (!configured[device].load()) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess)
            return (cudaGetLastError(), Q4Q_ERR_CUDA);
        configured[device].store(1);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(workers * cluster));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // behind the activation encoder
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster == 1 ? 1 : 2;
    if (cudaLaunchKernelEx(&cfg, kern, maps.w, maps.x, maps.sw, maps.sx, p) != cudaSuccess) return (cudaGetLastError(), Q4Q_ERR_CUDA);
    return launch_status();
}

template <bool E4M3>
q4q_status launch_bn(const Plan& q, const Maps& maps, const MxParams& p, int64_t workers, cudaStream_t stream, int device) {
    switch (q.bn) {
        case 8: return launch_t<8, E4M3, 1>(maps, p, workers, stream, device);
        case 16: return launch_t<16, E4M3, 1>(maps, p, workers, stream, device);
        case 32: return launch_t<32, E4M3, 1>(maps, p, workers, stream, device);
        case 64:
            return q.cg == 1 ? launch_t<64, E4M3, 1>(maps, p, workers, stream, device)
                             : launch_t<64, E4M3, 2>(maps, p, workers, stream, device);
        case 128: return launch_t<128, E4M3, 2>(maps, p, workers, stream, device);
        default: return launch_t<256, E4M3, 2>(maps, p, workers, stream, device);
    }
}

// 32-bit words of scales: {a chunk, 128-column chunks, row tiles, matrices}, boxes of `chunks` chunks
bool encode_scale_map(CUtensorMap* map, const void* base, int chunk_bytes, int64_t nkc, int64_t tiles, int64_t n_mats,
                      int64_t mat_stride, int chunks) {
    const cuuint64_t dims[4] = {(cuuint64_t)(chunk_bytes / 4), (cuuint64_t)nkc, (cuuint64_t)tiles, (cuuint64_t)n_mats};
    const cuuint64_t strides[3] = {(cuuint64_t)chunk_bytes, (cuuint64_t)(nkc * chunk_bytes), (cuuint64_t)mat_stride};
    const cuuint32_t box[4] = {(cuuint32_t)(chunk_bytes / 4), (cuuint32_t)chunks, 1, 1};
    const cuuint32_t one[4] = {1, 1, 1, 1};
    return g_encode(map, CU_TENSOR_MAP_DATA_TYPE_INT32, mat_stride ? 4 : 3, const_cast<void*>(base), dims, strides, box, one,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

q4q_status run(const void* src0, int64_t ne00, int64_t ne01, int n_mats, const MxActs& acts, int64_t n_tokens, void* dst,
               int dst_type, void* workspace, size_t workspace_bytes, bool pdl, cudaStream_t stream, const KernelDebug* dbg) {
    DeviceInfo info;
    q4q_status st = current_device_info(&info);
    if (st != Q4Q_OK) return st;
    if (info.cc_major != 10 || !get_encode()) return Q4Q_ERR_CUDA;
    const Plan q = make_plan(ne00, ne01, acts.n_rows, n_tokens, acts.first ? n_mats : 0, acts.acts, info.sm_count);
    if (workspace_bytes < q.total) return Q4Q_ERR_WORKSPACE;
    if (!workspace) return Q4Q_ERR_NULL;
    if (!aligned(workspace, 256)) return Q4Q_ERR_ALIGN;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const bool e4m3 = acts.acts == Q4Q_ACTS_MXFP8;
    const int64_t code_bytes = mx_code_bytes(ne00, ne01), stride = code_bytes + mx_scale_bytes(ne00, ne01);
    const uint8_t* w_scales = static_cast<const uint8_t*>(src0) + code_bytes;
    const int stage_atoms = atoms_of(q.bn), ch = e4m3 ? 1 : 2;
    const int64_t atoms = q.kp / (128 * ch), nkc = q.kp / 128;

    Maps maps{};
    if (!mx_encode_weight_map(&maps.w, src0, ne00, ne01, n_mats, e4m3, stage_atoms)) return Q4Q_ERR_CUDA;
    {
        // {128 bytes, tokens, atoms}
        const cuuint64_t dims[3] = {128, (cuuint64_t)(q.max_groups * q.bn), (cuuint64_t)atoms};
        const cuuint64_t strides[2] = {(cuuint64_t)(e4m3 ? q.kp : q.kp / 2), 128};
        const cuuint32_t box[3] = {128, (cuuint32_t)(q.bn / q.cg), (cuuint32_t)stage_atoms};
        const cuuint32_t one[3] = {1, 1, 1};
        if (g_encode(&maps.x, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, ws, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return Q4Q_ERR_CUDA;
    }
    if (q.cg == 2 && (!encode_scale_map(&maps.sw, w_scales, MX_CHUNK, nkc, (ne01 + BM - 1) / BM, n_mats, stride, stage_atoms * ch) ||
                      !encode_scale_map(&maps.sx, ws + q.scales, mx_chunk_bytes(q.bn), nkc, q.max_groups, 1, 0, stage_atoms * ch)))
        return Q4Q_ERR_CUDA;
    MxParams p;
    p.M = (int)ne01;
    p.n_mats = n_mats;
    p.n_rows = acts.n_rows;
    p.max_groups = q.max_groups;
    p.wait_first = pdl;
    p.split = q.split;
    p.mtiles = (int)((ne01 + BM * q.cg - 1) / (BM * q.cg));
    const int ks = 128 * ch * stage_atoms;
    p.kst = (int)((ne00 + ks - 1) / ks);
    p.nkc = (int)nkc;
    p.first = acts.first;
    p.w_scales = w_scales;
    p.mat_stride = stride;
    p.x_scales = ws + q.scales;
    p.dst = dst;
    p.dst_type = dst_type;
    p.abort_word = reinterpret_cast<unsigned int*>(ws + q.ctrl);
    p.limit_ns = dbg ? dbg->limit_ns : WAIT_LIMIT_NS;
    p.fault = dbg ? dbg->fault : 0;
    st = mx_encode_acts(acts, p.abort_word, ws, ws + q.scales, q.bn, q.max_groups, pdl, stream, info);
    if (st != Q4Q_OK) return st;
    // CTAs (pairs) that take tiles in turn, or a cluster for each tile that there may be
    const int64_t tiles = q.max_groups * p.mtiles;
    const int64_t workers = q.split > 1 ? tiles : std::min<int64_t>(info.sm_count / q.cg, tiles);
    if (workers * q.split >= (1ll << 31)) return Q4Q_ERR_SHAPE;
    return e4m3 ? launch_bn<true>(q, maps, p, workers, stream, info.device) : launch_bn<false>(q, maps, p, workers, stream, info.device);
}

q4q_status check_product(int64_t ne00, int64_t ne01, int src1_type, int64_t ne10, int64_t ne11, int acts, int dst_type, unsigned int flags) {
    if (flags & ~Q4Q_MUL_MAT_PDL) return Q4Q_ERR_ARG;
    if (!mx_type_ok(src1_type) || !mx_type_ok(dst_type) || !mx_acts_ok(acts)) return Q4Q_ERR_ARG;
    return check_mul_mat_shapes(ne00, ne01, ne10, ne11);
}

q4q_status mul_mat(const void* src0, int64_t ne00, int64_t ne01, const void* src1, int src1_type, int64_t ne10, int64_t ne11,
                   int acts, void* dst, int dst_type, void* workspace, size_t workspace_bytes, unsigned int flags,
                   q4q_stream_t stream, const KernelDebug* dbg) {
    q4q_status st = check_product(ne00, ne01, src1_type, ne10, ne11, acts, dst_type, flags);
    if (st != Q4Q_OK) return st;
    if (ne01 == 0 || ne11 == 0) return Q4Q_OK;
    if (!src0 || !src1 || !dst) return Q4Q_ERR_NULL;
    if (!aligned(src0, 256) || !aligned(src1, mx_type_bytes(src1_type)) || !aligned(dst, mx_type_bytes(dst_type))) return Q4Q_ERR_ALIGN;
    const MxActs a{src1, src1_type, acts, ne11, ne11, ne00, nullptr, nullptr, 0, 1};
    return run(src0, ne00, ne01, 1, a, ne11, dst, dst_type, workspace, workspace_bytes, (flags & Q4Q_MUL_MAT_PDL) != 0,
               (cudaStream_t)stream, dbg);
}

}  // namespace

// {128 elements (E4M3: widened to bytes) or bytes, weight rows, atoms along K, matrices}
bool mx_encode_weight_map(CUtensorMap* map, const void* src0, int64_t ne00, int64_t ne01, int n_mats, bool e4m3, int stage_atoms) {
    if (!get_encode()) return false;
    const int64_t kp = mx_up(ne00, MX_KP), stride = mx_code_bytes(ne00, ne01) + mx_scale_bytes(ne00, ne01);
    const cuuint64_t dims[4] = {128, (cuuint64_t)ne01, (cuuint64_t)(kp / (e4m3 ? 128 : 256)), (cuuint64_t)n_mats};
    const cuuint64_t strides[3] = {(cuuint64_t)(kp / 2), (cuuint64_t)(e4m3 ? 64 : 128), (cuuint64_t)stride};
    const cuuint32_t box[4] = {128, BM, (cuuint32_t)stage_atoms, 1};
    const cuuint32_t one[4] = {1, 1, 1, 1};
    return g_encode(map, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B : CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(src0),
                    dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

unsigned int mxmm_take_device_status() {
    unsigned int v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_mxmm_status, sizeof(v)) != cudaSuccess) return Q4Q_ERR_CUDA;
    if (v) cudaMemcpyToSymbol(g_mxmm_status, &z, sizeof(z));
    return v;
}

}  // namespace q4q

using namespace q4q;

extern "C" q4q_status q4q_mul_mat_mxfp4_workspace_size(int64_t ne00, int64_t ne01, int64_t ne11, int acts, size_t* bytes) {
    if (!bytes) return Q4Q_ERR_NULL;
    q4q_status st = check_product(ne00, ne01, Q4Q_TYPE_F32, ne00, ne11, acts, Q4Q_TYPE_F32, 0);
    if (st != Q4Q_OK) return st;
    *bytes = 0;
    if (ne01 == 0 || ne11 == 0) return Q4Q_OK;
    DeviceInfo info;
    if ((st = current_device_info(&info)) != Q4Q_OK) return st;
    *bytes = make_plan(ne00, ne01, ne11, ne11, 0, acts, info.sm_count).total;
    return Q4Q_OK;
}

extern "C" q4q_status q4q_mul_mat_mxfp4(const void* src0, int64_t ne00, int64_t ne01, const void* src1, int src1_type,
                                        int64_t ne10, int64_t ne11, int acts, void* dst, int dst_type, void* workspace,
                                        size_t workspace_bytes, unsigned int flags, q4q_stream_t stream) {
    return mul_mat(src0, ne00, ne01, src1, src1_type, ne10, ne11, acts, dst, dst_type, workspace, workspace_bytes, flags, stream, nullptr);
}

extern "C" q4q_status q4q_debug_mul_mat_mxfp4_timeout(const void* src0, int64_t ne00, int64_t ne01, const float* src1,
                                                      int64_t ne11, int acts, float* dst, void* workspace,
                                                      size_t workspace_bytes, uint64_t limit_ns, q4q_stream_t stream) {
    if (limit_ns == 0 || limit_ns > WAIT_LIMIT_NS) return Q4Q_ERR_ARG;
    if (ne01 == 0 || ne11 == 0) return Q4Q_ERR_SHAPE;
    const KernelDebug dbg{limit_ns, 1};
    return mul_mat(src0, ne00, ne01, src1, Q4Q_TYPE_F32, ne00, ne11, acts, dst, Q4Q_TYPE_F32, workspace, workspace_bytes, 0, stream, &dbg);
}

extern "C" q4q_status q4q_mul_mat_id_mxfp4_workspace_size(int64_t ne00, int64_t ne01, int64_t n_src1, int64_t n_rows,
                                                          int n_experts, int acts, size_t* bytes) {
    if (!bytes) return Q4Q_ERR_NULL;
    q4q_status st = check_product(ne00, ne01, Q4Q_TYPE_F32, ne00, 0, acts, Q4Q_TYPE_F32, 0);
    if (st != Q4Q_OK) return st;
    if (n_src1 < 0 || n_src1 >= (1 << 24) || n_rows < 0 || n_rows >= (1 << 24)) return Q4Q_ERR_SHAPE;
    if (n_experts < 1 || n_experts > MX_MAX_EXPERTS) return Q4Q_ERR_ARG;
    *bytes = 0;
    if (ne01 == 0 || n_rows == 0) return Q4Q_OK;
    DeviceInfo info;
    if ((st = current_device_info(&info)) != Q4Q_OK) return st;
    *bytes = make_plan(ne00, ne01, n_rows, n_src1, n_experts, acts, info.sm_count).total;
    return Q4Q_OK;
}

extern "C" q4q_status q4q_mul_mat_id_mxfp4(const void* src0, int64_t ne00, int64_t ne01, int n_experts, const void* src1,
                                           int src1_type, int64_t ne10, int64_t n_src1, const int32_t* first,
                                           const int32_t* slot, int64_t n_rows, int top_k, int acts, void* dst,
                                           int dst_type, void* workspace, size_t workspace_bytes, unsigned int flags,
                                           q4q_stream_t stream) {
    q4q_status st = check_product(ne00, ne01, src1_type, ne10, 0, acts, dst_type, flags);
    if (st != Q4Q_OK) return st;
    // tokens, or, without slots, sorted rows: as many as a call with slots may have made
    if (n_src1 < 0 || n_src1 >= (slot ? 1 << 20 : 1 << 24) || n_rows < 0 || n_rows >= (1 << 24)) return Q4Q_ERR_SHAPE;
    if (n_experts < 1 || n_experts > MX_MAX_EXPERTS || top_k < 1) return Q4Q_ERR_ARG;
    if (slot ? n_rows > n_src1 * top_k : n_rows > n_src1) return Q4Q_ERR_SHAPE;
    if (ne01 == 0 || n_rows == 0) return Q4Q_OK;
    if (!src0 || !src1 || !dst || !first) return Q4Q_ERR_NULL;
    if (!aligned(src0, 256) || !aligned(src1, mx_type_bytes(src1_type)) || !aligned(dst, mx_type_bytes(dst_type)) ||
        !aligned(first, 4) || !aligned(slot, 4))
        return Q4Q_ERR_ALIGN;
    const MxActs a{src1, src1_type, acts, n_src1, n_rows, ne00, first, slot, n_experts, top_k};
    return run(src0, ne00, ne01, n_experts, a, n_src1, dst, dst_type, workspace, workspace_bytes, (flags & Q4Q_MUL_MAT_PDL) != 0,
               (cudaStream_t)stream, nullptr);
}

extern "C" q4q_status q4q_debug_mxfp4_form(int64_t ne00, int64_t ne01, int64_t n_rows, int64_t n_src1, int n_experts, int acts,
                                           int sm_count, int* form) {
    if (!form) return Q4Q_ERR_NULL;
    q4q_status st = check_product(ne00, ne01, Q4Q_TYPE_F32, ne00, 0, acts, Q4Q_TYPE_F32, 0);
    if (st != Q4Q_OK) return st;
    if (ne01 == 0 || n_rows < 1 || n_rows >= (1 << 24) || n_src1 < 1 || n_src1 >= (1 << 24)) return Q4Q_ERR_SHAPE;
    if (n_experts < 0 || n_experts > MX_MAX_EXPERTS || sm_count < 2) return Q4Q_ERR_ARG;
    const Plan q = make_plan(ne00, ne01, n_rows, n_src1, n_experts, acts, sm_count);
    form[0] = q.bn;
    form[1] = q.cg;
    form[2] = q.split;
    return Q4Q_OK;
}
