// gemm_few.cuh -- qfp4_gemm_epilogue for up to 128 rows (decoding batches) and
// other small outputs: the weights as the wide operand of the tensor cores.
//
// With so few rows of A the call is the reading of B.  So B's rows take the
// 128 lanes of the accumulator and A's rows (padded to a multiple of 16) its
// columns: a CTA computes 128 outputs of every row, and the k range is split
// over a cluster of up to eight CTAs so that most SMs read.  Both operands
// come by TMA, a ring of k-tiles (128 bytes of a row) deep; the scales go from
// memory, as the quantize calls write them, through registers into tensor
// memory (tcgen05.st, as in the pair kernel) with no prepass and no workspace.
// The CTAs of a cluster add their sums through distributed shared memory, in
// the order of their k ranges; each then finishes some of the rows.
//
// On the device, bias and SiLU: 1 x 4096 x 4096 MXFP8 8.0 us (2.6 from memory
// alone), 8 x 11008 x 4096 MXFP4 8.5, 100 x 11008 x 4096 MXFP4 11.5 (4.0 from
// memory alone; its 86 tiles run on 86 SMs, and halves of K would need 172).
// What is left is the launch and a CTA's chain of barriers.
#pragma once

#include "epilogue.cuh"

namespace qfp4 {

constexpr int FW_ROWS = 128;               // rows of A a CTA
constexpr int FW_BN = 128;                 // output columns a CTA
// warps: 0 and 2 producers of B and A, 1 MMA, 3 idle, 4-7 and 8-11 scales of
// the even and the odd k-tiles; all twelve then finish the sums
constexpr int FW_THREADS = 384;
constexpr int FW_MAX_STAGES = 10;
constexpr int FW_SF_BUFS = 5;
__host__ __device__ constexpr int fw_ahead(int nx) { return nx == 1 ? 4 : 2; }   // k-tiles of scales in registers a warp
constexpr int FW_MAX_SPLIT = 8;
constexpr int FW_SMEM_MAX = 208 * 1024;
// At least this much, so that an SM never holds two CTAs of these kernels.  Each
// takes all of tensor memory and waits for its cluster at the end: two clusters
// of different streams on the same two SMs, each with one CTA that has tensor
// memory and one that waits for it, would never finish.
constexpr int FW_SMEM_MIN = 116 * 1024;
static_assert(2 * FW_SMEM_MIN > 228 * 1024, "one CTA an SM");
static_assert(FW_ROWS * FW_BN * 4 <= FW_SMEM_MIN, "the sums");

struct FewParams {
    const uint8_t *sA, *sB;                // row-major scales: M and N rows of Kg
    const float *tA, *tB;
    int M, N, Kg, KT;
    int tiles_n;
    int rows;                              // rows a CTA, rounded up to 16
    int split, stages;
    int aligned;                           // a k-tile's scales of a row are one aligned word group
    void *out;
};

__device__ __forceinline__ float4 ld_dsmem4(uint32_t cluster_addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(cluster_addr)
                 : "memory");
    return v;
}

// The epilogue of U quads of columns: quad u is elements i0 + u stride ..
// i0 + u stride + 3 (multiples of 4), the first nu of them exist.  Few quads at
// a time, so that the code stays short: with a row or two to finish, fetching
// it is what the epilogue costs.
__host__ __device__ constexpr int fw_quads(int nx) { return nx == 1 ? 1 : 2; }
template <int OUT, int U>
__device__ __forceinline__ void ep_quads(const EpParams &ep, void *out, int64_t i0, int64_t stride, int nu, float alpha,
                                         uint64_t step, const float4 *acc, float4 bias)
{
    alignas(16) float res[4 * U];
    float v[4 * U];
    if (ep.residual)
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (u < nu) {
                const int64_t i = i0 + u * stride;
                if (ep.residual_f32)
                    *reinterpret_cast<float4 *>(res + 4 * u) =
                        *reinterpret_cast<const float4 *>(static_cast<const float *>(ep.residual) + i);
                else {
                    const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(ep.residual) + i);
                    *reinterpret_cast<float4 *>(res + 4 * u) = make_float4(bf16lo(w.x), bf16hi(w.x), bf16lo(w.y), bf16hi(w.y));
                }
            }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        v[4 * u] = fmaf(acc[u].x, alpha, bias.x);
        v[4 * u + 1] = fmaf(acc[u].y, alpha, bias.y);
        v[4 * u + 2] = fmaf(acc[u].z, alpha, bias.z);
        v[4 * u + 3] = fmaf(acc[u].w, alpha, bias.w);
    }
    auto store = [&](void *p) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (u < nu) {
                const int64_t i = i0 + u * stride;
                if (OUT == QFP4_F32)
                    *reinterpret_cast<float4 *>(static_cast<float *>(p) + i) =
                        make_float4(v[4 * u], v[4 * u + 1], v[4 * u + 2], v[4 * u + 3]);
                else
                    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p) + i) =
                        make_uint2(pack_bf16(v[4 * u], v[4 * u + 1]), pack_bf16(v[4 * u + 2], v[4 * u + 3]));
            }
    };
    if (ep.preact) store(ep.preact);
    act_forward<4 * U>(v, ep.act);
    if (ep.drop.on)
#pragma unroll
        for (int u = 0; u < U; ++u) drop_values<4, true>(ep.drop, step, i0 + u * stride, v + 4 * u);
    if (ep.residual)
#pragma unroll
        for (int t = 0; t < 4 * U; ++t) v[t] += res[t];
    store(out);
}

// The epilogue without dropout of one column of the output: element i0 + t N
// is row t of the nm rows (at most EP) that exist.
template <int OUT, int EP>
__device__ __forceinline__ void ep_column(const EpParams &ep, void *out, int64_t i0, int64_t N, int nm, float alpha,
                                          const uint32_t *acc, float bias)
{
    float res[EP], v[EP];
    if (ep.residual)
#pragma unroll
        for (int t = 0; t < EP; ++t) res[t] = t < nm ? ld_as_float(ep.residual, ep.residual_f32, i0 + t * N) : 0.0f;
#pragma unroll
    for (int t = 0; t < EP; ++t) v[t] = fmaf(__uint_as_float(acc[t]), alpha, bias);
    auto store = [&](void *p) {
#pragma unroll
        for (int t = 0; t < EP; ++t)
            if (t < nm) {
                if (OUT == QFP4_F32) static_cast<float *>(p)[i0 + t * N] = v[t];
                else static_cast<__nv_bfloat16 *>(p)[i0 + t * N] = __float2bfloat16_rn(v[t]);
            }
    };
    if (ep.preact) store(ep.preact);
    act_forward<EP>(v, ep.act);
    if (ep.residual)
#pragma unroll
        for (int t = 0; t < EP; ++t) v[t] += res[t];
    store(out);
}

// NX: 32-row groups of A whose scales are loaded (1 for up to 32 rows, else 4).
// PLAIN: wide outputs without a split of K or dropout, scale rows of whole
// aligned words.  Such calls have kernels of their own because a block lives a
// few microseconds, of which fetching its code is a part: with both epilogues and
// both ways of loading scales in one kernel every call took 0.5 to 0.8 us more.
template <int FMT, int OUT, int NX, bool PLAIN>
__global__ void __launch_bounds__(FW_THREADS, 1)
    k_gemm_few(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, FewParams p, EpParams ep)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ __align__(8) uint64_t full[FW_MAX_STAGES], empty[FW_MAX_STAGES], acc_full;
    __shared__ uint32_t tmem_base_sh;
    __shared__ volatile int abort_flag;

    constexpr int CPS = gm_cps(FMT);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_ctarank()), tile = static_cast<int>(blockIdx.x / p.split);
    const int n0 = tile % p.tiles_n * FW_BN, r0 = tile / p.tiles_n * FW_ROWS;   // first column, first row
    const int live = imin(p.M - r0, FW_ROWS);                 // rows of this CTA
    const int kt0 = static_cast<int>(static_cast<int64_t>(p.KT) * rank / p.split);
    const int nkt = static_cast<int>(static_cast<int64_t>(p.KT) * (rank + 1) / p.split) - kt0;   // at least one
    const int w_bytes = FW_BN * GM_BKB, x_bytes = p.rows * GM_BKB, stage_bytes = w_bytes + x_bytes;

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(&full[s], 2 + 4);                       // two producers, four scale warps
            mbar_init(&empty[s], 1);
        }
        mbar_init(&acc_full, 1);
        abort_flag = 0;
        fence_mbar_init();
        prefetch_tensormap(&tmW);
        prefetch_tensormap(&tmX);
    }
    if (warp == 1) {
        tmem_alloc(&tmem_base_sh, GM_TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_sh;
    pdl_wait();
    pdl_trigger();

    auto buf_b = [&](int b) { return tmem + 256 + b * 32; };
    auto buf_a = [&](int b) { return tmem + 256 + FW_SF_BUFS * 32 + b * 16; };

    // A k-tile has one barrier (operands and scales) and one commit: each
    // instruction on a barrier or the tensor pipe takes the thread that issues
    // it 60 to 100 cycles, and with so few columns that is all a k-tile costs.
    if (warp == 0 || warp == 2) {
        // ------------------------------------------------ producers
        if (lane == 0) {
            const CUtensorMap *map = warp == 0 ? &tmW : &tmX;
            const int bytes = warp == 0 ? w_bytes : x_bytes, row = warp == 0 ? n0 : r0, off = warp == 0 ? 0 : w_bytes;
            int s = 0;
            uint32_t ph = 1;
            for (int i = 0; i < nkt; ++i) {
                if (i >= p.stages && !mbar_wait(&empty[s], ph)) { abort_flag = 1; break; }
                mbar_arrive_expect_tx(&full[s], bytes);
                tma_load_2d(smem + static_cast<size_t>(s) * stage_bytes + off, map, &full[s], (kt0 + i) * GM_BKB, row);
                if (++s == p.stages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            if (abort_flag) settle_ns(kSettleNs);   // loads already issued may still be landing
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer
        if (lane == 0) {
            const uint32_t id = idesc_blockscaled(FMT, FW_BN, p.rows, 0);
            int s = 0, b = 0;
            uint32_t ph = 0;
            bool ready = false;
            for (int i = 0; i < nkt; ++i) {
                if (!ready && !mbar_wait(&full[s], ph)) { abort_flag = 1; break; }
                tc_fence_after();
                const uint8_t *st = smem + static_cast<size_t>(s) * stage_bytes;
                const uint64_t wdesc = desc_k_sw128(st), xdesc = desc_k_sw128(st + w_bytes);
                const uint32_t sa = buf_a(b), sb = buf_b(b);
                uint64_t *done = &empty[s];
                if (++s == p.stages) {
                    s = 0;
                    ph ^= 1u;
                }
                if (++b == FW_SF_BUFS) b = 0;
                ready = mbar_test(&full[s], ph);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    umma_blockscaled<FMT>(tmem, wdesc + 2 * k, xdesc + 2 * k, id, sa + 4 * k, sb + 8 * k, (i | k) != 0);
                umma_commit(done);
            }
            // every MMA this thread issued has finished before the CTA can leave
            umma_commit(&acc_full);
            if (!mbar_wait(&acc_full, 0)) abort_flag = 1;
        }
    } else if (warp >= 4) {
        // ------------------------------------------------ scales: this quadrant's 32 rows of B, every row of A
        constexpr int AHEAD = fw_ahead(NX);
        const int q = warp & 3, odd = warp >= 8 ? 1 : 0;
        const uint32_t lane_base = static_cast<uint32_t>(32 * q) << 16;
        auto load_words = [&](const uint8_t *sc, int R, int row, int kt, uint32_t tail, uint32_t *w) {
#pragma unroll
            for (int c = 0; c < CPS; ++c) w[c] = 0u;
            if (row >= R || kt >= kt0 + nkt) return;
            const uint8_t *s = sc + static_cast<int64_t>(row) * p.Kg + 4 * CPS * kt;
            if (PLAIN || p.aligned) {
                if constexpr (CPS == 4) {
                    const uint4 u = *reinterpret_cast<const uint4 *>(s);
                    w[0] = u.x;
                    w[1] = u.y;
                    w[2] = u.z;
                    w[3] = u.w;
                } else if constexpr (CPS == 2) {
                    const uint2 u = *reinterpret_cast<const uint2 *>(s);
                    w[0] = u.x;
                    w[1] = u.y;
                } else
                    w[0] = *reinterpret_cast<const uint32_t *>(s);
            } else {
                // the aligned words around the row's bytes [s, last), shifted
                const int nb = imin(4 * CPS, p.Kg - 4 * CPS * kt), sh = 8 * static_cast<int>(reinterpret_cast<uintptr_t>(s) & 3);
                const uint8_t *last = s + nb, *end = sc + static_cast<int64_t>(R) * p.Kg, *a = s - sh / 8;
                auto word = [&](const uint8_t *at) -> uint32_t {
                    return at >= last ? 0u : at + 4 <= end ? *reinterpret_cast<const uint32_t *>(at) : tail;
                };
                uint32_t lo = word(a);
#pragma unroll
                for (int c = 0; c < CPS; ++c) {
                    const uint32_t hi = word(a + 4 * c + 4), v = __funnelshift_r(lo, hi, sh);
                    const int n = nb - 4 * c;                 // of this word's bytes, the row's
                    w[c] = n >= 4 ? v : n <= 0 ? 0u : v & ((1u << (8 * n)) - 1u);
                    lo = hi;
                }
            }
        };
        // the last, partial word of a scale array of that many bytes
        auto tail_word = [&](const uint8_t *sc, int64_t bytes) {
            uint32_t v = 0u;
            if (!PLAIN && !p.aligned)
                for (int i = 0; i < static_cast<int>(bytes & 3); ++i)
                    v |= static_cast<uint32_t>(sc[(bytes & ~int64_t(3)) + i]) << (8 * i);
            return v;
        };
        const uint32_t tail_b = tail_word(p.sB, static_cast<int64_t>(p.N) * p.Kg);
        const uint32_t tail_a = tail_word(p.sA, static_cast<int64_t>(p.M) * p.Kg);
        // the scale bytes of this thread's row of B, all of them, into L2: the
        // loads below reach only a few k-tiles, less than memory's latency
        if (n0 + 32 * q + lane < p.N && !odd) {
            const uint8_t *s = p.sB + static_cast<int64_t>(n0 + 32 * q + lane) * p.Kg;
            const int last = imin(4 * CPS * (kt0 + nkt), p.Kg);
            for (int o = 4 * CPS * kt0; o < last; o += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(s + o));
        }
        uint32_t rw[AHEAD][CPS], rx[AHEAD][NX][CPS];
        auto load_tile = [&](int i, int u) {                  // k-tile i of this CTA
            load_words(p.sB, p.N, n0 + 32 * q + lane, kt0 + i, tail_b, rw[u]);
#pragma unroll
            for (int m = 0; m < NX; ++m) load_words(p.sA, p.M, r0 + 32 * m + lane, kt0 + i, tail_a, rx[u][m]);
        };
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) load_tile(odd + 2 * u, u);
        // k-tile i has scale buffer i mod FW_SF_BUFS, which k-tile
        // i - FW_SF_BUFS has left when its stage is released, and arrives on
        // the barrier of stage i mod stages
        int b = odd, s = odd % p.stages, old_s = (odd + p.stages * FW_SF_BUFS - FW_SF_BUFS) % p.stages;
        int old_round = -((FW_SF_BUFS - odd + p.stages - 1) / p.stages);   // floor((odd - FW_SF_BUFS) / stages)
        bool ok = true;
        for (int i0 = odd; i0 < nkt && ok; i0 += 2 * AHEAD) {
#pragma unroll
            for (int u = 0; u < AHEAD; ++u) {
                const int i = i0 + 2 * u;
                if (i >= nkt || !ok) break;
                if (i >= FW_SF_BUFS && !warp_wait(&empty[old_s], static_cast<uint32_t>(old_round) & 1u)) {
                    abort_flag = 1;
                    ok = false;
                    break;
                }
                tc_fence_after();
                // one word per MMA k: a whole raw word (NVFP4), half of one
                // (MXFP4, its two scales in bytes 0-1) or a byte (MXFP8)
                auto mma_word = [&](const uint32_t *raw, int k) -> uint32_t {
                    if constexpr (FMT == QFP4_NVFP4) return raw[k];
                    else if constexpr (FMT == QFP4_MXFP4) return (raw[k >> 1] >> (16 * (k & 1))) & 0xFFFFu;
                    else return (raw[0] >> (8 * k)) & 0xFFu;
                };
                uint32_t av[16], bv[32];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t wa = mma_word(rw[u], k);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        av[4 * k + c] = wa;
                        bv[8 * k + c] = c < NX ? mma_word(rx[u][c < NX ? c : 0], k) : 0u;
                        bv[8 * k + 4 + c] = 0u;
                    }
                }
                tmem_st_x16(buf_a(b) + lane_base, av);
                tmem_st_x32(buf_b(b) + lane_base, bv);
                load_tile(i + 2 * AHEAD, u);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[s]);
                // two k-tiles on
                b = b + 2 >= FW_SF_BUFS ? b + 2 - FW_SF_BUFS : b + 2;
                s += 2;
                if (s >= p.stages) s -= p.stages;
                old_s += 2;
                if (old_s >= p.stages) {
                    old_s -= p.stages;
                    ++old_round;
                }
            }
        }
    }
    // ---------------------------------------------------- this CTA's sums, by
    // all twelve warps.  PLAIN: a thread a column, straight from tensor memory
    // (100 x 11008 x 4096 11.5 us on the device, the other way 13.6).  Else
    // through shared memory as [row][128], then quads of columns of this CTA's
    // rows over all threads: one generator call a quad, and no idle threads where
    // the output is narrow (100 x 11008 x 4096 with dropout 17.0 us, a thread a
    // column 20.5; 12440 x 32 x 704 9.6 and 18).
    __syncwarp();
    constexpr int U = fw_quads(NX);
    constexpr int SETS = FW_THREADS / 128;
    const int q = warp & 3, set = warp >> 2;
    const uint32_t acc_lane = tmem + (static_cast<uint32_t>(32 * q) << 16);
    const int quads = imin(FW_BN, p.N - n0) / 4, qd = static_cast<int>(threadIdx.x) % quads;
    const int n = n0 + 32 * q + lane;                         // PLAIN: this thread's column
    float4 bias = {};                                         // on its way while the sums are finished
    if (!PLAIN) bias = bias4_load(ep, n0 + 4 * qd, 4);
    else if (ep.bias && n < p.N) bias.x = ld_as_float(ep.bias, ep.bias_f32, n);
    const bool ok = warp_wait(&acc_full, 0) && !abort_flag;
    tc_fence_after();
    float alpha = 1.0f;
    if (FMT == QFP4_NVFP4) alpha = __fmul_rn(*p.tA, *p.tB);
    const uint64_t step = PLAIN ? 0ull : drop_step(ep.drop);
    float *sums = reinterpret_cast<float *>(smem);            // once every stage has been read (acc_full)
    if constexpr (PLAIN) {
        constexpr int EP = 4 * U;
        for (int m0 = EP * set; m0 < live; m0 += SETS * EP) {
            uint32_t r[EP];
            if constexpr (EP == 4) tmem_ld4(acc_lane + m0, r);
            else tmem_ld8(acc_lane + m0, r);
            tmem_ld_wait();
            reg_fence<EP>(r);
            if (ok && n < p.N)
                ep_column<OUT, EP>(ep, p.out, static_cast<int64_t>(r0 + m0) * p.N + n, p.N, live - m0, alpha, r, bias.x);
            __syncwarp();
        }
    } else {
        // (a CTA's rows, `rows` at a time: rank, rank + split, .., `count` of them)
        const int rows = FW_THREADS / quads, first = static_cast<int>(threadIdx.x) / quads;
        const int count = (live - rank + p.split - 1) / p.split;
        for (int m0 = 16 * set; m0 < live; m0 += 16 * SETS) {
            uint32_t r[16];
            tmem_ld16(acc_lane + m0, r);
            tmem_ld_wait();
            reg_fence<16>(r);
#pragma unroll
            for (int t = 0; t < 16; ++t) sums[(m0 + t) * FW_BN + 32 * q + lane] = __uint_as_float(r[t]);
        }
        // every CTA's sums are in its shared memory
        if (p.split == 1) __syncthreads();
        else cluster_sync();
        if (ok && first < rows && first < count) {
            const int64_t stride = static_cast<int64_t>(rows) * p.split * p.N;
#pragma unroll 1
            for (int k = first; k < count; k += rows * U) {
                const int row = rank + k * p.split, nu = imin(U, (count - k + rows - 1) / rows);
                float4 v[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const float *at = sums + (row + u * rows * p.split) * FW_BN + 4 * qd;
                    v[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (u >= nu) continue;
                    if (p.split == 1) v[u] = *reinterpret_cast<const float4 *>(at);
                    else {
                        float4 x[FW_MAX_SPLIT];
#pragma unroll
                        for (int r = 0; r < FW_MAX_SPLIT; ++r) {
                            x[r] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                            if (r < p.split) x[r] = ld_dsmem4(mapa_shared(smem_u32(at), r));
                        }
                        v[u] = x[0];
#pragma unroll
                        for (int r = 1; r < FW_MAX_SPLIT; ++r) {
                            v[u].x += x[r].x;
                            v[u].y += x[r].y;
                            v[u].z += x[r].z;
                            v[u].w += x[r].w;
                        }
                    }
                }
                ep_quads<OUT, U>(ep, p.out, static_cast<int64_t>(r0 + row) * p.N + n0 + 4 * qd, stride, nu, alpha, step, v, bias);
            }
        }
        __syncwarp();
        if (p.split > 1) cluster_sync();                      // nobody reads this CTA's shared memory any more
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, GM_TMEM_COLS);
}

template <int FMT, int OUT, int NX, bool PLAIN>
static int launch_few_nx(const CUtensorMap &tw, const CUtensorMap &tx, const FewParams &p, const EpParams &ep, int smem,
                      cudaStream_t s)
{
    if (ensure_dyn_smem<k_gemm_few<FMT, OUT, NX, PLAIN>>(FW_SMEM_MAX + 1024) != QFP4_OK) return QFP4_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.tiles_n * ((p.M + FW_ROWS - 1) / FW_ROWS) * p.split), 1, 1);
    cfg.blockDim = dim3(FW_THREADS, 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(p.split);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, k_gemm_few<FMT, OUT, NX, PLAIN>, tw, tx, p, ep) != cudaSuccess) {
        (void)cudaGetLastError();
        return QFP4_ERR_CUDA;
    }
    QFP4_LAUNCH_CHECK();
    return QFP4_OK;
}

template <int FMT, int OUT>
static int launch_few(const CUtensorMap &tw, const CUtensorMap &tx, const FewParams &p, const EpParams &ep, int smem,
                      cudaStream_t s)
{
    const bool plain = p.aligned && p.split == 1 && p.N > 4 * FW_BN && !ep.drop.on;
    if (p.rows <= 32)
        return plain ? launch_few_nx<FMT, OUT, 1, true>(tw, tx, p, ep, smem, s)
                     : launch_few_nx<FMT, OUT, 1, false>(tw, tx, p, ep, smem, s);
    return plain ? launch_few_nx<FMT, OUT, 4, true>(tw, tx, p, ep, smem, s)
                 : launch_few_nx<FMT, OUT, 4, false>(tw, tx, p, ep, smem, s);
}

static int64_t gemm_few_tiles(int64_t M, int64_t N)
{
    return ((N + FW_BN - 1) / FW_BN) * ((M + FW_ROWS - 1) / FW_ROWS);
}

// Up to 128 rows, and more where one tile an SM takes all of them: the pair
// kernel then has too few 256 x 256 tiles, and a prepass (512 x 4096 x 4096
// MXFP4 with bias and SiLU 18.2 us there, 13.2 here; 300 x 520 x 2080 16.7 and
// 10.2).  Larger outputs are the pair kernel's, which reads half the operand
// bytes from L2 for the same output.
static bool gemm_few_fits(int64_t M, int64_t N) { return M <= FW_ROWS || gemm_few_tiles(M, N) <= SMS; }

static int gemm_few(const uint8_t *A_codes, const uint8_t *A_scales, const float *A_tscale, const uint8_t *B_codes,
                    const uint8_t *B_scales, const float *B_tscale, int64_t M, int64_t N, int64_t K, qfp4_fmt fmt,
                    const EpParams &ep, qfp4_dtype out_dt, void *out, cudaStream_t stream)
{
    FewParams p;
    p.sA = A_scales;
    p.sB = B_scales;
    p.tA = A_tscale;
    p.tB = B_tscale;
    p.M = static_cast<int>(M);
    p.N = static_cast<int>(N);
    p.Kg = static_cast<int>(K / (fmt == QFP4_NVFP4 ? 16 : 32));
    p.KT = static_cast<int>((K + gm_bk(fmt) - 1) / gm_bk(fmt));
    p.tiles_n = static_cast<int>((N + FW_BN - 1) / FW_BN);
    p.rows = static_cast<int>(imin<int64_t>((M + 15) / 16 * 16, FW_ROWS));
    p.aligned = K % gm_bk(fmt) == 0;
    p.out = out;
    // as many CTAs as there are SMs, by splitting K (a CTA keeps two k-tiles at least)
    const int64_t tiles = gemm_few_tiles(M, N);
    p.split = static_cast<int>(imax<int64_t>(1, imin<int64_t>(imin<int64_t>(FW_MAX_SPLIT, SMS / tiles), p.KT / 2)));
    // all of a CTA's k-tiles under way at once, where shared memory allows
    const int stage = (FW_BN + p.rows) * GM_BKB;
    const int per = (p.KT + p.split - 1) / p.split;
    p.stages = imax(2, imin(imin(FW_MAX_STAGES, per), FW_SMEM_MAX / stage));
    const int smem = imax(p.stages * stage, FW_SMEM_MIN) + 1024;
    CUtensorMap tw, tx;
    const uint64_t row_bytes = static_cast<uint64_t>(fmt == QFP4_MXFP8 ? K : K / 2);
    {
        const uint64_t dims[2] = {row_bytes, static_cast<uint64_t>(N)}, strides[1] = {row_bytes};
        const uint32_t box[2] = {GM_BKB, FW_BN};
        const int st = encode_tensor_map(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(B_codes), dims,
                                         strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
        if (st != QFP4_OK) return st;
    }
    {
        const uint64_t dims[2] = {row_bytes, static_cast<uint64_t>(M)}, strides[1] = {row_bytes};
        const uint32_t box[2] = {GM_BKB, static_cast<uint32_t>(p.rows)};
        const int st = encode_tensor_map(&tx, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(A_codes), dims,
                                         strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
        if (st != QFP4_OK) return st;
    }
    const bool f32 = out_dt == QFP4_F32;
    if (fmt == QFP4_MXFP8)
        return f32 ? launch_few<QFP4_MXFP8, QFP4_F32>(tw, tx, p, ep, smem, stream)
                   : launch_few<QFP4_MXFP8, QFP4_BF16>(tw, tx, p, ep, smem, stream);
    if (fmt == QFP4_NVFP4)
        return f32 ? launch_few<QFP4_NVFP4, QFP4_F32>(tw, tx, p, ep, smem, stream)
                   : launch_few<QFP4_NVFP4, QFP4_BF16>(tw, tx, p, ep, smem, stream);
    return f32 ? launch_few<QFP4_MXFP4, QFP4_F32>(tw, tx, p, ep, smem, stream)
               : launch_few<QFP4_MXFP4, QFP4_BF16>(tw, tx, p, ep, smem, stream);
}

}  // namespace qfp4
