// gdr_bwd.cu -- sm_100a kernels for the gradients of the gated delta rule, in
// the chunked form (gdr_fwd.cu has the forward's formulas and names).
//
// From the forward, per chunk: T, Pm (the masked, scaled q.k), the decays,
// the state S at its start and the rows u it wrote.  With dS' the gradient
// reaching the state at the chunk's end, D_ij = e^(c_i - c_j) (j <= i), and
// rows i, j of the chunk:
//     du_j  = sum_{i>=j} Pm_ij do_i + e^(c_last - c_j) dS' k_j,    r = T^T du
//     dS    = e^(c_last) dS' + sum_i scale e^(c_i) do_i q_i^T - sum_j beta_j e^(c_j) r_j k_j^T
//     dv_j  = beta_j r_j
//     pd_ij = scale D_ij do_i.u_j (j <= i),   ad_ij = -beta_i D_ij r_i.u_j (j < i)
//     dq_i  = sum_j pd_ij k_j + scale e^(c_i) S^T do_i
//     dk_j  = sum_i pd_ij q_i + sum_i (ad_ij + ad_ji) k_i + e^(c_last - c_j) dS'^T u_j
//             - beta_j e^(c_j) S^T r_j
//     dbeta_i = r_i.v_i - e^(c_i) k_i.(S^T r_i) - sum_j D_ij (k_i.k_j) r_i.u_j
//     dc_i  = sum_j W_ij - sum_j W_ji + scale e^(c_i) q_i.(S^T do_i) - beta_i e^(c_i) k_i.(S^T r_i)
//             - e^(c_last - c_i) k_i.(dS'^T u_i),    W_ij = pd_ij q_i.k_j + ad_ij k_i.k_j  (j < i)
//     dc_last += e^(c_last) <S, dS'> + sum_i e^(c_last - c_i) k_i.(dS'^T u_i)
//     dg_t  = sum_{i >= t} dc_i over the chunk
// (the diagonal of W would cancel between its row and its column).
//
// Two launches: gdr_chain_kernel (gdr_chain.cu) walks the chunks backwards and
// writes dv, r and dS' per chunk; gdr_bwd_grad_kernel, parallel over chunks,
// forms the rest.  dq and dk of a group sum over its heads inside one block:
// no atomics, the same bits in every run.
//
// Precision: every gradient leaves as bf16 (2^-8).  The operands of the
// products are rounded to bf16 once each; products, sums, dS, the row sums
// and dc are fp32 or wider.  dh0 carries the products' operand rounding.
#include <cuda.h>

#include "gdr_common.cuh"

namespace mmscan {

static __device__ unsigned int g_grad_dev_err = 0;

namespace gdr {
namespace {

// ------------------------------------------------- everything else, by chunk ----
// One CTA an SM, on tensor cores (tcgen05 / TMEM); it goes from item to item (a
// batch row, group and chunk), the next one's first tiles loading while the
// last one's results leave.  As in the chain, k and q are stacked into one tile
// of 128 rows, and so are r and do: of every product the rows of k and dk are
// lanes 0-63, those of q and dq lanes 64-127.  Per head of the group:
//     1. [k; q] k^T (once)    2. [r; do] u^T     -> [ad; pd], the row and column sums of W
//     3. ACC += [ad; pd] k    5. ACC += [ad; pd]^T [k; q]  (lanes 0-63; zeros below)
//     4. Y = [r; do] S        6. Z = u dS'  (lanes 0-63)
//        dk += tail Z - beta e^c Y, dq += scale e^c Y, and their rows' products with k and q
// ACC stays in TMEM over the group's heads; what needs a factor of its row
// (Y, Z) the epilogue adds to it there, a thread a quarter of a row (held in
// registers instead, the sums spill, and with the shared memory in use what
// spills goes to L2: 147 us against 100).  Products 4 and 6 run while the
// epilogue forms [ad; pd], after 1 and 2.
//
// Roles (19 warps): 0-15 the epilogues, then one for the loads and the stores,
// one for the products, and one that sums up a head's decays before and its dg
// and dbeta after.  Loads are issued in the order of need, k and q (into the
// tile that the last item's dq and dk leave from) before S and dS'.  Waits are
// bounded as in the chain, and the two warps that issue copies and products see
// them complete before they leave.
//
// Bound: the latency of one chunk's steps (one CTA an SM: 190 KB of tiles and
// all of TMEM at P = N = 128): the last item's store, k and q, two products,
// [ad; pd], two products, the sums.  Measured: 100 us for 2048 chunks of one head
// of 128 x 128, 141 for 1040 of four heads of 64 x 128.  A CTA an item took 127
// and 149 us, with 8 epilogue warps 130 and 156; warp-level products (mma.sync)
// 174 for the first.  Products 3 and 5 before 4 and 6: 108 and 140 us.
constexpr int SLAB = 128 * 128;                        // 64 columns of a stacked tile
constexpr int GEPI = 16, NP = GEPI / 4, G_LOAD = GEPI, G_MMA = GEPI + 1, G_AUX = GEPI + 2, GTHREADS = 32 * (GEPI + 3);
// (B_CUM, B_ROWS: by head parity; B_RO, B_ST, B_FREE: by slot)
enum { B_QK = 0, B_G = 1, B_YZ = 2, B_YZF = 3, B_AP = 4, B_ACC = 5, B_DONE = 6, B_CUM = 7, B_ROWS = 9, B_RO = 11, B_ST = 13, B_FREE = 15, B_END = 17, NGBAR = 18 };

template <int DK, int DV>
struct GradSmem {
    static constexpr int KQ = 0, AP = DK / 64 * SLAB, Z0 = AP + SLAB, SLOTS0 = Z0 + SLAB;
    // a slot: the tiles of one head; two of them where they fit, so that the next head's loads run ahead
    static constexpr int RO = 0, U = DV / 64 * SLAB, S = U + DV / 64 * (SLAB / 2), DS = S + DV * DK * 2, V = DS + DV * DK * 2;
    static constexpr int F = V + DV / 64 * (SLAB / 2), SLOT = F + 1024;    // F: eg, tail, beta
    static constexpr int NS = DV == 64 ? 2 : 1;
    // by head parity: the decays (double c[C], float e^(c - mid), e^(mid - c), [C]) ...
    static constexpr int CUM = SLOTS0 + NS * SLOT, CUM_BYTES = C * 8 + 2 * C * 4;
    // ... and the sums: by column quarter, of dc by row of [k; q], of e^.. k.(dS' u) and of dbeta by row of k;
    // the column sums by lane quarter; <S, dS'> by warp
    static constexpr int ROW = CUM + 2 * CUM_BYTES, ROWS = NP * 4 * C * 4 + 4 * C * 4 + 128;
    static constexpr int WIDE = ROW + 2 * ROWS, BAR = WIDE + 16, TSLOT = BAR + NGBAR * 8, ABORT = TSLOT + 8;
    static constexpr int BYTES = ABORT + 8 + 1024;
    static_assert(BYTES <= 227 * 1024 && U % 1024 == 0 && S % 1024 == 0 && SLOT % 1024 == 0, "shared memory");
};
constexpr uint32_t TG_KQ = 0, TG_G = 64, TG_ACC = 128, TG_Y = 256, TG_Z = 384;

template <int DK, int DV>
__global__ void __launch_bounds__(GTHREADS, 1)
gdr_bwd_grad_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_q,
                    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                    const __grid_constant__ CUtensorMap tm_dk, const __grid_constant__ CUtensorMap tm_dq, const GDRArgs p) {
    using L = GradSmem<DK, DV>;
    constexpr int TV = DV / 64, HC = DK / NP;          // tiles of 64 p; columns of q and k a thread
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    const uint32_t base = (raw_addr + 1023u) & ~1023u;
    unsigned char* sm = smem_raw + (base - raw_addr);
    const int tid = threadIdx.x, lane = tid & 31, w = __shfl_sync(0xffffffffu, tid >> 5, 0);
    // The block's items m = 0 .. items - 1; their heads count on as n = 0 .. heads - 1.
    const int64_t all = p.batch * p.ngroups * p.nchunks;
    const int hpg = (int)(p.nheads / p.ngroups), items = (int)((all - blockIdx.x + gridDim.x - 1) / gridDim.x);
    const int heads = items * hpg;                            // (batch * nheads * chunks < 2^31)
    struct Item { int64_t b; int grp, t0; int64_t ch; };
    auto item_of = [&](int m) {
        const int64_t it = blockIdx.x + (int64_t)m * gridDim.x, bg = it / p.nchunks;
        Item x;
        x.ch = it - bg * p.nchunks;
        x.b = bg / p.ngroups;
        x.grp = (int)(bg - x.b * p.ngroups);
        x.t0 = (int)(x.ch * C);
        return x;
    };
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + L::ABORT);
    int* wide = reinterpret_cast<int*>(sm + L::WIDE);
    auto bar = [&](int i) { return base + L::BAR + 8u * (uint32_t)i; };
    if (tid == 0) {
        const int counts[NGBAR] = {1, 1, 1, GEPI, GEPI, 1, GEPI, 1, 1, GEPI, GEPI, 1, 1, 1, 1, GEPI + 1, GEPI + 1, 1};
        for (int i = 0; i < NGBAR; ++i) mbar_init(bar(i), counts[i]);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (w == 0) tmem_alloc(base + L::TSLOT, 512);
    for (int i = tid; i < SLAB / 16; i += GTHREADS) *reinterpret_cast<uint4*>(sm + L::Z0 + 16 * i) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sm + L::TSLOT);
    auto wait = [&](int i, int phase) -> bool {
        if (*abort_flag) return false;
        if (!mbar_wait_sleep(bar(i), (uint32_t)phase & 1u, &g_grad_dev_err)) {
            *abort_flag = 1;
            return false;
        }
        return true;
    };
    auto wwait = [&](int i, int phase) { return __all_sync(0xffffffffu, wait(i, phase)); };
    auto arrive = [&](int i) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(i));
    };

    if (w == G_LOAD) {
        if (lane == 0) {                                     // (stall: test only, only the first heads staged, every wait runs out)
            // dq, dk of item m, staged in the tile of k and q (rows past L are clipped)
            auto store = [&](int m) -> bool {
                if (!wait(B_DONE, m)) return false;
                const Item x = item_of(m);
#pragma unroll
                for (int s = 0; s < DK / 64; ++s) {
                    tma_store_4d(&tm_dk, base + L::KQ + s * SLAB, 64 * s, x.grp, x.t0, (int)x.b);
                    tma_store_4d(&tm_dq, base + L::KQ + s * SLAB + SLAB / 2, 64 * s, x.grp, x.t0, (int)x.b);
                }
                bulk_commit_group();
                bulk_wait_read_all();
                return true;
            };
            bool live = true;
            int n = 0, qks = 0, ros = 0, sts = 0;              // loads issued: items' k and q, heads' tiles, heads' S and dS'
            for (int m = 0; m < items && live; ++m) {
                const Item x = item_of(m);
                for (int hh = 0; hh < hpg; ++hh, ++n) {
                    const int sl = n % L::NS, h = x.grp * hpg + hh;
                    if (p.stall && n == p.stall - 1) {
                        live = false;
                        break;
                    }
                    if (n >= L::NS && !(live = wait(B_FREE + sl, n / L::NS - 1))) break;
                    const int64_t rec = (x.b * p.nheads + h) * p.nchunks + x.ch;
                    const uint32_t slot = base + L::SLOTS0 + sl * L::SLOT, ro = bar(B_RO + sl), st = bar(B_ST + sl);
                    mbar_expect_tx(ro, TV * 2 * SLAB + 3 * C * 4);
#pragma unroll
                    for (int t = 0; t < TV; ++t) {
                        bulk_load(slot + L::RO + t * SLAB, static_cast<const unsigned char*>(p.dr) + (rec * TV + t) * (SLAB / 2), SLAB / 2, ro);
                        tma_load_4d(slot + L::RO + t * SLAB + SLAB / 2, &tm_do, ro, 64 * t, h, x.t0, (int)x.b);
                        tma_load_4d(slot + L::V + t * (SLAB / 2), &tm_v, ro, 64 * t, h, x.t0, (int)x.b);
                    }
                    bulk_load(slot + L::U, static_cast<const unsigned char*>(p.u) + rec * TV * (SLAB / 2), TV * (SLAB / 2), ro);
                    bulk_load(slot + L::F, static_cast<const unsigned char*>(p.rec) + rec * REC_BYTES + REC_F, 3 * C * 4, ro);
                    ++ros;
                    if (hh == 0) {                           // k and q, once the tile has given up the last item's dq and dk: before
                                                             // S and dS', which are needed last (a store queues behind the loads)
                        if (m > 0 && !(live = store(m - 1))) break;
                        mbar_expect_tx(bar(B_QK), DK / 64 * SLAB);
#pragma unroll
                        for (int s = 0; s < DK / 64; ++s) {
                            tma_load_4d(base + L::KQ + s * SLAB, &tm_k, bar(B_QK), 64 * s, x.grp, x.t0, (int)x.b);
                            tma_load_4d(base + L::KQ + s * SLAB + SLAB / 2, &tm_q, bar(B_QK), 64 * s, x.grp, x.t0, (int)x.b);
                        }
                        ++qks;
                    }
                    mbar_expect_tx(st, 2 * DV * DK * 2);
                    bulk_load(slot + L::S, static_cast<const unsigned char*>(p.states) + rec * DV * DK * 2, DV * DK * 2, st);
                    bulk_load(slot + L::DS, static_cast<const unsigned char*>(p.dstates) + rec * DV * DK * 2, DV * DK * 2, st);
                    ++sts;
                }
            }
            if (live) store(items - 1);                      // (read out of shared memory: it is the kernel's end that completes it)
            for (int x = ros < L::NS ? 0 : ros - L::NS; x < ros; ++x) drain(bar(B_RO + x % L::NS), x / L::NS, &g_grad_dev_err);
            for (int x = sts < L::NS ? 0 : sts - L::NS; x < sts; ++x) drain(bar(B_ST + x % L::NS), x / L::NS, &g_grad_dev_err);
            if (qks > 0) drain(bar(B_QK), qks - 1, &g_grad_dev_err);
        }
    } else if (w == G_MMA) {
        const uint32_t kq = base + L::KQ, ap = base + L::AP;
        constexpr uint32_t ID64 = umma_idesc_bf16(128, 64, 0, 0), IDKK = umma_idesc_bf16(128, DK, 0, 0),
                           IDKN = umma_idesc_bf16(128, DK, 0, 1), IDNN = umma_idesc_bf16(128, DK, 1, 1);
        auto kmaj = [&](uint32_t tile, int s, uint32_t stride) { return umma_desc_sw128(tile + (s >> 2) * stride + (s & 3) * 32, 16, 1024); };
        bool live = true;
        int n = 0;
        for (int m = 0; m < items && live; ++m) {
            for (int hh = 0; hh < hpg; ++hh, ++n) {
                const int sl = n % L::NS, ph = (n & 1);
                const uint32_t slot = base + L::SLOTS0 + sl * L::SLOT, ro = slot + L::RO, u = slot + L::U;
                if (!(live = wwait(B_RO + sl, n / L::NS))) break;
                tc_fence_after();
#pragma unroll
                for (int s = 0; s < DV / 16; ++s) umma_elect(tmem + TG_G, kmaj(ro, s, SLAB), kmaj(u, s, SLAB / 2), ID64, s > 0);
                if (hh == 0) {                               // k and q come after the last item's results have left
                    if (!(live = wwait(B_QK, m))) break;
                    tc_fence_after();
#pragma unroll
                    for (int s = 0; s < DK / 16; ++s) umma_elect(tmem + TG_KQ, kmaj(kq, s, SLAB), kmaj(kq, s, SLAB), ID64, s > 0);
                }
                commit_elect(bar(B_G));
                if (!(live = wwait(B_ST + sl, n / L::NS) && (n == 0 || wwait(B_YZF, ph ^ 1)))) break;
                tc_fence_after();
#pragma unroll
                for (int s = 0; s < DV / 16; ++s) umma_elect(tmem + TG_Y, kmaj(ro, s, SLAB), kmaj(slot + L::S, s, DK * 128), IDKK, s > 0);
#pragma unroll
                for (int s = 0; s < DV / 16; ++s) umma_elect(tmem + TG_Z, kmaj(u, s, SLAB / 2), kmaj(slot + L::DS, s, DK * 128), IDKK, s > 0);
                commit_elect(bar(B_YZ));
                commit_elect(bar(B_FREE + sl));
                if (!(live = wwait(B_AP, ph))) break;
                tc_fence_after();
#pragma unroll
                for (int s = 0; s < C / 16; ++s)
                    umma_elect(tmem + TG_ACC, kmaj(ap, s, 0), umma_desc_sw128(kq + s * 2048, SLAB, 1024), IDKN, hh > 0 || s > 0);
#pragma unroll
                for (int s = 0; s < 2 * C / 16; ++s)
                    umma_elect(tmem + TG_ACC, umma_desc_sw128(ap + s * 2048, L::Z0 - L::AP, 1024), umma_desc_sw128(kq + s * 2048, SLAB, 1024), IDNN, 1u);
                commit_elect(bar(B_ACC));
            }
        }
        commit_elect(bar(B_END));                            // behind every product and commit before it
        drain(bar(B_END), 0, &g_grad_dev_err);
    } else if (w == G_AUX) {
        auto decays = [&](int n) {
            const Item x = item_of(n / hpg);
            const int h = x.grp * hpg + n % hpg, valid = (int)(p.seqlen - x.t0 < C ? p.seqlen - x.t0 : C);
            double* cum = reinterpret_cast<double*>(sm + L::CUM + (n & 1) * L::CUM_BYTES);
            float* ef = reinterpret_cast<float*>(cum + C);
            const int r = 2 * lane;
            double s0, s1, last;
            chunk_cumsum(static_cast<const bf16*>(p.g) + (x.b * p.seqlen + x.t0) * p.nheads + h, p.nheads, valid, lane, s0, s1, last);
            cum[r] = s0;
            cum[r + 1] = s1;
            // factors of e^(c_i - c_j), or ones (and then by element), as in the preparing kernel
            const double first = __shfl_sync(0xffffffffu, s0, 0), mid = 0.5 * (first + last);
            const double a0 = (s0 - mid) * kLog2e, a1 = (s1 - mid) * kLog2e;
            const bool far = __any_sync(0xffffffffu, !(fabs(a0) < 60.0) || !(fabs(a1) < 60.0));
            *reinterpret_cast<float2*>(ef + r) = far ? f2(1.0f, 1.0f) : f2(ex2_approx((float)a0), ex2_approx((float)a1));
            *reinterpret_cast<float2*>(ef + C + r) = far ? f2(1.0f, 1.0f) : f2(ex2_approx((float)-a0), ex2_approx((float)-a1));
            if (lane == 0) wide[n & 1] = far;
            arrive(B_CUM + (n & 1));
        };
        decays(0);
        for (int n = 0; n < heads; ++n) {
            if (n + 1 < heads) decays(n + 1);                // its buffer was head n - 1's, whose sums are taken
            if (!wwait(B_ROWS + (n & 1), n >> 1)) break;
            const Item x = item_of(n / hpg);
            const int h = x.grp * hpg + n % hpg, valid = (int)(p.seqlen - x.t0 < C ? p.seqlen - x.t0 : C);
            const float* rowc = reinterpret_cast<const float*>(sm + L::ROW + (n & 1) * L::ROWS);   // [part][128]
            const float* rowk = rowc + NP * 2 * C;                                                 // [part][C]
            const float* rowb = rowk + NP * C;
            const float* colv = rowb + NP * C;                                                     // [quarter][C]
            const float* red = colv + 4 * C;                                                       // [warp], then e^(c_last)
            float dc[2], ok[2], db[2], sums = 0.0f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = 2 * lane + e;
                float col = colv[C + i] + colv[3 * C + i];   // rows 32-63 of k and of q
                if (i < 32) col += colv[i] + colv[2 * C + i];
                ok[e] = db[e] = dc[e] = 0.0f;
#pragma unroll
                for (int m = 0; m < NP; ++m) {
                    ok[e] += rowk[m * C + i];
                    db[e] += rowb[m * C + i];
                    dc[e] += rowc[2 * m * C + i] + rowc[(2 * m + 1) * C + i];
                }
                dc[e] -= col + ok[e];
                sums += ok[e];
            }
#pragma unroll
            for (int m = 16; m >= 1; m >>= 1) sums += __shfl_xor_sync(0xffffffffu, sums, m);
            if (lane == 31) {
                float t = 0.0f;
#pragma unroll
                for (int m = 0; m < GEPI; ++m) t += red[m];
                dc[1] = fmaf(red[GEPI], t, dc[1] + sums);
            }
            // dg = the sums from each row to the chunk's end
            dc[0] += dc[1];
            float run = dc[0];
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const float dn = __shfl_down_sync(0xffffffffu, run, m);
                if (lane + m < 32) run += dn;
            }
            const float after = run - dc[0];
            const int64_t at = (x.b * p.seqlen + x.t0 + 2 * lane) * p.nheads + h;
            bf16* dg = static_cast<bf16*>(p.dg);
            bf16* dbeta = static_cast<bf16*>(p.dbeta);
            if (2 * lane < valid) {
                dg[at] = __float2bfloat16_rn(run);
                dbeta[at] = __float2bfloat16_rn(db[0]);
            }
            if (2 * lane + 1 < valid) {
                dg[at + p.nheads] = __float2bfloat16_rn(dc[1] + after);
                dbeta[at + p.nheads] = __float2bfloat16_rn(db[1]);
            }
        }
    } else {
        const int q = w & 3, part = w >> 2;
        const int t = 32 * q + lane, i = t & 63;             // TMEM lane: row of [k; q]; step of the chunk
        const bool krows = q < 2;
        const bool below = (q & 1) != 0 || part < NP / 2;    // this warp's 32 x 16 of [ad; pd] reaches the triangle
        const uint32_t lb = tmem + ((uint32_t)(q * 32) << 16);
        const int c0 = HC * part;                            // this thread's columns of q and k
        bool ok = true;
        int hh = 0, m = 0;
        for (int n = 0; n < heads; ++n, ++hh) {
            if (hh == hpg) {
                hh = 0;
                ++m;
            }
            const int sl = n % L::NS, ph = (n & 1);
            const double* cum = reinterpret_cast<const double*>(sm + L::CUM + ph * L::CUM_BYTES);
            const float* ef = reinterpret_cast<const float*>(cum + C);
            const unsigned char* slot = sm + L::SLOTS0 + sl * L::SLOT;
            const float* f = reinterpret_cast<const float*>(slot + L::F);
            float* rowc = reinterpret_cast<float*>(sm + L::ROW + ph * L::ROWS);
            float* rowk = rowc + NP * 2 * C;
            float* rowb = rowk + NP * C;
            float* colv = rowb + NP * C;
            float* red = colv + 4 * C;
            float rc = 0.0f, rk = 0.0f, rb = 0.0f;
            if (!(ok = wwait(B_CUM + ph, n >> 1) && wwait(B_RO + sl, n / L::NS))) break;
            const float eg = f[i], tail = f[C + i], beta = f[2 * C + i];
            if (krows) {                                     // r.v over this thread's part of p
#pragma unroll
                for (int m = 0; m < DV / 8 / NP; ++m) {
                    const int x = part * (DV / 8 / NP) + m;
                    const uint4 vv = *reinterpret_cast<const uint4*>(slot + L::V + (x >> 3) * (SLAB / 2) + tile_off<128>(i, x & 7));
                    const uint4 rr = *reinterpret_cast<const uint4*>(slot + L::RO + (x >> 3) * SLAB + tile_off<128>(i, x & 7));
                    rb = fmaf(bf16_lo(vv.x), bf16_lo(rr.x), fmaf(bf16_hi(vv.x), bf16_hi(rr.x), rb));
                    rb = fmaf(bf16_lo(vv.y), bf16_lo(rr.y), fmaf(bf16_hi(vv.y), bf16_hi(rr.y), rb));
                    rb = fmaf(bf16_lo(vv.z), bf16_lo(rr.z), fmaf(bf16_hi(vv.z), bf16_hi(rr.z), rb));
                    rb = fmaf(bf16_lo(vv.w), bf16_lo(rr.w), fmaf(bf16_hi(vv.w), bf16_hi(rr.w), rb));
                }
            }
            if (!(ok = wwait(B_G, ph))) break;
            tc_fence_after();
            if (below) {
                uint32_t g[16], kq[16], ap[8];
                tmem_ld16(lb + TG_G + 16 * part, g);
                tmem_ld16(lb + TG_KQ + 16 * part, kq);
                tmem_wait_ld();
                // d: what multiplies r.u (minus the decay) or do.u (scale times it)
                const float row = (krows ? -1.0f : p.scale) * ef[i];
                const bool apart = wide[ph] != 0;
                float wv[16];
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const float4 fj = *reinterpret_cast<const float4*>(ef + C + 16 * part + e);
                    float d[4] = {row * fj.x, row * fj.y, row * fj.z, row * fj.w};
                    if (apart) {
                        const float sgn = krows ? -1.0f : p.scale;
#pragma unroll 1
                        for (int k = 0; k < 4; ++k) {
                            const int j = 16 * part + e + k;
                            const float x = j <= i ? sgn * ex2_approx((float)((cum[i] - cum[j]) * kLog2e)) : 0.0f;
                            d[0] = k == 0 ? x : d[0];
                            d[1] = k == 1 ? x : d[1];
                            d[2] = k == 2 ? x : d[2];
                            d[3] = k == 3 ? x : d[3];
                        }
                    }
                    float a[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int j = 16 * part + e + k;
                        const float x = (krows ? j < i : j <= i) ? d[k] * __uint_as_float(g[e + k]) : 0.0f;
                        const float s = __uint_as_float(kq[e + k]);
                        if (krows) rb = fmaf(x, s, rb);
                        a[k] = krows ? beta * x : x;
                        wv[e + k] = j < i ? a[k] * s : 0.0f;
                        rc += wv[e + k];
                    }
                    ap[e / 2] = pack_bf16x2(a[0], a[1]);
                    ap[e / 2 + 1] = pack_bf16x2(a[2], a[3]);
                }
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    *reinterpret_cast<uint4*>(sm + L::AP + tile_off<128>(t, 2 * part + c)) = make_uint4(ap[4 * c], ap[4 * c + 1], ap[4 * c + 2], ap[4 * c + 3]);
                fence_proxy_async_smem();
                tc_fence_before();
                arrive(B_AP);
                float col[1];
                butterfly_sum<16, 16>(wv, col, lane & 15);   // lanes j, j + 16: column j's sum over half the warp's rows each
                col[0] += __shfl_xor_sync(0xffffffffu, col[0], 16);
                if (lane < 16) colv[q * C + 16 * part + lane] = col[0];
            } else {
#pragma unroll
                for (int c = 0; c < 2; ++c) *reinterpret_cast<uint4*>(sm + L::AP + tile_off<128>(t, 2 * part + c)) = make_uint4(0, 0, 0, 0);
                fence_proxy_async_smem();
                tc_fence_before();
                arrive(B_AP);
            }
            // <S, dS'>: both tiles have the same layout
            if (!(ok = wwait(B_ST + sl, n / L::NS))) break;
            float sd = 0.0f;
#pragma unroll 4
            for (int x = tid; x < DV * DK / 8; x += 32 * GEPI) {
                const uint4 a = *reinterpret_cast<const uint4*>(slot + L::S + x * 16), d = *reinterpret_cast<const uint4*>(slot + L::DS + x * 16);
                sd = fmaf(bf16_lo(a.x), bf16_lo(d.x), fmaf(bf16_hi(a.x), bf16_hi(d.x), sd));
                sd = fmaf(bf16_lo(a.y), bf16_lo(d.y), fmaf(bf16_hi(a.y), bf16_hi(d.y), sd));
                sd = fmaf(bf16_lo(a.z), bf16_lo(d.z), fmaf(bf16_hi(a.z), bf16_hi(d.z), sd));
                sd = fmaf(bf16_lo(a.w), bf16_lo(d.w), fmaf(bf16_hi(a.w), bf16_hi(d.w), sd));
            }
#pragma unroll
            for (int x = 16; x >= 1; x >>= 1) sd += __shfl_xor_sync(0xffffffffu, sd, x);
            if (lane == 0) red[w] = sd;
            if (tid == 0) red[GEPI] = f[C - 1];
            arrive(B_FREE + sl);
            // Y and Z, 16 columns at a time, onto ACC: back to TMEM for the group's next
            // head, or as dk and dq into the tile of k and q (of which a thread reads
            // and writes the same elements; the products have read them)
            if (!(ok = wwait(B_YZ, ph) && wwait(B_ACC, ph) && (hh > 0 || wwait(B_QK, m)))) break;
            tc_fence_after();
            float dy = 0.0f, dz = 0.0f;
            const float fy = krows ? -beta * eg : p.scale * eg;
            const bool last = hh + 1 == hpg;
#pragma unroll
            for (int cc = 0; cc < HC / 16; ++cc) {
                const int col = c0 + 16 * cc;
                uint32_t y[16], z[16], a[16];
                tmem_ld16(lb + TG_Y + col, y);
                tmem_ld16(lb + TG_ACC + col, a);
                if (krows) tmem_ld16(lb + TG_Z + col, z);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint4* at = reinterpret_cast<uint4*>(sm + L::KQ + (col >> 6) * SLAB + tile_off<128>(t, ((col & 63) >> 3) + c));
                    const uint4 row = *at;
                    const uint32_t r4[4] = {row.x, row.y, row.z, row.w};
                    uint32_t o[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int k = 8 * c + 2 * e;
                        const float2 yy = f2(__uint_as_float(y[k]), __uint_as_float(y[k + 1]));
                        const float2 kk = f2(bf16_lo(r4[e]), bf16_hi(r4[e]));
                        float2 g = fma2(f2(fy, fy), yy, f2(__uint_as_float(a[k]), __uint_as_float(a[k + 1])));
                        dy = fmaf(yy.x, kk.x, fmaf(yy.y, kk.y, dy));
                        if (krows) {
                            const float2 zz = f2(__uint_as_float(z[k]), __uint_as_float(z[k + 1]));
                            g = fma2(f2(tail, tail), zz, g);
                            dz = fmaf(zz.x, kk.x, fmaf(zz.y, kk.y, dz));
                        }
                        a[k] = __float_as_uint(g.x);
                        a[k + 1] = __float_as_uint(g.y);
                        o[e] = pack_bf16x2(g.x, g.y);
                    }
                    if (last) *at = make_uint4(o[0], o[1], o[2], o[3]);
                }
                if (!last) tmem_st16(lb + TG_ACC + col, a);
            }
            if (last) fence_proxy_async_smem();
            else tmem_wait_st();
            tc_fence_before();
            arrive(B_YZF);
            if (last) arrive(B_DONE);
            rc = fmaf(fy, dy, rc);
            if (krows) {
                rk = tail * dz;
                rb = fmaf(-eg, dy, rb);
                rowk[part * C + i] = rk;
                rowb[part * C + i] = rb;
            }
            rowc[part * 2 * C + t] = rc;
            arrive(B_ROWS + ph);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (w == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

unsigned int read_and_clear_grad_error() {
    unsigned int v = 0, z = 0;
    if (cudaMemcpyFromSymbol(&v, g_grad_dev_err, sizeof(v)) != cudaSuccess) return 0;
    if (v) cudaMemcpyToSymbol(g_grad_dev_err, &z, sizeof(z));
    return v;
}

[[maybe_unused]] const bool g_registered = (register_error_reader(read_and_clear_grad_error), true);

template <int DK, int DV>
cudaError_t launch_grad(const GDRArgs& a, const CallMaps& m, cudaStream_t s) {
    constexpr int bytes = GradSmem<DK, DV>::BYTES;
    CUtensorMap mv, mdk, mdq;
    cudaError_t e;
    if ((e = map_steps(&mdk, a.dk, DK, a.ngroups, a.seqlen, a.batch)) != cudaSuccess) return e;
    if ((e = map_steps(&mdq, a.dq, DK, a.ngroups, a.seqlen, a.batch)) != cudaSuccess) return e;
    if ((e = map_steps(&mv, a.v, DV, a.nheads, a.seqlen, a.batch)) != cudaSuccess) return e;
    static std::atomic<uint64_t> attr_done{0};
    if ((e = allow_dynamic_smem(reinterpret_cast<const void*>(gdr_bwd_grad_kernel<DK, DV>), bytes, attr_done)) != cudaSuccess) return e;
    const int64_t items = a.batch * a.ngroups * a.nchunks;
    gdr_bwd_grad_kernel<DK, DV><<<(unsigned)(items < 148 ? items : 148), GTHREADS, bytes, s>>>(m.k, m.q, mv, m.v, mdk, mdq, a);
    return cudaGetLastError();
}

template <int DK>
cudaError_t launch_bwd(const GDRArgs& a, cudaStream_t s) {
    CallMaps m;
    cudaError_t e;
    if ((e = map_call(&m, a, a.dout)) != cudaSuccess || (e = launch_gdr_chain(a, true, m, s)) != cudaSuccess) return e;
    return a.headdim == 64 ? launch_grad<DK, 64>(a, m, s) : launch_grad<DK, 128>(a, m, s);
}

}  // namespace
}  // namespace gdr

cudaError_t launch_gdr_bwd(const GDRArgs& a, cudaStream_t s) {
    return a.dstate == 64 ? gdr::launch_bwd<64>(a, s) : gdr::launch_bwd<128>(a, s);
}

}  // namespace mmscan
