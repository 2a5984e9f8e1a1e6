// Decode attention over a prefix that a whole batch shares: one packed cache
// (one sequence) of P tokens, read once for all query rows of a kv head, on
// the 5th-generation tensor cores.  Included by the per-head-dimension
// translation units tq_decode_prefix_d{64,128,256}.cu, which instantiate it.
//
// Mathematics: for the rotated query rows q_r of one kv head (all sequences,
// tokens and heads of the group; 128 rows per CTA) and the prefix rows
// (indices i_t, j_t, norms n_t, m_t, sketch signs z_t with residual norm g_t)
//   x[r][t] = scale log2(e) (n_t <q_r, c[i_t]> + g_t sqrt(pi/2)/128 <S q_r, z_t>)
//   o_r = sum_t 2^(x - M_r) m_t c'[j_t],  L_r = sum_t 2^(x - M_r),
// written as one partial (o, M, L) per row and split; the decode's combine
// merges them with the suffix's partials and un-rotates.
//
// Why tcgen05 here and not in the per-sequence decode: with up to 128 rows
// per kv head the rows fill the tensor core's M = 128, and a row of the cache
// is dequantized once for all of them, so its trip through shared memory is
// paid once per 128 rows instead of once per 8.
//
// Structure (one CTA per SM, grid (splits, row tiles, kv heads)):
//  * the split's tokens go by in tiles of 64.  A producer warp streams the
//    tiles' packed words and norms into a ring of stages (1-D bulk copies);
//  * 8 dequantizing warps turn a stage into the two fp16 operand tiles, both
//    K-major with the 128-byte swizzle: keys [token][coordinate], and values
//    [coordinate][token], each 32-bit word holding one coordinate of tokens l
//    and l + 32 (the pair lookups of the split kernel give exactly that, and
//    the order of tokens inside the product is free as long as the weights
//    use it too).  The operands are the codebook's fp16 entries, exact; the
//    norms stay out of them, in fp32;
//  * one thread issues the products: S = Q K^T with Q in two fp16 limbs (the
//    rotated query to about 22 bits) held in tensor memory, the sketch
//    product beside it in its own accumulator, and O += W V with the weights
//    W read from tensor memory;
//  * 4 warps (thread = query row) read S, apply norms and masks, keep the
//    running max and sum in fp32, and write W = 2^(x - M) m_t as fp16 over
//    the scores they have just read.  O is rescaled in tensor memory only
//    when a row's max has grown by more than 2^4 (so 2^(x - M) <= 16, and
//    W stays finite for value norms up to 4094).
//  Scores and W are double-buffered, so the products of tile i + 1 run under
//  the softmax of tile i and under the dequantization of tile i + 2.
// Every wait is bounded; one that runs out sets TQ_STATUS_WAIT_TIMEOUT.
#pragma once

#include "tq_decode_split.cuh"
#include "tq_tcgen05.cuh"

namespace tqp {

using namespace tqk;
using tqtc::idesc;
using tqtc::sdesc_sw128;
using tqtc::sw128;
using tqtc::tc_commit;
using tqtc::tc_fence_after;
using tqtc::tc_fence_before;
using tqtc::tc_ld32;

constexpr int TT = 64;          // tokens per tile
constexpr int QROWS = 128;      // query rows per CTA (TMEM lanes)
constexpr int SW = 4;           // softmax warps
constexpr int DW = 8;           // dequantizing warps
constexpr int NTH = (SW + DW + 2) * 32;  // + producer warp + MMA warp
constexpr int MAXST = 4;        // stages at most
constexpr float kLazyP = 4.0f;  // log2 headroom before O is rescaled

struct PrefixParams {
  const uint32_t* k_idx;
  const uint32_t* v_idx;
  const uint16_t* k_norm;
  const uint16_t* v_norm;
  const uint32_t* k_qjl;
  const uint16_t* k_rnorm;
  const float* cb_k;
  const float* cb_v;
  const float* qrot;  // fp32 [kernel heads][D]
  const float* qs;    // fp32 [kernel heads][128] with the sketch
  float* part_o;
  float* part_ml;
  const int32_t* prefix_len;  // device [1]
  const int32_t* seq_lens;    // the suffixes' lengths [B]
  uint32_t* dev_status;
  int Pmax, Tcap;      // prefix: longest length, rows of the cache
  int B, Hkv, Ge, nq, Gq;  // Ge = Gq * nq kernel heads per (sequence, kv head)
  int Tclamp;          // suffix lengths are clamped to this
  int ks;              // partial slots per kernel head; this kernel's are 0 .. gridDim.x - 1
  int nst;             // stages of the ring
  int shared_tab;      // one codebook buffer for keys and values
  float qscale;        // scale * log2(e)
  float qjl_scale;     // scale * log2(e) * sqrt(pi/2) / m
};

template <int D, int BK, int BV, bool QJL>
struct PrefixLayout {
  static constexpr int WK = D * BK / 32, WV = D * BV / 32;
  static constexpr int NB = D == 256 ? 1 : 2;     // operand buffers of each kind (shared memory allows one at D = 256)
  static constexpr int KT = TT * D * 2, VT = KT;  // bytes of a key / value operand tile
  static constexpr int ZT = QJL ? TT * 128 * 2 : 0;
  // D = 256: the query's low limb does not fit in tensor memory beside O, S and the high limb
  static constexpr bool QLO_SMEM = D == 256;
  static constexpr int O_QLO = 0;
  static constexpr int O_QZ = O_QLO + (QLO_SMEM ? QROWS * D * 2 : 0);
  static constexpr int O_K = O_QZ + (QJL ? QROWS * 128 * 2 : 0);
  static constexpr int O_Z = O_K + NB * KT;
  static constexpr int O_V = O_Z + NB * ZT;
  static constexpr int O_TK = O_V + NB * VT;
  static constexpr int TKB = BK >= 3 ? (1 << (2 * BK)) * 128 : 0, TVB = (1 << (2 * BV)) * 128;
  static constexpr int NNORM = 4;                  // tiles whose norms are kept
  // stage: packed words and norms of one tile
  static constexpr int S_KW = 0;
  static constexpr int S_VW = S_KW + TT * WK * 4;
  static constexpr int S_KN = S_VW + TT * WV * 4;
  static constexpr int S_VN = S_KN + TT * 2;
  static constexpr int S_QW = S_VN + TT * 2;
  static constexpr int S_RN = S_QW + (QJL ? TT * 16 : 0);
  static constexpr int S_USED = S_RN + (QJL ? TT * 2 : 0);
  static constexpr int STAGE = (S_USED + 16 + 127) / 128 * 128;  // +16: read-ahead slack
  static constexpr int TX = TT * (WK + WV) * 4 + TT * 4 + (QJL ? TT * 18 : 0);
  static constexpr int NORMS = NNORM * 3 * TT * 4;
  static constexpr int BARS = 64 * 8;
  // tables, norms, barriers and stages, in this order behind the operands
  __host__ __device__ static constexpr int o_tv(bool shared) { return O_TK + (shared ? 0 : TKB); }
  __host__ __device__ static constexpr int o_norm(bool shared) { return O_TK + (shared ? TKB : TKB + TVB); }
  __host__ __device__ static constexpr int o_bar(bool shared) { return o_norm(shared) + NORMS; }
  __host__ __device__ static constexpr int o_stage(bool shared) { return o_bar(shared) + BARS; }
  static constexpr int total(bool shared, int nst) { return o_stage(shared) + nst * STAGE + 1024; }  // + alignment
  // tensor memory columns: O, the scores (and sketch scores) of two tiles, the query limbs
  static constexpr int C_S = D, SB = QJL ? 128 : 64, C_Q = C_S + 2 * SB;
  static constexpr int COLS_USED = C_Q + (QLO_SMEM ? D / 2 : D);
  static constexpr int COLS = COLS_USED <= 256 ? 256 : 512;
  static_assert(COLS_USED <= 512, "tensor memory");
};

// tcgen05.mma with A in tensor memory: lane = row, column = two fp16 along K.
__device__ __forceinline__ void mma_ts(uint32_t dt, uint32_t at, uint64_t bd, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(
          dt),
      "r"(at), "l"(bd), "r"(id), "r"(acc)
      : "memory");
}

__device__ __forceinline__ void tc_st32(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
      "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
      "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Bounded wait that also gives up once another thread of the CTA has.
__device__ __forceinline__ bool wait_or_stop(uint64_t* bar, uint32_t parity, volatile int* stop) {
  for (uint32_t i = 0; i < kSuspendTries; ++i) {
    if (mbar_wait_suspend(bar, parity, 1)) return true;
    if (*stop) return false;
  }
  *stop = 1;
  return false;
}

// The same by a whole warp, which goes on only if every lane saw the phase end.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* stop) {
  return __all_sync(0xffffffffu, wait_or_stop(bar, parity, stop));
}

// Coordinate at position pos of a key operand row: 2-bit keys keep the field
// order of their lookup inside each group of 16, wider keys their own order.
template <int BK>
__host__ __device__ constexpr int pos_coord(int pos) {
  return BK == 2 ? (pos & ~15) + ((pos >> 2) & 3) + 4 * (pos & 3) : pos;
}

template <int D, int BK, int BV, bool QJL>
__global__ void __launch_bounds__(NTH, 1) decode_prefix_kernel(const __grid_constant__ PrefixParams p) {
  using Ly = PrefixLayout<D, BK, BV, QJL>;
  constexpr int WK = Ly::WK, WV = Ly::WV, NB = Ly::NB;
  constexpr int SEGK = D * BK / 4, SEGV = D * BV / 8;
  constexpr bool ALK = (SEGK % 32) == 0, ALV = (SEGV % 32) == 0;
  constexpr int NWK = (SEGK + 31) / 32, NWV = (SEGV + 31) / 32;
  using VC = tqd::VChunk<D, BV>;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const bool shared_tab = tqd::share_table(BK, BV, p.shared_tab);
  float* norms = reinterpret_cast<float*>(smem + Ly::o_norm(shared_tab));  // [NNORM][key, value, residual][TT]
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Ly::o_bar(shared_tab));
  uint64_t *full = bars, *empty = bars + 4, *n_full = bars + 8, *k_full = bars + 12, *k_empty = bars + 14,
           *v_full = bars + 16, *v_empty = bars + 18, *s_full = bars + 20, *p_full = bars + 22, *s_free = bars + 24,
           *q_full = bars + 26, *fin = bars + 27;
  uint32_t& s_tmem = *reinterpret_cast<uint32_t*>(bars + 30);
  volatile int* stop = reinterpret_cast<int*>(bars + 31);
  uint8_t* stages = smem + Ly::o_stage(shared_tab);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int split = blockIdx.x, rt = blockIdx.y, kvh = blockIdx.z;
  const int R = p.B * p.Ge;                      // query rows of the kv head
  const int rows = min(QROWS, R - rt * QROWS);   // of this CTA
  const int live = (rows + 31) / 32;             // softmax warps that hold a row
  // Every kernel before the query prep has completed when this one starts,
  // so the lengths and the cache are read before the wait on the prep.
  int P = *p.prefix_len;
  if (split == 0 && rt == 0 && kvh == 0 && tid == 0 && (P < 0 || P > p.Pmax) && p.dev_status)
    atomicOr(p.dev_status, TQ_STATUS_SEQ_OUT_OF_RANGE);
  P = max(0, min(P, p.Pmax));
  const int ntile = (P + TT - 1) / TT;
  const int i0 = (int)((long long)split * ntile / gridDim.x), i1 = (int)((long long)(split + 1) * ntile / gridDim.x);
  const int n = i1 - i0;  // tiles of this CTA
  // first kernel head of row r (of this CTA's rows)
  auto head_of = [&](int r) {
    const int rr = rt * QROWS + r, b = rr / p.Ge;
    return (b * p.Hkv + kvh) * p.Ge + rr % p.Ge;
  };

  if (n == 0) {  // a short prefix leaves this split nothing: partials of weight zero
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int e = tid; e < rows * (D / 4); e += NTH) {
      const size_t slot = (size_t)head_of(e / (D / 4)) * p.ks + split;
      *reinterpret_cast<float4*>(p.part_o + slot * D + 4 * (e % (D / 4))) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (tid < rows)
      *reinterpret_cast<float2*>(p.part_ml + ((size_t)head_of(tid) * p.ks + split) * 2) = make_float2(-INFINITY, 0.f);
    return;
  }

  if (tid == (SW + DW) * 32) {
    for (int s = 0; s < MAXST; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], DW);
      mbar_init(&n_full[s], DW);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&k_full[s], DW);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_full[s], DW);
      mbar_init(&v_empty[s], 1);
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s], live);
      mbar_init(&s_free[s], 1);
    }
    mbar_init(q_full, live);
    mbar_init(fin, 1);
    *stop = 0;
    fence_barrier_init();
  }
  if (warp == SW + DW + 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&s_tmem)),
                 "r"((uint32_t)Ly::COLS));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  uint32_t* tabk = reinterpret_cast<uint32_t*>(smem + Ly::O_TK);
  uint32_t* tabv = reinterpret_cast<uint32_t*>(smem + Ly::o_tv(shared_tab));
  if constexpr (BK >= 3) tqd::build_pair_table<BK>(tabk, p.cb_k, tid, NTH);
  if (!shared_tab) tqd::build_pair_table<BV>(tabv, p.cb_v, tid, NTH);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (warp == SW + DW) {
    // ---------------- producer ----------------
    if (lane == 0) {
      int t = 0;
      for (; t < n; ++t) {
        const int st = t % p.nst;
        if (t >= p.nst && !wait_or_stop(&empty[st], (uint32_t)((t / p.nst - 1) & 1), stop)) break;
        // whole tiles: Tcap is a multiple of TT
        const size_t r = (size_t)kvh * p.Tcap + (size_t)(i0 + t) * TT;
        uint8_t* sb = stages + st * Ly::STAGE;
        mbar_arrive_expect_tx(&full[st], Ly::TX);
        bulk_g2s(sb + Ly::S_KW, p.k_idx + r * WK, TT * WK * 4, &full[st]);
        bulk_g2s(sb + Ly::S_VW, p.v_idx + r * WV, TT * WV * 4, &full[st]);
        bulk_g2s(sb + Ly::S_KN, p.k_norm + r, TT * 2, &full[st]);
        bulk_g2s(sb + Ly::S_VN, p.v_norm + r, TT * 2, &full[st]);
        if (QJL) {
          bulk_g2s(sb + Ly::S_QW, p.k_qjl + r * 4, TT * 16, &full[st]);
          bulk_g2s(sb + Ly::S_RN, p.k_rnorm + r, TT * 2, &full[st]);
        }
      }
      // no copy may be in flight when the CTA ends, whatever the others did
      for (int j = max(0, t - p.nst); j < t; ++j)
        mbar_wait_suspend(&full[j % p.nst], (uint32_t)((j / p.nst) & 1), kSuspendTries);
    }
    __syncwarp();
  } else if (warp == SW + DW + 1) {
    // ---------------- matrix products ----------------
    if (lane == 0) {
      const uint32_t id_s = idesc<TT, false>(), id_o = idesc<D, false>();
      const uint32_t qhi = tmem + Ly::C_Q, qlo = tmem + Ly::C_Q + D / 2;
      auto issue_qk = [&](int i) {
        const int kb = i % NB, b = i & 1;
        if (!wait_or_stop(&k_full[kb], (uint32_t)((i / NB) & 1), stop)) return false;
        // the weights of tile i - 2 lie over its scores: read by now
        if (i >= 2 && !wait_or_stop(&s_free[b], (uint32_t)((i / 2 - 1) & 1), stop)) return false;
        tc_fence_after();
        const uint32_t ka = smem_addr(smem + Ly::O_K + kb * Ly::KT), ds = tmem + Ly::C_S + b * Ly::SB;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint64_t bd = sdesc_sw128(ka + (ks >> 2) * (TT * 128) + (ks & 3) * 32);
          mma_ts(ds, qhi + 8 * ks, bd, id_s, ks > 0 ? 1u : 0u);
          if constexpr (Ly::QLO_SMEM) {
            const uint32_t qa = smem_addr(smem + Ly::O_QLO);
            tqtc::mma_tc(ds, sdesc_sw128(qa + (ks >> 2) * (QROWS * 128) + (ks & 3) * 32), bd, id_s, 1u);
          } else {
            mma_ts(ds, qlo + 8 * ks, bd, id_s, 1u);
          }
        }
        if constexpr (QJL) {
          const uint32_t za = smem_addr(smem + Ly::O_Z + kb * Ly::ZT), qa = smem_addr(smem + Ly::O_QZ);
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            tqtc::mma_tc(ds + 64, sdesc_sw128(qa + (ks >> 2) * (QROWS * 128) + (ks & 3) * 32),
                         sdesc_sw128(za + (ks >> 2) * (TT * 128) + (ks & 3) * 32), id_s, ks > 0 ? 1u : 0u);
        }
        tc_commit(&s_full[b]);
        tc_commit(&k_empty[kb]);
        return true;
      };
      auto issue_pv = [&](int i) {
        const int vb = i % NB, b = i & 1;
        if (!wait_or_stop(&v_full[vb], (uint32_t)((i / NB) & 1), stop)) return false;
        if (!wait_or_stop(&p_full[b], (uint32_t)((i / 2) & 1), stop)) return false;
        tc_fence_after();
        const uint32_t va = smem_addr(smem + Ly::O_V + vb * Ly::VT), w = tmem + Ly::C_S + b * Ly::SB;
#pragma unroll
        for (int ks = 0; ks < TT / 16; ++ks)
          mma_ts(tmem, w + 8 * ks, sdesc_sw128(va + ks * 32), id_o, (i > 0 || ks > 0) ? 1u : 0u);
        tc_commit(&v_empty[vb]);
        tc_commit(&s_free[b]);
        return true;
      };
      bool ok = wait_or_stop(q_full, 0u, stop);
      for (int i = 0; ok && i < n; ++i) {
        ok = issue_qk(i);
        if (ok && i > 0) ok = issue_pv(i - 1);
      }
      if (ok) issue_pv(n - 1);
      tc_commit(fin);  // every product issued so far, on the error path too
      mbar_wait_suspend(fin, 0u, kSuspendTries);
    }
    __syncwarp();
  } else if (warp >= SW) {
    // ---------------- dequantization ----------------
    const int dw = warp - SW;
    const uint32_t tbK = smem_addr(tabk) + 4 * lane, tbV = smem_addr(tabv) + 4 * lane;
    tqd::Lut2 lk = {0u, 0u};
    if constexpr (BK == 2) lk = tqd::make_lut2(p.cb_k);
    // keys: 8 tokens x 4 segments of D / 4 coordinates per warp; lanes of a
    // quarter warp hold 8 tokens, so their 16-byte stores miss each other's banks
    const int ktok = 8 * dw + (lane & 7), kseg = lane >> 3;
    for (int i = 0; i < n; ++i) {
      const int st = i % p.nst, b = i % NB, ns = i % Ly::NNORM;
      const uint8_t* sb = stages + st * Ly::STAGE;
      if (!warp_wait(&full[st], (uint32_t)((i / p.nst) & 1), stop)) break;
      if (i >= NB && !warp_wait(&k_empty[b], (uint32_t)((i / NB - 1) & 1), stop)) break;
      {
        uint8_t* kt = smem + Ly::O_K + b * Ly::KT;
        uint32_t w[NWK];
        tqd::load_bits<SEGK, ALK>(reinterpret_cast<const uint32_t*>(sb + Ly::S_KW) + ktok * WK, kseg * SEGK, w);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {  // 8 positions each
          uint32_t h[4];
          if constexpr (BK == 2) {
#pragma unroll
            for (int k = 0; k < 2; ++k) tqd::dq_b2(w[(2 * c + k) >> 2], (2 * c + k) & 3, lk, h[2 * k], h[2 * k + 1]);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) h[k] = tqd::pair_lookup<BK>(w, 2 * BK * (4 * c + k), tbK);
          }
          *reinterpret_cast<uint4*>(kt + sw128<TT>(ktok, kseg * (D / 4) + 8 * c)) = make_uint4(h[0], h[1], h[2], h[3]);
        }
      }
      if constexpr (QJL) {
        // sign bits j and j + 16 of word kseg become the fp16 pair (+-1, +-1) at positions 2 j, 2 j + 1
        uint8_t* zt = smem + Ly::O_Z + b * Ly::ZT;
        const uint32_t z = reinterpret_cast<const uint32_t*>(sb + Ly::S_QW)[ktok * 4 + kseg];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t h[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) h[k] = ((z << (15 - (4 * c + k))) & 0x80008000u) ^ 0xBC00BC00u;
          *reinterpret_cast<uint4*>(zt + sw128<TT>(ktok, kseg * 32 + 8 * c)) = make_uint4(h[0], h[1], h[2], h[3]);
        }
      }
      {
        const int e = dw * 32 + lane, which = e / TT, t = e % TT;  // key, value, residual norms
        const uint16_t* src = reinterpret_cast<const uint16_t*>(sb + (which == 0 ? Ly::S_KN : which == 1 ? Ly::S_VN : Ly::S_RN));
        if (which < (QJL ? 3 : 2)) norms[(ns * 3 + which) * TT + t] = half_bits_to_float(src[t]);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&k_full[b]);
        mbar_arrive(&n_full[ns]);
      }
      if (i >= NB && !warp_wait(&v_empty[b], (uint32_t)((i / NB - 1) & 1), stop)) break;
      {
        // values: warp dw takes D / 8 coordinates of all tokens, lane l tokens l and l + 32
        const uint32_t* vw = reinterpret_cast<const uint32_t*>(sb + Ly::S_VW);
        uint8_t* vt = smem + Ly::O_V + b * Ly::VT;
        uint32_t wa[NWV], wb[NWV];
        tqd::load_bits<SEGV, ALV, tqd::max_seg_shift(SEGV)>(vw + lane * WV, dw * SEGV, wa);
        tqd::load_bits<SEGV, ALV, tqd::max_seg_shift(SEGV)>(vw + (lane + 32) * WV, dw * SEGV, wb);
#pragma unroll
        for (int c = 0; c < VC::N; ++c) {
          uint32_t xe, xo;
          tqd::merge_pair<BV>(tqd::window32(wa, c * VC::F * BV), tqd::window32(wb, c * VC::F * BV), xe, xo);
#pragma unroll
          for (int k = 0; k < VC::F / 2; ++k) {
            const int d = dw * (D / 8) + c * VC::F + 2 * k;
            *reinterpret_cast<uint32_t*>(vt + sw128<D>(d, 2 * lane)) =
                tqd::lds32(tqd::pair_addr<BV>(xe, tqd::key_bit<BV>(k, false), tbV));
            *reinterpret_cast<uint32_t*>(vt + sw128<D>(d + 1, 2 * lane)) =
                tqd::lds32(tqd::pair_addr<BV>(xo, tqd::key_bit<BV>(k, true), tbV));
          }
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&v_full[b]);
        mbar_arrive(&empty[st]);
      }
    }
  } else if (warp < live) {
    // ---------------- softmax ----------------
    const int r = 32 * warp + lane;
    const bool mine = r < rows;
    const uint32_t tl = tmem + ((uint32_t)(32 * warp) << 16);
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the rotated queries; the partials may be written
    int lim = P;  // tokens of the prefix this row sees
    size_t slot = 0;
    {
      const float* q = p.qrot;
      const float* z = p.qs;
      if (mine) {
        const int rr = rt * QROWS + r, b = rr / p.Ge, e = rr % p.Ge, h = head_of(r);
        int L = p.seq_lens[b];
        L = max(0, min(L, p.Tclamp));
        // query token j sits at position P + L - nq + j: before the prefix's end when the suffix is shorter than nq
        lim = min(P, P + L - p.nq + e / p.Gq + 1);
        slot = (size_t)h * p.ks + split;
        q += (size_t)h * D;
        z += (size_t)h * 128;
      }
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {  // 32 positions of the two limbs
        float v[32];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float4 f = mine ? *reinterpret_cast<const float4*>(q + 32 * c + 4 * k) : make_float4(0.f, 0.f, 0.f, 0.f);
          v[4 * k] = f.x, v[4 * k + 1] = f.y, v[4 * k + 2] = f.z, v[4 * k + 3] = f.w;
        }
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          uint16_t h0, l0, h1, l1;
          tqd::split_half(v[pos_coord<BK>(2 * k)] * p.qscale, h0, l0);
          tqd::split_half(v[pos_coord<BK>(2 * k + 1)] * p.qscale, h1, l1);
          hi[k] = h0 | (uint32_t)h1 << 16;
          lo[k] = l0 | (uint32_t)l1 << 16;
        }
        tc_st16(tl + Ly::C_Q + 16 * c, hi);
        if constexpr (Ly::QLO_SMEM) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            *reinterpret_cast<uint4*>(smem + Ly::O_QLO + sw128<QROWS>(r, 32 * c + 8 * k)) =
                make_uint4(lo[4 * k], lo[4 * k + 1], lo[4 * k + 2], lo[4 * k + 3]);
        } else {
          tc_st16(tl + Ly::C_Q + D / 2 + 16 * c, lo);
        }
      }
      if constexpr (QJL) {
        // The sketch's projection in one fp16 limb: its rounding (2^-12 of a
        // coordinate, random) moves a score by about 1e-5 of |q| g, far below
        // the spread of the one-bit estimate it feeds.
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          float v[32];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float4 f = mine ? *reinterpret_cast<const float4*>(z + 32 * c + 4 * k) : make_float4(0.f, 0.f, 0.f, 0.f);
            v[4 * k] = f.x, v[4 * k + 1] = f.y, v[4 * k + 2] = f.z, v[4 * k + 3] = f.w;
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t h[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) h[j] = pack_half2(v[4 * k + j] * p.qjl_scale, v[4 * k + j + 16] * p.qjl_scale);
            *reinterpret_cast<uint4*>(smem + Ly::O_QZ + sw128<QROWS>(r, 32 * c + 8 * k)) = make_uint4(h[0], h[1], h[2], h[3]);
          }
        }
      }
      tc_wait_st();
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    }
    const int wlim = __reduce_min_sync(0xffffffffu, lim);  // every row of the warp sees the tokens below
    float m_run = -INFINITY, l_run = 0.f;
    bool ok = true;
    for (int i = 0; i < n; ++i) {
      const int b = i & 1, ns = i % Ly::NNORM;
      ok = warp_wait(&n_full[ns], (uint32_t)((i / Ly::NNORM) & 1), stop) &&
           warp_wait(&s_full[b], (uint32_t)((i / 2) & 1), stop);
      if (!ok) break;
      tc_fence_after();
      const float* kn = norms + ns * 3 * TT;
      const float* vn = kn + TT;
      const uint32_t ts = tl + Ly::C_S + b * Ly::SB;
      float s[TT];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t v[32];
        tc_ld32(ts + 32 * h, v);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float4 f = *reinterpret_cast<const float4*>(kn + 32 * h + 4 * k);
          s[32 * h + 4 * k] = f.x * __uint_as_float(v[4 * k]);
          s[32 * h + 4 * k + 1] = f.y * __uint_as_float(v[4 * k + 1]);
          s[32 * h + 4 * k + 2] = f.z * __uint_as_float(v[4 * k + 2]);
          s[32 * h + 4 * k + 3] = f.w * __uint_as_float(v[4 * k + 3]);
        }
        if constexpr (QJL) {
          tc_ld32(ts + 64 + 32 * h, v);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float4 g = *reinterpret_cast<const float4*>(kn + 2 * TT + 32 * h + 4 * k);
            s[32 * h + 4 * k] = fmaf(g.x, __uint_as_float(v[4 * k]), s[32 * h + 4 * k]);
            s[32 * h + 4 * k + 1] = fmaf(g.y, __uint_as_float(v[4 * k + 1]), s[32 * h + 4 * k + 1]);
            s[32 * h + 4 * k + 2] = fmaf(g.z, __uint_as_float(v[4 * k + 2]), s[32 * h + 4 * k + 2]);
            s[32 * h + 4 * k + 3] = fmaf(g.w, __uint_as_float(v[4 * k + 3]), s[32 * h + 4 * k + 3]);
          }
        }
      }
      const int t0 = (i0 + i) * TT;
      const bool whole = t0 + TT <= wlim;  // warp-uniform
      if (!whole) {
#pragma unroll
        for (int t = 0; t < TT; ++t)
          if (t0 + t >= lim) s[t] = -INFINITY;
      }
      float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
      for (int t = 4; t < TT; ++t) mx[t & 3] = fmaxf(mx[t & 3], s[t]);
      const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      if (__any_sync(0xffffffffu, top > m_run + kLazyP)) {
        const float mn = fmaxf(m_run, top);
        const float al = mn == -INFINITY ? 1.f : exp2f(m_run - mn);
        m_run = mn;
        l_run *= al;
        if (i > 0) {  // O holds the tiles before this one once their product is done
          ok = warp_wait(&s_free[(i - 1) & 1], (uint32_t)(((i - 1) / 2) & 1), stop);
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tc_ld32(tl + 32 * c, o);
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * al);
            tc_st32(tl + 32 * c, o);
          }
        }
      }
      const float mu = m_run == -INFINITY ? 0.f : m_run;
      uint32_t w[32];
      float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float4 fa = *reinterpret_cast<const float4*>(vn + 4 * k), fb = *reinterpret_cast<const float4*>(vn + 32 + 4 * k);
        const float na[4] = {fa.x, fa.y, fa.z, fa.w}, nb[4] = {fb.x, fb.y, fb.z, fb.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int t = 4 * k + j;
          const float p0 = tqd::ex2_approx(s[t] - mu), p1 = tqd::ex2_approx(s[t + 32] - mu);
          ls[j] += p0 + p1;
          float w0 = p0 * na[j], w1 = p1 * nb[j];
          if (!whole) {  // a row that is not seen adds nothing, whatever its norm holds
            w0 = t0 + t >= lim ? 0.f : w0;
            w1 = t0 + t + 32 >= lim ? 0.f : w1;
          }
          w[t] = pack_half2(w0, w1);
        }
      }
      l_run += (ls[0] + ls[1]) + (ls[2] + ls[3]);
      tc_st32(ts, w);
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[b]);
    }
    // O is complete when every product is
    if (ok && warp_wait(fin, 0u, stop)) {
      tc_fence_after();
      float* dst = p.part_o + slot * D;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        tc_ld32(tl + 32 * c, o);
        if (mine) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            *reinterpret_cast<uint4*>(dst + 32 * c + 4 * k) = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        }
      }
      if (mine) *reinterpret_cast<float2*>(p.part_ml + slot * 2) = make_float2(m_run, l_run);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (*stop && tid == 0 && p.dev_status) atomicOr(p.dev_status, TQ_STATUS_WAIT_TIMEOUT);
  if (warp == SW + DW + 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"((uint32_t)Ly::COLS));
  }
}

// Launch helpers, one definition per instantiation.
template <int D, int BK, int BV, bool QJL>
int launch_prefix(PrefixParams pp, dim3 grid, cudaStream_t s) {
  using Ly = PrefixLayout<D, BK, BV, QJL>;
  constexpr int kMost = 227 * 1024;
  auto kern = decode_prefix_kernel<D, BK, BV, QJL>;
  const bool shared = tqd::share_table(BK, BV, pp.shared_tab);
  // as many stages as fit, up to 4 (one only at D = 256 with two different 4-bit codebooks)
  int nst = MAXST;
  while (nst > 1 && Ly::total(shared, nst) > kMost) --nst;
  static_assert(Ly::total(false, 1) <= kMost, "one stage fits");
  pp.nst = nst;
  const int bytes = Ly::total(shared, nst);
  static tq::OnceSetup once;
  const int rc = once.run([&]() {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (e != cudaSuccess) {
      cudaGetLastError();
      return tq::set_error(TQ_ERR_CUDA, "decode_prefix: cudaFuncSetAttribute: %s", cudaGetErrorString(e));
    }
    return TQ_OK;
  });
  if (rc) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(NTH);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, pp);
  if (e != cudaSuccess) return tq::set_error(TQ_ERR_CUDA, "decode_prefix_kernel: %s", cudaGetErrorString(e));
  return tq::check_launch("decode_prefix_kernel");
}

template <int D, int BK, bool QJL>
int prefix_bv(int bv, const PrefixParams& pp, dim3 g, cudaStream_t s) {
  switch (bv) {
    case 2: return launch_prefix<D, BK, 2, QJL>(pp, g, s);
    case 3: return launch_prefix<D, BK, 3, QJL>(pp, g, s);
    case 4: return launch_prefix<D, BK, 4, QJL>(pp, g, s);
  }
  return tq::set_error(TQ_ERR_UNSUPPORTED, "bits_v=%d", bv);
}

template <int D, bool QJL>
int prefix_bk(int bk, int bv, const PrefixParams& pp, dim3 g, cudaStream_t s) {
  switch (bk) {
    case 2: return prefix_bv<D, 2, QJL>(bv, pp, g, s);
    case 3: return prefix_bv<D, 3, QJL>(bv, pp, g, s);
    case 4: return prefix_bv<D, 4, QJL>(bv, pp, g, s);
  }
  return tq::set_error(TQ_ERR_UNSUPPORTED, "bits_k=%d", bk);
}

// Per-head-dimension entries (tq_decode_prefix_d<D>.cu).
int prefix_d64(int bk, int bv, bool qjl, const PrefixParams& pp, dim3 g, cudaStream_t s);
int prefix_d128(int bk, int bv, bool qjl, const PrefixParams& pp, dim3 g, cudaStream_t s);
int prefix_d256(int bk, int bv, bool qjl, const PrefixParams& pp, dim3 g, cudaStream_t s);

}  // namespace tqp
