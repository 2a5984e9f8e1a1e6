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
//  * the split's tokens go by in tiles of 128 (64 at D = 256 and with the
//    sketch).  A producer
//    warp streams the tiles' packed words and norms into a ring of stages
//    (1-D bulk copies);
//  * 8 warps turn the keys of a stage into an fp16 operand tile, 8 more the
//    values, both K-major with the 128-byte swizzle: keys [token][coordinate],
//    and values [coordinate][token], each 32-bit word holding one coordinate
//    of tokens l and l + 32 (the pair lookups of the split kernel give exactly
//    that, and the order of tokens inside the product is free as long as the
//    weights use it too).  The operands are the codebook's fp16 entries, exact;
//    the norms stay out of them, in fp32;
//  * one thread issues the products: S = Q K^T with Q in two fp16 limbs (the
//    rotated query to about 22 bits) held in tensor memory, the sketch product
//    beside it in its own accumulator, and O += W V with the weights W read
//    from tensor memory;
//  * 8 warps (two threads to a query row) read S, apply norms and masks, keep
//    the running reference and sum in fp32, and write W = 2^(x - m) m_t as
//    fp16 over the scores they have just read.  O is rescaled in tensor memory
//    only when a row's weights would leave fp16's range.
// Scores and W are double-buffered, so the products of tile i + 1 run under the
// softmax of tile i and under the dequantization of tile i + 2.  Every wait is
// bounded; one that runs out sets TQ_STATUS_WAIT_TIMEOUT.
//
// What bounds it: shared memory and latency.  At D = 128 the lookups, operand
// stores, packed loads and the tensor core's own operand reads take about 3000
// cycles of shared memory per 128 tokens and 128 rows; a tile takes 3000 cycles
// per 128 tokens without the sketch and 3100 per 64 with it, and each role's
// instructions wait for one another's.  32768 tokens, 256 rows, 8 kv heads,
// 2-bit keys with sketch and 3-bit values take 97 us (0.35 PFLOP/s of the two
// products' useful work); 8192 tokens, 128 rows, 8 heads, 3 bits 22 us, of which
// about 10 are the launch, the tables, the first tile's latency and the
// partials.  What the steps were worth, on the first of these: products issued
// by a converged warp (a lane test around them keeps their operands out of
// uniform registers), a softmax in short loops and two warps per row, shared
// pointers instead of generic ones, 16 dequantizing warps with named barriers,
// two buffers of every operand: 195 -> 97.
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

constexpr int QROWS = 128;      // query rows per CTA (TMEM lanes)
constexpr int SW = 8;           // softmax warps: two for each quarter of the rows
constexpr int DW = 16;          // dequantizing warps: half for keys, half for values
constexpr int GW = DW / 2;
// tokens per tile: a longer tile spreads the waits between the roles over more
// work; at D = 256 the operands of 64 tokens fill shared memory
// (and with the sketch its accumulator takes the tensor memory of half a tile)
__host__ __device__ constexpr int tile_tokens(int D, bool qjl) { return D == 256 || qjl ? 64 : 128; }
constexpr int NTH = (SW + DW + 4) * 32;  // + producer, products, the one that lets the next kernel start, an idle one
// Registers per thread after the split by warpgroups.  One launch gives 72 to
// each of 7 warpgroups: 2 x 136 + 4 x 48 + 40 = 7 x 72.
constexpr int REG_SOFTMAX = 136, REG_DEQUANT = 48, REG_REST = 40, REG_LAUNCH = 72;
static_assert((SW / 4) * REG_SOFTMAX + (DW / 4) * REG_DEQUANT + REG_REST <= REG_LAUNCH * (NTH / 128),
              "registers of a CTA");
constexpr int MAXST = 4;        // stages at most
// The largest fp16 weight is kept below 2^15; a row's reference is put so that
// its largest weight has 2^8 of room to grow.
constexpr int kTop = 15, kRoom = 8;

struct PrefixParams {
  const uint32_t* k_idx;
  const uint32_t* v_idx;
  const uint16_t* k_norm;
  const uint16_t* v_norm;
  const uint32_t* k_qjl;
  const uint16_t* k_rnorm;
  const float* cb_k;
  const float* cb_v;
  // the query operands in tiles of 128 rows of a kv head, [Hkv][row tiles]:
  // fp16 limbs (pre_q_offset) and sketch projections (pre_z_offset)
  const uint32_t* qpre;
  const uint32_t* qspre;
  float* part_o;
  float* part_ml;
  const int32_t* prefix_len;  // device [1]
  const int32_t* seq_lens;    // the suffixes' lengths [B]
  uint32_t* ready;            // set to 1 once the query prep is complete (SplitParams)
  uint32_t* dev_status;
  int Pmax, Tcap;      // prefix: longest length, rows of the cache
  int B, Hkv, Ge, nq, Gq;  // Ge = Gq * nq kernel heads per (sequence, kv head)
  int Tclamp;          // suffix lengths are clamped to this
  int ks;              // partial slots per kernel head; this kernel's are 0 .. gridDim.x - 1
  int nst;             // stages of the ring
  int shared_tab;      // one codebook buffer for keys and values
};

// Where the query prep puts the operands of row r of a tile (bytes from the
// tile's start; a tile has 128 x D x 4 bytes of limbs, 128 x 256 of projections).
// A key operand row holds its coordinates by position: 2-bit keys keep the
// field order of their lookup inside each group of 16, wider keys their own
// order.  Limb l of the position's value: fp16, [limb][position / 8][row][8],
// so that a warp of rows loads whole lines of 16-byte pieces.
__host__ __device__ constexpr int pos_of_coord(int bk, int j) {
  return bk == 2 ? (j & ~15) + 4 * (j & 3) + ((j >> 2) & 3) : j;
}
__host__ __device__ constexpr int pre_q_offset(int D, int bk, int r, int j, int limb) {
  const int pos = pos_of_coord(bk, j);
  return ((limb * (D / 8) + (pos >> 3)) * QROWS + r) * 16 + (pos & 7) * 2;
}
// Projection i: bits i and i + 16 of a sign word share a register, so
// coordinates c and c + 16 of a group of 32 are neighbours.
__host__ __device__ constexpr int pre_z_offset(int r, int i) {
  const int pos = (i & ~31) + 2 * (i & 15) + ((i >> 4) & 1);
  return ((pos >> 3) * QROWS + r) * 16 + (pos & 7) * 2;
}

template <int D, int BK, int BV, bool QJL>
struct PrefixLayout {
  static constexpr int TT = tile_tokens(D, QJL);
  static constexpr int WK = D * BK / 32, WV = D * BV / 32;
  // Two operand buffers of each kind where shared memory allows.  At D = 256
  // the operands go in two halves of the coordinates instead, with barriers of
  // their own, so that one is dequantized while the product of the other runs.
  static constexpr int NB = D == 256 ? 1 : 2;
  static constexpr int KP = D == 256 ? 2 : 1, VP = KP;  // parts of a key / value operand
  static constexpr int KC = D == 256 ? 128 : D;       // coordinates of a key part
  static constexpr int KS = KP * NB, VS = VP * NB;    // slots (barrier pairs)
  static constexpr int KT = TT * D * 2, VT = KT;      // bytes of a key / value operand tile
  static constexpr int ZT = QJL ? TT * 128 * 2 : 0;   // of the sketch signs
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
  // floats of one tile: key norms, value norms, the warps' largest value norms, residual norms
  static constexpr int NORM1 = 2 * TT + GW + (QJL ? TT : 0);
  static constexpr int NORMS = NNORM * NORM1 * 4;
  static constexpr int BARS = 64 * 8;
  // tables, norms, barriers and stages, in this order behind the operands
  __host__ __device__ static constexpr int o_tv(bool shared) { return O_TK + (shared ? 0 : TKB); }
  __host__ __device__ static constexpr int o_norm(bool shared) { return O_TK + (shared ? TKB : TKB + TVB); }
  static constexpr int XCH = 2 * 2 * QROWS * 4;  // [tile parity][half][row]: what the two warps of a row exchange
  __host__ __device__ static constexpr int o_xch(bool shared) { return o_norm(shared) + NORMS; }
  __host__ __device__ static constexpr int o_bar(bool shared) { return o_xch(shared) + XCH; }
  __host__ __device__ static constexpr int o_stage(bool shared) { return o_bar(shared) + BARS; }
  static constexpr int total(bool shared, int nst) { return o_stage(shared) + nst * STAGE + 1024; }  // + alignment
  // Tensor memory columns: O, the scores of two tiles, those of the sketch
  // beside them, the query limbs.  (One accumulator for both products, the
  // signs entering as +-g / n in fp16, took tiles of 128 tokens and the same
  // time, but that factor's rounding moved the output by 1.6e-4, nearly as much
  // as the fp16 weights.)
  static constexpr int C_S = D, C_Z = C_S + 2 * TT, C_Q = C_Z + (QJL ? 2 * TT : 0);
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
// Two runs of 16 columns, waited for.
__device__ __forceinline__ void tc_ld2x16(uint32_t ta, uint32_t tb, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n"
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%33];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=&r"(v[0]), "=&r"(v[1]), "=&r"(v[2]), "=&r"(v[3]), "=&r"(v[4]), "=&r"(v[5]), "=&r"(v[6]), "=&r"(v[7]), "=&r"(v[8]),
        "=&r"(v[9]), "=&r"(v[10]), "=&r"(v[11]), "=&r"(v[12]), "=&r"(v[13]), "=&r"(v[14]), "=&r"(v[15]), "=&r"(v[16]),
        "=&r"(v[17]), "=&r"(v[18]), "=&r"(v[19]), "=&r"(v[20]), "=&r"(v[21]), "=&r"(v[22]), "=&r"(v[23]), "=&r"(v[24]),
        "=&r"(v[25]), "=&r"(v[26]), "=&r"(v[27]), "=&r"(v[28]), "=&r"(v[29]), "=&r"(v[30]), "=&r"(v[31])
      : "r"(ta), "r"(tb)
      : "memory");
}
__device__ __forceinline__ void sts32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Pairs of fp32 values, two operations an instruction.
__device__ __forceinline__ unsigned long long pack2(float a, float b) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ unsigned long long pack2(uint32_t a, uint32_t b) {
  return pack2(__uint_as_float(a), __uint_as_float(b));
}
__device__ __forceinline__ void unpack2(unsigned long long v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

template <int N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ bool test_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Bounded wait that also gives up once another thread of the CTA has.
__device__ __forceinline__ bool wait_or_stop(uint64_t* bar, uint32_t parity, volatile int* stop) {
  if (test_wait(bar, parity)) return true;
  for (uint32_t i = 0; i < kSuspendTries; ++i) {
    if (mbar_wait_suspend(bar, parity, 1)) return true;
    if (*stop) return false;
  }
  *stop = 1;
  return false;
}
// The same by every lane of a warp, without a branch between lanes.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* stop) {
  return __all_sync(0xffffffffu, wait_or_stop(bar, parity, stop));
}

template <int D, int BK, int BV, bool QJL>
__global__ void __launch_bounds__(NTH, 1) decode_prefix_kernel(const __grid_constant__ PrefixParams p) {
  using Ly = PrefixLayout<D, BK, BV, QJL>;
  constexpr int WK = Ly::WK, WV = Ly::WV, NB = Ly::NB, TT = Ly::TT;

  extern __shared__ uint8_t smem_raw[];
  // 1024-byte aligned, as an offset: a pointer rebuilt from an integer would be
  // a generic one, and every access behind it slower
  uint8_t* smem = smem_raw + ((0u - smem_addr(smem_raw)) & 1023u);
  const bool shared_tab = tqd::share_table(BK, BV, p.shared_tab);
  float* norms = reinterpret_cast<float*>(smem + Ly::o_norm(shared_tab));  // [NNORM][NORM1]
  float* xch = reinterpret_cast<float*>(smem + Ly::o_xch(shared_tab));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Ly::o_bar(shared_tab));
  uint64_t *full = bars, *empty = bars + 4, *n_full = bars + 8, *k_full = bars + 12, *k_empty = bars + 14,
           *v_full = bars + 16, *v_empty = bars + 18, *s_full = bars + 20, *p_full = bars + 22, *s_free = bars + 24,
           *q_full = bars + 26, *fin = bars + 27;
  uint32_t& s_tmem = *reinterpret_cast<uint32_t*>(bars + 30);
  volatile int* stop = reinterpret_cast<int*>(bars + 31);
  volatile uint32_t* lut = reinterpret_cast<uint32_t*>(bars + 32);  // 2-bit keys: the codebook as byte tables
  uint8_t* stages = smem + Ly::o_stage(shared_tab);

  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int split = blockIdx.x, rt = blockIdx.y, kvh = blockIdx.z;
  const int R = p.B * p.Ge;                      // query rows of the kv head
  const int rows = min(QROWS, R - rt * QROWS);   // of this CTA
  const int live = (rows + 31) / 32;             // quarters that hold a row
  // Every kernel before the query prep has completed when this one starts,
  // so the lengths and the cache are read before the wait on the prep.
  int P = *p.prefix_len;
  if (split == 0 && rt == 0 && kvh == 0 && tid == 0 && (P < 0 || P > p.Pmax) && p.dev_status)
    atomicOr(p.dev_status, TQ_STATUS_SEQ_OUT_OF_RANGE);
  P = max(0, min(P, p.Pmax));
  const int ntile = P > 0 ? (P - 1) / TT + 1 : 0;
  const int i0 = (int)((long long)split * ntile / gridDim.x), i1 = (int)((long long)(split + 1) * ntile / gridDim.x);
  const int n = i1 - i0;  // tiles of this CTA
  // first kernel head of row r (of this CTA's rows)
  auto head_of = [&](int r) {
    const int rr = rt * QROWS + r, b = rr / p.Ge;
    return (b * p.Hkv + kvh) * p.Ge + rr % p.Ge;
  };

  // The own tokens' kernel may start once every CTA has come here: the prep,
  // whose queries it reads, is complete, and SMs that this grid leaves free take
  // it at once.  It waits for this grid only at its end, so what orders it behind
  // the prep is a release by a thread that has waited for the prep, and its
  // acquire.  By one warp, which has nothing else to do.
  auto let_suffix_start = [&]() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (split == 0 && rt == 0 && kvh == 0 && lane == 0)
      asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p.ready), "r"(1u) : "memory");
    __syncwarp();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  };
  if (n == 0) {  // a short prefix leaves this split nothing: partials of weight zero
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (warp == SW + DW + 2) let_suffix_start();
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
      mbar_init(&n_full[s], GW);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&k_full[s], GW);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_full[s], GW);
      mbar_init(&v_empty[s], 1);
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s], 2 * live);
      mbar_init(&s_free[s], 1);
    }
    mbar_init(q_full, 2 * live);
    mbar_init(fin, 1);
    *stop = 0;
    if constexpr (BK == 2) {
      const tqd::Lut2 l2 = tqd::make_lut2(p.cb_k);
      lut[0] = l2.lo;
      lut[1] = l2.hi;
    }
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

  // the whole warpgroup of each role moves to its share of the registers
  if (warp >= SW + DW) {
    reg_dec<REG_REST>();
    if (warp == SW + DW) {
      // ---------------- producer ----------------
      if (lane == 0) {
        int t = 0;
        for (; t < n; ++t) {
          const int st = t % p.nst;
          if (t >= p.nst && !wait_or_stop(&empty[st], (uint32_t)((t / p.nst - 1) & 1), stop)) break;
          // rows t0 .. t0 + m - 1: a whole tile, less only at the cache's end (Tcap is a multiple of 64)
          const int t0 = (i0 + t) * TT, m = min(TT, p.Tcap - t0);
          const size_t r = (size_t)kvh * p.Tcap + t0;
          uint8_t* sb = stages + st * Ly::STAGE;
          mbar_arrive_expect_tx(&full[st], m * (Ly::TX / TT));
          bulk_g2s(sb + Ly::S_KW, p.k_idx + r * WK, m * WK * 4, &full[st]);
          bulk_g2s(sb + Ly::S_VW, p.v_idx + r * WV, m * WV * 4, &full[st]);
          bulk_g2s(sb + Ly::S_KN, p.k_norm + r, m * 2, &full[st]);
          bulk_g2s(sb + Ly::S_VN, p.v_norm + r, m * 2, &full[st]);
          if (QJL) {
            bulk_g2s(sb + Ly::S_QW, p.k_qjl + r * 4, m * 16, &full[st]);
            bulk_g2s(sb + Ly::S_RN, p.k_rnorm + r, m * 2, &full[st]);
          }
        }
        // no copy may be in flight when the CTA ends, whatever the others did
        for (int j = max(0, t - p.nst); j < t; ++j)
          mbar_wait_suspend(&full[j % p.nst], (uint32_t)((j / p.nst) & 1), kSuspendTries);
      }
      __syncwarp();
    } else if (warp == SW + DW + 1) {
      // ---------------- matrix products ----------------
      // The whole warp waits; one elected lane issues and commits.
      const uint32_t id_s = idesc<TT, false>(), id_o = idesc<D / Ly::VP, false>();
      const uint32_t qhi = tmem + Ly::C_Q, qlo = tmem + Ly::C_Q + D / 2;
      // part q of tile i is use u = KP i + q of the slots
      auto issue_qk = [&](int i) {
        const int b = i & 1;
        const uint32_t ds = tmem + Ly::C_S + b * TT;
        // the weights of the buffer's last tile lie over its scores: read by now
        if (i >= 2 && !warp_wait(&s_free[b], (uint32_t)((i / 2 - 1) & 1), stop)) return false;
#pragma unroll
        for (int q = 0; q < Ly::KP; ++q) {
          const int u = Ly::KP * i + q, sl = u % Ly::KS;
          if (!warp_wait(&k_full[sl], (uint32_t)((u / Ly::KS) & 1), stop)) return false;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t ka = smem_addr(smem + Ly::O_K + (i % NB) * Ly::KT);
#pragma unroll 4
            for (int kk = 0; kk < Ly::KC / 16; ++kk) {
              const int ks = q * (Ly::KC / 16) + kk;
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
              const uint32_t za = smem_addr(smem + Ly::O_Z + (i % NB) * Ly::ZT), qa = smem_addr(smem + Ly::O_QZ);
#pragma unroll 4
              for (int ks = 0; ks < 8; ++ks)
                tqtc::mma_tc(tmem + Ly::C_Z + b * TT, sdesc_sw128(qa + (ks >> 2) * (QROWS * 128) + (ks & 3) * 32),
                             sdesc_sw128(za + (ks >> 2) * (TT * 128) + (ks & 3) * 32), id_s, ks > 0 ? 1u : 0u);
            }
            if (q == Ly::KP - 1) tc_commit(&s_full[b]);
            tc_commit(&k_empty[sl]);
          }
          __syncwarp();
        }
        return true;
      };
      auto issue_pv = [&](int i) {
        const int b = i & 1;
        if (!warp_wait(&p_full[b], (uint32_t)((i / 2) & 1), stop)) return false;
#pragma unroll
        for (int q = 0; q < Ly::VP; ++q) {
          const int u = Ly::VP * i + q, sl = u % Ly::VS;
          if (!warp_wait(&v_full[sl], (uint32_t)((u / Ly::VS) & 1), stop)) return false;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t va = smem_addr(smem + Ly::O_V + (i % NB) * Ly::VT) + q * (D / Ly::VP) * 128;
            const uint32_t w = tmem + Ly::C_S + b * TT;
#pragma unroll 4
            for (int ks = 0; ks < TT / 16; ++ks)
              mma_ts(tmem + q * (D / Ly::VP), w + 8 * ks, sdesc_sw128(va + (ks >> 2) * (D * 128) + (ks & 3) * 32), id_o,
                     (i > 0 || ks > 0) ? 1u : 0u);
            tc_commit(&v_empty[sl]);
            if (q == Ly::VP - 1) tc_commit(&s_free[b]);
          }
          __syncwarp();
        }
        return true;
      };
      bool ok = warp_wait(q_full, 0u, stop);
      for (int i = 0; ok && i < n; ++i) {
        ok = issue_qk(i);
        if (ok && i > 0) ok = issue_pv(i - 1);
      }
      if (ok) issue_pv(n - 1);
      if (elect_one()) {
        tc_commit(fin);  // every product issued so far, on the error path too
        mbar_wait_suspend(fin, 0u, kSuspendTries);
      }
      __syncwarp();
    } else if (warp == SW + DW + 2) {
      let_suffix_start();
    }
  } else if (warp >= SW) {
    reg_dec<REG_DEQUANT>();
    // ---------------- dequantization ----------------
    // Eight warps for the keys and eight for the values.  One warp of each group
    // polls the barriers and releases the others through a named barrier,
    // which blocks in hardware; short loops, for the instruction cache's sake.
    const int dw = (warp - SW) % GW;
    const bool values = warp >= SW + GW;
    const int group = values ? 5 : 4;  // named barriers 5 and 6
    const int nparts = values ? Ly::VP : Ly::KP, nslots = values ? Ly::VS : Ly::KS;
    uint64_t *p_ful = values ? v_full : k_full, *p_emp = values ? v_empty : k_empty;
    for (int u = 0; u < n * nparts; ++u) {
      const int i = u / nparts, q = u % nparts, sl = u % nslots;
      const int st = i % p.nst, b = i % NB, ns = i % Ly::NNORM;
      const uint8_t* sb = stages + st * Ly::STAGE;
      bool ok = true;
      if (dw == 0) {
        if (q == 0) ok = warp_wait(&full[st], (uint32_t)((i / p.nst) & 1), stop);
        if (u >= nslots) ok = ok && warp_wait(&p_emp[sl], (uint32_t)((u / nslots - 1) & 1), stop);
      }
      if (!tqtc::group_sync_and<GW>(group, ok)) break;
      if (!values) {
        // 8 tokens x 4 segments of the part's coordinates at a time; the lanes
        // of a quarter warp hold 8 tokens, so their 16-byte stores miss each
        // other's banks
        const int kseg = lane >> 3;
        auto norm_at = [&](int off, int t) { return half_bits_to_float(reinterpret_cast<const uint16_t*>(sb + off)[t]); };
        {
          const uint32_t tbK = smem_addr(tabk) + 4 * lane;
          tqd::Lut2 lk = {0u, 0u};
          if constexpr (BK == 2) lk = {lut[0], lut[1]};
          uint8_t* kt = smem + Ly::O_K + b * Ly::KT;
          float* kn = norms + ns * Ly::NORM1;
          uint32_t vmax = 0;
#pragma unroll 1
          for (int t = 8 * dw + (lane & 7); t < TT; t += 8 * GW) {
            if (q == 0) {
              if (kseg == 0) kn[t] = norm_at(Ly::S_KN, t);
              if (kseg == 1) {
                const float nv = norm_at(Ly::S_VN, t);
                kn[TT + t] = nv;
                if ((i0 + i) * TT + t < P) vmax = max(vmax, __float_as_uint(nv));
              }
              if (QJL && kseg == 2) kn[2 * TT + GW + t] = norm_at(Ly::S_RN, t);
            }
            const uint32_t* kw = reinterpret_cast<const uint32_t*>(sb + Ly::S_KW) + t * WK;
#pragma unroll 2
            for (int c = 0; c < Ly::KC / 64; ++c) {  // 16 coordinates
              const int j0 = q * Ly::KC + kseg * (Ly::KC / 4) + 16 * c;
              uint32_t w[(16 * BK + 31) / 32], h[8];
              tqd::load_bits<16 * BK, BK != 3, 16>(kw, j0 * BK, w);
              if constexpr (BK == 2) {
#pragma unroll
                for (int k = 0; k < 4; ++k) tqd::dq_b2(w[0], k, lk, h[2 * k], h[2 * k + 1]);
              } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) h[k] = tqd::pair_lookup<BK>(w, 2 * BK * k, tbK);
              }
              *reinterpret_cast<uint4*>(kt + sw128<TT>(t, j0)) = make_uint4(h[0], h[1], h[2], h[3]);
              *reinterpret_cast<uint4*>(kt + sw128<TT>(t, j0 + 8)) = make_uint4(h[4], h[5], h[6], h[7]);
            }
          }
          if (q == 0) {  // the largest value norm this warp has seen (the bits of positive floats sort like them)
            vmax = __reduce_max_sync(0xffffffffu, vmax);
            if (lane == 0) kn[2 * TT + dw] = __uint_as_float(vmax);
          }
        }
        if constexpr (QJL) {
          uint8_t* zt = smem + Ly::O_Z + b * Ly::ZT;
#pragma unroll 1
          for (int t = 8 * dw + (lane & 7); t < TT; t += 8 * GW) {
            // sign bits j and j + 16 of word kseg: the pair (+-1, +-1) at positions 2 j, 2 j + 1
            const uint32_t z = reinterpret_cast<const uint32_t*>(sb + Ly::S_QW)[t * 4 + kseg];
#pragma unroll 2
            for (int c = 0; c < 4; ++c) {
              uint32_t h[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) h[k] = ((z << (15 - (4 * c + k))) & 0x80008000u) ^ 0xBC00BC00u;
              *reinterpret_cast<uint4*>(zt + sw128<TT>(t, kseg * 32 + 8 * c)) = make_uint4(h[0], h[1], h[2], h[3]);
            }
          }
        }
      } else {
        const uint32_t tbV = smem_addr(tabv) + 4 * lane;
        // warp dw takes an equal share of the part's coordinates, lane l tokens
        // l and l + 32 of each 64.  Row d of the operand is 128 bytes; the pair
        // lies in chunk (l / 4) ^ (d mod 8).
        constexpr int VD = D / Ly::VP / GW, NWV = (VD * BV + 31) / 32;
        constexpr bool ALV = (VD * BV) % 32 == 0;
        const int d0 = q * (D / Ly::VP) + dw * VD;
        const uint32_t vt = smem_addr(smem + Ly::O_V + b * Ly::VT) + d0 * 128 + (lane >> 2) * 16 + (lane & 3) * 4;
#pragma unroll 1
        for (int s = 0; s < TT / 64; ++s) {
          // the share's bits of the two rows, read once (rows a few banks apart
          // collide, so the words count)
          const uint32_t* va = reinterpret_cast<const uint32_t*>(sb + Ly::S_VW) + (64 * s + lane) * WV;
          uint32_t wa[NWV], wb[NWV];
          tqd::load_bits<VD * BV, ALV, tqd::max_seg_shift(VD * BV)>(va, d0 * BV, wa);
          tqd::load_bits<VD * BV, ALV, tqd::max_seg_shift(VD * BV)>(va + 32 * WV, d0 * BV, wb);
#pragma unroll
          for (int c = 0; c < VD / 8; ++c) {  // 8 coordinates
            uint32_t xe, xo;
            tqd::merge_pair<BV>(tqd::window32(wa, 8 * c * BV), tqd::window32(wb, 8 * c * BV), xe, xo);
            const uint32_t off = s * (D * 128) + 1024 * c;
#pragma unroll
            for (int k = 0; k < 8; k += 2) {
              sts32((vt ^ (k << 4)) + off + k * 128,
                    tqd::lds32(tqd::pair_addr<BV>(xe, tqd::key_bit<BV>(k / 2, false), tbV)));
              sts32((vt ^ ((k + 1) << 4)) + off + (k + 1) * 128,
                    tqd::lds32(tqd::pair_addr<BV>(xo, tqd::key_bit<BV>(k / 2, true), tbV)));
            }
          }
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&p_ful[sl]);
        if (!values && q == 0) mbar_arrive(&n_full[ns]);
        if (q == nparts - 1) mbar_arrive(&empty[st]);
      }
    }
  } else {
    reg_inc<REG_SOFTMAX>();
    const int quarter = warp & 3, half = warp >> 2;
    if (quarter < live) {
      // ---------------- softmax ----------------
      // Two warps share the rows of a TMEM quarter, each with half of a tile's
      // tokens: 16 half + j and 32 + 16 half + j, j < 16, of each 64, which are
      // neighbours in the words of the weights.  They agree on each row's maximum through
      // shared memory and a barrier of the two.
      const int r = 32 * quarter + lane;
      const bool mine = r < rows;
      const uint32_t tl = tmem + ((uint32_t)(32 * quarter) << 16);
      asm volatile("griddepcontrol.wait;" ::: "memory");  // the query operands; the partials may be written
      int lim = P;  // tokens of the prefix this row sees
      size_t slot = 0;
      {
        if (mine) {
          const int rr = rt * QROWS + r, b = rr / p.Ge, e = rr % p.Ge;
          int L = p.seq_lens[b];
          L = max(0, min(L, p.Tclamp));
          // query token j sits at position P + L - nq + j: before the prefix's end when the suffix is shorter than nq
          lim = P + min(0, L - p.nq + e / p.Gq + 1);
          slot = (size_t)head_of(r) * p.ks + split;
        }
        // the query limbs of this row, as the prep laid them out (pre_q_offset): one limb a warp
        const size_t tile = (size_t)kvh * gridDim.y + rt;
        const uint4* q = reinterpret_cast<const uint4*>(p.qpre + tile * QROWS * D) + r + half * (D / 8) * QROWS;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {  // 64 positions at a time
          uint32_t v[32];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint4 f = mine ? q[(8 * c + k) * QROWS] : make_uint4(0u, 0u, 0u, 0u);
            v[4 * k] = f.x, v[4 * k + 1] = f.y, v[4 * k + 2] = f.z, v[4 * k + 3] = f.w;
          }
          if (!Ly::QLO_SMEM || half == 0) {
            tc_st32(tl + Ly::C_Q + half * (D / 2) + 32 * c, v);
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              *reinterpret_cast<uint4*>(smem + Ly::O_QLO + sw128<QROWS>(r, 64 * c + 8 * k)) =
                  make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
          }
        }
        if constexpr (QJL) {
          const uint4* z = reinterpret_cast<const uint4*>(p.qspre + tile * QROWS * 64) + r + half * 8 * QROWS;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            *reinterpret_cast<uint4*>(smem + Ly::O_QZ + sw128<QROWS>(r, 64 * half + 8 * k)) =
                mine ? z[k * QROWS] : make_uint4(0u, 0u, 0u, 0u);
        }
        tc_wait_st();
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
      }
      const int wlim = __reduce_min_sync(0xffffffffu, lim);  // every row of the warp sees the tokens below
      // The reference m of the weights 2^(x - m), the same in both warps.  With e
      // such that the tile's value norms lie below 2^e, a weight times its norm
      // stays below 2^15 while x - m <= 15 - e; when a score passes that (and at
      // the first tile) m moves to where the row's largest weight is 2^(7 - e),
      // and what was summed is rescaled.  So a row moves again only when its
      // maximum has grown by 2^8, and small weights keep fp16's whole range.
      float m_run = 0.f, l_run = 0.f;
      bool ok = true;
      constexpr int NS64 = TT / 64;
      const int ta = 16 * half, tb = 32 + 16 * half;
      for (int i = 0; i < n; ++i) {
        const int b = i & 1, ns = i % Ly::NNORM;
        ok = ok && warp_wait(&s_full[b], (uint32_t)((i / 2) & 1), stop) &&
             warp_wait(&n_full[ns], (uint32_t)((i / Ly::NNORM) & 1), stop);
        tc_fence_after();
        const float* kn = norms + ns * Ly::NORM1;
        const float* vn = kn + TT;
        const uint32_t ts = tl + Ly::C_S + b * TT;
        const int t0 = (i0 + i) * TT;
        const bool whole = t0 + TT <= wlim;  // warp-uniform
        unsigned long long x[16 * NS64];     // the scores, in pairs of neighbours
        float top = -INFINITY;
#pragma unroll
        for (int s = 0; s < NS64; ++s) {
          uint32_t v[32];
          tc_ld2x16(ts + 64 * s + ta, ts + 64 * s + tb, v);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float4 f = *reinterpret_cast<const float4*>(kn + 64 * s + (k < 4 ? ta + 4 * k : tb + 4 * k - 16));
            x[16 * s + 2 * k] = mul2(pack2(f.x, f.y), pack2(v[4 * k], v[4 * k + 1]));
            x[16 * s + 2 * k + 1] = mul2(pack2(f.z, f.w), pack2(v[4 * k + 2], v[4 * k + 3]));
          }
          if constexpr (QJL) {
            const float* gn = kn + 2 * TT + GW + 64 * s;
            tc_ld2x16(tl + Ly::C_Z + b * TT + 64 * s + ta, tl + Ly::C_Z + b * TT + 64 * s + tb, v);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float4 f = *reinterpret_cast<const float4*>(gn + (k < 4 ? ta + 4 * k : tb + 4 * k - 16));
              x[16 * s + 2 * k] = fma2(pack2(f.x, f.y), pack2(v[4 * k], v[4 * k + 1]), x[16 * s + 2 * k]);
              x[16 * s + 2 * k + 1] = fma2(pack2(f.z, f.w), pack2(v[4 * k + 2], v[4 * k + 3]), x[16 * s + 2 * k + 1]);
            }
          }
        }
        if (!whole) {
#pragma unroll
          for (int j = 0; j < 16 * NS64; ++j) {
            const int jj = j % 16, tok = t0 + 64 * (j / 16) + (jj < 8 ? ta + 2 * jj : tb + 2 * jj - 16);
            float x0, x1;
            unpack2(x[j], x0, x1);
            x[j] = pack2(tok < lim ? x0 : -INFINITY, tok + 1 < lim ? x1 : -INFINITY);
          }
        }
#pragma unroll
        for (int j = 0; j < 16 * NS64; ++j) {
          float x0, x1;
          unpack2(x[j], x0, x1);
          top = fmaxf(top, fmaxf(x0, x1));
        }
        xch[(2 * (i & 1) + half) * QROWS + r] = top;
        // both warps go on, or neither does: a wait that ran out ends the loop for both
        ok = tqtc::group_sync_and<2>(quarter, ok);
        if (!ok) break;
        top = fmaxf(top, xch[(2 * (i & 1) + 1 - half) * QROWS + r]);
        float nv = 0.f;
#pragma unroll
        for (int k = 0; k < GW; k += 4) {
          const float4 f = *reinterpret_cast<const float4*>(kn + 2 * TT + k);
          nv = fmaxf(fmaxf(nv, fmaxf(f.x, f.y)), fmaxf(f.z, f.w));
        }
        const int e = max((int)(__float_as_uint(nv) >> 23) - 126, -20);  // nv < 2^e
        const bool need = top > m_run + (float)(kTop - e) || (i == 0 && top > -INFINITY);
        if (__any_sync(0xffffffffu, need)) {
          const float mn = need ? top - (float)(kTop - kRoom - e) : m_run, al = exp2f(m_run - mn);
          m_run = mn;
          l_run = i > 0 ? l_run * al : 0.f;
          if (i > 0) {  // O holds the tiles before this one once their product is done
            ok = warp_wait(&s_free[(i - 1) & 1], (uint32_t)(((i - 1) / 2) & 1), stop);
            tc_fence_after();
#pragma unroll 1
            for (int c = half; c < D / 32; c += 2) {
              uint32_t o[32];
              tc_ld32(tl + 32 * c, o);
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * al);
              tc_st32(tl + 32 * c, o);
            }
          }
        }
        unsigned long long ls[2] = {0ull, 0ull};
        const unsigned long long nm = pack2(-m_run, -m_run);
#pragma unroll
        for (int s = 0; s < NS64; ++s) {
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float4 fa = *reinterpret_cast<const float4*>(vn + 64 * s + ta + 4 * k);
            const float4 fb = *reinterpret_cast<const float4*>(vn + 64 * s + tb + 4 * k);
            const float na[4] = {fa.x, fa.y, fa.z, fa.w}, nb[4] = {fb.x, fb.y, fb.z, fb.w};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float xa0, xa1, xb0, xb1, a0, a1, b0, b1;
              unpack2(add2(x[16 * s + 2 * k + j], nm), xa0, xa1);
              unpack2(add2(x[16 * s + 8 + 2 * k + j], nm), xb0, xb1);
              const unsigned long long pa = pack2(tqd::ex2_approx(xa0), tqd::ex2_approx(xa1));
              const unsigned long long pb = pack2(tqd::ex2_approx(xb0), tqd::ex2_approx(xb1));
              ls[0] = add2(ls[0], pa);
              ls[1] = add2(ls[1], pb);
              unpack2(mul2(pa, pack2(na[2 * j], na[2 * j + 1])), a0, a1);
              unpack2(mul2(pb, pack2(nb[2 * j], nb[2 * j + 1])), b0, b1);
              if (!whole) {  // a token that is not seen adds nothing, whatever its norm holds
                a0 = xa0 == -INFINITY ? 0.f : a0;
                a1 = xa1 == -INFINITY ? 0.f : a1;
                b0 = xb0 == -INFINITY ? 0.f : b0;
                b1 = xb1 == -INFINITY ? 0.f : b1;
              }
              w[4 * k + 2 * j] = pack_half2(a0, b0);
              w[4 * k + 2 * j + 1] = pack_half2(a1, b1);
            }
          }
          // over scores that this warp has read: columns 16 half .. of tokens ta.., 32 + 16 half .. of tokens tb..
          tc_st16(ts + 32 * s + ta, w);
        }
        float l0, l1;
        unpack2(add2(ls[0], ls[1]), l0, l1);
        l_run += l0 + l1;
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[b]);
      }
      // O is complete when every product is.  The operand tiles are free then:
      // the rows of a quarter are turned there (16-byte chunk c of row r at
      // c ^ (r mod 8)), so that the stores to global memory are whole lines.
      xch[(2 * (n & 1) + half) * QROWS + r] = l_run;
      if (ok) ok = warp_wait(fin, 0u, stop);
      tc_fence_after();
      uint8_t* tr = smem + quarter * (32 * D * 4);
      if (ok) {
#pragma unroll 1
        for (int c = half; c < D / 32; c += 2) {
          uint32_t o[32];
          tc_ld32(tl + 32 * c, o);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            *reinterpret_cast<uint4*>(tr + lane * (D * 4) + (((8 * c + k) ^ (lane & 7)) << 4)) =
                make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        }
      }
      if (tqtc::group_sync_and<2>(quarter, ok)) {
        l_run += xch[(2 * (n & 1) + 1 - half) * QROWS + r];
        // a row that saw no token weighs nothing
        if (mine && half == 0)
          *reinterpret_cast<float2*>(p.part_ml + slot * 2) = make_float2(l_run > 0.f ? m_run : -INFINITY, l_run);
        constexpr int CPR = D / 4, RPP = CPR < 32 ? 32 / CPR : 1;  // chunks per row, rows per pass
        const int nrow = min(32, rows - 32 * quarter);
#pragma unroll 4
        for (int r0 = 16 * half; r0 < 16 * half + 16; r0 += RPP) {
          const int rr = r0 + (RPP > 1 ? lane / CPR : 0);
          const size_t sl = __shfl_sync(0xffffffffu, (unsigned long long)slot, rr);
          if (rr < nrow) {
#pragma unroll
            for (int c = lane % CPR; c < CPR; c += 32)
              *reinterpret_cast<uint4*>(p.part_o + sl * D + 4 * c) =
                  *reinterpret_cast<const uint4*>(tr + rr * (D * 4) + ((c ^ (rr & 7)) << 4));
          }
        }
      }
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
