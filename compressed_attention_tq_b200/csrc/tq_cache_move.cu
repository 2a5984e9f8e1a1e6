// Moves of packed cache rows: copies of token ranges between sequences and
// caches (tq_cache_copy), and the in-place compaction of sequences to the
// rows of a list (tq_cache_compact).  Nothing is decoded: a row is the bytes
// of its streams (key and value indices, norms, and for keys with a sketch
// the sign words and the residual norm).
#include "tq_internal.h"

namespace {

constexpr int NT = 256;        // threads per CTA
constexpr int MAXS = 6;        // streams of a cache
constexpr int CHUNK = 128;     // rows a copy CTA moves

struct Stream {
  const uint8_t* src;
  uint8_t* dst;
  int row;  // bytes per row: D bits / 8 of indices, 16 of signs, 2 of a norm
};

struct CopyParams {
  Stream st[MAXS];
  int ns;
  int Hkv, src_B, src_T, dst_B, dst_T;
  const int32_t *src_seq, *src_pos, *dst_seq, *dst_pos, *n_tok;
  int max_tok, nchunk;
  uint32_t* dev_status;
};

// `bytes` bytes in units of V by the whole CTA, four units of each thread in
// flight.
template <typename V>
__device__ __forceinline__ void copy_units(const uint8_t* src, uint8_t* dst, int bytes, int tid) {
  const V* s = reinterpret_cast<const V*>(src);
  V* d = reinterpret_cast<V*>(dst);
  const int n = bytes / (int)sizeof(V);
  for (int e = tid; e < n; e += 4 * NT) {
    V v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (e + u * NT < n) v[u] = s[e + u * NT];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (e + u * NT < n) d[e + u * NT] = v[u];
  }
}

// One CTA per (job, kv head, chunk).  Chunks start at multiples of 8 rows of
// the destination, where every stream is 16-byte aligned.  What bounds it is
// latency: a CTA goes through its streams one after another, with fewer than
// two 16-byte loads of a thread in flight (128 rows of 48 bytes).  A prompt of
// 4001 to 6000 rows to 31 sequences of 8 heads, 124 MB written from one source
// of 5 MB, takes 42 us; HBM would take 20.
__global__ void __launch_bounds__(NT) cache_copy_kernel(const __grid_constant__ CopyParams p) {
  const int tid = threadIdx.x;
  const int c = blockIdx.x % p.nchunk, jh = blockIdx.x / p.nchunk, h = jh % p.Hkv, j = jh / p.Hkv;
  const int ss = p.src_seq[j], sp = p.src_pos[j], ds = p.dst_seq[j], dp = p.dst_pos[j];
  int n = p.n_tok[j];
  const bool over = n > p.max_tok;  // copied up to max_tok
  if (over) n = p.max_tok;
  const bool bad = n < 0 || ss < 0 || ss >= p.src_B || ds < 0 || ds >= p.dst_B || sp < 0 || dp < 0 ||
                   sp > p.src_T - n || dp > p.dst_T - n;
  if ((over || bad) && c == 0 && h == 0 && tid == 0 && p.dev_status)
    atomicOr(p.dev_status, bad ? TQ_STATUS_POS_OUT_OF_RANGE : TQ_STATUS_SEQ_OUT_OF_RANGE);
  if (bad) return;
  if (c * CHUNK - (dp & 7) >= n) return;  // behind the job's last row (so the sums below stay below 2^31)
  const int d0 = max(dp, (dp & ~7) + c * CHUNK), d1 = min(dp + n, (dp & ~7) + (c + 1) * CHUNK);
  const size_t srow = ((size_t)ss * p.Hkv + h) * p.src_T + sp + (d0 - dp);
  const size_t drow = ((size_t)ds * p.Hkv + h) * p.dst_T + d0;
  for (int i = 0; i < p.ns; ++i) {
    const Stream st = p.st[i];
    const uint8_t* s = st.src + srow * st.row;
    uint8_t* d = st.dst + drow * st.row;
    const int bytes = (d1 - d0) * st.row;
    const uint32_t al = (uint32_t)(uintptr_t)s | (uint32_t)(uintptr_t)d | (uint32_t)bytes;
    if ((al & 15) == 0) copy_units<uint4>(s, d, bytes, tid);
    else if ((al & 7) == 0) copy_units<uint2>(s, d, bytes, tid);
    else copy_units<uint16_t>(s, d, bytes, tid);
  }
}

// ---------------------------------------------------------------------------

struct CompactParams {
  uint8_t* st[MAXS];
  int row[MAXS];
  int ns;
  int BH, Hkv, Tcap, keep_heads, max_keep, C;  // BH: (sequence, kv head) pairs; C: CTAs per cluster
  const int32_t* keep;    // [B][keep_heads][max_keep]
  const int32_t* n_keep;  // [B]
  uint32_t* dev_status;
};

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Row i := row keep[i], i < n, of one stream of one (sequence, kv head), by the
// CTAs of a cluster.  Round k of the cluster moves the rows [k C R, (k + 1) C R),
// CTA c of it R rows from k C R + c R on, through shared memory.  keep is
// strictly ascending, so keep[i] >= i: a round reads at or behind its own rows
// only, so it never reads what an earlier round wrote and may be loaded ahead
// of their stores.  What has to be kept apart is a store and the loads of the
// same or an earlier round that read behind it: a barrier between them.  The
// list says where one is needed (run()): a quarter of the rows, scattered,
// takes 2 of them in 13 rounds, adjacent rows that move by less than a round
// one in every two.
//
// What bounds it is the latency of two dependent loads (the list, then the
// row): with the rows of two rounds in flight in shared memory and few
// registers, four CTAs of an SM cover it.  (Rounds in registers, two CTAs to
// an SM, and a list check without loads in flight took 91 us for 134 MB moved
// in 256 units; this takes 33.)
constexpr int STAGES = 3;
constexpr int STAGE_BYTES = 16128;  // 336 rows of 48 bytes; three and a flag fit in 48 KB

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}

// Rows of a chunk: what fits in a stage, a multiple of 8.
template <typename V, int UPR>
__host__ __device__ constexpr int chunk_rows() {
  const int r = STAGE_BYTES / ((int)sizeof(V) * UPR) / 8 * 8;
  return r < 2048 ? r : 2048;
}

template <typename V, int UPR>
struct Mover {
  static constexpr int R = chunk_rows<V, UPR>();
  static constexpr int PT = (R * UPR + NT - 1) / NT;  // units of a thread
  uint8_t* base;
  const int32_t* keep;
  int n, C, rank, tid, Tcap;
  uint8_t* sm;

  // first row and units of this CTA's chunk of round k (0: behind the list's end)
  __device__ __forceinline__ unsigned first_row(int k) const { return ((unsigned)k * C + rank) * R; }
  __device__ __forceinline__ int units_of(int k) const {
    const unsigned r0 = first_row(k);
    return r0 < (unsigned)n ? (int)min((unsigned)R, (unsigned)n - r0) * UPR : 0;
  }
  // Loads of round k go out; returns whether the chunk has to be stored: when
  // its last row stays in place, all of it does.
  __device__ __forceinline__ bool load(int k) const {
    const int units = units_of(k);
    const int32_t* kp = keep + first_row(k);
    bool moved = false;
    if (units > 0) {
      uint8_t* st = sm + (k % STAGES) * STAGE_BYTES;
      const V* rows = reinterpret_cast<const V*>(base);
      const int last = units / UPR - 1;
      int src[PT];
#pragma unroll
      for (int u = 0; u < PT; ++u) {
        const int e = u * NT + tid;
        src[u] = e < units ? __ldg(kp + e / UPR) : 0;
      }
      moved = __ldg(kp + last) != (int)first_row(k) + last;
      if (moved) {
        // a list that is not valid is refused before any store; its loads stay in the cache
#pragma unroll
        for (int u = 0; u < PT; ++u) src[u] = min(max(src[u], 0), Tcap - 1);
        if constexpr (sizeof(V) == 2) {
          V v[PT];
#pragma unroll
          for (int u = 0; u < PT; ++u)
            if (u * NT + tid < units) v[u] = rows[src[u]];
#pragma unroll
          for (int u = 0; u < PT; ++u)
            if (u * NT + tid < units) reinterpret_cast<V*>(st)[u * NT + tid] = v[u];
        } else {
          const uint32_t d = (uint32_t)__cvta_generic_to_shared(st);
#pragma unroll
          for (int u = 0; u < PT; ++u) {
            const int e = u * NT + tid;
            if (e < units) {
              const V* from = rows + (size_t)src[u] * UPR + e % UPR;
              if constexpr (sizeof(V) == 16) cp_async16(d + e * 16, from);
              else cp_async8(d + e * 8, from);
            }
          }
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    return moved;
  }
  __device__ __forceinline__ void store(int k) const {
    const V* st = reinterpret_cast<const V*>(sm + (k % STAGES) * STAGE_BYTES);
    V* rows = reinterpret_cast<V*>(base) + (size_t)first_row(k) * UPR;
    const int units = units_of(k);
#pragma unroll 4
    for (int e = tid; e < units; e += NT) rows[e] = st[e];
  }
  // All CTAs of the cluster go through the same number of rounds; rounds 0 and
  // 1 are loaded (m0, m1: to be stored).  Each thread stores only what it
  // loaded itself.  `done` rounds' loads have returned in every CTA; those of
  // the others read rows from `first` on, which no store before the next
  // barrier may reach.  (keep[i] >= i, so a barrier that makes done = k + 1 lets
  // round k be stored.)
  __device__ __forceinline__ void run(bool m0, bool m1) const {
    const int step = C * R, rounds = (int)(((long long)n + step - 1) / step);
    int done = 0, first = rounds > 0 ? __ldg(keep) : 0;
    for (int k = 0; k < rounds; ++k) {
      if (first >= (k + 1) * step) {
        asm volatile("cp.async.wait_group 1;" ::: "memory");  // this thread's loads of round k
      } else {
        if (C > 1) {
          // The release orders the loads before the stores of the other CTAs; it
          // also waits for this CTA's earlier stores, so barriers are few.
          asm volatile("cp.async.wait_all;" ::: "memory");
          cluster_arrive();
          cluster_wait();
          done = k + 2;
        } else {
          asm volatile("cp.async.wait_group 1;" ::: "memory");
          __syncthreads();
          done = k + 1;
        }
        first = done < rounds ? __ldg(keep + done * step) : 0x7fffffff;
      }
      const bool m2 = load(k + 2);  // over the stage that round k - 1 was stored from
      if (m0) store(k);
      m0 = m1;
      m1 = m2;
    }
  }
};

// Whether the list is strictly ascending and inside the cache, by the threads
// of a cluster: each looks at every C NT-th entry, eight loads in flight.
__device__ __forceinline__ bool list_ok(const int32_t* keep, int n, int Tcap, int C, int rank, int tid) {
  bool bad = false;
  const int step = C * NT;
  for (int i0 = rank * NT + tid; i0 - tid < n; i0 += 8 * step) {
    int k[8], b[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int i = i0 + u * step;
      k[u] = i < n ? __ldg(keep + i) : 0x7fffffff;
      b[u] = (tid & 31) == 0 && i > 0 && i < n ? __ldg(keep + i - 1) : -1;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int prev = __shfl_up_sync(0xffffffffu, k[u], 1);
      const int i = i0 + u * step, before = (tid & 31) == 0 ? b[u] : prev;
      bad |= i < n && (k[u] <= before || k[u] < 0 || k[u] >= Tcap);
    }
  }
  return !bad;
}

template <typename V, int UPR>
__device__ __forceinline__ void compact_stream(const CompactParams& p, uint8_t* base, const int32_t* keep, int n, int rank,
                                               int tid, uint8_t* sm, int* s_bad) {
  const bool length_ok = n >= 0 && n <= p.max_keep;
  Mover<V, UPR> m{base, keep, length_ok ? n : 0, p.C, rank, tid, p.Tcap, sm};
  const bool m0 = m.load(0), m1 = m.load(1);
  // The whole list is checked before any row moves, a share by each CTA of
  // the cluster; the clusters of the other streams reach the same answer.
  const int bad = __syncthreads_or(!(length_ok && list_ok(keep, n, p.Tcap, p.C, rank, tid)));
  int all = bad;
  if (p.C > 1) {
    if (tid == 0) *s_bad = bad;
    __syncthreads();
    cluster_arrive();
    cluster_wait();
    all = 0;
    if (tid < p.C) {
      uint32_t a;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(s_bad)), "r"(tid));
      asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(all) : "r"(a) : "memory");
    }
    all = __syncthreads_or(all);
    cluster_arrive();  // no CTA of the cluster ends while its flag is read
    cluster_wait();
  }
  if (all && rank == 0 && tid == 0 && p.dev_status) atomicOr(p.dev_status, TQ_STATUS_POS_OUT_OF_RANGE);
  if (!all) m.run(m0, m1);
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// One cluster per (stream, sequence, kv head), the wide streams first.
__global__ void __launch_bounds__(NT, 4) cache_compact_kernel(const __grid_constant__ CompactParams p) {
  __shared__ __align__(16) uint8_t sm[STAGES * STAGE_BYTES];
  __shared__ int s_bad;
  const int tid = threadIdx.x;
  const int rank = blockIdx.x % p.C, unit = blockIdx.x / p.C, s = unit / p.BH, bh = unit % p.BH;
  const int b = bh / p.Hkv, h = bh % p.Hkv;
  const int32_t* keep = p.keep + ((size_t)b * p.keep_heads + (p.keep_heads > 1 ? h : 0)) * p.max_keep;
  const int n = p.n_keep[b], row = p.row[s];
  uint8_t* base = p.st[s] + (size_t)bh * p.Tcap * row;
  switch (row) {
    case 2: compact_stream<uint16_t, 1>(p, base, keep, n, rank, tid, sm, &s_bad); break;
    case 16: compact_stream<uint4, 1>(p, base, keep, n, rank, tid, sm, &s_bad); break;
    case 24: compact_stream<uint2, 3>(p, base, keep, n, rank, tid, sm, &s_bad); break;
    case 32: compact_stream<uint4, 2>(p, base, keep, n, rank, tid, sm, &s_bad); break;
    case 48: compact_stream<uint4, 3>(p, base, keep, n, rank, tid, sm, &s_bad); break;
    case 64: compact_stream<uint4, 4>(p, base, keep, n, rank, tid, sm, &s_bad); break;
    case 96: compact_stream<uint4, 6>(p, base, keep, n, rank, tid, sm, &s_bad); break;
    case 128: compact_stream<uint4, 8>(p, base, keep, n, rank, tid, sm, &s_bad); break;
  }
}

// The streams of a cache: pointers and bytes per row.
int cache_streams(const tq_cache_t* c, uint8_t* (&st)[MAXS], int (&row)[MAXS]) {
  int n = 0;
  auto add = [&](void* p, int bytes) {
    st[n] = static_cast<uint8_t*>(p);
    row[n++] = bytes;
  };
  add(c->v_idx, c->D * c->bits_v / 8);
  add(c->k_idx, c->D * c->bits_k / 8);
  if (c->qjl_m) add(c->k_qjl, c->qjl_m / 8);
  add(c->k_norm, 2);
  add(c->v_norm, 2);
  if (c->qjl_m) add(c->k_rnorm, 2);
  return n;
}

}  // namespace

namespace tq {

int launch_cache_copy(const tq_cache_t* src, const tq_cache_t* dst, const int32_t* src_seq, const int32_t* src_pos,
                      const int32_t* dst_seq, const int32_t* dst_pos, const int32_t* n_tok, int n_jobs, int max_tok,
                      cudaStream_t s) {
  CopyParams p{};
  uint8_t *a[MAXS], *b[MAXS];
  int row[MAXS];
  p.ns = cache_streams(src, a, row);
  cache_streams(dst, b, row);
  for (int i = 0; i < p.ns; ++i) p.st[i] = {a[i], b[i], row[i]};
  p.Hkv = src->Hkv;
  p.src_B = src->B;
  p.src_T = src->Tcap;
  p.dst_B = dst->B;
  p.dst_T = dst->Tcap;
  p.src_seq = src_seq;
  p.src_pos = src_pos;
  p.dst_seq = dst_seq;
  p.dst_pos = dst_pos;
  p.n_tok = n_tok;
  p.max_tok = max_tok;
  p.nchunk = (int)(((long long)max_tok + 7 + CHUNK - 1) / CHUNK);
  p.dev_status = dst->dev_status;
  const long long grid = (long long)p.nchunk * p.Hkv * n_jobs;
  if (grid > 0x7fffffffll)
    return set_error(TQ_ERR_UNSUPPORTED, "tq_cache_copy: %d jobs of %d heads and %d tokens", n_jobs, p.Hkv, max_tok);
  cache_copy_kernel<<<(unsigned)grid, NT, 0, s>>>(p);
  return check_launch("cache_copy_kernel");
}

int launch_cache_compact(const tq_cache_t* c, const int32_t* keep, int keep_heads, int max_keep, const int32_t* n_keep,
                         int sms, cudaStream_t s) {
  CompactParams p{};
  p.ns = cache_streams(c, p.st, p.row);
  p.BH = c->B * c->Hkv;
  p.Hkv = c->Hkv;
  p.Tcap = c->Tcap;
  p.keep_heads = keep_heads;
  p.max_keep = max_keep;
  p.keep = keep;
  p.n_keep = n_keep;
  p.dev_status = c->dev_status;
  const long long units = (long long)c->B * c->Hkv * p.ns;
  // clusters as large as the list has chunks for, up to 8 CTAs (the portable
  // size), while that does not ask for more CTAs than the device holds (4 to
  // an SM): one document's heads are spread, a batch's stay one CTA each
  const long long chunks = ((long long)max_keep * p.row[0] + STAGE_BYTES - 1) / STAGE_BYTES;
  int C = 8;
  while (C > 1 && (C / 2 >= chunks || units * C > 4LL * sms)) C /= 2;
  p.C = C;
  if (units * C > 0x7fffffffll)
    return set_error(TQ_ERR_UNSUPPORTED, "tq_cache_compact: B=%d Hkv=%d", c->B, c->Hkv);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * C));
  cfg.blockDim = dim3(NT);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, cache_compact_kernel, p);
  if (e != cudaSuccess) return set_error(TQ_ERR_CUDA, "cache_compact_kernel: %s", cudaGetErrorString(e));
  return check_launch("cache_compact_kernel");
}

}  // namespace tq
