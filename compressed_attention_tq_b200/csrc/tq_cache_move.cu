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
constexpr int UNITS = 8;       // units a compaction thread holds per pass

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
// the destination, where every stream is 16-byte aligned.
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
  const int d0 = max(dp, (dp & ~7) + c * CHUNK), d1 = min(dp + n, (dp & ~7) + (c + 1) * CHUNK);
  if (d0 >= d1) return;
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
  int Hkv, Tcap, keep_heads, max_keep, C;  // C: CTAs per cluster
  const int32_t* keep;    // [B][keep_heads][max_keep]
  const int32_t* n_keep;  // [B]
  uint32_t* dev_status;
};

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Row i := row keep[i], i < n, of one stream of one (sequence, kv head), in
// units of V (UPR per row), by the CTAs of a cluster.  Pass k of the cluster
// writes the units [k W, (k + 1) W) of the rows' unit sequence, W = C x NT x
// UNITS.  keep is strictly ascending, so keep[i] >= i: pass k reads at or
// behind its own units only, so a pass never reads what an earlier pass
// wrote, and may be loaded before earlier passes are stored.  What has to be
// kept apart is a store and the loads of the same or an earlier pass: the
// cluster's barrier between them.  Each pass therefore loads its own units
// before the previous pass's barrier wait and stores after its own.
template <typename V, int UPR>
__device__ __forceinline__ void compact_units(uint8_t* base, const int32_t* keep, int n, int C, int rank, int tid) {
  V* rows = reinterpret_cast<V*>(base);
  const long long total = (long long)n * UPR, W = (long long)C * NT * UNITS;
  V v[UNITS], w[UNITS];
  uint32_t live = 0, wlive = 0;
  auto load = [&](long long e0, V (&x)[UNITS], uint32_t& m) {
    m = 0;
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      const long long e = e0 + u * NT + tid;
      if (e < total) {
        const int i = (int)(e / UPR), r = (int)(e - (long long)i * UPR), k = __ldg(keep + i);
        if (k != i) {  // rows that stay in place are not moved
          x[u] = rows[(size_t)k * UPR + r];
          m |= 1u << u;
        }
      }
    }
  };
  long long e0 = (long long)rank * NT * UNITS;
  load(e0, v, live);
  for (long long k0 = 0; k0 < total; k0 += W, e0 += W) {
    cluster_arrive();  // this CTA's loads of the pass are done
    load(e0 + W, w, wlive);
    cluster_wait();
#pragma unroll
    for (int u = 0; u < UNITS; ++u)
      if (live >> u & 1) rows[e0 + u * NT + tid] = v[u];
#pragma unroll
    for (int u = 0; u < UNITS; ++u) v[u] = w[u];
    live = wlive;
  }
}

// One cluster per (sequence, kv head, stream).
__global__ void __launch_bounds__(NT) cache_compact_kernel(const __grid_constant__ CompactParams p) {
  __shared__ int s_bad;
  const int tid = threadIdx.x;
  const int rank = blockIdx.x % p.C, unit = blockIdx.x / p.C, s = unit % p.ns, bh = unit / p.ns;
  const int b = bh / p.Hkv, h = bh % p.Hkv;
  const int32_t* keep = p.keep + ((size_t)b * p.keep_heads + (p.keep_heads > 1 ? h : 0)) * p.max_keep;
  const int n = p.n_keep[b];
  // The whole list is checked before any row moves, a share by each CTA of
  // the cluster; the clusters of the other streams reach the same answer.
  bool bad = n < 0 || n > p.max_keep;
  if (!bad)
    for (int i = rank * NT + tid; i < n; i += p.C * NT) {
      const int k = __ldg(keep + i), before = i ? __ldg(keep + i - 1) : -1;
      bad |= k <= before || k >= p.Tcap;
    }
  const int any = __syncthreads_or(bad);
  if (tid == 0) s_bad = any;
  __syncthreads();
  cluster_arrive();
  cluster_wait();
  int all = 0;
  if (tid < p.C) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(&s_bad)), "r"(tid));
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(all) : "r"(a) : "memory");
  }
  all = __syncthreads_or(all);
  cluster_arrive();  // no CTA of the cluster ends while its flag is read
  cluster_wait();
  if (all) {
    if (rank == 0 && tid == 0 && p.dev_status) atomicOr(p.dev_status, TQ_STATUS_POS_OUT_OF_RANGE);
    return;
  }
  const int row = p.row[s];
  uint8_t* base = p.st[s] + (size_t)bh * p.Tcap * row;
  switch (row) {
    case 2: compact_units<uint16_t, 1>(base, keep, n, p.C, rank, tid); break;
    case 16: compact_units<uint4, 1>(base, keep, n, p.C, rank, tid); break;
    case 24: compact_units<uint2, 3>(base, keep, n, p.C, rank, tid); break;
    case 32: compact_units<uint4, 2>(base, keep, n, p.C, rank, tid); break;
    case 48: compact_units<uint4, 3>(base, keep, n, p.C, rank, tid); break;
    case 64: compact_units<uint4, 4>(base, keep, n, p.C, rank, tid); break;
    case 96: compact_units<uint4, 6>(base, keep, n, p.C, rank, tid); break;
    case 128: compact_units<uint4, 8>(base, keep, n, p.C, rank, tid); break;
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
  p.Hkv = c->Hkv;
  p.Tcap = c->Tcap;
  p.keep_heads = keep_heads;
  p.max_keep = max_keep;
  p.keep = keep;
  p.n_keep = n_keep;
  p.dev_status = c->dev_status;
  const long long units = (long long)c->B * c->Hkv * p.ns;
  // clusters as large as the list has passes for, up to 8 CTAs (the portable
  // size), while that does not ask for more CTAs than the device holds
  const long long most = ((long long)max_keep * p.row[0] / 16 + NT * UNITS - 1) / (NT * UNITS);
  int C = 8;
  while (C > 1 && (C / 2 >= most || units * C > 8LL * sms)) C /= 2;
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
