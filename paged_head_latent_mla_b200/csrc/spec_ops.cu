// The operators around a speculative step's attention: verification of the drafted trees,
// the move of the accepted nodes' latent rows, and page copies.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "mla_launch.h"
#include "sm100_ptx.cuh"

namespace mla {

namespace {

// ------------------------------------------------------------------ verification
// Row b's tree is walked from node 0 (include/mla.h, mla_verify_tree).  The tests along
// the walk need single weights only: p and q at each child's token.  Whole rows of V
// weights are read where a sum over the vocabulary is needed: after a rejected child that
// has a next sibling (Z = sum of max(w - Z q, 0)), and once at the end, where the next
// token is found in the running sum of w.
//
// One cluster of C blocks works on a row.  Block 0 gathers the tree's single weights (all
// nodes at once), walks it, and publishes a command for every pass over a row of weights;
// the other blocks only follow commands, so that the cluster's barriers match whatever the
// inputs hold.  In a pass block r sums its C-th of the vocabulary, each warp a contiguous
// segment of that, and the warps' sums go to block 0's shared memory.  Block 0 finds the
// segment in which the running sum crosses the target and reads that segment again.
//
// Weights are held in 64 bits from the first subtraction on: acceptance and the next token
// are decided at borders, and a sum rounded to 32 bits over a large vocabulary would move
// a border by more than a token's weight.  Every sum has one fixed order.
constexpr int kVThreads = 512;
constexpr int kVWarps = kVThreads / 32;
constexpr int kVMaxCluster = 8;
constexpr int kVMaxNodes = MLA_TREE_MAX_NODES;

enum : int32_t { kCmdSum = 0, kCmdExit = 1 };

struct VerifyShared {
  // block 0: the tree
  int32_t tok[kVMaxNodes];
  float u[kVMaxNodes], p[kVMaxNodes], q[kVMaxNodes];  // p, q: weights of tok at the parent
  int32_t first[kVMaxNodes], next[kVMaxNodes];
  // every block: the command (written by block 0) and the rejections at its node
  int32_t cmd, cmd_token, cmd_rejected;
  double z[kVMaxNodes];        // draft: Z of each rejection
  int32_t zero[kVMaxNodes];    // point masses: the rejected tokens
  // block 0: warps' segment sums of the pass
  double seg[kVMaxCluster * kVWarps];
  // block 0: search of the crossing
  double warp_sum[kVWarps];
  int32_t warp_first[kVWarps], warp_last[kVWarps];
};

template <typename T>
__device__ __forceinline__ float to_float(T x);
template <>
__device__ __forceinline__ float to_float<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 x) {
  return __bfloat162float(x);
}

// Negative, infinite and NaN weights count as 0.
__device__ __forceinline__ float weight(float x) {
  return (x > 0.f && x < __int_as_float(0x7f800000)) ? x : 0.f;
}

// kVec consecutive weights of a row, chunk c of it: elements [c * kVec - head, + kVec) of
// which those in [0, V) exist (the others are 0).  `head` makes every whole chunk start on
// a 16-byte boundary.
template <typename T, int kVec>
__device__ __forceinline__ void load_chunk(const T* row, int head, int c, int V, float (&w)[kVec]) {
  const int e0 = c * kVec - head;
  if (kVec > 1 && e0 >= 0 && e0 + kVec <= V) {
    const uint4 raw = __ldg(reinterpret_cast<const uint4*>(row + e0));
    const uint32_t r[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      if (sizeof(T) == 4)
        w[i] = weight(__uint_as_float(r[i & 3]));
      else
        w[i] = weight(__uint_as_float((i & 1) ? (r[(i >> 1) & 3] & 0xffff0000u) : (r[(i >> 1) & 3] << 16)));
    }
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i) w[i] = (e0 + i >= 0 && e0 + i < V) ? weight(to_float(row[e0 + i])) : 0.f;
  }
}

// What the rejections at a node leave of a weight.
__device__ __forceinline__ double left_of(float p, float q, const double* z, int n) {
  double w = static_cast<double>(p);
  if (n > 0) {
    const double dq = static_cast<double>(q);
    w = fmax(w - dq, 0.0);  // the first Z is 1
    for (int k = 1; k < n; ++k) w = fmax(__dadd_rn(w, -__dmul_rn(z[k], dq)), 0.0);
  }
  return w;
}

template <typename T, int kVec, bool kDraft>
struct RowPass {
  const T* p;
  const T* q;
  int head, V, chunks;        // chunks of the row
  int per_block, per_warp;    // chunks of a block and of a warp's segment
  const double* z;
  const int32_t* zero;
  int rejected;

  __device__ RowPass(const VerifyParams& a, int64_t token, int nrej, const VerifyShared& s, int cluster) {
    p = static_cast<const T*>(a.target) + token * a.ld_target;
    q = kDraft ? static_cast<const T*>(a.draft) + token * a.ld_draft : nullptr;
    V = a.vocab;
    head = kVec > 1 ? static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T)) : 0;
    chunks = static_cast<int>((static_cast<int64_t>(V) + head + kVec - 1) / kVec);
    per_block = (chunks + cluster - 1) / cluster;
    per_warp = (per_block + kVWarps - 1) / kVWarps;
    z = s.z;
    zero = s.zero;
    rejected = nrej;
  }
  // chunks [lo, hi) of warp `w` of block `r`
  __device__ void segment(int r, int w, int* lo, int* hi) const {
    const int b1 = min(chunks, (r + 1) * per_block);
    *lo = min(b1, r * per_block + w * per_warp);
    *hi = min(b1, *lo + per_warp);
  }
  __device__ __forceinline__ void weights(const float (&fp)[kVec], const float (&fq)[kVec], int c,
                                          double (&w)[kVec]) const {
#pragma unroll
    for (int i = 0; i < kVec; ++i) w[i] = kDraft ? left_of(fp[i], fq[i], z, rejected) : static_cast<double>(fp[i]);
    if (!kDraft) {
      const int e0 = c * kVec - head;
      for (int k = 0; k < rejected; ++k) {
        const int at = zero[k] - e0;
#pragma unroll
        for (int i = 0; i < kVec; ++i)
          if (at == i) w[i] = 0.0;
      }
    }
  }
  // Sum over chunks lo + lane, lo + lane + 32, ...: kBatch chunks' loads in flight.
  __device__ __forceinline__ double sum(int lo, int hi, int lane) const {
    constexpr int kBatch = kVec > 1 ? 4 : 8;
    double acc[kVec > 1 ? 4 : 1] = {};
    for (int c0 = lo + lane; c0 < hi; c0 += 32 * kBatch) {
      float fp[kBatch][kVec], fq[kBatch][kVec];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int c = c0 + 32 * k;
        if (c < hi) {
          load_chunk<T, kVec>(p, head, c, V, fp[k]);
          if (kDraft) load_chunk<T, kVec>(q, head, c, V, fq[k]);
        } else {
#pragma unroll
          for (int i = 0; i < kVec; ++i) fp[k][i] = fq[k][i] = 0.f;
        }
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        double w[kVec];
        weights(fp[k], fq[k], c0 + 32 * k, w);
#pragma unroll
        for (int i = 0; i < kVec; ++i) acc[kVec > 1 ? i & 3 : 0] += w[i];
      }
    }
    double t = acc[0];
    if (kVec > 1) t = (acc[0] + acc[1 % (kVec > 1 ? 4 : 1)]) + (acc[2 % (kVec > 1 ? 4 : 1)] + acc[3 % (kVec > 1 ? 4 : 1)]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
    return t;
  }
};

__device__ __forceinline__ void st_cluster_f64(uint32_t addr, double v) {
  asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(addr), "d"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ void cluster_sync() {
  ptx::cluster_arrive();
  ptx::cluster_wait();
}

__device__ __forceinline__ double warp_scan(double x, int lane) {
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const double y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  return x;
}

template <typename T, int kVec, bool kDraft>
__global__ void __launch_bounds__(kVThreads, 2) mla_verify_kernel(const VerifyParams a) {
  extern __shared__ uint8_t verify_smem[];
  VerifyShared& s = *reinterpret_cast<VerifyShared*>(verify_smem);
  uint32_t C;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(C));
  const int rank = static_cast<int>(ptx::cluster_ctarank());
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.x / C;
  const TreeRow row = a.rows[b];
  const int n = row.n_nodes;
  if (n < 0) return;  // an unused row of a graph plan: the whole cluster leaves
  if (n == 0 || n > kVMaxNodes) {
    if (rank == 0) {
      if (tid == 0) {
        a.num_accepted[b] = 0;
        a.next_token[b] = -1;
      }
      for (int i = tid; i < n; i += kVThreads) a.accept_index[row.token0 + i] = -1;
    }
    return;
  }
  const int64_t t0 = row.token0;
  ptx::cluster_arrive();  // a block's shared memory may be written once it is known to run

  // One pass over the row of weights of node `node` by the whole cluster (block 0 calls it
  // with the command published): the warps' sums land in block 0's s.seg.
  auto pass = [&](int64_t token, int rejected) {
    const RowPass<T, kVec, kDraft> rp(a, token, rejected, s, C);
    int lo, hi;
    rp.segment(rank, warp, &lo, &hi);
    const double t = rp.sum(lo, hi, lane);
    if (lane == 0) st_cluster_f64(ptx::map_to_cta(ptx::smem_addr(&s.seg[rank * kVWarps + warp]), 0), t);
    __syncwarp();
    cluster_sync();
  };

  if (rank != 0) {
    ptx::cluster_wait();
    while (true) {
      cluster_sync();  // the command is there
      if (s.cmd == kCmdExit) return;
      pass(t0 + s.cmd_token, s.cmd_rejected);
    }
  }

  // ---------------------------------------------------------------- block 0
  for (int i = tid; i < n; i += kVThreads) {
    const TreeNode nd = a.nodes[t0 + i];
    const int x = i > 0 ? a.draft_tokens[t0 + i] : -1;
    s.tok[i] = x;
    s.u[i] = a.uniform[t0 + i];
    s.first[i] = nd.first_child;
    s.next[i] = nd.next_sibling;
    float p = 0.f, q = 0.f;
    if (nd.parent >= 0 && x >= 0 && x < a.vocab) {
      p = weight(to_float(static_cast<const T*>(a.target)[(t0 + nd.parent) * a.ld_target + x]));
      if (kDraft) q = weight(to_float(static_cast<const T*>(a.draft)[(t0 + nd.parent) * a.ld_draft + x]));
    }
    s.p[i] = p;
    s.q[i] = q;
    a.accept_index[t0 + i] = i == 0 ? 0 : -1;
  }
  __syncthreads();
  ptx::cluster_wait();

  // Publish a pass and run it; afterwards every thread may read s.seg.  The rejections
  // (s.z or s.zero) are copied to the other blocks with the command.
  auto run_pass = [&](int node, int rejected) {
    __syncthreads();
    for (uint32_t r = 1 + warp; r < C; r += kVWarps) {
      for (int k = lane; k < rejected; k += 32) {
        if (kDraft)
          st_cluster_f64(ptx::map_to_cta(ptx::smem_addr(&s.z[k]), r), s.z[k]);
        else
          st_cluster_u32(ptx::map_to_cta(ptx::smem_addr(&s.zero[k]), r), static_cast<uint32_t>(s.zero[k]));
      }
      if (lane == 0) {
        st_cluster_u32(ptx::map_to_cta(ptx::smem_addr(&s.cmd), r), kCmdSum);
        st_cluster_u32(ptx::map_to_cta(ptx::smem_addr(&s.cmd_token), r), static_cast<uint32_t>(node));
        st_cluster_u32(ptx::map_to_cta(ptx::smem_addr(&s.cmd_rejected), r), static_cast<uint32_t>(rejected));
      }
    }
    __syncwarp();
    cluster_sync();
    pass(t0 + node, rejected);
  };
  const int segs = static_cast<int>(C) * kVWarps;
  // Inclusive running sum at segment i of this lane's share (lane l owns segments [l * per,
  // (l + 1) * per)); the same in every warp.
  const int per = (segs + 31) / 32;
  auto total = [&]() -> double {
    double t = 0.0;
    for (int i = 0; i < per; ++i)
      if (lane * per + i < segs) t += s.seg[lane * per + i];
    return __shfl_sync(0xffffffffu, warp_scan(t, lane), 31);
  };

  int v = 0, kept = 1, rejected = 0;
  while (true) {
    // every thread walks alike over the same shared values
    int c = s.first[v], got = -1;
    double Z = 1.0;
    rejected = 0;
    for (; c >= 0; c = s.next[c]) {
      const int x = s.tok[c];
      if (x < 0) {  // given
        got = c;
        break;
      }
      double w;
      if (kDraft) {
        w = left_of(s.p[c], s.q[c], s.z, rejected);
      } else {
        w = s.p[c];
        for (int k = 0; k < rejected; ++k)
          if (s.zero[k] == x) w = 0.0;
      }
      const double u = s.u[c];
      const double limit = kDraft ? __dmul_rn(__dmul_rn(u, static_cast<double>(s.q[c])), Z) : __dmul_rn(u, Z);
      if (limit < w) {
        got = c;
        break;
      }
      __syncthreads();  // all have read the list
      if (kDraft) {
        if (tid == 0) s.z[rejected] = Z;
        ++rejected;
        if (s.next[c] >= 0) {
          run_pass(v, rejected);
          Z = total();
        } else {
          __syncthreads();
        }
      } else {
        if (tid == 0) s.zero[rejected] = x;
        ++rejected;
        Z = fmax(Z - w, 0.0);
        __syncthreads();
      }
    }
    if (got < 0) break;
    v = got;
    if (tid == 0) a.accept_index[t0 + kept] = v;
    ++kept;
  }

  run_pass(v, rejected);
  double W = total();
  if (!(W > 0.0) && rejected > 0) {
    rejected = 0;
    run_pass(v, 0);
    W = total();
  }
  // dismiss the other blocks
  for (uint32_t r = 1 + warp; r < C; r += kVWarps)
    if (lane == 0) st_cluster_u32(ptx::map_to_cta(ptx::smem_addr(&s.cmd), r), kCmdExit);
  __syncwarp();
  ptx::cluster_arrive();

  int token = -1;
  if (W > 0.0) {
    const double target = __dmul_rn(static_cast<double>(a.uniform_next[b]), W);
    // the first segment whose inclusive running sum exceeds the target, else the last one
    // that holds any weight
    double mine = 0.0;
    for (int i = 0; i < per; ++i)
      if (lane * per + i < segs) mine += s.seg[lane * per + i];
    double run = warp_scan(mine, lane);
    run = __shfl_up_sync(0xffffffffu, run, 1);
    if (lane == 0) run = 0.0;
    int hit = segs, last = -1;
    double before_hit = 0.0, before_last = 0.0;
    for (int i = 0; i < per; ++i) {
      const int g = lane * per + i;
      if (g >= segs) break;
      const double t = s.seg[g];
      if (t > 0.0) {
        if (hit == segs && run + t > target) {
          hit = g;
          before_hit = run;
        }
        last = g;
        before_last = run;
      }
      run += t;
    }
    const int best = __reduce_min_sync(0xffffffffu, hit);
    const int tail = __reduce_max_sync(0xffffffffu, last);
    const int g = best < segs ? best : tail;
    double base = best < segs ? before_hit : before_last;
    const unsigned owner = __ballot_sync(0xffffffffu, (best < segs ? hit : last) == g);
    base = __shfl_sync(0xffffffffu, base, __ffs(owner) - 1);

    // read the segment again, the whole block at once, in order
    const RowPass<T, kVec, kDraft> rp(a, t0 + v, rejected, s, C);
    int lo, hi;
    rp.segment(g / kVWarps, g % kVWarps, &lo, &hi);
    int last_seen = -1;
    for (int c0 = lo; c0 < hi && token < 0; c0 += kVThreads) {
      const int c = c0 + tid;
      float fp[kVec], fq[kVec];
      double w[kVec];
#pragma unroll
      for (int i = 0; i < kVec; ++i) fp[i] = fq[i] = 0.f;
      if (c < hi) {
        load_chunk<T, kVec>(rp.p, rp.head, c, rp.V, fp);
        if (kDraft) load_chunk<T, kVec>(rp.q, rp.head, c, rp.V, fq);
      }
      rp.weights(fp, fq, c, w);
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < kVec; ++i) sum += w[i];
      const double incl = warp_scan(sum, lane);
      if (lane == 31) s.warp_sum[warp] = incl;
      __syncthreads();
      double run2 = base;
      for (int k = 0; k < warp; ++k) run2 += s.warp_sum[k];
      double all = base;
      for (int k = 0; k < kVWarps; ++k) all += s.warp_sum[k];
      const double prev = __shfl_up_sync(0xffffffffu, incl, 1);
      run2 += lane > 0 ? prev : 0.0;
      int first = 0x7fffffff, fin = -1;
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        run2 += w[i];
        if (w[i] > 0.0) {
          const int e = c * kVec - rp.head + i;
          if (first == 0x7fffffff && run2 > target) first = e;
          fin = e;
        }
      }
      first = __reduce_min_sync(0xffffffffu, first);
      fin = __reduce_max_sync(0xffffffffu, fin);
      if (lane == 0) {
        s.warp_first[warp] = first;
        s.warp_last[warp] = fin;
      }
      __syncthreads();
      for (int k = kVWarps - 1; k >= 0; --k) {
        if (s.warp_first[k] != 0x7fffffff) token = s.warp_first[k];
        last_seen = max(last_seen, s.warp_last[k]);
      }
      base = all;
      __syncthreads();
    }
    // rounding may leave the crossing just past the segment's last weight
    if (token < 0) token = last_seen;
  }
  if (tid == 0) {
    a.num_accepted[b] = kept;
    a.next_token[b] = token;
  }
  __syncwarp();
  ptx::cluster_wait();
}

// ------------------------------------------------------------------ compaction
// Row b's accepted rows move to the row's first step slots, one thread per 16-byte piece.
// A thread moves its piece of every path entry, in order: entry k's destination is at or
// before its source (a >= k), and every source before it has been read, so the move is
// right in place.  Up to eight entries are in flight.
constexpr int kCompactThreads = 288;  // 4 caches' rows of 72 pieces (4 of 64 without kpe)

__global__ void __launch_bounds__(kCompactThreads) mla_compact_kernel(const __grid_constant__ CompactParams p) {
  const int pieces = p.width / 8;
  const int layer = blockIdx.y * 4 + threadIdx.x / pieces;
  const int c = threadIdx.x % pieces;
  if (layer >= p.num_caches) return;
  const TreeRow row = p.rows[blockIdx.x];
  if (row.n_nodes <= 0) return;
  const int count = min(p.num_accepted[blockIdx.x], row.n_nodes);
  const int32_t* path = p.accept_index + row.token0;
  const int32_t* slot = p.append_rows + row.token0;
  uint4* cache = static_cast<uint4*>(p.caches[layer]) + c;
  for (int k0 = 0; k0 < count; k0 += 8) {
    uint4 v[8];
    int32_t to[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int k = k0 + u;
      to[u] = -1;
      const int a = k < count ? path[k] : -1;
      if (a > k && a < row.n_nodes) {
        const int32_t from = slot[a], dst = slot[k];
        if (from >= 0 && dst >= 0) {
          v[u] = cache[static_cast<int64_t>(from) * pieces];
          to[u] = dst;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (to[u] >= 0) cache[static_cast<int64_t>(to[u]) * pieces] = v[u];
  }
}

// ------------------------------------------------------------------ page copies
// The first tokens of a page are one contiguous run of bytes on both sides.  A block
// copies one 16 KB part of one pair in one cache, four 16-byte pieces per thread in
// flight.
constexpr int kCopyThreads = 256;
constexpr int kCopyPart = kCopyThreads * 16 * 4;

__global__ void __launch_bounds__(kCopyThreads) mla_copy_pages_kernel(const __grid_constant__ CopyParams p) {
  const CopyPair pr = p.pairs[blockIdx.y];
  const int off = blockIdx.x * kCopyPart;
  if (off >= pr.bytes) return;
  uint8_t* cache = static_cast<uint8_t*>(p.caches[blockIdx.z]);
  const uint4* src = reinterpret_cast<const uint4*>(cache + pr.src * p.page_bytes + off) + threadIdx.x;
  uint4* dst = reinterpret_cast<uint4*>(cache + pr.dst * p.page_bytes + off) + threadIdx.x;
  const int n = (pr.bytes - off) / 16 - static_cast<int>(threadIdx.x);
  uint4 v[4];
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (u * kCopyThreads < n) v[u] = src[u * kCopyThreads];
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (u * kCopyThreads < n) dst[u * kCopyThreads] = v[u];
}

template <typename T, int kVec>
cudaError_t launch_verify_as(const VerifyParams& p, int rows, int cluster, cudaStream_t stream) {
  const auto kernel = p.draft ? mla_verify_kernel<T, kVec, true> : mla_verify_kernel<T, kVec, false>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows) * static_cast<unsigned>(cluster));
  cfg.blockDim = dim3(kVThreads);
  cfg.dynamicSmemBytes = sizeof(VerifyShared);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}
static_assert(sizeof(VerifyShared) <= 48 * 1024, "fits without an opt-in");

}  // namespace

cudaError_t launch_verify(const VerifyParams& p, int rows, bool bf16, int num_sms, cudaStream_t stream) {
  // As many blocks to a row as keep every cluster resident at once (two blocks to an SM).
  int cluster = kVMaxCluster;
  while (cluster > 1 && static_cast<int64_t>(rows) * cluster > 2 * static_cast<int64_t>(num_sms)) cluster /= 2;
  // Whole 16-byte loads where p's and q's rows have the same offset from a 16-byte boundary.
  const int64_t es = bf16 ? 2 : 4;
  const bool vec = !p.draft || (((p.ld_target - p.ld_draft) * es) % 16 == 0 &&
                                ((reinterpret_cast<uintptr_t>(p.target) ^ reinterpret_cast<uintptr_t>(p.draft)) & 15u) == 0);
  if (bf16)
    return vec ? launch_verify_as<__nv_bfloat16, 8>(p, rows, cluster, stream)
               : launch_verify_as<__nv_bfloat16, 1>(p, rows, cluster, stream);
  return vec ? launch_verify_as<float, 4>(p, rows, cluster, stream)
             : launch_verify_as<float, 1>(p, rows, cluster, stream);
}

cudaError_t launch_compact(const CompactParams& p, int rows, cudaStream_t stream) {
  const int threads = 4 * (p.width / 8);
  const dim3 grid(static_cast<unsigned>(rows), static_cast<unsigned>((p.num_caches + 3) / 4));
  mla_compact_kernel<<<grid, threads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_copy_pages(const CopyParams& p, int32_t max_bytes, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((max_bytes + kCopyPart - 1) / kCopyPart), static_cast<unsigned>(p.num_pairs),
                  static_cast<unsigned>(p.num_caches));
  mla_copy_pages_kernel<<<grid, kCopyThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace mla
