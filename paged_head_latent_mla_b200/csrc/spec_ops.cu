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
// token is found in the running sum of w.  q is read only where a child was rejected.
//
// One cluster of C blocks works on a row.  Block 0 gathers the tree's single weights (all
// nodes at once) into every block's shared memory.  All blocks then walk alike over these
// copies: what decides a step was written once, to all of them, so that their barriers
// match whatever the inputs hold.  In a pass block r sums its C-th of the vocabulary, each
// warp a contiguous segment of that, and every warp's sum goes to all blocks; one cluster
// barrier per pass (the sums of two passes have buffers of their own: a block can be one
// barrier ahead of another at most).  The block whose segment the running sum crosses reads
// that segment again.
//
// Weights are held in 64 bits from the first subtraction on (one rounding): acceptance and
// the next token are decided at borders, and a sum rounded to 32 bits over a large
// vocabulary would move a border by more than a token's weight.  Every sum has one fixed
// order.
//
// Measured (device time, replayed from a graph): one chain of five over 32768 fp32 tokens
// 10.2 us (three passes), 64 trees of 16 nodes over 131072 fp32 tokens 24.9 us (10.3 us of
// bytes at the copy rate), 128 point-mass trees over 65537 bf16 tokens 12.5 us (2.6).  A call with one pass is a
// chain of about ten dependent memory latencies (the gather's three, the pass, two cluster
// barriers, the crossing).  Rows with several rejections then bound a batch: their passes
// follow one another, about 4 us each over 131072 tokens, with two warps to a scheduler.
// Measured when the 64 trees took 26.7 us: 512-thread blocks 28.3, two chunks in flight
// instead of four 29.6, clusters beyond what is resident 34.4.
constexpr int kVThreads = 256;
constexpr int kVWarps = kVThreads / 32;
constexpr int kVBlocksPerSm = 4;
constexpr int kVMaxCluster = 8;
constexpr int kVMaxNodes = MLA_TREE_MAX_NODES;

// A node as the walk needs it; p, q: the weights of its token at its parent.
struct WalkNode {
  int32_t tok;
  float u, p, q;
  int32_t first, next;
};

struct VerifyShared {
  WalkNode node[kVMaxNodes];
  int32_t n;       // tokens of the row
  int32_t token0;  // its first
  int32_t zero[kVMaxNodes];  // point masses: the tokens rejected at the walk's node
  double seg[2][kVMaxCluster * kVWarps];  // warps' sums of a pass
  // search of the crossing
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

// The doubles that a pass adds up are weights divided by this (the difference of a double's
// and a float's exponent bias).
constexpr double kUp = 0x1p896;

// kVec consecutive weights of a row, kept as loaded until they are used.
template <typename T, int kVec>
struct Chunk {
  static_assert(kVec == 1 || kVec * sizeof(T) == 16, "one element or 16 bytes");
  uint32_t r[kVec > 1 ? 4 : 1];

  // Chunk c of the row: elements [c * kVec - head, + kVec) of which those in [0, V) exist
  // (the others are 0).  `head` makes every whole chunk start on a 16-byte boundary.
  __device__ __forceinline__ void load(const T* row, int head, int c, int V) {
    const int e0 = c * kVec - head;
    if (kVec > 1) {
      if (e0 >= 0 && e0 + kVec <= V) {
        load_whole(row + e0);
        return;
      }
      clear();
      for (int i = 0; i < kVec; ++i)
        if (e0 + i >= 0 && e0 + i < V) put(i, row[e0 + i]);
    } else {
      clear();
      if (e0 < V) put(0, row[e0]);
    }
  }
  // All of a chunk's elements exist; a 16-byte chunk is aligned.
  __device__ __forceinline__ void load_whole(const T* at) {
    if (kVec > 1) {
      const uint4 x = __ldg(reinterpret_cast<const uint4*>(at));
      r[0] = x.x;
      r[1 % (kVec > 1 ? 4 : 1)] = x.y;
      r[2 % (kVec > 1 ? 4 : 1)] = x.z;
      r[3 % (kVec > 1 ? 4 : 1)] = x.w;
    } else {
      clear();
      put(0, *at);
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < (kVec > 1 ? 4 : 1); ++i) r[i] = 0u;
  }
  // Element i as it is stored.
  __device__ __forceinline__ float get(int i) const {
    if (sizeof(T) == 4) return __uint_as_float(r[i]);
    return __uint_as_float((i & 1) ? (r[i >> 1] & 0xffff0000u) : (r[i >> 1] << 16));
  }
  // Element i (finite, not negative) as a double, divided by kUp: a float's or a bf16's bits
  // shifted to where a double has them differ from its conversion in the exponent's bias
  // alone, zeros and subnormals included.  Conversion instructions run at an eighth of the
  // rate (128 trees over 131072 bf16 tokens: 32.6 us with them, 28.2 without).
  __device__ __forceinline__ double scaled(int i) const {
    if (sizeof(T) == 4) return __hiloint2double(static_cast<int>(r[i] >> 3), static_cast<int>(r[i] << 29));
    return __hiloint2double(static_cast<int>(((i & 1) ? r[i >> 1] >> 3 : r[i >> 1] << 13) & 0x1fffe000u), 0);
  }
  // All elements' bits: no sign and no top exponent bit among them means that every one is
  // in [0, 2), which probabilities are, and a weight as it stands.
  __device__ __forceinline__ uint32_t bits() const {
    return kVec > 1 ? (r[0] | r[1 % (kVec > 1 ? 4 : 1)]) | (r[2 % (kVec > 1 ? 4 : 1)] | r[3 % (kVec > 1 ? 4 : 1)])
                    : r[0];
  }
  static constexpr uint32_t kOddBits = sizeof(T) == 4 ? 0xc0000000u : 0xc000c000u;
  // Replace elements that count as 0.
  __device__ __forceinline__ void clean() {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      if (weight(get(i)) != 0.f) continue;
      if (sizeof(T) == 4)
        r[i] = 0u;
      else
        r[i >> 1] &= (i & 1) ? 0x0000ffffu : 0xffff0000u;
    }
  }

 private:
  __device__ __forceinline__ void put(int i, T x) {
    const float w = to_float(x);
    const uint32_t bits = __float_as_uint(w);
#pragma unroll
    for (int k = 0; k < kVec; ++k) {  // (registers are not indexed by a variable)
      if (k != i) continue;
      if (sizeof(T) == 4)
        r[k] = bits;
      else
        r[k >> 1] |= (k & 1) ? bits : (bits >> 16);
    }
  }
};

// What rejections at a node leave of a weight.  Taking Z q off and cutting at 0, once per
// rejection, is taking off the sum S of all Z at once: max(max(w - a, 0) - b, 0) is
// max(w - a - b, 0) for a, b >= 0.  So a pass costs the same after any number of
// rejections.
__device__ __forceinline__ double left_of(double p, double q, double S) {
  const double d = __fma_rn(-S, q, p);
  return d > 0.0 ? d : 0.0;
}

template <typename T, int kVec, bool kDraft>
struct RowPass {
  const T* p;
  const T* q;
  int head, V, chunks;      // chunks of the row
  int per_block, per_warp;  // chunks of a block and of a warp's segment
  double S;             // draft: sum of the rejections' Z, 0 without one
  const int32_t* zero;  // point masses: the rejected tokens
  int rejected;

  __device__ RowPass(const VerifyParams& a, int64_t token, int nrej, double sum_z, const VerifyShared& s,
                     int cluster) {
    p = static_cast<const T*>(a.target) + token * a.ld_target;
    q = kDraft ? static_cast<const T*>(a.draft) + token * a.ld_draft : nullptr;
    V = a.vocab;
    head = kVec > 1 ? static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T)) : 0;
    chunks = static_cast<int>((static_cast<int64_t>(V) + head + kVec - 1) / kVec);
    per_block = (chunks + cluster - 1) >> (__ffs(cluster) - 1);  // clusters are powers of two
    per_warp = (per_block + kVWarps - 1) / kVWarps;
    S = sum_z;
    zero = s.zero;
    rejected = nrej;
  }
  // chunks [lo, hi) of warp `w` of block `r`
  __device__ void segment(int r, int w, int* lo, int* hi) const {
    const int b1 = min(chunks, (r + 1) * per_block);
    *lo = min(b1, r * per_block + w * per_warp);
    *hi = min(b1, *lo + per_warp);
  }
  // What is left of a (clean) chunk's weights, divided by kUp; kQ: a child was rejected.
  template <bool kQ>
  __device__ __forceinline__ void weights(const Chunk<T, kVec>& cp, const Chunk<T, kVec>& cq,
                                          double (&w)[kVec]) const {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      w[i] = cp.scaled(i);
      if (kQ) w[i] = left_of(w[i], cq.scaled(i), S);
    }
  }
  // Point masses: the first chunk of c, c + step, ... (below hi) that holds a rejected
  // token.  Looked up once and again behind every such chunk, not for each chunk.
  __device__ int zero_chunk(int c, int step, int hi) const {
    int best = hi;
    if (!kDraft)
      for (int k = 0; k < rejected; ++k) {
        if (zero[k] >= V) continue;
        const int at = (zero[k] + head) / kVec;
        if (at >= c && at < best && ((at - c) & (step - 1)) == 0) best = at;
      }
    return best;
  }
  __device__ void clear_zeros(int c, double (&w)[kVec]) const {
    for (int k = 0; k < rejected; ++k) {
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        if (zero[k] == c * kVec - head + i) w[i] = 0.0;
    }
  }
  // The warp's sum over chunks [lo, hi): batches of 32 * kBatch whole chunks with all their
  // loads in flight, then single ones, then the row's ragged ends.
  template <int kBatch, bool kQ>
  __device__ __forceinline__ double sum(int lo, int hi, int lane) const {
    using C = Chunk<T, kVec>;
    constexpr int kAcc = kVec > 1 ? 4 : 1;
    double acc[kAcc] = {};
    const int first = max(lo, head > 0 ? 1 : 0), end = min(hi, (V + head) / kVec);  // whole chunks
    int special = kDraft ? hi : zero_chunk(first + lane, 32, end);
    auto add = [&](C& cp, C& cq, int c) {
      if (!kDraft && c == special) {
        double w[kVec];
        cp.clean();
        weights<false>(cp, cq, w);
        clear_zeros(c, w);
#pragma unroll
        for (int i = 0; i < kVec; ++i) acc[i % kAcc] += w[i];
        special = zero_chunk(c + 32, 32, end);
        return;
      }
      if ((cp.bits() | (kQ ? cq.bits() : 0u)) & C::kOddBits) {
        cp.clean();
        if (kQ) cq.clean();
      }
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const double p1 = cp.scaled(i);
        if (kQ) {
          const double d = __fma_rn(-S, cq.scaled(i), p1);
          if (d > 0.0) acc[i % kAcc] += d;  // (one predicated addition)
        } else {
          acc[i % kAcc] += p1;
        }
      }
    };
    const T* p0 = p + (static_cast<int64_t>(first + lane) * kVec - head);
    const T* q0 = kQ ? q + (static_cast<int64_t>(first + lane) * kVec - head) : nullptr;
    int b = first;
    for (; b + 32 * kBatch <= end; b += 32 * kBatch, p0 += 32 * kBatch * kVec, q0 += kQ ? 32 * kBatch * kVec : 0) {
      C cp[kBatch], cq[kQ ? kBatch : 1];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        cp[k].load_whole(p0 + 32 * k * kVec);
        if (kQ) cq[kQ ? k : 0].load_whole(q0 + 32 * k * kVec);
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) add(cp[k], cq[kQ ? k : 0], b + lane + 32 * k);
    }
#pragma unroll 1
    for (int c = b + lane; c < end; c += 32, p0 += 32 * kVec, q0 += kQ ? 32 * kVec : 0) {
      C cp, cq;
      cp.load_whole(p0);
      if (kQ) cq.load_whole(q0);
      add(cp, cq, c);
    }
    if (kVec > 1 && lane < 2) {  // the row's first chunk where it is ragged, and its last
      const int c = lane == 0 ? 0 : (V + head) / kVec;
      if (c >= lo && c < hi && (lane == 0 ? head > 0 : c > 0 || head == 0)) {
        C cp, cq;
        cp.load(p, head, c, V);
        cp.clean();
        cq.clear();
        if (kQ) {
          cq.load(q, head, c, V);
          cq.clean();
        }
        double w[kVec];
        weights<kQ>(cp, cq, w);
        if (!kDraft) clear_zeros(c, w);
#pragma unroll
        for (int i = 0; i < kVec; ++i) acc[i % kAcc] += w[i];
      }
    }
    __syncwarp();
    double t = acc[0];
    if (kAcc == 4) t = (acc[0] + acc[1 % kAcc]) + (acc[2 % kAcc] + acc[3 % kAcc]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
    return t * kUp;
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
__global__ void __launch_bounds__(kVThreads, kVBlocksPerSm) mla_verify_kernel(const VerifyParams a) {
  extern __shared__ __align__(16) uint8_t verify_smem[];
  VerifyShared& s = *reinterpret_cast<VerifyShared*>(verify_smem);
  uint32_t C;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(C));
  const int rank = static_cast<int>(ptx::cluster_ctarank());
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.x / C;
  ptx::cluster_arrive();  // a block's shared memory may be written once it is known to run

  // ---------------------------------------------------------------- gather (block 0)
  TreeRow row{0, -1};
  if (rank == 0) {
    row = a.rows[b];
    const int n = row.n_nodes, held = n <= kVMaxNodes ? n : 0;
    const int64_t t0 = row.token0;
    for (int i = tid; i < n; i += kVThreads) a.accept_index[t0 + i] = (i == 0 && held > 0) ? 0 : -1;
    for (int i = tid; i < held; i += kVThreads) {
      const TreeNode nd = a.nodes[t0 + i];
      WalkNode w{i > 0 ? a.draft_tokens[t0 + i] : -1, a.uniform[t0 + i], 0.f, 0.f, nd.first_child, nd.next_sibling};
      if (nd.parent >= 0 && w.tok >= 0 && w.tok < a.vocab) {
        w.p = weight(to_float(static_cast<const T*>(a.target)[(t0 + nd.parent) * a.ld_target + w.tok]));
        if (kDraft) w.q = weight(to_float(static_cast<const T*>(a.draft)[(t0 + nd.parent) * a.ld_draft + w.tok]));
      }
      s.node[i] = w;
    }
    if (tid == 0) {
      s.n = n;
      s.token0 = row.token0;
    }
    __syncthreads();
  }
  ptx::cluster_wait();
  if (rank == 0 && C > 1) {
    // copy to the other blocks: the nodes' words, block by block across the warps
    const int words = s.n > 0 && s.n <= kVMaxNodes ? s.n * static_cast<int>(sizeof(WalkNode) / 4) : 0;
    const uint32_t* src = reinterpret_cast<const uint32_t*>(s.node);
    const uint32_t at = ptx::smem_addr(s.node), at_n = ptx::smem_addr(&s.n),
                   at_t = ptx::smem_addr(&s.token0);
    for (int i = tid; i < words; i += kVThreads) {
      const uint32_t x = src[i];
      for (uint32_t r = 1; r < C; ++r) st_cluster_u32(ptx::map_to_cta(at + 4u * i, r), x);
    }
    if (tid > 0 && tid < static_cast<int>(C)) {
      st_cluster_u32(ptx::map_to_cta(at_n, tid), static_cast<uint32_t>(s.n));
      st_cluster_u32(ptx::map_to_cta(at_t, tid), static_cast<uint32_t>(s.token0));
    }
    __syncwarp();
  }
  cluster_sync();

  const int n = s.n;
  if (n < 0) return;  // an unused row of a graph plan
  if (n == 0 || n > kVMaxNodes) {
    if (rank == 0 && tid == 0) {
      a.num_accepted[b] = 0;
      a.next_token[b] = -1;
    }
    return;
  }
  const int64_t t0 = s.token0;
  // (read now, needed at the end)
  const double u_next = static_cast<double>(a.uniform_next[b]);
  const int segs = static_cast<int>(C) * kVWarps;
  const int per = (segs + 31) / 32;  // segments of a lane, in order
  int flip = 0;                      // the buffer of the last pass's sums

  // ---------------------------------------------------------------- walk (all blocks alike)
  // Children are tried until one is accepted (its children are next), a pass has to give
  // the next Z, or none is left and a pass gives the sum W of what is left.  One place calls
  // for all passes: copies of that code would evict one another from the instruction cache.
  int v = 0, c = s.node[0].first, kept = 1, rejected = 0;
  double S = 0.0, Z = 1.0, W;  // S: the sum of the rejections' Z (draft)
  while (true) {
    while (c >= 0) {
      const WalkNode nd = s.node[c];
      bool accept = nd.tok < 0;  // given
      double w = nd.p;
      if (!accept) {
        const double u = nd.u;
        double limit;
        if (kDraft) {
          w = left_of(w, nd.q, S);
          limit = __dmul_rn(__dmul_rn(u, static_cast<double>(nd.q)), Z);
        } else {
          for (int k = 0; k < rejected; ++k)
            if (s.zero[k] == nd.tok) w = 0.0;
          limit = __dmul_rn(u, Z);
        }
        accept = limit < w;
      }
      if (accept) {
        v = c;
        if (rank == 0 && tid == 0) a.accept_index[t0 + kept] = v;
        ++kept;
        c = s.node[v].first;
        rejected = 0;
        S = 0.0;
        Z = 1.0;
        continue;
      }
      ++rejected;
      c = nd.next;
      if (kDraft) {
        S += Z;
        if (c >= 0) break;  // its Z
      } else {
        __syncthreads();  // all have read the list
        if (tid == 0) s.zero[rejected - 1] = nd.tok;
        Z = fmax(Z - w, 0.0);
        __syncthreads();
      }
    }

    // a pass over node v's row of weights by the whole cluster: every warp's sum goes to
    // all blocks
    flip ^= 1;
    {
      const RowPass<T, kVec, kDraft> rp(a, t0 + v, rejected, S, s, C);
      int lo, hi;
      rp.segment(rank, warp, &lo, &hi);
      double t;
      if (kDraft && rejected > 0)
        t = rp.template sum<(kVec > 4 ? 2 : 4), kDraft>(lo, hi, lane);
      else
        t = rp.template sum<(kVec > 1 ? 4 : 8), false>(lo, hi, lane);
      if (lane < static_cast<int>(C))
        st_cluster_f64(ptx::map_to_cta(ptx::smem_addr(&s.seg[flip][rank * kVWarps + warp]), lane), t);
      __syncwarp();
      cluster_sync();
    }
    double mine = 0.0;
    for (int i = 0; i < per; ++i)
      if (lane * per + i < segs) mine += s.seg[flip][lane * per + i];
    W = __shfl_sync(0xffffffffu, warp_scan(mine, lane), 31);
    if (c >= 0) {
      Z = W;
      continue;
    }
    if (W > 0.0 || rejected == 0) break;
    rejected = 0;  // the rejections left nothing: p itself
    S = 0.0;
  }
  if (rank == 0 && tid == 0) a.num_accepted[b] = kept;
  if (!(W > 0.0)) {
    if (rank == 0 && tid == 0) a.next_token[b] = -1;
    return;
  }

  // ---------------------------------------------------------------- the next token
  // The first segment whose inclusive running sum exceeds the target, else the last one
  // that holds any weight; the same in every warp.
  const double target = __dmul_rn(u_next, W);
  const double* seg = s.seg[flip];
  double mine = 0.0;
  for (int i = 0; i < per; ++i)
    if (lane * per + i < segs) mine += seg[lane * per + i];
  double run = warp_scan(mine, lane);
  run = __shfl_up_sync(0xffffffffu, run, 1);
  if (lane == 0) run = 0.0;
  int hit = segs, last = -1;
  double before_hit = 0.0, before_last = 0.0;
  for (int i = 0; i < per; ++i) {
    const int g = lane * per + i;
    if (g >= segs) break;
    const double t = seg[g];
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
  if (g / kVWarps != rank) return;
  double base = best < segs ? before_hit : before_last;
  const unsigned owner = __ballot_sync(0xffffffffu, (best < segs ? hit : last) == g);
  base = __shfl_sync(0xffffffffu, base, __ffs(owner) - 1);

  // read the segment again, the whole block at once, in order
  const RowPass<T, kVec, kDraft> rp(a, t0 + v, rejected, S, s, C);
  int lo, hi;
  rp.segment(rank, g % kVWarps, &lo, &hi);
  int token = -1, last_seen = -1;
  for (int c0 = lo; c0 < hi && token < 0; c0 += kVThreads) {
    const int c = c0 + tid;
    Chunk<T, kVec> cp, cq;
    cp.clear();
    cq.clear();
    if (c < hi) {
      cp.load(rp.p, rp.head, c, rp.V);
      if (kDraft && rejected > 0) cq.load(rp.q, rp.head, c, rp.V);
    }
    cp.clean();
    cq.clean();
    double w[kVec];
    if (kDraft && rejected > 0)
      rp.template weights<kDraft>(cp, cq, w);
    else
      rp.template weights<false>(cp, cq, w);
    if (!kDraft) rp.clear_zeros(c, w);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      w[i] *= kUp;
      sum += w[i];
    }
    const double incl = warp_scan(sum, lane);
    if (lane == 31) s.warp_sum[warp] = incl;
    __syncthreads();
    double run2 = base, all = base;
    for (int k = 0; k < kVWarps; ++k) {
      if (k < warp) run2 += s.warp_sum[k];
      all += s.warp_sum[k];
    }
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
  if (tid == 0) a.next_token[b] = token < 0 ? last_seen : token;
}

// ------------------------------------------------------------------ compaction
// Row b's accepted rows move to the row's first step slots, one thread per 16-byte piece.
// A thread moves its piece of every path entry, in order: entry k's destination is at or
// before its source (a >= k), and every source before it has been read, so the move is
// right in place.  Up to eight entries are in flight.  Bound by the launch and three
// dependent latencies (the row's record, path and slots, the rows): one row in one cache
// 2.4 us, 64 rows in 48 caches (8 MB moved) 5.3 us, captured in a graph.
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
// flight.  64 whole pages of 64 tokens in 48 caches (453 MB read and written) take 70.2 us,
// 6.45 TB/s: the copy rate of the memory.
constexpr int kCopyThreads = 256;
constexpr int kCopyPart = kCopyThreads * 16 * 4;

template <typename Params>
__global__ void __launch_bounds__(kCopyThreads) mla_copy_pages_kernel(const __grid_constant__ Params p) {
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
  // As many blocks to a row as keep every cluster resident at once: 64 rows over 131072
  // tokens take 24 us with 8, 29 with 4 and 44 with 2 blocks; 512 rows over 32768 bf16
  // tokens 27 us with 1 and 57 with 8.  `rows` is a graph plan's bucket, whatever its step
  // holds: 64 rows take 18 us in a bucket of 64, 28 in one of 256 and 59 in one of 512
  // (another draw of the same sizes).
  int cluster = kVMaxCluster;
  while (cluster > 1 && static_cast<int64_t>(rows) * cluster > int64_t(kVBlocksPerSm) * num_sms) cluster /= 2;
  // Whole 16-byte loads where p's and q's rows have the same offset from a 16-byte boundary
  // (64 rows over 131072 tokens 24 us, element by element 33).
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

template <typename Params>
cudaError_t launch_copy_pages(const Params& p, int32_t max_bytes, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((max_bytes + kCopyPart - 1) / kCopyPart), static_cast<unsigned>(p.num_pairs),
                  static_cast<unsigned>(p.num_caches));
  mla_copy_pages_kernel<<<grid, kCopyThreads, 0, stream>>>(p);
  return cudaGetLastError();
}
template cudaError_t launch_copy_pages(const CopyParamsSmall&, int32_t, cudaStream_t);
template cudaError_t launch_copy_pages(const CopyParamsLarge&, int32_t, cudaStream_t);

}  // namespace mla
