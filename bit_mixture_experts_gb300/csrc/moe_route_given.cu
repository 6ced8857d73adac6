// GPU-resident routing where the experts have been chosen already (by a gate, or with the router's logits): counts,
// offsets, stable permutation and block map of ids [T, k] with T k > 1024.
#include "moe_common.cuh"
#include "moe_route_dev.cuh"

namespace moe {

using namespace route_dev;

namespace {

__device__ __forceinline__ int ld_acquire_gpu(const int* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

struct GivenParams {
  const int32_t* ids;
  int T, E, A, per, bn;
  int32_t* cc;  // [chunks][E] counts
  int* ctr;     // grid barrier, CTAs done
  int32_t* counts;
  int32_t* offsets;
  int32_t* perm;
  int32_t* inv_perm;
  int32_t* block_map;
  int32_t* num_blocks;
  int cap;
  int* err;
  unsigned long long wait_cycles;
};

}  // namespace

// A counting sort in one cooperative launch; chunk c = assignments [c per, (c + 1) per).
//   1. each assignment's rank among those of its chunk with the same expert (warps: __match_any_sync; their group
//      sizes are summed per expert over the warps and rounds of the chunk) and the chunk's counts;
//   -  grid barrier;
//   2. every CTA: counts of all chunks and of the earlier ones per expert, scanned over the experts; CTA 0 also
//      writes counts, offsets and the block map;
//   3. position = the expert's offset + earlier chunks' count + rank.
// A chunk's first round keeps its ranks in registers, later ones in inv_perm.  All of an expert's chunks are read
// by every CTA, chunks^2 E counts in all, so that few and large chunks are better than many.  What bounds it: launch,
// barrier and the counts' way through L2; then the rounds (2097152 assignments 103 us, 25 MB).
template <int WARPS>
__global__ void __launch_bounds__(32 * WARPS) route_given_kernel(const GivenParams p) {
  constexpr int THREADS = 32 * WARPS;
  extern __shared__ int smem_i[];
  const int E = p.E, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int* s_hist = smem_i;      // [E] the chunk's counts, then its first position per expert
  int* s_tot = smem_i + E;   // [E] counts of all chunks
  int* s_wc = s_tot + E;     // [WARPS][E] group sizes, then first ranks
  __shared__ uint64_t s_scan[33];
  const int c = blockIdx.x, nch = gridDim.x;
  const int a0 = c * p.per, a1 = min(p.A, a0 + p.per);

  auto expert = [&](int a) {
    const int e = __ldg(p.ids + a);
    if (e >= 0 && e < E) return e;
    set_device_error(p.err, MOE_DEV_BAD_INDEX);
    return 0;
  };

  // ---- 1: ranks in the chunk and its counts
  for (int i = tid; i < 2 * E; i += THREADS) smem_i[i] = 0;
  int e_first = 0, rank_first = 0;
  for (int ab = a0; ab < a1; ab += THREADS) {
    const int a = ab + tid, e = a < a1 ? expert(a) : -1;
    for (int i = tid; i < WARPS * E; i += THREADS) s_wc[i] = 0;
    __syncthreads();
    const unsigned mask = __match_any_sync(FULL, e);
    if (e >= 0 && lane == __ffs(mask) - 1) s_wc[warp * E + e] = __popc(mask);
    __syncthreads();
    for (int i = tid; i < E; i += THREADS) {
      int run = s_hist[i];
#pragma unroll 8
      for (int w = 0; w < WARPS; ++w) {
        const int n = s_wc[w * E + i];
        s_wc[w * E + i] = run;
        run += n;
      }
      s_hist[i] = run;
    }
    __syncthreads();
    if (e >= 0) {
      const int rank = s_wc[warp * E + e] + __popc(mask & ((1u << lane) - 1u));
      if (ab == a0) {
        e_first = e;
        rank_first = rank;
      } else {
        p.inv_perm[a] = rank;
      }
    }
    __syncthreads();
  }
  for (int i = tid; i < E; i += THREADS) {
    p.cc[static_cast<size_t>(c) * E + i] = s_hist[i];
    s_hist[i] = 0;
  }

  // ---- grid barrier: every chunk's counts are written
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    const int before_me = atomicAdd(p.ctr, 1);
    if (before_me < 0 || before_me >= nch) set_device_error(p.err, MOE_DEV_BAD_WORKSPACE);  // not zero at the start
    const long long w0 = clock64();
    while (ld_acquire_gpu(p.ctr) < nch) {
      if (static_cast<unsigned long long>(clock64() - w0) > p.wait_cycles) {
        set_device_error(p.err, MOE_DEV_TIMEOUT);
        break;
      }
      __nanosleep(32);
    }
  }
  __syncthreads();

  // ---- 2: totals, this chunk's start per expert, offsets and the block map
  {
    const int cols = min((E + 31) & ~31, THREADS), parts = THREADS / cols, part = tid / cols;
    for (int e = tid % cols; e < E && part < parts; e += cols) {
      int tot = 0, before = 0;
      for (int q0 = part; q0 < nch; q0 += 16 * parts) {
        int v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int q = q0 + i * parts;
          v[i] = q < nch ? __ldcg(p.cc + static_cast<size_t>(q) * E + e) : 0;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          tot += v[i];
          before += q0 + i * parts < c ? v[i] : 0;
        }
      }
      atomicAdd(&s_tot[e], tot);  // integers: any order
      atomicAdd(&s_hist[e], before);
    }
  }
  __syncthreads();
  // Counts that cannot come from this call (a workspace that was not zero when it began): nothing more is written.
  bool bad = false;
  for (int e = tid; e < E; e += THREADS) bad |= s_tot[e] < 0 || s_hist[e] < 0 || s_hist[e] > s_tot[e];
  bad = __syncthreads_or(bad);
  {
    const int each = ceil_div(E, THREADS);
    const int e0 = min(E, tid * each), e1 = min(E, e0 + each);
    uint64_t loc = 0;
    for (int e = e0; e < e1; ++e)
      loc += (static_cast<uint64_t>(s_tot[e]) << 32) | static_cast<uint32_t>(ceil_div(s_tot[e], p.bn));
    uint64_t total;
    uint64_t run = block_exclusive_scan(loc, s_scan, &total);
    const int ntiles = static_cast<int>(total & 0xffffffffu);
    bad = bad || static_cast<int>(total >> 32) != p.A || ntiles + ceil_div(p.T, p.bn) > p.cap;
    if (bad && tid == 0) set_device_error(p.err, MOE_DEV_BAD_WORKSPACE);
    for (int e = e0; e < e1 && !bad; ++e) {
      const int cnt = s_tot[e];
      const int off = static_cast<int>(run >> 32), tile0 = static_cast<int>(run & 0xffffffffu);
      s_hist[e] += off;
      if (c == 0) {
        p.counts[e] = cnt;
        p.offsets[e] = off;
        emit_expert_tiles(p.block_map, tile0, e, off, cnt, p.bn);
      }
      run += (static_cast<uint64_t>(cnt) << 32) | static_cast<uint32_t>(ceil_div(cnt, p.bn));
    }
    if (c == 0 && !bad) {
      if (tid == 0) {
        p.offsets[E] = p.A;
        p.num_blocks[0] = ntiles + ceil_div(p.T, p.bn);
      }
      for (int i = tid, r = tid * p.bn; r < p.T; i += THREADS, r += THREADS * p.bn) {
        int32_t* m = p.block_map + 3 * (ntiles + i);
        m[0] = E;
        m[1] = p.A + r;
        m[2] = min(p.bn, p.T - r);
      }
    }
  }
  __syncthreads();

  // ---- 3: positions (bad is the same in every thread of the CTA)
  for (int a = a0 + tid; a < a1 && !bad; a += THREADS) {
    const bool first = a < a0 + THREADS;
    const int e = first ? e_first : expert(a), rank = first ? rank_first : p.inv_perm[a];
    const int pos = s_hist[e] + rank;
    if (pos >= 0 && pos < p.A) {
      p.perm[pos] = a;
      p.inv_perm[a] = pos;
    } else {
      set_device_error(p.err, MOE_DEV_BAD_INDEX);
    }
  }

  // ---- the last CTA returns the counters to zero
  if (tid == 0 && atomicAdd(p.ctr + 1, 1) == nch - 1) {
    p.ctr[0] = 0;
    p.ctr[1] = 0;
  }
}

namespace {

// Fewer than the GPU has SMs, so that any CTA has one to itself (131072 assignments in 64, 96, 128 and 152 chunks: 13.9, 14.0, 12.4
// and 12.4 us).
constexpr int GIVEN_CHUNKS = 128;

template <int WARPS>
cudaError_t launch_given(GivenParams& p, int least, cudaStream_t s) {
  const auto kernel = route_given_kernel<WARPS>;
  p.per = max(least, max(ceil_div(p.A, GIVEN_CHUNKS), 32 * WARPS));
  const size_t sm = static_cast<size_t>(WARPS + 2) * p.E * sizeof(int);
  if (sm > 48 * 1024) {
    const cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(kernel), sm);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ceil_div(p.A, p.per));
  cfg.blockDim = dim3(32 * WARPS);
  cfg.dynamicSmemBytes = sm;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;  // every chunk's CTA is resident
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  note_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

unsigned long long wait_limit_ns();

// `least`: assignments of a chunk at least (the workspace has room for as many chunks as that makes).
cudaError_t launch_route_given(const int32_t* ids, int T, int E, int k, int least, int bn, int32_t* counts,
                               int32_t* offsets, int32_t* perm, int32_t* inv_perm, int32_t* bm, int32_t* nb, void* ws,
                               size_t ws_bytes, cudaStream_t s) {
  const unsigned long long ns = wait_limit_ns();
  GivenParams p = {};
  p.ids = ids;
  p.T = T;
  p.E = E;
  p.A = T * k;
  p.bn = bn;
  p.cc = static_cast<int32_t*>(ws);
  p.ctr = reinterpret_cast<int*>(static_cast<char*>(ws) + ((ws_bytes - 16) & ~static_cast<size_t>(3)));
  p.counts = counts;
  p.offsets = offsets;
  p.perm = perm;
  p.inv_perm = inv_perm;
  p.block_map = bm;
  p.num_blocks = nb;
  p.cap = moe_block_map_capacity(T, E, k, bn);
  p.err = device_error_ptr();
  p.wait_cycles = ns > (~0ull) / 3 ? ~0ull : ns * 21 / 10;
  // Larger CTAs take more assignments a round and clear more tables; 1280 assignments to 256 experts with 8, 16 and 32
  // warps 5.2, 5.9 and 7.1 us, 32768 11.1, 8.0 and 8.2, 131072 18.6, 14.4 and 12.4, 32768 to 1024 experts 30, 15 and 11.
  // (Chunks of a few tokens that every CTA counted, as moe_route's, took 5.8, 11.5, 17.7 and 30.)
  if (p.A < 8192) return launch_given<8>(p, least, s);
  if (p.A < 131072 && E <= 512) return launch_given<16>(p, least, s);
  return launch_given<32>(p, least, s);
}

}  // namespace moe
