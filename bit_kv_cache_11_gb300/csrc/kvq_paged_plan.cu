// kvq_paged_plan.cu — block tables, sequence lengths and slots of a serving
// step from the requests' lengths (kvq_paged_plan).
//
// With have = ceil(ctx / ps) and tot = ceil((ctx + new) / ps) pages before
// and after the step, request b needs tot - have fresh pages.  The inclusive
// prefix sum A_b of the needs places them: request b takes stack entries
// n_free - 1 - (A_b - need_b) - j, j < need_b, and fits when A_b <= n_free.
// The prefix sum of new gives cu_new, and token t of request b lies at
// position ctx_b + t - cu_new[b], whose page is an old table entry or one of
// the fresh ones.
//
// Bound: latency (4.0 us for 256 prompts and 140791 tokens, 0.6 MB; 5.5 us for
// 64 requests).  A step moves a few KB (a large admission 0.6 MB), so the
// kernel is one launch, and no CTA waits for another: every CTA reads all
// lengths (at most 4096) and redoes the prefix sum, then fills its share of
// the slots and table rows.  A fresh page's id comes from the stack itself,
// never from a table entry another CTA writes.
#include "kvq_paged.cuh"

namespace kvq {
namespace {

constexpr int kPlanThreads = 256;
constexpr int kTokensPerThread = 4;

// Inclusive sums of (a, b) over the CTA's threads; total of both in *ta, *tb.
__device__ __forceinline__ void block_scan2(long long& a, long long& b, long long* ta,
                                            long long* tb) {
  __shared__ long long wa[kPlanThreads / 32], wb[kPlanThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
    if (lane >= o) {
      a += x;
      b += y;
    }
  }
  if (lane == 31) {
    wa[warp] = a;
    wb[warp] = b;
  }
  __syncthreads();
  long long sa = 0, sb = 0;
  *ta = 0;
  *tb = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w < warp) {
      sa += wa[w];
      sb += wb[w];
    }
    *ta += wa[w];
    *tb += wb[w];
  }
  a += sa;
  b += sb;
}

__device__ __forceinline__ int sat_int(long long v) {
  return v > 0x7fffffffLL ? 0x7fffffff : static_cast<int>(v);
}

__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(const PagedPlanParams p) {
  // per request: first token (cu_new) and the stack depth of its first fresh
  // page (-1: it does not fit, its tokens get no slot)
  extern __shared__ int sm[];
  int* cu = sm;                    // [batch + 1]
  int* depth = sm + p.batch + 1;   // [batch]
  grid_dep_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.batch + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(tid * per, p.batch), b1 = min(b0 + per, p.batch);
  const int ps1 = (1 << p.lg_ps) - 1;
  const int free_raw = *p.n_free;
  const int n_free = max(0, min(free_raw, p.free_cap));
  int flag = free_raw != n_free ? KVQ_PAGED_ERR_LENGTH : 0;
  auto lengths = [&](int b, long long* c, long long* n, long long* need, bool* bad) {
    const long long ctx = p.ctx_len[b], nw = p.new_len[b];
    *c = ctx;
    *n = nw > 0 ? nw : 0;
    const long long tot = (ctx + nw + ps1) >> p.lg_ps;
    *bad = ctx < 0 || nw < 0 || tot > p.max_pages;
    *need = *bad ? 0 : tot - ((ctx + ps1) >> p.lg_ps);
  };
  long long s_new = 0, s_need = 0;
  for (int b = b0; b < b1; ++b) {
    long long c, n, need;
    bool bad;
    lengths(b, &c, &n, &need, &bad);
    s_new += n;
    s_need += need;
  }
  long long e_new = s_new, e_need = s_need, t_new, t_need;
  block_scan2(e_new, e_need, &t_new, &t_need);
  long long at = e_new - s_new, got = e_need - s_need;
  const bool lead = blockIdx.x == 0;
  long long taken = 0;
  for (int b = b0; b < b1; ++b) {
    long long c, n, need;
    bool bad;
    lengths(b, &c, &n, &need, &bad);
    const bool fits = !bad && (need == 0 || got + need <= n_free);
    if (bad) flag |= KVQ_PAGED_ERR_LENGTH;
    if (!bad && !fits) flag |= KVQ_PAGED_ERR_NO_PAGES;
    cu[b] = sat_int(at);
    depth[b] = fits ? static_cast<int>(got) : -1;
    if (lead) {
      p.cu_new[b] = sat_int(at);
      p.seq_len[b] = static_cast<int>(fits ? c + n : c);
    }
    if (fits) taken += need;
    at += n;
    got += need;
  }
  if (tid == 0) {
    cu[p.batch] = sat_int(t_new);
    if (t_new > p.n_tokens) flag |= KVQ_PAGED_ERR_LENGTH;
    if (lead) p.cu_new[p.batch] = sat_int(t_new);
  }
  if (lead) {
    // pages taken: the needs of the requests that fit
    long long dummy = 0, sum = taken, all, none;
    __syncthreads();  // block_scan2's shared sums are read above
    block_scan2(sum, dummy, &all, &none);
    if (tid == 0) *p.n_left = n_free - static_cast<int>(all);
    if (flag) set_err(p.err, flag);
  }
  __syncthreads();
  grid_dep_launch();

  // table rows: one warp per request, fresh entries only
  const int n_warps = gridDim.x * (kPlanThreads / 32);
  for (int b = blockIdx.x * (kPlanThreads / 32) + warp; b < p.batch; b += n_warps) {
    const int d = depth[b];
    if (d < 0) continue;
    const int ctx = p.ctx_len[b], n = cu[b + 1] - cu[b];
    const int have = (ctx + ps1) >> p.lg_ps;
    const int need = static_cast<int>((static_cast<long long>(ctx) + n + ps1) >> p.lg_ps) - have;
    int* row = p.table + static_cast<size_t>(b) * p.max_pages + have;
    for (int j = lane; j < need; j += 32) row[j] = p.free_pages[n_free - 1 - d - j];
  }
  // slots: kTokensPerThread consecutive tokens a thread
  const int total = cu[p.batch];
  for (long long t0 = (static_cast<long long>(blockIdx.x) * kPlanThreads + tid) * kTokensPerThread;
       t0 < p.n_tokens; t0 += static_cast<long long>(gridDim.x) * kPlanThreads * kTokensPerThread) {
    int lo = 0, hi = p.batch;  // the request of token t0: the last b with cu[b] <= t0
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (cu[mid] <= t0) lo = mid;
      else hi = mid;
    }
    int b = lo;
    int last_pg = -1, page = 0;  // page index of the cached table entry
    int s[kTokensPerThread], at[kTokensPerThread];
#pragma unroll
    for (int i = 0; i < kTokensPerThread; ++i) {
      const long long t = t0 + i;
      s[i] = -1;
      at[i] = 0;
      if (t >= total) continue;
      while (cu[b + 1] <= t) {
        ++b;
        last_pg = -1;
      }
      // (unsigned: a request whose length breaks the contract may pass 31 bits)
      const int pos = static_cast<int>(static_cast<uint32_t>(p.ctx_len[b]) + static_cast<uint32_t>(t) - cu[b]);
      at[i] = pos;
      if (depth[b] < 0) continue;
      const int have = (p.ctx_len[b] + ps1) >> p.lg_ps;
      const int pg = pos >> p.lg_ps;
      if (pg != last_pg) {
        last_pg = pg;
        page = pg < have ? p.table[static_cast<size_t>(b) * p.max_pages + pg]
                         : p.free_pages[n_free - 1 - depth[b] - (pg - have)];
      }
      // (an entry whose slots do not fit 31 bits, or a negative one, is no page)
      s[i] = (page >> (31 - p.lg_ps)) != 0 ? -1 : (page << p.lg_ps) + (pos & ps1);
    }
    if (t0 + kTokensPerThread <= p.n_tokens) {
      *reinterpret_cast<int4*>(p.slots + t0) = make_int4(s[0], s[1], s[2], s[3]);
      if (p.positions) *reinterpret_cast<int4*>(p.positions + t0) = make_int4(at[0], at[1], at[2], at[3]);
    } else {
      for (int i = 0; i < kTokensPerThread && t0 + i < p.n_tokens; ++i) {
        p.slots[t0 + i] = s[i];
        if (p.positions) p.positions[t0 + i] = at[i];
      }
    }
  }
}

}  // namespace

cudaError_t launch_paged_plan(const PagedPlanParams& p, cudaStream_t st) {
  const long long per_cta = kPlanThreads * kTokensPerThread;
  long long grid = (p.n_tokens + per_cta - 1) / per_cta;
  const long long rows = (p.batch + 63) / 64;  // eight table rows a warp
  if (grid < rows) grid = rows;
  if (grid < 1) grid = 1;
  if (grid > 304) grid = 304;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = sizeof(int) * (2 * static_cast<size_t>(p.batch) + 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_plan_kernel, p);
}

}  // namespace kvq
