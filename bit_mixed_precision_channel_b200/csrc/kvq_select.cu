// kvq_select.cu — choice of the pages a decode step reads (sm_100a).
//
// The stored key ranges of a page bound every logit it can give: with the largest code in
// plane A and plane B, channel c of a token is at most z_c + 3 sA_c (+ 3 sB_j on boosted
// row j of channel idx(j)), with code 0 it is z_c, and so
//   sum_h q_h . k_t  <=  sum_c pos_c (z_c + 3 sA_c) + sum_j pos_idx(j) 3 sB_j + sum_c neg_c z_c,
//   pos_c = sum_h max(q_hc, 0), neg_c = sum_h min(q_hc, 0) over the query heads of the kv head.
// The score of a page is the largest such bound over its 32-token groups.
//
// One cluster of up to 8 CTAs per (sequence, kv head): each CTA scores its share of the pages
// (a warp per page, the next page's scales and zeros loading meanwhile; they, 2 KB of the
// record's 12, are all it reads), the keys stay in shared memory, and the choice is made
// there, so there is one launch and no workspace.  Few units take 8 CTAs each, many fewer (the
// rule and its timings are at the launch).  Up to 256 pages, CTA 0 gathers the keys and ranks
// them by counting (a thread per page); above, the cluster runs a radix select, 8 bits a pass, summing the CTAs'
// histograms through distributed shared memory.
//
// The sums are carried in 64 bits: a choice is a whole-number result, and in 32 bits the
// rounding of two orders of summation would swap pages of almost equal score.
#include <cooperative_groups.h>

#include "kvq_internal.cuh"

namespace kvq {
namespace cg = cooperative_groups;

namespace {

constexpr int kSelThreads = 256;
constexpr int kSelRankMax = kSelThreads;  // pages ranked by counting

// A 16-bit value as a double times 2^-kBias: its exponent and mantissa bits moved into
// place, which is exact for subnormals too and cheaper than a conversion.
__device__ __forceinline__ double biased(uint32_t b, __half) {
  return __hiloint2double(int(((b & 0x8000u) << 16) | ((b & 0x7fffu) << 10)), 0);  // * 2^-1008
}
__device__ __forceinline__ double biased(uint32_t b, __nv_bfloat16) {
  return __hiloint2double(int(((b & 0x8000u) << 16) | ((b & 0x7fffu) << 13)), 0);  // * 2^-896
}
// The power of two the query weights carry against the bias above: products stay far from
// the ends of the exponent range, and the common factor does not change any order.
__device__ __forceinline__ double unbias(__half) { return 0x1p1000; }
__device__ __forceinline__ double unbias(__nv_bfloat16) { return 0x1p880; }

// Scores as unsigned keys of the same order; a score that is no number is the lowest.
__device__ __forceinline__ unsigned long long order_key(double x) {
  if (x != x) return 0ull;
  const unsigned long long u = (unsigned long long)__double_as_longlong(x + 0.0);  // -0 -> +0
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

__device__ __forceinline__ double shfl_xor_d(double x, int m) {
  return __hiloint2double(__shfl_xor_sync(kFull, __double2hiint(x), m), __shfl_xor_sync(kFull, __double2loint(x), m));
}

struct SelShared {
  double wa[kHeadDim];   // 3 pos at the stored position of the channel
  double wz[kHeadDim];   // pos + neg, the same order
  double wb[kHeadDim];   // 3 pos in channel order, for the boosted rows
  __align__(16) uint32_t hist[2][256];
  uint32_t cnt[2];       // own pages above / at the threshold
  uint32_t warp_sum[2][kSelThreads / 32];
  int bin, rest;
};

// Inclusive prefix sums of two flags over the CTA's threads, and their totals.
__device__ __forceinline__ void scan2(SelShared& sh, bool a, bool b, int tid, uint32_t& ia, uint32_t& ib, uint32_t& ta,
                                      uint32_t& tb) {
  const int lane = tid & 31, warp = tid >> 5;
  const uint32_t ba = __ballot_sync(kFull, a), bb = __ballot_sync(kFull, b), le = 0xffffffffu >> (31 - lane);
  ia = __popc(ba & le);
  ib = __popc(bb & le);
  if (lane == 0) {
    sh.warp_sum[0][warp] = __popc(ba);
    sh.warp_sum[1][warp] = __popc(bb);
  }
  __syncthreads();
  ta = tb = 0;
#pragma unroll
  for (int w = 0; w < kSelThreads / 32; ++w) {
    if (w < warp) {
      ia += sh.warp_sum[0][w];
      ib += sh.warp_sum[1][w];
    }
    ta += sh.warp_sum[0][w];
    tb += sh.warp_sum[1][w];
  }
  __syncthreads();
}

}  // namespace

// What the score of a page needs of its record, GP groups of 32 tokens.  Lane i holds the
// stored positions 4i .. 4i + 3 of the scales and zeros, and the boosted rows i, i + 32, ...
template <int GP, int JN>
struct PageMeta {
  uint2 sc[GP], ze[GP];
  uint32_t sb[JN > 0 ? JN : 1][GP];
  uint32_t idx[JN > 0 ? JN : 1];
};

template <int GP, int JN>
__device__ __forceinline__ void page_load(const uint8_t* rec, const SelectParams& p, PageMeta<GP, JN>& m, int lane) {
#pragma unroll
  for (int g = 0; g < GP; ++g) {
    m.sc[g] = __ldcg(reinterpret_cast<const uint2*>(rec + p.L.k_scale + g * 256) + lane);
    m.ze[g] = __ldcg(reinterpret_cast<const uint2*>(rec + p.L.k_zero + g * 256) + lane);
  }
#pragma unroll
  for (int i = 0; i < JN; ++i) {
    const int j = lane + 32 * i;
    const bool in = j < p.k;
    m.idx[i] = in ? __ldcg(rec + p.L.boost_idx + j) : 0u;
#pragma unroll
    for (int g = 0; g < GP; ++g)
      m.sb[i][g] = in ? __ldcg(reinterpret_cast<const uint16_t*>(rec + p.L.kb_scale) + g * p.k + j) : 0u;
  }
}

// Score of one page (all lanes return it).
template <typename T, int GP, int JN>
__device__ __forceinline__ double page_score(const PageMeta<GP, JN>& m, const double (&wa)[4], const double (&wz)[4],
                                             const double* wb, int lane) {
  double x[GP];
#pragma unroll
  for (int g = 0; g < GP; ++g) {
    x[g] = biased(m.sc[g].x & 0xffffu, T()) * wa[0];
    x[g] = fma(biased(m.sc[g].x >> 16, T()), wa[1], x[g]);
    x[g] = fma(biased(m.sc[g].y & 0xffffu, T()), wa[2], x[g]);
    x[g] = fma(biased(m.sc[g].y >> 16, T()), wa[3], x[g]);
    x[g] = fma(biased(m.ze[g].x & 0xffffu, T()), wz[0], x[g]);
    x[g] = fma(biased(m.ze[g].x >> 16, T()), wz[1], x[g]);
    x[g] = fma(biased(m.ze[g].y & 0xffffu, T()), wz[2], x[g]);
    x[g] = fma(biased(m.ze[g].y >> 16, T()), wz[3], x[g]);
  }
#pragma unroll
  for (int i = 0; i < JN; ++i) {
    const double w = wb[m.idx[i] & 127];
#pragma unroll
    for (int g = 0; g < GP; ++g) x[g] = fma(biased(m.sb[i][g], T()), w, x[g]);
  }
  // the lanes' parts of the GP sums: halve the number of sums a lane carries while there
  // are several, so that four groups take 6 exchanges instead of 20
  int h = 16;
#pragma unroll
  for (int n = GP; n > 1; n >>= 1, h >>= 1) {
    const bool up = lane & h;
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
      const double keep = up ? x[i + n / 2] : x[i], give = up ? x[i] : x[i + n / 2];
      x[i] = keep + shfl_xor_d(give, h);
    }
  }
  for (; h > 0; h >>= 1) x[0] += shfl_xor_d(x[0], h);
  double best = x[0];
#pragma unroll
  for (int n = GP, b = 16; n > 1; n >>= 1, b >>= 1) {
    const double o = shfl_xor_d(best, b);
    best = (o > best || o != o) ? o : best;
  }
  return best;
}

template <typename T, int GP, int JN>
__global__ void __launch_bounds__(kSelThreads) select_pages_kernel(const __grid_constant__ SelectParams p) {
  extern __shared__ __align__(16) unsigned long long keys[];  // own pages' keys; in CTA 0 room for kSelRankMax
  __shared__ SelShared sh;
  cg::cluster_group cl = cg::this_cluster();
  const int rank = int(cl.block_rank()), ctas = int(cl.num_blocks());
  const int u = blockIdx.x / ctas, b = u / p.Hkv, h = u - b * p.Hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_trigger();
  const int np = __ldcg(p.num_pages + b);
  const int n = p.n_select;
  int32_t* sel = p.sel + size_t(u) * n;
  const bool bad = np < 0 || np > p.max_pages;
  if (bad || np <= n) {  // every page, in order
    if (rank == 0) {
      const int have = bad ? 0 : np;
      for (int i = tid; i < n; i += kSelThreads) sel[i] = i < have ? i : -1;
      if (tid == 0 && h == 0) {
        p.n_sel[b] = have;
        if (bad) flag_error(p.err, KVQ_DEV_ERR_LENGTH);
      }
    }
    return;
  }
  if (rank == 0 && tid == 0 && h == 0) p.n_sel[b] = n;

  // ---- the query's weights
  if (tid < kHeadDim) {
    double pos = 0.0, neg = 0.0;
    for (int i = 0; i < p.gqa; ++i) {
      const double x = double(bits_to_float(p.q[((size_t(b) * p.Hkv + h) * p.gqa + i) * kHeadDim + tid], T()));
      if (x < 0.0)
        neg += x;
      else
        pos += x;  // also what is no number
    }
    // (infinite bounds of one sign are in no order, and no NaN among them shows it)
    if (!(pos < INFINITY && neg > -INFINITY)) flag_error(p.err, KVQ_DEV_ERR_RANGE);
    const int at = key_meta_pos(tid);
    sh.wa[at] = 3.0 * pos * unbias(T());
    sh.wz[at] = (pos + neg) * unbias(T());
    sh.wb[tid] = 3.0 * pos * unbias(T());
  }
  __syncthreads();
  double wa[4], wz[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    wa[i] = sh.wa[4 * lane + i];
    wz[i] = sh.wz[4 * lane + i];
  }

  // ---- scores of the own pages [s0, s1); pages that are kept anyway get the largest key
  const int per = (np + ctas - 1) / ctas;
  const int s0 = min(np, rank * per), s1 = min(np, s0 + per);
  // (a page that is kept anyway is read like the others: no branch around the loads)
  auto load = [&](int s, PageMeta<GP, JN>& m) {
    int id = __ldcg(p.page_table + size_t(b) * p.max_pages + s);
    if (id < 0 || id >= p.pool_pages) {
      if (lane == 0 && s >= p.n_first && s < np - p.n_recent) flag_error(p.err, KVQ_DEV_ERR_PAGE_RANGE);
      id = 0;
    }
    page_load<GP, JN>(p.pool + (size_t(id) * p.Hkv + h) * p.L.record, p, m, lane);
  };
  PageMeta<GP, JN> m;
  if (s0 + warp < s1) load(s0 + warp, m);
  for (int s = s0 + warp; s < s1; s += kSelThreads / 32) {
    const PageMeta<GP, JN> now = m;
    if (s + kSelThreads / 32 < s1) load(s + kSelThreads / 32, m);
    unsigned long long key = ~0ull;
    if (s >= p.n_first && s < np - p.n_recent) {
      const double x = page_score<T, GP, JN>(now, wa, wz, sh.wb, lane);
      if (x != x && lane == 0) flag_error(p.err, KVQ_DEV_ERR_RANGE);
      key = order_key(x);
    }
    if (lane == 0) keys[s - s0] = key;
  }

  if (np <= kSelRankMax) {
    cl.sync();
    unsigned long long mine = 0;
    if (rank == 0 && tid < np) mine = cl.map_shared_rank(keys, tid / per)[tid % per];
    cl.sync();  // the other CTAs' shared memory is no longer read
    if (rank != 0) return;
    // pages before this one: by the upper halves of the keys, four at a time; where two of
    // them are equal, by the keys and then the slots
    uint32_t* upper = sh.hist[0];
    const uint32_t up = uint32_t(mine >> 32);
    upper[tid] = up;
    if (tid < np) keys[tid] = mine;
    __syncthreads();
    int before = 0;
    if (tid < np) {
      int same = 0;
      for (int j = 0; j < np; j += 4) {
        const uint4 o = lds128(upper + j);  // behind the last page: 0
        before += (o.x > up) + (o.y > up) + (o.z > up) + (o.w > up);
        same += (o.x == up) + (o.y == up) + (o.z == up) + (o.w == up);
      }
      if (same > 1) {
        before = 0;
        for (int j = 0; j < np; ++j) {
          const unsigned long long o = keys[j];
          before += (o > mine || (o == mine && j < tid)) ? 1 : 0;
        }
      }
    }
    const bool keep = tid < np && before < n;
    uint32_t at, none, total, zero;
    scan2(sh, keep, false, tid, at, none, total, zero);
    if (keep) sel[at - 1] = tid;
    return;
  }

  // ---- radix select over the cluster: the n-th largest key's leading bits
  unsigned long long prefix = 0;  // the bits fixed so far, at their place
  int rest = n;                   // pages still to take among those with this prefix
  int shift = 64;
  for (int pass = 0; pass < 8; ++pass) {
    uint32_t* hist = sh.hist[pass & 1];
    hist[tid] = 0;
    __syncthreads();
    const int lo = shift - 8;
    for (int i = tid; i < s1 - s0; i += kSelThreads) {
      const unsigned long long k = keys[i];
      if (shift == 64 || (k >> shift) == (prefix >> shift)) atomicAdd(&hist[int(k >> lo) & 255], 1u);
    }
    cl.sync();
    uint32_t c = 0;
    for (int r = 0; r < ctas; ++r) c += cl.map_shared_rank(hist, r)[tid];
    // bins from the top: thread t holds bin t; pages in higher bins
    uint32_t incl = c;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t y = __shfl_down_sync(kFull, incl, off);
      if (lane + off < 32) incl += y;
    }
    if (lane == 0) sh.warp_sum[0][warp] = incl;
    __syncthreads();
    for (int w = warp + 1; w < kSelThreads / 32; ++w) incl += sh.warp_sum[0][w];
    const uint32_t above = incl - c;
    if (above < uint32_t(rest) && uint32_t(rest) <= incl) {
      sh.bin = tid;
      sh.rest = rest - int(above);
      sh.cnt[0] = c;
    }
    __syncthreads();
    prefix |= (unsigned long long)(sh.bin) << lo;
    rest = sh.rest;
    shift = lo;
    const bool done = sh.cnt[0] == uint32_t(rest);
    __syncthreads();
    if (done) break;  // the whole bin is taken
  }
  // ---- own pages above the threshold and at it, then the places of those taken
  uint32_t gt = 0, eq = 0;
  for (int i = tid; i < s1 - s0; i += kSelThreads) {
    const unsigned long long a = keys[i] >> shift, t = prefix >> shift;
    gt += a > t;
    eq += a == t;
  }
  gt = __reduce_add_sync(kFull, gt);
  eq = __reduce_add_sync(kFull, eq);
  if (tid < 2) sh.cnt[tid] = 0;
  __syncthreads();
  if (lane == 0) {
    atomicAdd(&sh.cnt[0], gt);
    atomicAdd(&sh.cnt[1], eq);
  }
  cl.sync();
  uint32_t at = 0, eq_before = 0;
  for (int r = 0; r < rank; ++r) {
    const uint32_t* c = cl.map_shared_rank(sh.cnt, r);
    const uint32_t left = uint32_t(rest) > eq_before ? uint32_t(rest) - eq_before : 0u;
    at += c[0] + min(c[1], left);
    eq_before += c[1];
  }
  cl.sync();  // no CTA's shared memory is read after this
  for (int base = 0; base < s1 - s0; base += kSelThreads) {
    const int i = base + tid;
    const bool in = i < s1 - s0;
    const unsigned long long a = in ? keys[i] >> shift : 0, t = prefix >> shift;
    const bool is_gt = in && a > t, is_eq = in && a == t;
    uint32_t ig, ie, tg, te;
    scan2(sh, is_gt, is_eq, tid, ig, ie, tg, te);
    const bool keep = is_gt || (is_eq && eq_before + ie <= uint32_t(rest));
    uint32_t ik, in_, tk, tn;
    scan2(sh, keep, false, tid, ik, in_, tk, tn);
    if (keep) sel[at + ik - 1] = s0 + i;
    at += tk;
    eq_before += te;
  }
}

template <typename T, int GP, int JN>
static cudaError_t launch_select_t(const SelectParams& p, int sms, cudaStream_t stream) {
  // The largest power of two up to 8 with at most 8 CTAs an SM in the grid.  At 48 to 128
  // registers a thread 2 to 5 of them reside; the rest start as those end.  Timed on one shape,
  // pages of 64: 512 units of 30 to 250 pages on 1, 2, 4, 8 CTAs each take 57, 51, 59, 72 us
  // (fewer pages a warp would only repeat the CTAs' set-up), 8 units finish soonest on 64 CTAs.
  // Long tables take more, because a CTA's keys have to fit its shared memory.
  const long long units = (long long)p.batch * p.Hkv;
  int ctas = 8;
  while (ctas > 1 && units * ctas > 8ll * sms) ctas /= 2;
  while (ctas < 8 && (long long)p.max_pages > 1024ll * ctas) ctas *= 2;
  const size_t own = (size_t(p.max_pages) + ctas - 1) / ctas;
  const size_t smem = (own > kSelRankMax ? own : size_t(kSelRankMax)) * sizeof(unsigned long long);
  static int seen[64];
  cudaError_t e = ensure_dynamic_smem(select_pages_kernel<T, GP, JN>, int(smem), seen);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(units) * unsigned(ctas));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, select_pages_kernel<T, GP, JN>, p);
}

template <typename T, int GP>
static cudaError_t launch_select_k(const SelectParams& p, int sms, cudaStream_t stream) {
  switch (p.k) {
    case 0: return launch_select_t<T, GP, 0>(p, sms, stream);
    case 16:
    case 32: return launch_select_t<T, GP, 1>(p, sms, stream);
    case 64: return launch_select_t<T, GP, 2>(p, sms, stream);
    case 128: return launch_select_t<T, GP, 4>(p, sms, stream);
  }
  return cudaErrorInvalidValue;
}

template <typename T>
static cudaError_t launch_select_p(const SelectParams& p, int P, int sms, cudaStream_t stream) {
  switch (P) {
    case 32: return launch_select_k<T, 1>(p, sms, stream);
    case 64: return launch_select_k<T, 2>(p, sms, stream);
    case 128: return launch_select_k<T, 4>(p, sms, stream);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_select_pages(const SelectParams& p, int P, int dtype, int sms, cudaStream_t stream) {
  return dtype == KVQ_BF16 ? launch_select_p<__nv_bfloat16>(p, P, sms, stream)
                           : launch_select_p<__half>(p, P, sms, stream);
}

}  // namespace kvq
