// kvq_tree.cu — attention of a tree of drafted tokens over the paged 2-bit cache (sm_100a).
//
// Row (i, head) of sequence b, drafted token i < draft_len[b], attends to every token of
// the quantized pages and of the residual window, and to the drafted tokens j that bit j of
// its mask names (its ancestors in the tree and itself):
//   out = sum_t p_t v_t / sum_t p_t,  p_t = exp(sm_scale q . k_t - max).
//
// One warp per row: 32 keys at a time, a lane per key for the logits, then a lane per four
// channels for the sum of the values.  Everything is carried in 32 bits.
#include "kvq_internal.cuh"

namespace kvq {

namespace {

constexpr int kRowWarps = 8;

struct RowState {
  float m, l, o[4];
};

// 32 logits (one a lane, log2 units, -inf where not seen) into the running softmax; returns
// the lane's probability.
__device__ __forceinline__ float online(RowState& st, float x) {
  float mx = x;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, off));
  const float m = fmaxf(st.m, mx);
  if (m == -INFINITY) return 0.0f;  // nothing seen so far
  const float a = ex2(st.m - m), pr = ex2(x - m);
  st.m = m;
  float s = pr;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(kFull, s, off);
  st.l = st.l * a + s;
#pragma unroll
  for (int c = 0; c < 4; ++c) st.o[c] *= a;
  return pr;
}

// Up to 32 tokens of unquantized rows (token t at k + t * stride); bit t of `seen` set where
// token t is attended to.
template <typename T>
__device__ __forceinline__ void raw_tokens(RowState& st, const uint16_t* k, const uint16_t* v, size_t stride, int n,
                                           uint32_t seen, const float* q, float c_log2, int lane) {
  float x = -INFINITY;
  if (lane < n && ((seen >> lane) & 1u)) {
    x = 0.0f;
    for (int c = 0; c < kHeadDim; ++c) x = fmaf(q[c], bits_to_float(k[lane * stride + c], T()), x);
    x *= c_log2;
  }
  const float pr = online(st, x);
  for (int t = 0; t < n; ++t) {
    const float pt = __shfl_sync(kFull, pr, t);
    if (pt == 0.0f) continue;  // the value of a token that is not seen is not read
#pragma unroll
    for (int c = 0; c < 4; ++c) st.o[c] = fmaf(pt, bits_to_float(v[t * stride + 4 * lane + c], T()), st.o[c]);
  }
}

}  // namespace

template <typename T>
__global__ void __launch_bounds__(32 * kRowWarps) tree_rows_kernel(const __grid_constant__ TreeParams p) {
  __shared__ float qs[kRowWarps][kHeadDim];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_trigger();
  const int hq = blockIdx.y, b = blockIdx.z, h = hq / p.gqa;
  const int i = blockIdx.x * kRowWarps + warp;  // drafted token
  const int np = p.num_pages[b], rl = p.res_len[b], dl = p.draft_len[b];
  if (np < 0 || np > p.max_pages || rl < 0 || rl > p.P || dl < 0 || dl > p.T) {
    if (tid == 0) flag_error(p.err, KVQ_DEV_ERR_LENGTH);
    return;
  }
  if (i >= dl) return;
  const size_t row = (size_t(b) * p.T + i) * p.Hq + hq;
  float* q = qs[warp];
  for (int c = lane; c < kHeadDim; c += 32) q[c] = bits_to_float(p.q[row * kHeadDim + c], T());
  __syncwarp();
  RowState st{-INFINITY, 0.0f, {0.0f, 0.0f, 0.0f, 0.0f}};

  for (int pg = 0; pg < np; ++pg) {
    int id = p.page_table[size_t(b) * p.max_pages + pg];
    if (id < 0 || id >= p.pool_pages) {
      if (lane == 0) flag_error(p.err, KVQ_DEV_ERR_PAGE_RANGE);
      id = 0;
    }
    const uint8_t* rec = p.pool + (size_t(id) * p.Hkv + h) * p.L.record;
    for (int g = 0; g < p.P / 32; ++g) {
      const int t = 32 * g + lane;
      const uint32_t* kw = reinterpret_cast<const uint32_t*>(rec + p.L.k_codes) + t * (kHeadDim / 16);
      const uint16_t* sc = reinterpret_cast<const uint16_t*>(rec + p.L.k_scale) + g * kHeadDim;
      const uint16_t* ze = reinterpret_cast<const uint16_t*>(rec + p.L.k_zero) + g * kHeadDim;
      float x = 0.0f;
      for (int c = 0; c < kHeadDim; ++c) {
        const int pos = key_pos(c), mp = key_meta_pos(c);
        const float code = float((kw[pos >> 4] >> elem_bit(pos & 15)) & 3u);
        x = fmaf(q[c], fmaf(code, bits_to_float(sc[mp], T()), bits_to_float(ze[mp], T())), x);
      }
      const int KB = p.k / 16;
      const uint32_t* bw = reinterpret_cast<const uint32_t*>(rec + p.L.kb_codes) + t * KB;
      for (int j = 0; j < p.k; ++j) {
        const int pos = boost_pos(j, KB);
        const float code = float((bw[pos >> 4] >> elem_bit(pos & 15)) & 3u);
        const float sb = bits_to_float(reinterpret_cast<const uint16_t*>(rec + p.L.kb_scale)[g * p.k + j], T());
        x = fmaf(q[rec[p.L.boost_idx + j] & 127], code * sb, x);
      }
      const float pr = online(st, x * p.c_log2);
      for (int tt = 0; tt < 32; ++tt) {
        const float pt = __shfl_sync(kFull, pr, tt);
        const int tok = 32 * g + tt, vp = value_meta_pos(tok);
        const float vs = bits_to_float(reinterpret_cast<const uint16_t*>(rec + p.L.v_scale)[vp], T());
        const float vz = bits_to_float(reinterpret_cast<const uint16_t*>(rec + p.L.v_zero)[vp], T());
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int c = 4 * lane + e, m = c >> 4, v = (c >> 3) & 1, w = c & 7;
          const int a = tt >> 4, u = (tt >> 3) & 1, qq = (tt >> 1) & 3, f = tt & 1;
          const uint32_t word =
              reinterpret_cast<const uint32_t*>(rec + p.L.v_codes)[((2 * g + (m >> 2)) * 32 + 4 * w + qq) * 4 + (m & 3)];
          const float code = float((word >> elem_bit(8 * a + 2 * (2 * u + v) + f)) & 3u);
          st.o[e] = fmaf(pt, fmaf(code, vs, vz), st.o[e]);
        }
      }
    }
  }
  const uint16_t* rk = p.res_k + (size_t(b) * p.Hkv + h) * p.P * kHeadDim;
  const uint16_t* rv = p.res_v + (size_t(b) * p.Hkv + h) * p.P * kHeadDim;
  for (int t = 0; t < rl; t += 32)
    raw_tokens<T>(st, rk + size_t(t) * kHeadDim, rv + size_t(t) * kHeadDim, kHeadDim, min(32, rl - t), kFull, q, p.c_log2, lane);
  const size_t stride = size_t(p.Hkv) * kHeadDim;
  for (int t = 0; t < dl; t += 32) {
    const size_t at = (size_t(b) * p.T + t) * stride + size_t(h) * kHeadDim;
    raw_tokens<T>(st, p.k_draft + at, p.v_draft + at, stride, min(32, dl - t),
                  p.mask[(size_t(b) * p.T + i) * p.W + t / 32], q, p.c_log2, lane);
  }
  const float inv = st.l > 0.0f ? 1.0f / st.l : 0.0f;
  reinterpret_cast<float4*>(p.out + row * kHeadDim)[lane] =
      make_float4(st.o[0] * inv, st.o[1] * inv, st.o[2] * inv, st.o[3] * inv);
}

cudaError_t launch_tree(const TreeParams& p, int dtype, cudaStream_t stream) {
  const dim3 grid((p.T + kRowWarps - 1) / kRowWarps, p.Hq, p.batch);
  return dtype == KVQ_BF16 ? launch_pdl(tree_rows_kernel<__nv_bfloat16>, grid, dim3(32 * kRowWarps), 0, stream, p)
                           : launch_pdl(tree_rows_kernel<__half>, grid, dim3(32 * kRowWarps), 0, stream, p);
}

}  // namespace kvq
