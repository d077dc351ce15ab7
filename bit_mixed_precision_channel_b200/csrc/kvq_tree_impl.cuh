// kvq_tree_impl.cuh — attention of a tree of drafted tokens over the paged 2-bit cache on
// the fifth-generation tensor cores (sm_100a).  Kernel templates; kvq_tree_<dtype>.cu
// instantiate them, kvq_tree.cu holds the host side.
//
// Row (i, head) of sequence b, drafted token i < draft_len[b], attends to every token of
// the quantized pages and of the residual window, and to the drafted tokens j that bit j of
// its mask names:  out = sum_t p_t v_t / sum_t p_t,  p_t = 2^(c q . k_t - M).
//
// Work.  A unit is (sequence, kv head, 128 rows); its items are tiles of 128 tokens: the
// pages' (128 / P pages each), then the window and the drafted tokens end to end as raw
// tiles.  The units' tiles are laid end to end and cut into one equal range per SM.  A CTA
// that holds a whole unit writes its rows; the parts of a unit that was cut go to the
// workspace, and merge_kernel joins them.
//
// Per tile, with thread roles that run ahead of one another through mbarriers:
//   producer   1 warp    copies the page records (one bulk copy each, three tiles ahead);
//   mover      1 warp    lists where the boosted channels' plane-B codes go;
//   dequant   16 warps   write the keys of a tile, then the value codes of the tile before,
//                        as fp16 operands;
//   issuer     1 warp    S = Q K^T, then O += P V of the tile before (tcgen05, M = 128);
//   softmax    8 warps   16 rows each, four lanes a row: S from tensor memory, running
//                        maximum, P back over S.
// Two S / P buffers of 144 columns, O (128 columns) and Q (64 columns) fill tensor memory.
//
// Arithmetic.  Everything is carried to about 22 bits, as the decode kernel does, so that a
// drafted token verified here sees the logits that the decode step would give it:
//  * a key is u * s + z with u = codeA + codeB / 4 (plane-A scale = 4 x plane-B scale).
//    The fp16 product u * s / 2 is split exactly into its rounding and the remainder (one
//    HMUL2, one HFMA2 for two elements): two operand tiles.  The zero points depend on the
//    32-token group alone, so they are 4 more rows of the key operand, and q . z comes out
//    in columns 128..131 of S;
//  * the query enters as q * 2^-e (exact), e from its largest element;
//  * the value scale is folded into the probability, P = p * sV as a high and a low fp16
//    part, so the value operand is the 2-bit codes themselves, centred (code - 1.5) so that
//    sums do not cancel against the zero points; sum p (z + 1.5 sV) is added in fp32.
//    The running reference M covers the largest logit of a tile with its largest sV (of raw
//    bf16 tokens the largest p * sV that the row sees), so P stays inside fp16 whatever the
//    value scales are;
//  * window and drafted tokens go through the same products: K / 2 and V * 2^-e_t in fp16,
//    with 2^e_t (bf16 only; the token's largest value) in the place of the value scale.
#pragma once
#include <type_traits>

#include "kvq_internal.cuh"
#include "kvq_tc.cuh"

namespace kvq {
namespace tree {

// The code of all roles together has to stay in the instruction caches, so the roles' loops
// are rolled: with 16 x 4096 tokens and 32 drafted ones the unrolled form of an earlier
// version, 130 KB of code, took 182 us and the rolled one 149.
constexpr int kSoftWarps = 8, kDeqWarps = 16;
constexpr int kIssuer = kSoftWarps + kDeqWarps, kProducer = kIssuer + 1, kMover = kIssuer + 2;
constexpr int kThreads = 896;  // 7 warpgroups: two of softmax, four of dequant, one of single warps
// Registers a thread: at launch, then by role (setmaxnreg): 2 x 112 + 4 x 56 + 56 = 7 x 72,
// so the split draws on exactly what the block was launched with.  The shared memory leaves
// next to no L1, so a register spilled in a role's loop costs an L2 access.  bf16, whose dequant
// warps also convert the scales: 2 x 104 + 4 x 64 + 40 (ragged 32 x 8192 of 61 nodes, 32 boosted
// channels: 672 against 700 us; fp16 16 x 4096 of 32 nodes: 113.2 against 111.8).
constexpr int kRegsLaunch = 72;
template <bool BF>
struct Regs {
  static constexpr int soft = BF ? 104 : 112, deq = BF ? 64 : 56, rest = BF ? 40 : 56;
  static_assert(2 * soft + 4 * deq + rest <= 7 * kRegsLaunch, "register split");
};
// (two where every channel may be boosted: the moves take the third's place)
constexpr int rec_stages(int KB) { return KB == 8 ? 2 : 3; }
// The tensor cores round their fp32 accumulator toward zero: 16 products a tile shrink a long
// sum by about 2^-24 each.  O is therefore moved every kFlush tiles into fp32 sums in shared
// memory, which round to nearest.  (Left in tensor memory over 28 tiles of a 4096-token
// cache, the output was off by 3.6e-5 against 64 bits.)
constexpr int kFlush = 4;
constexpr uint32_t kAccStride = 544;  // bytes of an output row's sums: 128 floats, padded against bank conflicts
// shared-memory offsets: key operand (high parts and zero points, remainders), value operand,
// output sums, record stages
constexpr uint32_t kKhi = 0, kKlo = 144 * 256, kV = kKlo + 128 * 256, kAcc = kV + 128 * 256, kRec = kAcc + 128 * kAccStride;
constexpr int kColS = 144, kColO = 288, kColQ = 416;  // tensor-memory columns: S at 0 and 144

__device__ __forceinline__ uint32_t tco(int r, int c) { return uint32_t((r >> 3) * 2048 + c * 128 + (r & 7) * 16); }

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// True in one lane of a converged warp.  The tensor-core products are issued under it by a
// warp whose lanes all walk the same loop: the operands then sit in uniform registers, and a
// product of N = 128 columns takes 64 cycles; issued under `if (lane == 0)`, where each
// operand is moved there first, it took 150 to 220 whatever its size (measured).
__device__ __forceinline__ bool elect_one() {
  uint32_t x;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(x));
  return x != 0;
}
// Tensor memory of the 16 lanes at `a`, as the matrix instructions of a warp lay a tile out:
// lane i of the warp holds rows i / 4 and i / 4 + 8.  ld32: 32 columns of 32 bits, columns
// 8 c + 2 (i % 4) and the next in r[4 c], r[4 c + 1] (row i / 4) and r[4 c + 2], r[4 c + 3].
// The loads are complete on return: the wait names the registers, which keeps uses behind it.
__device__ __forceinline__ void ld32(uint32_t a, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(a)
      : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}
__device__ __forceinline__ void st32(uint32_t a, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(a),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// 4 columns: column i % 4 of rows i / 4 and i / 4 + 8.
__device__ __forceinline__ void ld4(uint32_t a, uint32_t (&r)[2]) {
  asm volatile("tcgen05.ld.sync.aligned.16x128b.x1.b32 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(a) : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(r[0]), "+r"(r[1])::"memory");
}
// 8 columns: column 4 c + i % 4 in r[2 c] (row i / 4) and r[2 c + 1].
__device__ __forceinline__ void st8(uint32_t a, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(r0), "r"(r1), "r"(r2), "r"(r3)
               : "memory");
}
// 32 columns: column 4 c + i % 4 in r[2 c] (row i / 4) and r[2 c + 1].
__device__ __forceinline__ void st32x4(uint32_t a, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(a),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// Two fp32 values in one 64-bit register: sm_100 adds, multiplies and fuses them in one
// instruction.
__device__ __forceinline__ uint64_t f2(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float2 f2_get(uint64_t x) {
  float2 d;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(x));
  return d;
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(kFull, x, 1));
  return fmaxf(x, __shfl_xor_sync(kFull, x, 2));
}
__device__ __forceinline__ float quad_sum(float x) {
  x += __shfl_xor_sync(kFull, x, 1);
  return x + __shfl_xor_sync(kFull, x, 2);
}

template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

__device__ __forceinline__ float pow2i(int e) { return __int_as_float((127 + e) << 23); }  // e in [-126, 127]

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ float2 unpack2(uint32_t u, __half) { return __half22float2(u32_as_h2(u)); }
__device__ __forceinline__ float2 unpack2(uint32_t u, __nv_bfloat16) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
// Two scales or zero points as fp16 (bf16: exact inside fp16's normal range).
__device__ __forceinline__ uint32_t meta_h2(uint32_t x, __half) { return x; }
__device__ __forceinline__ uint32_t meta_h2(uint32_t x, __nv_bfloat16) {
  const float2 f = unpack2(x, __nv_bfloat16());
  return pack_h2(f.x, f.y);
}
// A pair of the cache dtype times a power of two f, as fp16.
__device__ __forceinline__ uint32_t scaled_h2(uint32_t x, float f, __half) {
  return h2_as_u32(__hmul2(u32_as_h2(x), __float2half2_rn(f)));
}
__device__ __forceinline__ uint32_t scaled_h2(uint32_t x, float f, __nv_bfloat16) {
  const float2 y = unpack2(x, __nv_bfloat16());
  return pack_h2(y.x * f, y.y * f);
}

// The least integer n >= -20 with a value scale below 2^n.
__device__ __forceinline__ float scale_log2(float s) { return float(max(-20, int((__float_as_uint(s) >> 23) & 0xff) - 126)); }

// Not zero if an element of the fp16 pair is no finite number: an exponent of ones carries
// into the place of the sign.
__device__ __forceinline__ uint32_t not_finite2(uint32_t x) { return ((x & 0x7c007c00u) + 0x04000400u) & 0x80008000u; }

// Tiles of one unit of sequence b; 0 units for invalid lengths or no drafted token.
struct Seq {
  int np, rl, dl;
  int ntp, nt, nrt;  // page tiles, tiles, row tiles
};
__device__ __forceinline__ void seq_tiles_of(const TreeParams& p, Seq& s) {
  s.ntp = (s.np * p.P + 127) >> 7;
  s.nt = s.ntp + ((s.rl + s.dl + 127) >> 7);
  s.nrt = ((s.dl << p.gqa_log2) + 127) >> 7;
}
__device__ __forceinline__ bool seq_load(const TreeParams& p, int b, Seq& s) {
  s.np = __ldcg(p.num_pages + b);
  s.rl = __ldcg(p.res_len + b);
  s.dl = __ldcg(p.draft_len + b);
  const bool ok = s.np >= 0 && s.np <= p.max_pages && s.rl >= 0 && s.rl <= p.P && s.dl >= 0 && s.dl <= p.T;
  if (!ok) s.np = s.rl = s.dl = 0;
  seq_tiles_of(p, s);
  return ok;
}
__device__ __forceinline__ int seq_tiles(const TreeParams& p, const Seq& s) { return s.nrt * s.nt * p.Hkv; }

// A walk over the tiles [pos, end) of the line.
struct Walk {
  Seq s;
  int b, h, r, k;  // sequence, kv head, row tile, tile of the unit
  int pos, end;
  bool first;        // of this CTA's part of the unit
  template <typename L>
  __device__ __forceinline__ void start(const TreeParams& p, const L& ln, int from, int to) {
    b = ln.b0;
    s.np = ln.np;
    s.rl = ln.rl;
    s.dl = ln.dl;
    seq_tiles_of(p, s);
    const int off = from - ln.base0, u = off / s.nt;
    k = off - u * s.nt;
    h = u / s.nrt;
    r = u - h * s.nrt;
    pos = from;
    end = to;
    first = true;
  }
  __device__ __forceinline__ bool next(const TreeParams& p) {
    if (++pos >= end) return false;
    first = ++k == s.nt;
    if (first) next_unit(p);
    return true;
  }
  __device__ __forceinline__ void next_unit(const TreeParams& p) {
    k = 0;
    if (++r < s.nrt) return;
    r = 0;
    if (++h < p.Hkv) return;
    h = 0;
    do {
      ++b;
      seq_load(p, b, s);
    } while (s.nrt == 0 && b < p.batch - 1);
  }
  __device__ __forceinline__ bool raw() const { return k >= s.ntp; }
};

// Range of CTA i of n (n < 2^15) over W tiles: floor(W i / n).
__device__ __forceinline__ int range_at(int i, int W, int n) {
  const int q = W / n, rest = W - q * n;
  return q * i + rest * i / n;
}
// The CTA whose range holds tile x.
__device__ __forceinline__ int range_owner(int x, int W, int n) {
  int i = min(n - 1, int(float(x) * float(n) / float(W)));
  while (range_at(i, W, n) > x) --i;
  while (i + 1 < n && range_at(i + 1, W, n) <= x) ++i;
  return i;
}

// Total tiles of the line, and the sequence (with its first tile) that holds tile range_at(
// cta): every thread of a block of NT threads takes part.
struct Line {
  int W, n, b0, base0;
  int np, rl, dl;  // of sequence b0
  int sums[32];
};
template <int NT>
__device__ __forceinline__ void line_find(const TreeParams& p, Line& ln, int cta, int ctas, bool flag) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int total = 0, x = 0, incl = 0;
  Seq s;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    int run = 0, at = 0;
    if (pass == 1) {
      if (tid == 0) {
        ln.W = total;
        ln.n = min(ctas, total);
      }
      if (cta >= min(ctas, total)) break;
      at = range_at(cta, total, min(ctas, total));
    }
#pragma unroll 1
    for (int base = 0; base < p.batch; base += NT) {
      const int b = base + tid;
      if (pass == 0 || p.batch > NT) {  // (with a sequence a thread its tiles and their sums stay)
        x = 0;
        if (b < p.batch) {
          if (!seq_load(p, b, s) && flag && pass == 0) flag_error(p.err, KVQ_DEV_ERR_LENGTH);
          x = seq_tiles(p, s);
        }
        incl = x;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int y = __shfl_up_sync(kFull, incl, off);
          if (lane >= off) incl += y;
        }
        if (lane == 31) ln.sums[warp] = incl;
        __syncthreads();
      }
      int before = run, all = 0;
#pragma unroll 4
      for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) before += ln.sums[w];
        all += ln.sums[w];
      }
      run += all;
      if (pass == 1 && x > 0 && before + incl - x <= at && at < before + incl) {
        ln.b0 = b;
        ln.base0 = before + incl - x;
        ln.np = s.np;
        ln.rl = s.rl;
        ln.dl = s.dl;
      }
      if (p.batch > NT) __syncthreads();
    }
    total = run;
  }
  __syncthreads();
}

// Moves of one page's boosted codes, by the words that receive them (8 lists, see
// list_moves): {rotation | source word << 8, mask}, padded to an even length.
// n[0] = -1: every channel boosted, row j of plane B being channel j.
struct Moves {
  uint2 m[8][18];
  int n[8];
};

template <int KB>
struct Shared {
  static constexpr int kRecStages = rec_stages(KB);
  uint64_t rec_full[kRecStages], rec_empty[kRecStages], mv_full[kRecStages], k_full, k_empty, v_full, v_empty, s_full[2],
      p_full[2], pv_done[2], q_full;
  uint32_t tmem;
  int abort;
  // of two tokens {s, s', z, z'}: value scale (raw tiles: 2^e_t / 2), zero point + 1.5 s (raw
  // tiles have none: 0, in bf16 scale_log2(s))
  float4 sz[3][64];
  float smax[3][4];                     // largest value scale of a page tile's groups
  Line line;
  __align__(16) Moves moves[KB > 0 ? kRecStages : 1][KB > 0 ? 4 : 1];  // [stage][page of the tile]
};

// Waits for a phase (about a second at most); false once any wait of the CTA has given up,
// which the end of the kernel reports.
template <typename S>
__device__ __forceinline__ bool wait(S& sh, uint64_t* bar, uint32_t parity) {
  bool ok = mbar_try_wait_suspend(bar, parity, 20000u);
  if (!ok) {
    const uint32_t t0 = uint32_t(clock());
    volatile int* abort = &sh.abort;
    do {
      if (*abort) break;
      ok = mbar_try_wait_suspend(bar, parity, 20000u);
    } while (!ok && uint32_t(clock()) - t0 < (1u << 31));
    if (!ok) *abort = 1;
  }
  return ok;
}
// The same by a whole warp, with one answer for all lanes.
template <typename S>
__device__ __forceinline__ bool wait_warp(S& sh, uint64_t* bar, uint32_t parity) {
  return __all_sync(kFull, wait(sh, bar, parity));
}

constexpr int kPart = 132;  // floats of a partial row: unnormalised output, reference M, sum

// ---------------------------------------------------------------- dequantization

// A dequant warp takes one pass a (0, 1) of the plane-A words 2q + half (q = 0..3) of a
// token: channels 16 s + 8 r + 2 q + f with s = 4 half + 2 a + (0, 1).  The plane-B codes of
// its boosted channels are gathered into two words, for q = 2 qp and 2 qp + 1: code of byte
// i = 2 (s & 1) + r, f at bit 8 i + 4 f + 2 (q & 1).  List 4 half + 2 a + qp of a page's
// moves holds, for each of its boosted channels there, the rotation that brings the plane-B
// code to that bit.  One warp lists a page's moves; the indices are those of the record.
template <int KB>
__device__ __forceinline__ void list_moves(const uint8_t* idx, Moves& mv, int lane) {
  if constexpr (KB == 8) {
    // (not so with fewer boosted channels of a head than the record has rows)
    if (__all_sync(kFull, lds32(idx + 4 * lane) == 0x03020100u + 0x04040404u * uint32_t(lane))) {
      if (lane == 0) mv.n[0] = -1;
      __syncwarp();
      return;
    }
  }
  int count = 0;  // of list `lane`
#pragma unroll 1
  for (int j0 = 0; j0 < 16 * KB; j0 += 32) {
    const int j = j0 + lane;
    int list = 8 + (lane & 7);  // none
    uint2 m = make_uint2(0u, 0u);
    if (j < 16 * KB) {
      const int c = idx[j] & 127, s = c >> 4, r = (c >> 3) & 1, q = (c >> 1) & 3, f = c & 1;
      const int src = boost_pos(j, KB), db = 8 * (2 * (s & 1) + r) + 4 * f + 2 * (q & 1);
      list = 4 * (s >> 2) + 2 * ((s >> 1) & 1) + (q >> 1);
      m = make_uint2(uint32_t((elem_bit(src & 15) - db) & 31) | (uint32_t(src >> 4) << 8), 3u << db);
    }
    const uint32_t same = __match_any_sync(kFull, list);
    const int at = __shfl_sync(kFull, count, list & 7) + __popc(same & ((1u << lane) - 1u));
    // 16 channels a list; more only where a record repeats an index (unused rows, code zero)
    if (list < 8 && at < 16) mv.m[list][at] = m;
#pragma unroll
    for (int l = 0; l < 8; ++l) {
      const int n = __popc(__ballot_sync(kFull, list == l));
      if (lane == l) count = min(count + n, 16);
    }
  }
  __syncwarp();
  if (lane < 8) {
    if (count & 1) mv.m[lane][count] = make_uint2(0u, 0u);
    mv.n[lane] = count;
  }
  __syncwarp();
}

// Keys of token `row` of the tile (token tp of the page record): the 32 channels of (half, a).
// The operands' contraction axis has its own order of channels, the one in which the record
// keeps scales and zero points: 16 bytes number 4 cc + q of a row are the pairs q of the four
// groups of 8 channels 4 cc .. 4 cc + 3 (cc = 2 half + a).
template <typename T, int KB>
__device__ __forceinline__ void key_row(const TreeParams& p, const uint8_t* rec, int tp, int row, int half, int a,
                                        uint8_t* smem, const Moves& mv) {
  const uint4 w0 = lds128(rec + p.L.k_codes + tp * 32), w1 = lds128(rec + p.L.k_codes + tp * 32 + 16);
  const uint32_t w[4] = {half ? w0.y : w0.x, half ? w0.w : w0.z, half ? w1.y : w1.x, half ? w1.w : w1.z};
  uint32_t wb[4];
  if (KB == 8 && mv.n[0] < 0) {  // plane B has the layout of plane A
    const uint4 b0 = lds128(rec + p.L.kb_codes + tp * 32), b1 = lds128(rec + p.L.kb_codes + tp * 32 + 16);
    wb[0] = (half ? b0.y : b0.x) >> (2 * a);
    wb[1] = (half ? b0.w : b0.z) >> (2 * a);
    wb[2] = (half ? b1.y : b1.x) >> (2 * a);
    wb[3] = (half ? b1.w : b1.z) >> (2 * a);
  } else if (KB > 0) {
    const uint8_t* brow = rec + p.L.kb_codes + tp * (4 * KB);
    uint32_t src0 = 0u, src1 = 0u;
    if constexpr (KB == 1) src0 = lds32(brow);
    if constexpr (KB == 2) {
      const uint2 x = lds64(brow);
      src0 = x.x;
      src1 = x.y;
    }
#pragma unroll
    for (int qp = 0; qp < 2; ++qp) {
      const int list = 4 * half + 2 * a + qp, n = mv.n[list];
      uint32_t acc = 0u;
#pragma unroll 2
      for (int e = 0; e < n; e += 2) {
        const uint4 m = *reinterpret_cast<const uint4*>(&mv.m[list][e]);
        uint32_t x, y;
        if constexpr (KB == 1) {
          x = y = src0;
        } else if constexpr (KB == 2) {
          x = (m.x >> 8) ? src1 : src0;
          y = (m.z >> 8) ? src1 : src0;
        } else {
          x = lds32(brow + 4 * (m.x >> 8));
          y = lds32(brow + 4 * (m.z >> 8));
        }
        acc |= (__funnelshift_r(x, x, m.x) & m.y) | (__funnelshift_r(y, y, m.z) & m.w);
      }
      wb[2 * qp] = acc;
      wb[2 * qp + 1] = acc >> 2;
    }
  }
  const uint8_t* sc = rec + p.L.k_scale + (tp >> 5) * 256 + 64 * (2 * half + a);
  uint8_t* dst = smem + tco(row, 4 * (2 * half + a));
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t u[4], lo[4];
    e2m1_pairs(code_pass(w[q], a), u[0], u[1], u[2], u[3]);
    if constexpr (KB > 0) {
      uint32_t ub[4];
      e2m1_pairs(wb[q] & 0x33333333u, ub[0], ub[1], ub[2], ub[3]);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        u[i] = h2_as_u32(__hfma2(u32_as_h2(ub[i]), __float2half2_rn(0.25f), u32_as_h2(u[i])));
    }
    const uint4 s4 = lds128(sc + 16 * q);
    const uint32_t s[4] = {meta_h2(s4.x, T()), meta_h2(s4.y, T()), meta_h2(s4.z, T()), meta_h2(s4.w, T())};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 x = __hmul2(u32_as_h2(u[i]), u32_as_h2(s[i]));
      lo[i] = h2_as_u32(__hfma2(u32_as_h2(u[i]), u32_as_h2(s[i]), __hneg2(x)));
      u[i] = h2_as_u32(x);
    }
    *reinterpret_cast<uint4*>(dst + kKhi + 128 * q) = make_uint4(u[0], u[1], u[2], u[3]);
    *reinterpret_cast<uint4*>(dst + kKlo + 128 * q) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
}

// Value codes of group g of the tile (group gp of the page record), pass a: channels of
// m-tiles 4 mh .. 4 mh + 3, tokens contiguous (K-major operand of the second product), as
// (code - 1.5) / 2.
__device__ __forceinline__ void value_codes(const TreeParams& p, const uint8_t* rec, int gp, int g, int mh, int a,
                                            uint8_t* smem, int lane) {
  const int w = lane & 7, m3 = lane >> 3, m = 4 * mh + m3;
  const uint8_t* vq = rec + p.L.v_codes + (((2 * gp + mh) * 32 + 4 * w) * 4 + m3) * 4;
  const __half2 mid = __float2half2_rn(-0.75f);
  uint32_t u[4][4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    e2m1_pairs(code_pass(lds32(vq + 16 * q), a), u[q][0], u[q][1], u[q][2], u[q][3]);
#pragma unroll
    for (int i = 0; i < 4; ++i) u[q][i] = h2_as_u32(__hadd2(u32_as_h2(u[q][i]), mid));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)  // byte 2u + v: tokens 8u.., channels 8v..
    *reinterpret_cast<uint4*>(smem + kV + (2 * m + (i & 1)) * 2048 + (4 * g + 2 * a + (i >> 1)) * 128 + w * 16) =
        make_uint4(u[0][i], u[1][i], u[2][i], u[3][i]);
}

// Window and drafted tokens: source row of token x of the raw sequence.
__device__ __forceinline__ size_t raw_row(const TreeParams& p, int b, int h, int rl, int x, bool& draft) {
  draft = x >= rl;
  return draft ? ((size_t(b) * p.T + (x - rl)) * p.Hkv + h) * 16 : ((size_t(b) * p.Hkv + h) * p.P + x) * 16;
}

// Raises the range flag if a row sees one of the raw tokens x0 + 2 i, bit i of `which`.
static __device__ __noinline__ void flag_seen(const TreeParams& p, int b, int rl, int dl, int x0, uint32_t which) {
  for (int t = 0; t < 4; ++t) {
    const int j = x0 + 2 * t - rl;  // the drafted token
    if (!((which >> t) & 1u) || j >= dl) continue;
    bool seen = j < 0;
    for (int i = 0; i < dl && !seen; ++i) seen = (__ldcg(p.mask + (size_t(b) * p.T + i) * p.W + (j >> 5)) >> (j & 31)) & 1u;
    if (seen) flag_error(p.err, KVQ_DEV_ERR_RANGE);
  }
}

// An fp16 pair / bf16 pair with the elements that are no finite number set to zero.
__device__ __forceinline__ uint32_t finite2(uint32_t x, uint32_t expo, bool& bad) {
  const bool a = (x & expo) == expo, b = (x & (expo << 16)) == (expo << 16);
  bad |= a | b;
  return (a ? 0u : x & 0xffffu) | (b ? 0u : x & 0xffff0000u);
}

// ---------------------------------------------------------------- softmax

// 32 logits of the lane's two rows at columns tR .. tR + 31, as 2^(cl S + off), times the
// tokens' value scales, back in the same columns as fp16: 16 columns of high parts, 16 of low
// parts.  sz: {s, s', z, z'} of the tokens' pairs, from the lane's first on.  The sums (also
// with z) go to l and zs.
__device__ __forceinline__ void weights(uint32_t tR, const uint64_t (&cl)[2], const uint64_t (&off)[2], const float4* sz,
                                        uint64_t (&l)[2], uint64_t (&zs)[2]) {
  const uint64_t neg = f2(-1.0f, -1.0f);
  uint32_t x[16], out[16];
  ld32(tR, x);
#pragma unroll
  for (int c = 0; c < 4; ++c) {  // 8 tokens
    const float4 v = sz[4 * c];
    const uint64_t s2 = f2(v.x, v.y), z2 = f2(v.z, v.w);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float2 t =
          f2_get(f2_fma(f2(__uint_as_float(x[4 * c + 2 * r]), __uint_as_float(x[4 * c + 2 * r + 1])), cl[r], off[r]));
      uint64_t p = f2(ex2(t.x), ex2(t.y));
      l[r] = f2_add(l[r], p);
      zs[r] = f2_fma(p, z2, zs[r]);
      p = f2_mul(p, s2);
      const float2 y = f2_get(p);
      const uint32_t h = pack_h2(y.x, y.y);
      const float2 f = __half22float2(u32_as_h2(h));
      const float2 e = f2_get(f2_fma(f2(f.x, f.y), neg, p));
      out[2 * c + r] = h;
      out[8 + 2 * c + r] = pack_h2(e.x, e.y);
    }
  }
  st32x4(tR, out);
}

// ---------------------------------------------------------------- the kernel

template <typename T, int KB>
__global__ void __launch_bounds__(kThreads, 1) tree_kernel(const __grid_constant__ TreeParams p) {
  constexpr bool BF = std::is_same<T, __nv_bfloat16>::value;
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr bool kMoves = KB > 0;
  constexpr int kRecStages = rec_stages(KB);
  __shared__ Shared<KB> sh;
  // (taken from lane 0, so that the compiler knows the roles' branches to be uniform)
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(kFull, tid >> 5, 0);

  if (warp == kIssuer) tc::alloc(&sh.tmem, 512);
  if (tid == 0) {
    for (int i = 0; i < kRecStages; ++i) {
      mbar_init(&sh.rec_full[i], 1);
      mbar_init(&sh.rec_empty[i], kDeqWarps);
      mbar_init(&sh.mv_full[i], 1);
    }
    mbar_init(&sh.k_full, kDeqWarps);
    mbar_init(&sh.k_empty, 1);
    mbar_init(&sh.v_full, kDeqWarps);
    mbar_init(&sh.v_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_full[i], kSoftWarps);
      mbar_init(&sh.pv_done[i], 1);
    }
    mbar_init(&sh.q_full, kSoftWarps);
    fence_mbar_init();
    sh.abort = 0;
  }
  // a probability of zero meets whatever the value operand holds: start from finite contents
  for (int i = tid; i < int((kAcc - kV) / 16); i += kThreads)
    reinterpret_cast<uint4*>(smem + kV)[i] = make_uint4(0u, 0u, 0u, 0u);
  pdl_wait();
  line_find<kThreads>(p, sh.line, blockIdx.x, p.n_ctas, blockIdx.x == 0);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tm = __shfl_sync(kFull, sh.tmem, 0);
  const int W = sh.line.W, n_ctas = sh.line.n, cta = blockIdx.x;
  const bool idle = cta >= n_ctas;
  Walk wk{};
  if (!idle) wk.start(p, sh.line, range_at(cta, W, n_ctas), range_at(cta + 1, W, n_ctas));
  if (tid == 0 && cta > 0) {
    // where this range's first boundary cuts a unit, and is the first to do so, merge_kernel joins its parts
    int4 cut = make_int4(-1, 0, 0, 0);
    if (!idle && wk.k > 0) {
      const int c0 = range_owner(wk.pos - wk.k, W, n_ctas);
      if (c0 == cta - 1) cut = make_int4(wk.b, wk.h * wk.s.nrt + wk.r, c0, range_owner(wk.pos - wk.k + wk.s.nt - 1, W, n_ctas));
    }
    p.cuts[cta] = cut;
  }
  const int PPT = 4 >> p.gpp_log2;  // pages of a tile
  const uint32_t stage_bytes = uint32_t(PPT) * p.L.record;

  if (idle) {
    // nothing to do
  } else if (warp >= kIssuer) {
    regs_dec<Regs<BF>::rest>();
    if (warp == kProducer) {
    // ------------------------------------------------------------ producer
    const uint64_t policy = l2_evict_first_policy();
    int n = 0;
    bool more = true;
    while (more) {
      if (wk.first)  // the unit's query rows into L2
        for (int i = lane; i < 128; i += 32) {
          const int R = 128 * wk.r + i, t = R >> p.gqa_log2;
          if (t < wk.s.dl) {
            const uint16_t* q = p.q + ((size_t(wk.b) * p.T + t) * p.Hq + (wk.h << p.gqa_log2) + (R - (t << p.gqa_log2))) * kHeadDim;
            asm volatile("prefetch.global.L2 [%0];" ::"l"(q));
            asm volatile("prefetch.global.L2 [%0];" ::"l"(q + 64));
          }
        }
      if (!wk.raw()) {
        const int st = n % kRecStages, npg = min(PPT, wk.s.np - wk.k * PPT);
        int id = 0;
        if (lane < npg) {
          id = __ldcg(p.page_table + size_t(wk.b) * p.max_pages + wk.k * PPT + lane);
          if (id < 0 || id >= p.pool_pages) {
            flag_error(p.err, KVQ_DEV_ERR_PAGE_RANGE);
            id = 0;
          }
        }
        if (n >= kRecStages && !wait_warp(sh, &sh.rec_empty[st], uint32_t(n / kRecStages - 1) & 1u)) break;
        if (lane == 0) {
          tc::fence_async_smem();
          mbar_arrive_expect_tx(&sh.rec_full[st], uint32_t(npg) * p.L.payload);
        }
        __syncwarp();
        if (lane < npg)
          bulk_g2s(smem + kRec + st * stage_bytes + lane * p.L.record, p.pool + (size_t(id) * p.Hkv + wk.h) * p.L.record,
                   p.L.payload, &sh.rec_full[st], policy);
        ++n;
      } else {
        // window and drafted tokens: into L2 ahead of the dequant warps' loads
        const int x0 = 128 * (wk.k - wk.s.ntp), nx = min(wk.s.rl + wk.s.dl, x0 + 128);
        for (int x = x0 + lane; x < nx; x += 32) {
          bool draft;
          const size_t at = raw_row(p, wk.b, wk.h, wk.s.rl, x, draft);
          const uint4* k = reinterpret_cast<const uint4*>(draft ? p.k_draft : p.res_k) + at;
          const uint4* v = reinterpret_cast<const uint4*>(draft ? p.v_draft : p.res_v) + at;
          asm volatile("prefetch.global.L2 [%0];" ::"l"(k));
          asm volatile("prefetch.global.L2 [%0];" ::"l"(k + 8));
          asm volatile("prefetch.global.L2 [%0];" ::"l"(v));
          asm volatile("prefetch.global.L2 [%0];" ::"l"(v + 8));
        }
      }
      more = wk.next(p);
    }
    // every copy has landed before the shared memory is released
    __syncwarp();
    if (lane == 0)
      for (int y = max(0, n - kRecStages); y < n; ++y)
        mbar_wait_bounded(&sh.rec_full[y % kRecStages], uint32_t(y / kRecStages) & 1u);
    } else if (warp == kIssuer) {
    // ------------------------------------------------------------ issuer
    const uint32_t sKh = smem_addr(smem + kKhi), sKl = smem_addr(smem + kKlo), sV = smem_addr(smem + kV);
    constexpr uint32_t kIdHi = tc::idesc_f16(144, false, false), kIdLo = tc::idesc_f16(128, false, false),
                       kIdMn = tc::idesc_f16(128, false, true);
    // QK of tile `it`, one tile ahead of PV of tile j; at a unit's first tile PV catches up
    // first, because the new query waits for the rows of the old one to be done with S
    int it = 0, j = 0, seg = 0, run = 0;  // run: tiles of this CTA's part of the unit so far
    bool more = true, ok = true;
    uint32_t raws = 0, fresh = 0;  // by the tile's parity: raw; O starts anew with it
    while (true) {
      const bool first = __any_sync(kFull, wk.first), raw = __any_sync(kFull, wk.raw());  // the same in all lanes
      if (more && it - j < (first ? 1 : 2)) {
        if (first) {
          ok = ok && wait_warp(sh, &sh.q_full, uint32_t(seg++) & 1u);
          run = 0;
        }
        ok = ok && wait_warp(sh, &sh.k_full, uint32_t(it) & 1u);
        if (!ok) break;
        tc::fence_after();
        const uint32_t dS = tm + uint32_t(it & 1) * kColS;
        if (elect_one()) {
          uint64_t bd = tc::smem_desc(sKh, 128, 2048);
          const int steps = raw ? 8 : 16;
#pragma unroll 1
          for (int s = 0; s < steps; ++s) {
            if (s == 8) bd = tc::smem_desc(sKl, 128, 2048);  // the remainders
            tc::mma(dS, tm + kColQ + 8 * (s & 7), bd, s < 8 ? kIdHi : kIdLo, s > 0);
            bd += 256 / 16;
          }
          tc::commit(&sh.k_empty);
          tc::commit(&sh.s_full[it & 1]);
        }
        __syncwarp();
        const uint32_t bit = 1u << (it & 1);
        raws = raw ? raws | bit : raws & ~bit;
        fresh = run++ % kFlush == 0 ? fresh | bit : fresh & ~bit;
        ++it;
        more = __any_sync(kFull, wk.next(p));
      } else if (j < it) {
        const uint32_t tP = tm + uint32_t(j & 1) * kColS;
        ok = ok && wait_warp(sh, &sh.p_full[j & 1], uint32_t(j >> 1) & 1u) && wait_warp(sh, &sh.v_full, uint32_t(j) & 1u);
        if (!ok) break;
        tc::fence_after();
        const bool praw = (raws >> (j & 1)) & 1u, pfresh = (fresh >> (j & 1)) & 1u;
        if (elect_one()) {
          // 16 tokens a step: the raw tile's rows are tokens (MN-major), the codes' are channels
          uint64_t bd = praw ? tc::smem_desc(sV, 2048, 128) : tc::smem_desc(sV, 128, 2048);
          const uint32_t step = praw ? 4096 / 16 : 256 / 16, id = praw ? kIdMn : kIdLo;
#pragma unroll 1
          for (uint32_t s = 0; s < 8; ++s) {
            const uint32_t a = tP + 32 * (s >> 1) + 8 * (s & 1);
            tc::mma(tm + kColO, a, bd, id, s > 0 || !pfresh);
            tc::mma(tm + kColO, a + 16, bd, id, 1u);
            bd += step;
          }
          tc::commit(&sh.v_empty);
          tc::commit(&sh.pv_done[j & 1]);
        }
        __syncwarp();
        ++j;
      } else {
        break;
      }
    }
    // the products have completed before the operands' memory is released
    if (ok && j > 0) wait_warp(sh, &sh.pv_done[(j - 1) & 1], uint32_t((j - 1) >> 1) & 1u);
    } else if (kMoves && warp == kMover) {
      // ---------------------------------------------------------- moves of boosted codes
      if constexpr (kMoves) {
        int n = 0;
        bool more = true;
        while (more) {
          if (!wk.raw()) {
            const int st = n % kRecStages, npg = min(PPT, wk.s.np - wk.k * PPT);
            // (a stage that is full again has been read out, its moves too)
            if (!wait_warp(sh, &sh.rec_full[st], uint32_t(n / kRecStages) & 1u)) break;
            for (int i = 0; i < npg; ++i)
              list_moves<KB>(smem + kRec + st * stage_bytes + i * p.L.record + p.L.boost_idx, sh.moves[st][i], lane);
            if (lane == 0) mbar_arrive(&sh.mv_full[st]);
            ++n;
          }
          more = wk.next(p);
        }
      }
    }
  } else if (warp >= kSoftWarps) {
    // ------------------------------------------------------------ dequantization
    regs_dec<Regs<BF>::deq>();
    const int dw = warp - kSoftWarps, g = dw >> 2, half = (dw >> 1) & 1, a = dw & 1;
    const int pg = g >> p.gpp_log2, gp = g - (pg << p.gpp_log2);  // page of the tile, group of the page
    int it = 0, n = 0;  // tiles whose keys are written; page tiles among them
    bool more = true, ok = true, pend = false, phave = false;
    uint32_t badz = 0u;  // not zero once a zero point was no finite number
    // the values of the page tile before, whose record is in stage (n - 1) % kRecStages
    auto values = [&](int j) {
      if (j > 0) ok = wait_warp(sh, &sh.v_empty, uint32_t(j - 1) & 1u);
      if (!ok) return;
      const int st = (n - 1) % kRecStages;
      if (phave)
        value_codes(p, smem + kRec + st * stage_bytes + pg * p.L.record, gp, g, half, a, smem, lane);
      tc::fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sh.v_full);
        mbar_arrive(&sh.rec_empty[st]);
      }
      pend = false;
    };
    while (more) {
      const int v3 = it % 3;
      if (!wk.raw()) {
        const int st = n % kRecStages;
        if (kMoves && !wait_warp(sh, &sh.mv_full[st], uint32_t(n / kRecStages) & 1u)) break;
        if (!wait_warp(sh, &sh.rec_full[st], uint32_t(n / kRecStages) & 1u)) break;
        const bool have = pg < wk.s.np - wk.k * PPT;
        const uint8_t* rec = smem + kRec + st * stage_bytes + pg * p.L.record;
        if (it > 0 && !wait_warp(sh, &sh.k_empty, uint32_t(it - 1) & 1u)) break;
        if (have)
          key_row<T, KB>(p, rec, 32 * gp + lane, 32 * g + lane, half, a, smem, sh.moves[kMoves ? st : 0][kMoves ? pg : 0]);
        if (half == 0 && a == 0) {
          if (have && lane < 16) {  // zero points: row 128 + g of the key operand
            const uint4 z = lds128(rec + p.L.k_zero + gp * 256 + 16 * lane);
            const uint4 o = make_uint4(scaled_h2(z.x, 0.5f, T()), scaled_h2(z.y, 0.5f, T()),
                                       scaled_h2(z.z, 0.5f, T()), scaled_h2(z.w, 0.5f, T()));
            *reinterpret_cast<uint4*>(smem + kKhi + tco(128 + g, lane)) = o;
            // (a scale beyond fp16 makes the sums no number; a zero point could leave a weight of
            // zero.  Looked at once, behind the loop: a flag raised here took 2% more time.)
            if constexpr (BF) badz |= not_finite2(o.x) | not_finite2(o.y) | not_finite2(o.z) | not_finite2(o.w);
          }
        } else if (half == 1 && a == 0) {
          float s = 0.0f, z = 0.0f;
          if (have) {
            const int at = 2 * value_meta_pos(32 * gp + lane);
            s = bits_to_float(*reinterpret_cast<const uint16_t*>(rec + p.L.v_scale + at), T());
            z = bits_to_float(*reinterpret_cast<const uint16_t*>(rec + p.L.v_zero + at), T());
          }
          float* sz = reinterpret_cast<float*>(sh.sz[v3]) + 4 * (16 * g + (lane >> 1)) + (lane & 1);
          sz[0] = s;
          sz[2] = fmaf(1.5f, s, z);
          const uint32_t mx = __reduce_max_sync(kFull, __float_as_uint(fabsf(s)));
          if (lane == 0) sh.smax[v3][g] = __uint_as_float(mx);
        }
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.k_full);
        if (pend) values(it - 1);
        if (!ok) break;
        pend = true;
        phave = have;
        ++n;
      } else {
        // window and drafted tokens: warp dw takes tokens 8 dw .. 8 dw + 7 of the tile, two at a
        // time, 16 lanes a token
        const int x0 = 128 * (wk.k - wk.s.ntp) + 8 * dw + (lane >> 4), nx = wk.s.rl + wk.s.dl, c = lane & 15;
        const int t0 = 8 * dw + (lane >> 4);  // token of the tile, and the 3 that follow it two by two
        auto rows = [&](const uint16_t* window, const uint16_t* drafted, uint4 (&x)[4]) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[i] = make_uint4(0u, 0u, 0u, 0u);
            if (x0 + 2 * i < nx) {
              bool draft;
              const size_t at = raw_row(p, wk.b, wk.h, wk.s.rl, x0 + 2 * i, draft) + c;
              x[i] = __ldcg(reinterpret_cast<const uint4*>(draft ? drafted : window) + at);
            }
          }
        };
        uint4 x[4];
        rows(p.res_k, p.k_draft, x);
        if (it > 0 && !wait_warp(sh, &sh.k_empty, uint32_t(it - 1) & 1u)) break;
        uint32_t which = 0u;  // of the lane's tokens those of which something is no finite number
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t k[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
          uint8_t* dst = smem + kKhi + tco(t0 + 2 * i, c & ~3) + 4 * (c & 3);
#pragma unroll
          for (int e = 0; e < 4; ++e) {  // pair e of 8 channels c: the operand's order
            k[e] = scaled_h2(k[e], 0.5f, T());
            *reinterpret_cast<uint32_t*>(dst + 128 * e) = k[e];
          }
          if (not_finite2(k[0]) | not_finite2(k[1]) | not_finite2(k[2]) | not_finite2(k[3])) which |= 1u << i;
        }
        // the values: what is no number is zero (a probability of zero has to stay zero), and
        // bf16 is brought below 2 by the token's power of two
        rows(p.res_v, p.v_draft, x);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int xi = x0 + 2 * i;
          uint32_t v[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
          bool bad = false;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = finite2(v[e], BF ? 0x7f80u : 0x7c00u, bad);
          if (bad) which |= 1u << i;
          float s = xi < nx ? 0.5f : 0.0f;
          if constexpr (BF) {
            float m = 0.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 y = unpack2(v[e], T());
              m = fmaxf(m, fmaxf(fabsf(y.x), fabsf(y.y)));
            }
#pragma unroll
            for (int off = 8; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, off));
            const int e2 = max(-90, min(126, int((__float_as_uint(m) >> 23) & 0xff) - 127));  // (below 4 at 2^127)
            s *= pow2i(e2);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = scaled_h2(v[e], pow2i(-e2), T());
          }
          x[i] = make_uint4(v[0], v[1], v[2], v[3]);
          if (c == 0) {
            const int t = t0 + 2 * i;
            float* sz = reinterpret_cast<float*>(sh.sz[v3]) + 4 * (t >> 1) + (t & 1);
            sz[0] = s;
            sz[2] = BF ? scale_log2(s) : 0.0f;
          }
        }
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.k_full);
        if (pend) values(it - 1);
        if (!ok) break;
        if (it > 0 && !wait_warp(sh, &sh.v_empty, uint32_t(it - 1) & 1u)) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(smem + kV + tco(t0 + 2 * i, c)) = x[i];
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.v_full);
        if (which) flag_seen(p, wk.b, wk.s.rl, wk.s.dl, x0, which);  // (earlier, the call took registers from the loops)
      }
      ++it;
      more = wk.next(p);
    }
    if (!more && pend && ok) values(it - 1);
    if (BF && badz) flag_error(p.err, KVQ_DEV_ERR_RANGE);
  } else {
    // ------------------------------------------------------------ softmax
    regs_inc<Regs<BF>::soft>();
    const int row0 = 32 * (warp & 3) + 16 * (warp >> 2), quad = lane & 3;  // of the warp's rows the first; the lane's place
    const int row = row0 + (lane >> 2);                                    // ... and row + 8
    const uint32_t at = uint32_t(row0) << 16;                              // the warp's tensor-memory lanes
    int it = 0, run = 0, k0 = 0;  // tiles; tiles of this part of the unit, and its first
    bool some = false, to_end = false;
    bool valid[2] = {false, false};
    size_t orow[2] = {0, 0};
    float M[2], l[2], zs[2], cl[2];
    float asc[2];     // factor of the sums in shared memory against O (0: nothing there yet)
    // Waits until the second product of tile j is complete.  A parity names a phase only
    // among two: with a barrier for every other tile, and tile it - 2 waited for at tile it,
    // the phase asked for is always the current one or the one before.  (After a wait that
    // gave up every other one returns at once, and the loop runs out by itself.)
    auto wait_pv = [&](int j) {
      wait(sh, &sh.pv_done[j & 1], uint32_t(j >> 1) & 1u);
      __syncwarp();
      tc::fence_after();
    };
    auto sums = [&](int c2, int r) -> float2& {  // output sums of columns 2 c2, 2 c2 + 1
      return *reinterpret_cast<float2*>(smem + kAcc + (row + 8 * r) * kAccStride + c2 * 8);
    };
    bool done = false;
    while (true) {
      if (wk.first || done) {
        // the unit before is complete but for its second products; first the next unit's query,
        // so that its products start while these rows are written
        const bool some0 = some, whole = k0 == 0 && to_end;
        const bool v0[2] = {valid[0], valid[1]};
        float* dst[2];
#pragma unroll
        for (int r = 0; r < 2; ++r)
          dst[r] = whole ? p.out + orow[r] * kHeadDim
                         : p.part + (size_t(2 * cta + (k0 == 0 ? 1 : 0)) * 128 + row + 8 * r) * kPart;
        float ncl[2] = {0.0f, 0.0f};
        if (!done) {
          some = 128 * wk.r + row0 < wk.s.dl << p.gqa_log2;  // any row of this warp
          if (some) {
            // 16 bytes c of a row: channels 8 (4 c + quad) .., the operand's order
            uint4 v[2][4];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const int R = 128 * wk.r + row + 8 * r, i = R >> p.gqa_log2;
              valid[r] = i < wk.s.dl;
              orow[r] = (size_t(wk.b) * p.T + i) * p.Hq + (wk.h << p.gqa_log2) + (R - (i << p.gqa_log2));
              const uint4* src = reinterpret_cast<const uint4*>(p.q + orow[r] * kHeadDim) + quad;
#pragma unroll
              for (int c = 0; c < 4; ++c) v[r][c] = valid[r] ? __ldcg(src + 4 * c) : make_uint4(0u, 0u, 0u, 0u);
            }
            float f[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              uint32_t m2 = 0u;  // magnitudes as integers: the order of their bits
#pragma unroll
              for (int c = 0; c < 4; ++c)
                m2 = __vmaxu2(m2, __vmaxu2(__vmaxu2(v[r][c].x & 0x7fff7fffu, v[r][c].y & 0x7fff7fffu),
                                           __vmaxu2(v[r][c].z & 0x7fff7fffu, v[r][c].w & 0x7fff7fffu)));
              const float2 m = unpack2(m2, T());
              const float top = quad_max(fmaxf(m.x, m.y));
              // (its logits may all be minus infinity, which looks like a row that sees nothing; NaN shows in the sums)
              if (valid[r] && !(top < INFINITY)) flag_error(p.err, KVQ_DEV_ERR_RANGE);
              // |q| < 2^e; e = 0 below 1
              const int e = min(max(int((__float_as_uint(top) >> 23) & 0xff) - 126, 0), 126);
              f[r] = p.c_log2 < 0.0f ? -pow2i(-e) : pow2i(-e);
              ncl[r] = fmaxf(2.0f * fabsf(p.c_log2) * pow2i(e), 1e-30f);  // above 0: a masked -inf stays one
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              st8(tm + kColQ + at + 16 * c, scaled_h2(v[0][c].x, f[0], T()), scaled_h2(v[1][c].x, f[1], T()),
                  scaled_h2(v[0][c].y, f[0], T()), scaled_h2(v[1][c].y, f[1], T()));
              st8(tm + kColQ + at + 16 * c + 8, scaled_h2(v[0][c].z, f[0], T()), scaled_h2(v[1][c].z, f[1], T()),
                  scaled_h2(v[0][c].w, f[0], T()), scaled_h2(v[1][c].w, f[1], T()));
            }
            tc::wait_st();
          }
          tc::fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.q_full);
        }
        if (it > 0) {
          wait_pv(it - 1);
          if (some0) {
            asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the rows before have left their place
            __syncwarp();
            uint64_t inv[2], z2[2], a2[2], chk = 0ull;  // chk: 0, or no number once a result is none
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              l[r] = quad_sum(l[r]);
              zs[r] = quad_sum(zs[r]);
              const float x = whole ? (l[r] > 0.0f ? 1.0f / l[r] : 0.0f) : 1.0f;
              inv[r] = f2(x, x);
              z2[r] = f2(zs[r], zs[r]);
              a2[r] = f2(asc[r], asc[r]);
              if (v0[r]) chk = f2_fma(z2[r], 0ull, f2_fma(f2(l[r], l[r]), 0ull, chk));
            }
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
              uint32_t o[16];
              ld32(tm + kColO + at + 32 * i, o);
#pragma unroll
              for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                  float2& sum = sums(16 * i + 4 * c + quad, r);
                  uint64_t x = f2(__uint_as_float(o[4 * c + 2 * r]), __uint_as_float(o[4 * c + 2 * r + 1]));
                  const float2 a = asc[r] != 0.0f ? sum : make_float2(0.0f, 0.0f);
                  x = f2_mul(f2_fma(f2_fma(f2(a.x, a.y), a2[r], x), f2(2.0f, 2.0f), z2[r]), inv[r]);
                  if (v0[r]) chk = f2_fma(x, 0ull, chk);
                  sum = f2_get(x);
                }
            }
            // the rows leave from where their sums were, one bulk copy each (written from the
            // registers, 32 bytes of eight rows at a time, a unit's rows took 10000 cycles)
            tc::fence_async_smem();
            __syncwarp();
#pragma unroll
            for (int r = 0; r < 2; ++r)
              if (quad == 0 && v0[r])
                asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], 512;" ::"l"(dst[r]),
                             "r"(smem_addr(&sums(0, r)))
                             : "memory");
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            const float2 ck = f2_get(chk);
            if (ck.x != 0.0f || ck.y != 0.0f) flag_error(p.err, KVQ_DEV_ERR_RANGE);
#pragma unroll
            for (int r = 0; r < 2; ++r)
              if (!whole && v0[r] && quad == 0) {
                dst[r][128] = M[r];
                dst[r][129] = l[r];
              }
          }
        }
        if (done) {
          asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
          break;
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          M[r] = -INFINITY;
          l[r] = zs[r] = asc[r] = 0.0f;
          cl[r] = ncl[r];
        }
        run = 0;
        k0 = wk.k;
      }
      const int buf = it & 1, v3 = it % 3;
      const uint32_t tS = tm + uint32_t(buf) * kColS + at;
      const bool raw = wk.raw();
      wait(sh, &sh.s_full[buf], uint32_t(it >> 1) & 1u);
      if (it >= 2) wait_pv(it - 2);
      __syncwarp();
      tc::fence_after();
      if (some) {
        uint32_t zr[2] = {0u, 0u};  // q . z of group `quad`
        if (!raw) ld4(tS + 128, zr);
        if (raw || wk.s.np - wk.k * PPT < PPT) {
          // masked places, whatever they hold, become -inf: tokens that are not there or not seen
          const int ng = raw ? 0 : (wk.s.np - wk.k * PPT) << p.gpp_log2;  // groups that hold tokens
          if (quad >= ng) zr[0] = zr[1] = 0u;
          uint32_t mine[2] = {0u, 0u};  // bits of the tokens of group `quad` that the rows see
          if (raw) {
            const int xw = 128 * (wk.k - wk.s.ntp) + 32 * quad, in_window = wk.s.rl - xw;
            const int d = xw - wk.s.rl, wd = d >> 5;  // d: first drafted token of the group
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const uint32_t* mask = p.mask + (size_t(wk.b) * p.T + ((128 * wk.r + row + 8 * r) >> p.gqa_log2)) * p.W;
              auto word = [&](int j) {  // of the row's mask, without what is behind draft_len
                const int left = wk.s.dl - 32 * j;
                return valid[r] && j >= 0 && left > 0 ? __ldcg(mask + j) & (left >= 32 ? kFull : (1u << left) - 1u) : 0u;
              };
              const uint32_t drafted = d > -32 ? __funnelshift_r(word(wd), word(wd + 1), uint32_t(d) & 31u) : 0u;
              mine[r] = in_window >= 32 ? kFull : drafted | (in_window > 0 ? (1u << in_window) - 1u : 0u);
            }
          }
#pragma unroll 1
          for (int g = ng; g < 4; ++g) {
            uint32_t x[16], see[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) see[r] = __shfl_sync(kFull, mine[r], (lane & ~3) + g);
            if (__all_sync(kFull, (see[0] & see[1]) == kFull)) continue;
            see[0] >>= 2 * quad;  // the lane's first token lowest
            see[1] >>= 2 * quad;
            ld32(tS + 32 * g, x);
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (!((see[(j >> 1) & 1] >> (8 * (j >> 2) + (j & 1))) & 1u)) x[j] = 0xff800000u;
            st32(tS + 32 * g, x);
          }
          tc::wait_st();
        }
        // first pass: the rows' largest logits (S is read again for the second).  Raw bf16 tokens
        // have scales of any size, hidden ones too: there each logit counts with its own token's
        // scale, in the units of M, so that what a row does not see cannot move its reference
        float mx[2] = {-INFINITY, -INFINITY};
        const float4* sz = &sh.sz[v3][quad];
#pragma unroll 1
        for (int g = 0; g < 4; ++g) {
          uint32_t x[16];
          ld32(tS + 32 * g, x);
          if (BF && raw) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const float4 v = sz[16 * g + 4 * c];
#pragma unroll
              for (int r = 0; r < 2; ++r)
                mx[r] = fmaxf(mx[r], fmaxf(fmaf(__uint_as_float(x[4 * c + 2 * r]), cl[r], v.z),
                                           fmaf(__uint_as_float(x[4 * c + 2 * r + 1]), cl[r], v.w)));
            }
            continue;
          }
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float m = -INFINITY;
#pragma unroll
            for (int c = 0; c < 4; ++c)
              m = fmaxf(m, fmaxf(__uint_as_float(x[4 * c + 2 * r]), __uint_as_float(x[4 * c + 2 * r + 1])));
            mx[r] = fmaxf(mx[r], m + __shfl_sync(kFull, __uint_as_float(zr[r]), (lane & ~3) + g));
          }
        }
        // probabilities are carried as 2^(x - M + 7), so p * s starts below 2^7 (raw fp16: s = 1/2)
        const float lg = raw ? 0.0f
                             : scale_log2(fmaxf(fmaxf(sh.smax[v3][0], sh.smax[v3][1]), fmaxf(sh.smax[v3][2], sh.smax[v3][3])));
        float alpha[2], nm[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float top = BF && raw ? quad_max(mx[r]) : fmaf(quad_max(mx[r]), cl[r], lg);
          alpha[r] = 1.0f;
          if (top > M[r] + 8.0f) {  // p * s could pass 2^15
            alpha[r] = ex2(M[r] - top);  // M = -inf: 0
            l[r] *= alpha[r];
            zs[r] *= alpha[r];
            asc[r] *= alpha[r];
            M[r] = top;
          }
          nm[r] = M[r] == -INFINITY ? 0.0f : 7.0f - M[r];
        }
        // second pass
        uint64_t tl[2] = {0ull, 0ull}, tz[2] = {0ull, 0ull};
        const uint64_t cl2[2] = {f2(cl[0], cl[0]), f2(cl[1], cl[1])};
#pragma unroll 1
        for (int g = 0; g < 4; ++g) {
          uint64_t off[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float o = fmaf(__shfl_sync(kFull, __uint_as_float(zr[r]), (lane & ~3) + g), cl[r], nm[r]);
            off[r] = f2(o, o);
          }
          weights(tS + 32 * g, cl2, off, sz + 16 * g, tl, tz);
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float2 a = f2_get(tl[r]), z = f2_get(tz[r]);
          l[r] += a.x + a.y;
          if (!(BF && raw)) zs[r] += z.x + z.y;
        }
        const bool flush = run > 0 && run % kFlush == 0;
        if (flush && run == kFlush) {  // the rows of the unit before have left
          asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
          __syncwarp();
        }
        if (flush || (run > 0 && __any_sync(kFull, alpha[0] != 1.0f || alpha[1] != 1.0f))) {
          // O into the sums, to start anew with this tile; or only to the new reference
          wait_pv(it - 1);
#pragma unroll 1
          for (int i = 0; i < 4; ++i) {
            uint32_t o[16];
            ld32(tm + kColO + at + 32 * i, o);
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha[(j >> 1) & 1]);
            if (flush) {
#pragma unroll
              for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                  float2& a = sums(16 * i + 4 * c + quad, r);
                  const float2 x = asc[r] != 0.0f ? a : make_float2(0.f, 0.f);
                  a = make_float2(fmaf(x.x, asc[r], __uint_as_float(o[4 * c + 2 * r])),
                                  fmaf(x.y, asc[r], __uint_as_float(o[4 * c + 2 * r + 1])));
                }
            } else {
              st32(tm + kColO + at + 32 * i, o);
            }
          }
          if (flush) asc[0] = asc[1] = 1.0f;
        }
        tc::wait_st();
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.p_full[buf]);
      to_end = wk.k == wk.s.nt - 1;
      done = !wk.next(p);
      ++it;
      ++run;
    }
  }
  // ---------------------------------------------------------------- leave
  pdl_trigger();
  tc::fence_before();
  __syncwarp();
  __syncthreads();
  if (tid == 0 && sh.abort) flag_error(p.err, KVQ_DEV_ERR_TIMEOUT);
  if (warp == kIssuer) tc::dealloc(tm, 512);
}

// Joins the parts of the units that were cut (cuts[i], i = 1 .. n_ctas - 1), 16 rows a block.
static __global__ void __launch_bounds__(256) merge_kernel(const __grid_constant__ TreeParams p) {
  pdl_wait();
  pdl_trigger();
  const int4 cut = __ldcg(reinterpret_cast<const int4*>(p.cuts) + blockIdx.x + 1);
  if (cut.x < 0) return;
  const int b = cut.x, c0 = cut.z, c1 = cut.w, lane = threadIdx.x & 31;
  const int dl = __ldcg(p.draft_len + b), nrt = (dl * p.gqa + 127) / 128, h = cut.y / nrt, rt = cut.y - h * nrt;
  for (int r = 16 * blockIdx.y + (threadIdx.x >> 5); r < 16 * blockIdx.y + 16; r += 8) {
    const int R = 128 * rt + r, i = R / p.gqa;
    if (i >= dl) return;
    const float* part = p.part + size_t(r) * kPart;
    constexpr size_t kSlot = 128 * kPart;
    float M = -INFINITY;
    for (int c = c0 + lane; c <= c1; c += 32) M = fmaxf(M, __ldcg(part + size_t(2 * c + (c == c0)) * kSlot + 128));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, off));
    float l = 0.0f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int c = c0; c <= c1; ++c) {
      const float* pc = part + size_t(2 * c + (c == c0)) * kSlot;
      const float f = M == -INFINITY ? 0.0f : ex2(__ldcg(pc + 128) - M);
      const float4 x = __ldcg(reinterpret_cast<const float4*>(pc) + lane);
      l = fmaf(f, __ldcg(pc + 129), l);
      o.x = fmaf(f, x.x, o.x);
      o.y = fmaf(f, x.y, o.y);
      o.z = fmaf(f, x.z, o.z);
      o.w = fmaf(f, x.w, o.w);
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    const size_t row = (size_t(b) * p.T + i) * p.Hq + h * p.gqa + (R - i * p.gqa);
    reinterpret_cast<float4*>(p.out + row * kHeadDim)[lane] = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  }
}

template <typename T, int KB>
cudaError_t launch_t(const TreeParams& p, cudaStream_t stream) {
  static int seen[64];
  const int bytes = int(kRec + rec_stages(KB) * uint32_t(128 / p.P) * p.L.record);
  cudaError_t e = ensure_dynamic_smem(tree_kernel<T, KB>, bytes, seen);
  if (e != cudaSuccess) return e;
  // the register split waits for good on a build that launches with fewer registers
  static int regs;
  int r = __atomic_load_n(&regs, __ATOMIC_ACQUIRE);
  if (r == 0) {
    cudaFuncAttributes a;
    e = cudaFuncGetAttributes(&a, tree_kernel<T, KB>);
    if (e != cudaSuccess) return e;
    r = a.numRegs;
    __atomic_store_n(&regs, r, __ATOMIC_RELEASE);
  }
  if (r < kRegsLaunch) return cudaErrorInvalidConfiguration;
  e = launch_pdl(tree_kernel<T, KB>, dim3(p.n_ctas), dim3(kThreads), size_t(bytes), stream, p);
  if (e != cudaSuccess || p.n_ctas < 2) return e;
  return launch_pdl(merge_kernel, dim3(p.n_ctas - 1, 8), dim3(256), 0, stream, p);
}

template <typename T>
cudaError_t launch(const TreeParams& p, cudaStream_t stream) {
  switch (p.k / 16) {
    case 0: return launch_t<T, 0>(p, stream);
    case 1: return launch_t<T, 1>(p, stream);
    case 2: return launch_t<T, 2>(p, stream);
    case 4: return launch_t<T, 4>(p, stream);
    case 8: return launch_t<T, 8>(p, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace tree
}  // namespace kvq
