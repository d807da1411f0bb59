// The matrix products behind the cross entropy of an output head, for gfx950:
//   logits  z = H · W^T           (tile of z never leaves the workgroup: it becomes
//                                  softmax statistics, or the gradient G in bf16)
//   dH      = G · W               (split over the vocabulary, float32 partial sums)
//   dW      = G^T · H
// One main loop serves all three.  Four waves (one per SIMD) share a tile through LDS;
// each computes TA x TB MFMA tiles of 32 x 32 (v_mfma_f32_32x32x16_bf16), 64 deep per
// step.  Both operands go from memory straight into LDS (buffer_load ... lds, 16 bytes
// per lane) in a ring of stages.  An operand is stored in one of two ways:
//   rows   k runs along memory: a stage is [rows][64 k] in 128-byte rows whose 16-byte
//          chunks are XOR-swizzled by row; a fragment (8 consecutive k of one row) is
//          one 16-byte read;
//   cols   the tile's own index runs along memory: a stage is [64 k][cols] as it is,
//          whose 64-byte units are XOR-swizzled by k % 4; a fragment is two transposing
//          reads (ds_read_b64_tr_b16), whose 32-lane phases name 4 rows k of one unit
//          and so cover the 64 banks once.
// Within a step lane group g = lane / 32 owns k in [32 g, 32 g + 32) and MFMA group kk
// takes k = 32 g + 8 kk + 0..7 for both operands.  The fragments of group kk + 1 are
// read while group kk's MFMAs run.  One barrier per step, after the third group: by then
// the step's last fragments are read, so its slot takes the copy S stages ahead, and the
// fourth group's MFMAs cover those copies and the next step's first reads.
// Rows past an operand's end read as zero (buffer bounds).

#include "loss.h"

#include "gemm.h"

#include <type_traits>

namespace ql {
namespace {

typedef short ls16x4 __attribute__((ext_vector_type(4)));

QL_DEV __amdgpu_buffer_rsrc_t lrsrc(const void *base, int64_t bytes) {
  const int64_t cap = 0x7FFFFFF0;
  const int32_t n = (int32_t)(bytes < 0 ? 0 : (bytes > cap ? cap : bytes));
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, n, 0x00020000);
}
QL_DEV f32x16 lmfma(u32x4 a, u32x4 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                0, 0);
}
// (device functions, not builtins inline in a kernel template's lambda, where the host
// pass of this compiler drops the kernel's launch stub)
QL_DEV void lload_lds(__amdgpu_buffer_rsrc_t r, uint16_t *dst, int voff, int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)dst, 16, voff, soff, 0, 0);
}
QL_DEV u32x4 ltr_pair(const uint16_t *lo, const uint16_t *hi) {
  typedef __attribute__((address_space(3))) ls16x4 lds_s16x4;
  const ls16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(lo));
  const ls16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(hi));
  const u32x2 ua = __builtin_bit_cast(u32x2, a), ub = __builtin_bit_cast(u32x2, b);
  return u32x4{ua[0], ua[1], ub[0], ub[1]};
}
// Workgroup barrier without the fences of __syncthreads(), which would wait for the
// copies in flight; the loop waits for what it needs itself.
QL_DEV void lbarrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

constexpr int kThreads = 256;
constexpr int kBK = 64;

// An operand stored in rows: R rows of the tile, k along memory.  `base`: the tile's
// first row, `bytes`: from there to the operand's end.
template <int R>
struct RowOperand {
  static constexpr int kElems = R * kBK;
  static constexpr int kCopies = R / 32;  // 1 KB copies (8 rows) per wave and stage
  static_assert(kCopies == 1 || kCopies % 2 == 0, "the swizzle of a copy depends on its parity");
  __amdgpu_buffer_rsrc_t rsrc;
  int voff[2], step;
  int frag;  // element offset of the lane's row in a stage
  int swz;
  QL_DEV void init(const uint16_t *base, int64_t ld, int64_t bytes, int lane, int wv, int first_row) {
    rsrc = lrsrc(base, bytes);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int r = 8 * (wv * kCopies + c) + (lane >> 3), lc = (lane & 7) ^ ((r >> 1) & 7);
      voff[c] = (int)((r * ld + lc * 8) * 2);
    }
    step = __builtin_amdgcn_readfirstlane((int)(8 * ld * 2));
    const int r = first_row + (lane & 31);  // the tile rows are multiples of 32, so row % 16 is the lane's
    frag = r * kBK;
    swz = (r >> 1) & 7;
  }
  QL_DEV void copy(uint16_t *stage, int wv, int kt_) const {
    const int kt = __builtin_amdgcn_readfirstlane(kt_);
#pragma unroll
    for (int c = 0; c < kCopies; ++c)
      lload_lds(rsrc, stage + (wv * kCopies + c) * 512, voff[c & 1], kt * kBK * 2 + (c & ~1) * step);
  }
  QL_DEV u32x4 read(const uint16_t *stage, int lane, int t, int kk) const {
    return *reinterpret_cast<const u32x4 *>(stage + frag + t * 32 * kBK + (((4 * (lane >> 5) + kk) ^ swz) << 3));
  }
};

// An operand stored in columns: C columns of the tile along memory, k down the rows.
template <int C>
struct ColOperand {
  static constexpr int kElems = C * kBK;
  static constexpr int kCopies = C / 32;
  static constexpr int kPerCopy = 512 / C;        // rows k per 1 KB copy
  static constexpr int kLanes = 64 / kPerCopy;    // lanes (16-byte chunks) per row
  const uint16_t *base;
  int64_t ld, bytes;
  int voff[2], step;
  int frag, frag2;  // element offsets of the lane's unit for tiles of even and odd index
  QL_DEV void init(const uint16_t *b, int64_t l, int64_t n, int lane, int wv, int first_col) {
    base = b, ld = l, bytes = n;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int k = kPerCopy * (wv * kCopies + c) + lane / kLanes, pc = lane % kLanes;
      const int lc = (((pc >> 2) ^ (k & 3)) << 2) | (pc & 3);
      voff[c] = (int)((k * ld + lc * 8) * 2);
    }
    step = __builtin_amdgcn_readfirstlane((int)(kPerCopy * ld * 2));
    const int c = lane & 15, half = (lane >> 4) & 1, g = lane >> 5;
    frag = (32 * g + (c >> 2)) * C + 16 * half + 4 * (c & 3);
    frag2 = ((first_col >> 5) ^ (c >> 2));
  }
  QL_DEV void copy(uint16_t *stage, int wv, int kt_) const {
    const int kt = __builtin_amdgcn_readfirstlane(kt_);
    const int64_t at = (int64_t)kt * kBK * ld;
    const auto r = lrsrc(base + at, bytes - at * 2);
#pragma unroll
    for (int c = 0; c < kCopies; ++c)
      lload_lds(r, stage + (wv * kCopies + c) * 512, voff[c & 1], (c & ~1) * step);
  }
  // the first column's unit is a multiple of the wave's TA or TB (a power of two), so
  // unit + t is unit ^ t and the swizzle of tile t is the lane's with t XORed in
  QL_DEV u32x4 read(const uint16_t *stage, int, int t, int kk) const {
    const uint16_t *lo = stage + frag + 8 * kk * C + ((frag2 ^ t) << 5);
    return ltr_pair(lo, lo + 4 * C);
  }
};

// acc[i][j] += sum over nk steps of A tile i times B tile j.  S slots of OpA::kElems +
// OpB::kElems elements at `ring`.
template <int S, int TA, int TB, typename OpA, typename OpB>
QL_DEV void product(const OpA &A, const OpB &B, uint16_t *ring, int nk, int lane, int wv, f32x16 (&acc)[TA][TB]) {
  constexpr int kStage = OpA::kElems + OpB::kElems;
  constexpr int NC = OpA::kCopies + OpB::kCopies;
  constexpr int kReadsA = std::is_same_v<OpA, RowOperand<OpA::kElems / kBK>> ? 1 : 2;
  constexpr int kReadsB = std::is_same_v<OpB, RowOperand<OpB::kElems / kBK>> ? 1 : 2;
  constexpr int NM = TA * TB, NR = TA * kReadsA + TB * kReadsB;
  u32x4 fa[2][TA], fb[2][TB];
  auto copy = [&](int kt, int slot) {
    A.copy(ring + slot * kStage, wv, kt);
    B.copy(ring + slot * kStage + OpA::kElems, wv, kt);
  };
  auto read = [&](int slot, int kk, int set) {
#pragma unroll
    for (int i = 0; i < TA; ++i) fa[set][i] = A.read(ring + slot * kStage, lane, i, kk);
#pragma unroll
    for (int j = 0; j < TB; ++j) fb[set][j] = B.read(ring + slot * kStage + OpA::kElems, lane, j, kk);
  };
  // vmcnt(n) and lgkmcnt(0)
  auto wait = [](auto nconst) {
    constexpr int n = decltype(nconst)::value;
    __builtin_amdgcn_s_waitcnt((n & 15) | (7 << 4) | ((n >> 4) << 14));
  };
#pragma unroll
  for (int s = 0; s < S; ++s) copy(s, s);
  __builtin_amdgcn_sched_barrier(0);
  wait(std::integral_constant<int, (S - 1) * NC>{});  // stage 0's copies
  lbarrier();
  __builtin_amdgcn_sched_barrier(0);
  read(0, 0, 0);
  auto step = [&](auto slotc, int kt) {
    constexpr int SLOT = decltype(slotc)::value;
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      if (kk < 3) {
        read(SLOT, kk + 1, (kk + 1) & 1);
      } else {
        copy(kt + S, SLOT);
        read((SLOT + 1) % S, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < TA; ++i)
#pragma unroll
        for (int j = 0; j < TB; ++j) acc[i][j] = lmfma(fa[kk & 1][i], fb[kk & 1][j], acc[i][j]);
#pragma unroll
      for (int i = 0; i < NM; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                                          // MFMA
        if (kk == 3 && i < NC) __builtin_amdgcn_sched_group_barrier(0x010, (NC + NM - 1) / NM, 0);  // VMEM
        __builtin_amdgcn_sched_group_barrier(0x100, (NR + NM - 1) / NM, 0);                         // LDS read
      }
      __builtin_amdgcn_sched_barrier(0);
      if (kk == 2) {
        // this wave's copies of stage kt + 1 (S - 2 younger stages may be in flight) and
        // its reads of this slot; with that in every wave, stage kt + 1 is whole and the
        // slot is free
        wait(std::integral_constant<int, (S - 2) * NC>{});
        lbarrier();
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  int kt = 0;
  for (; kt + S - 1 < nk; kt += S) {
    step(std::integral_constant<int, 0>{}, kt);
    step(std::integral_constant<int, 1>{}, kt + 1);
    if constexpr (S > 2) step(std::integral_constant<int, 2 % S>{}, kt + 2);
    if constexpr (S > 3) step(std::integral_constant<int, 3 % S>{}, kt + 3);
  }
  if (kt < nk) step(std::integral_constant<int, 0>{}, kt);
  if constexpr (S > 2)
    if (kt + 1 < nk) step(std::integral_constant<int, 1>{}, kt + 1);
  if constexpr (S > 3)
    if (kt + 2 < nk) step(std::integral_constant<int, 2>{}, kt + 2);
  __builtin_amdgcn_s_waitcnt(0);  // no copy of a stage past the end may still land in LDS
  __syncthreads();
}

template <int TA, int TB>
QL_DEV void clear(f32x16 (&acc)[TA][TB]) {
#pragma unroll
  for (int i = 0; i < TA; ++i)
#pragma unroll
    for (int j = 0; j < TB; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
}

constexpr int lmax(int a, int b) { return a > b ? a : b; }

// the row of accumulator element v in its 32 x 32 tile
QL_DEV int acc_row(int v, int g) { return 8 * (v >> 2) + 4 * g + (v & 3); }

}  // namespace

// Logits of a tile of BV vocabulary rows x BT tokens, WV x (4 / WV) waves.  The
// vocabulary is on the MFMA's rows, so most of a token's values are in one lane and
// its softmax statistics need one exchange between lanes.
// GRAD false: part[tile][token] = (max, sum of exp(z - max)) over the tile's rows, and
// zlab of the tokens whose label is among them.
// GRAD true: G[token][v] = bf16((exp(z - lse) - [v is the label]) * (dloss / top)).
template <int BV, int BT, int WV, int S, bool GRAD>
__global__ __launch_bounds__(kThreads) void head_logits_kernel(LogitParams p) {
  constexpr int WT = 4 / WV, TA = BV / WV / 32, TB = BT / WT / 32;
  constexpr int kRing = S * (BV + BT) * kBK;       // elements
  constexpr int kLdg = BV + 8;                     // staging of G: [token][BV]
  constexpr int kBytes = lmax(kRing * 2, GRAD ? BT * kLdg * 2 : WV * BT * 8);
  __shared__ __attribute__((aligned(16))) char lds[kBytes];
  uint16_t *ring = reinterpret_cast<uint16_t *>(lds);
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 5, l32 = lane & 31;
  const int n = *p.count;
  const int tiles_t = (n + BT - 1) / BT;
  if ((int64_t)blockIdx.x >= (int64_t)tiles_t * p.tiles_v) return;
  int tv, tt;
  gemm_tile_of(blockIdx.x, p.tiles_v, tiles_t, 4, tv, tt);
  const int64_t v0 = (int64_t)tv * BV, t0 = (int64_t)tt * BT;
  const int wa = wv / WT * (BV / WV), wb = wv % WT * (BT / WT);  // the wave's first row and column
  RowOperand<BV> A;
  RowOperand<BT> B;
  A.init(p.W + v0 * p.h, p.h, (p.nvoc - v0) * p.h * 2, lane, wv, wa);
  B.init(p.H + t0 * p.h, p.h, ((int64_t)n - t0) * p.h * 2, lane, wv, wb);
  f32x16 acc[TA][TB];
  clear(acc);
  product<S, TA, TB>(A, B, ring, (int)(p.h / kBK), lane, wv, acc);

  const int rows = (int)(p.nvoc - v0 < BV ? p.nvoc - v0 : BV);  // vocabulary rows of this tile
  if constexpr (!GRAD) {
    f32x2 *red = reinterpret_cast<f32x2 *>(lds);  // [WV][BT]
#pragma unroll
    for (int j = 0; j < TB; ++j) {
      const int64_t t = t0 + wb + 32 * j + l32;
      // the label's row in this tile (none: a row that no lane has)
      const int64_t lab = t < n ? (int64_t)p.label[t] - p.v0 - v0 : -1;
      float mx = -__builtin_inff();
#pragma unroll
      for (int i = 0; i < TA; ++i)
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const int row = wa + 32 * i + acc_row(v, g);
          if (row == lab) p.zlab[t] = acc[i][j][v];
          if (row >= rows) acc[i][j][v] = -__builtin_inff();
          mx = fmaxf(mx, acc[i][j][v]);
        }
      mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
      // a wave whose rows are all past the vocabulary has no maximum: its sum is 0
      const float top = mx == -__builtin_inff() ? 0.0f : mx;
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < TA; ++i)
#pragma unroll
        for (int v = 0; v < 16; ++v) s += __expf(acc[i][j][v] - top);
      s += __shfl_xor(s, 32, 64);
      if (g == 0) red[wv / WT * BT + wb + 32 * j + l32] = f32x2{mx, s};
    }
    __syncthreads();
    if (threadIdx.x < BT) {
      const int64_t t = t0 + threadIdx.x;
      f32x2 a = red[threadIdx.x];  // rows 0.. of the tile: never empty
#pragma unroll
      for (int w = 1; w < WV; ++w) {
        const f32x2 b = red[w * BT + threadIdx.x];
        const float m = fmaxf(a[0], b[0]);
        a = f32x2{m, a[1] * __expf(a[0] - m) + b[1] * __expf(b[0] - m)};
      }
      if (t < n) p.part[(int64_t)tv * p.ldp + t] = a;
    }
  } else {
    uint16_t *cs = reinterpret_cast<uint16_t *>(lds);
    const float top = *p.top;
#pragma unroll
    for (int j = 0; j < TB; ++j) {
      const int col = wb + 32 * j + l32;
      const int64_t t = t0 + col;
      const bool live = t < n;
      const float lse = live ? p.lse[t] : 0.0f, dl = live && top > 0.0f ? p.dloss[t] / top : 0.0f;
      const int64_t lab = live ? (int64_t)p.label[t] - p.v0 - v0 : -1;
#pragma unroll
      for (int i = 0; i < TA; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int row = wa + 32 * i + 8 * q + 4 * g + e;
            const float pr = __expf(acc[i][j][4 * q + e] - lse);
            o[e] = row < rows ? (row == lab ? pr - 1.0f : pr) * dl : 0.0f;
          }
          *reinterpret_cast<u32x2 *>(cs + col * kLdg + wa + 32 * i + 8 * q + 4 * g) =
              u32x2{pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3])};
        }
    }
    __syncthreads();
    for (int ch = threadIdx.x; ch < BT * BV / 8; ch += kThreads) {
      const int col = ch / (BV / 8), c8 = ch % (BV / 8);
      if (t0 + col < n)
        *reinterpret_cast<u32x4 *>(p.G + (t0 + col) * p.ldg + v0 + c8 * 8) =
            *reinterpret_cast<const u32x4 *>(cs + col * kLdg + c8 * 8);
    }
  }
}

// dH partial sums: part[split][token][k] (+)= sum over the split's vocabulary entries v
// of G[token][v] W[v][k].  G's columns past the piece are zero and W's rows past it read
// as zero, so the last step may be short.
template <int BM, int S>
__global__ __launch_bounds__(kThreads) void head_dh_kernel(HeadGradParams p) {
  constexpr int BN = 256, WM = BM == 256 ? 2 : 1, WN = 4 / WM;
  constexpr int TA = BM / WM / 32, TB = BN / WN / 32;
  __shared__ __attribute__((aligned(16))) uint16_t ring[S * (BM + BN) * kBK];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 5, l32 = lane & 31;
  const int n = *p.count;
  const int tiles_m = (n + BM - 1) / BM;
  if ((int)blockIdx.x >= tiles_m * p.tiles_n) return;
  int tm, tn;
  gemm_tile_of(blockIdx.x, tiles_m, p.tiles_n, 4, tm, tn);
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
  const int64_t k0 = (int64_t)blockIdx.y * p.kper;
  const int64_t k1 = k0 + p.kper < p.nvoc ? k0 + p.kper : p.nvoc;
  const int wa = wv / WN * (BM / WM), wb = wv % WN * (BN / WN);
  RowOperand<BM> A;
  ColOperand<BN> B;
  A.init(p.G + m0 * p.ldg + k0, p.ldg, ((int64_t)n - m0) * p.ldg * 2 - k0 * 2, lane, wv, wa);
  B.init(p.W + k0 * p.h + n0, p.h, (p.nvoc - k0) * p.h * 2 - n0 * 2, lane, wv, wb);
  f32x16 acc[TA][TB];
  clear(acc);
  product<S, TA, TB>(A, B, ring, (int)((k1 - k0 + kBK - 1) / kBK), lane, wv, acc);
  float *out = p.part + (int64_t)blockIdx.y * p.rows * p.h;
#pragma unroll
  for (int i = 0; i < TA; ++i)
#pragma unroll
    for (int j = 0; j < TB; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        const int64_t m = m0 + wa + 32 * i + acc_row(v, g), c = n0 + wb + 32 * j + l32;
        if (m >= n || c >= p.h) continue;
        float *dst = out + m * p.h + c;
        *dst = p.add ? *dst + acc[i][j][v] : acc[i][j][v];
      }
}

// dW[v][k] = bf16(top * sum over the tokens of G[token][v] H[token][k]).
template <int S>
__global__ __launch_bounds__(kThreads) void head_dw_kernel(HeadGradParams p) {
  constexpr int BM = 256, BN = 256, TA = 4, TB = 4, kLdc = BN + 8;
  constexpr int kBytes = lmax(S * (BM + BN) * kBK * 2, BM * kLdc * 2);
  __shared__ __attribute__((aligned(16))) char lds[kBytes];
  uint16_t *ring = reinterpret_cast<uint16_t *>(lds);
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 5, l32 = lane & 31;
  const int n = *p.count;
  int tm, tn;
  gemm_tile_of(blockIdx.x, p.tiles_m, p.tiles_n, 4, tm, tn);
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
  const int wa = wv / 2 * 128, wb = wv % 2 * 128;
  ColOperand<BM> A;
  ColOperand<BN> B;
  A.init(p.G + m0, p.ldg, (int64_t)n * p.ldg * 2 - m0 * 2, lane, wv, wa);
  B.init(p.H + n0, p.h, (int64_t)n * p.h * 2 - n0 * 2, lane, wv, wb);
  f32x16 acc[TA][TB];
  clear(acc);
  product<S, TA, TB>(A, B, ring, (n + kBK - 1) / kBK, lane, wv, acc);
  uint16_t *cs = reinterpret_cast<uint16_t *>(lds);
  const float top = n > 0 ? *p.top : 0.0f;
#pragma unroll
  for (int i = 0; i < TA; ++i)
#pragma unroll
    for (int j = 0; j < TB; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v)
        cs[(wa + 32 * i + acc_row(v, g)) * kLdc + wb + 32 * j + l32] =
            (uint16_t)(pack_bf16x2(top * acc[i][j][v], 0.0f) & 0xFFFFu);
  __syncthreads();
  for (int ch = threadIdx.x; ch < BM * BN / 8; ch += kThreads) {
    const int row = ch / (BN / 8), c8 = ch % (BN / 8);
    const int64_t m = m0 + row, c = n0 + c8 * 8;
    if (m < p.nvoc && c < p.h)
      *reinterpret_cast<u32x4 *>(p.dW + m * p.h + c) = *reinterpret_cast<const u32x4 *>(cs + row * kLdc + c8 * 8);
  }
}

namespace {
inline int64_t cdiv(int64_t x, int64_t m) { return (x + m - 1) / m; }
}  // namespace

int logit_tile_v(int64_t max_tokens) { return max_tokens <= 128 ? 128 : 256; }

hipError_t launch_logit_stats(LogitParams &p, int64_t max_tokens, hipStream_t st) {
  p.tiles_v = (int)cdiv(p.nvoc, logit_tile_v(max_tokens));
  if (max_tokens <= 32) return launch(head_logits_kernel<128, 32, 4, 4, false>, (unsigned)p.tiles_v, kThreads, st, p);
  if (max_tokens <= 128)
    return launch(head_logits_kernel<128, 128, 2, 2, false>, (unsigned)p.tiles_v, kThreads, st, p);
  return launch(head_logits_kernel<256, 256, 2, 2, false>, (unsigned)(p.tiles_v * cdiv(max_tokens, 256)), kThreads, st,
                p);
}

hipError_t launch_logit_grad(LogitParams &p, int64_t max_tokens, hipStream_t st) {
  if (max_tokens <= 32) {
    p.tiles_v = (int)cdiv(p.nvoc, 128);
    return launch(head_logits_kernel<128, 32, 4, 4, true>, (unsigned)p.tiles_v, kThreads, st, p);
  }
  if (max_tokens <= 128) {
    p.tiles_v = (int)cdiv(p.nvoc, 128);
    return launch(head_logits_kernel<128, 128, 2, 2, true>, (unsigned)p.tiles_v, kThreads, st, p);
  }
  p.tiles_v = (int)cdiv(p.nvoc, 256);
  return launch(head_logits_kernel<256, 256, 2, 2, true>, (unsigned)(p.tiles_v * cdiv(max_tokens, 256)), kThreads, st,
                p);
}

hipError_t launch_head_dh(HeadGradParams &p, int splits, int64_t max_tokens, hipStream_t st) {
  p.tiles_n = (int)cdiv(p.h, 256);
  if (max_tokens <= 64)
    return launch(head_dh_kernel<64, 2>, dim3((unsigned)(cdiv(max_tokens, 64) * p.tiles_n), (unsigned)splits), kThreads,
                  st, p);
  return launch(head_dh_kernel<256, 2>, dim3((unsigned)(cdiv(max_tokens, 256) * p.tiles_n), (unsigned)splits), kThreads,
                st, p);
}

hipError_t launch_head_dw(HeadGradParams &p, hipStream_t st) {
  p.tiles_m = (int)cdiv(p.nvoc, 256);
  p.tiles_n = (int)cdiv(p.h, 256);
  return launch(head_dw_kernel<2>, (unsigned)(p.tiles_m * p.tiles_n), kThreads, st, p);
}

}  // namespace ql
