// Attention of new tokens over a paged K/V cache, for few query rows a K/V head: single
// tokens, proposed tokens, short chunks, and every fp32 call.
//
//   out[r] = sum_j p_rj V_j / sum_j p_rj,  p_rj = 2^(s_rj - m_r),
//   s_rj = scale * log2(e) * q_r . K_j  over the keys j that row r may see,
//
// in one pass with the running reference m_r. Bound by memory: K and V are read once for
// the 16 query rows of a tile (query heads of one K/V head times new tokens; 32 in fp32
// chunks). 64 single tokens over 4400 keys of 8 heads of 128 channels, 4 query heads each:
// 181 us, 6.5 TB/s; one token over 262144 keys of 4 heads of 64: 56 us, of which some 16 are
// start, merge and imbalance; 5 fp32 tokens in each of 16 sequences: 38 us, 3.6 TB/s, in 64
// sequences 133 us, 4.3 TB/s: two warps a scheduler wait for each other's products.
//
// A warp takes 16 keys a step, which it streams into a ring of its own in shared memory
// (cp.async, two or three steps; no barrier but the warp's), and multiplies on the tensor cores
// with m16n8k16 products. A product does not care which channel carries which index as long
// as both operands agree, so operands are read 16 bytes a lane: lane (g, t) of the K operand
// takes 16 consecutive bytes of key g, the query operand being laid out to match, and for
// P.V lane (g, t) takes 16 consecutive bytes of keys 2t and 2t + 1 and pairs them up by byte
// permutes. The 16-byte pieces of a row are stored permuted so that both reads are free of
// bank conflicts.
//
// Rounding: fp32 values enter the products as sums of three bf16 parts (8 + 8 + 8 bits,
// by truncation, so exactly), of whose products the six largest are taken: what is left
// out (second by third part both ways, third by third) is below 2^-21 of a term. With bf16 tensors q, K and V are exact as they are and the
// probabilities keep two parts (16 bits), which leaves the output's own rounding as the
// only one that shows. Sums, references and accumulators are fp32. The products round their
// running sums towards zero; in fp32, where that would show (2e-6 of the result after 100
// steps, against 4e-7), each step's products start from zero, smallest first, and are added
// to the sums by ordinary additions.
#include <cuda_bf16.h>

#include <cmath>

#include "paged.cuh"
#include "paged_work.cuh"
#include "ptx.cuh"

namespace cxa {
namespace {

constexpr int kRows = 16;            // query rows of a product
constexpr int kStep = 16;            // keys a warp takes at a time
constexpr int kMaxBlocks = kRowsMaxBlocks;
// Parts of an item that are merged at once, and then of those. One token over 262144 keys: 8 at a
// time 55.7 us, 6 55.7, 10 56.5, 16 57.1.
constexpr int kGroup = 8;
constexpr int kMaxParts = (kMaxBlocks + kGroup - 1) / kGroup;
constexpr int kWideItems = 1;        // items an SM below which wide blocks run (see launch)
constexpr float kMoveLog2 = 8.f;     // a row's reference moves only past this margin

struct RowsParams {
  const void* q;
  void* out;
  long long q_stride, o_stride;
  float qscale;                      // scale * log2(e)
  unsigned int* counters;            // [grid][3], zero between calls
  float* part;                       // [2 * grid][rows of a tile][kDh + 2]
  unsigned int* status;
  PagedBatch batch;
  PagedLayer layer;
  WorkShape shape;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

// The high halves of two words: (lo's, hi's) as a bf16 pair, that is, both truncated.
__device__ __forceinline__ uint32_t high_halves(uint32_t lo, uint32_t hi) { return __byte_perm(lo, hi, 0x7632); }
__device__ __forceinline__ uint32_t low_halves(uint32_t lo, uint32_t hi) { return __byte_perm(lo, hi, 0x5410); }

// A pair of fp32 values as N bf16 pairs that add up to them (exactly, for N = 3).
template <int N>
__device__ __forceinline__ void split_pair(float a, float b, uint32_t (&w)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
    w[i] = high_halves(ua, ub);
    a -= __uint_as_float(ua & 0xFFFF0000u);
    b -= __uint_as_float(ub & 0xFFFF0000u);
  }
}

__device__ __forceinline__ bool nonfinite(uint32_t w, bool bf16_pair) {
  if (bf16_pair) return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
  return (w & 0x7F800000u) == 0x7F800000u;
}

template <typename TQ, typename TP, int kDh, bool kWide, int kMt>
struct Shape {
  static constexpr int rows = kMt * kRows;         // query rows a tile
  static constexpr bool q32 = sizeof(TQ) == 4, p32 = sizeof(TP) == 4;
  static constexpr int QP = q32 ? 3 : 1;           // bf16 parts of a query value,
  static constexpr int KP = p32 ? 3 : 1;           // of a K or V value
  static constexpr int PP = q32 ? 3 : 2;           // and of a probability
  static constexpr int KS = kDh / 16;              // products along a head
  static constexpr int NB = kDh / 8;               // accumulator blocks of 8 channels
  static constexpr int row_bytes = kDh * static_cast<int>(sizeof(TP));
  static constexpr int KV = row_bytes / 64;        // 16-byte loads of a lane along a K row
  static constexpr int VV = row_bytes / 128;       // and along a V row
  static constexpr int PE = kDh + 4;               // floats of a row in the block's merge
  static constexpr int half_bytes = kStep * row_bytes;     // K or V of a step
  // One block of many warps an SM (kWide), or several of four; a chunk is a step of each
  // warp. The rings hold three steps a warp, and as many warps run as that leaves room for; two
  // of the 8 KB steps of fp32 rows of 64 channels do (5 tokens in each of 16 sequences: 37.6 us,
  // three steps 38.5; two steps and half as many warps again, whose registers spill: 40.3).
  static constexpr int stages = p32 && kDh == 64 && kMt == 1 ? 2 : 3;
  static constexpr int warps_sm = kMt > 1 && row_bytes <= 128 ? 8 : 2048 / row_bytes;
  static constexpr int warps = kWide ? warps_sm : 4, blocks = warps_sm / warps, threads = warps * 32;
  static constexpr int chunk_shift = warps == 16 ? 8 : warps == 8 ? 7 : 6;
  static constexpr int ring_bytes = warps * stages * 2 * half_bytes;
  static constexpr int q_bytes = kMt * QP * KS * 32 * 16;
  static constexpr int merge_bytes = warps * rows * PE * 4 + 2 * warps * rows * 4;
  static_assert(2 * kMaxParts * rows * 4 <= merge_bytes, "the weights of a merge fit");
  static constexpr int smem = q_bytes + (ring_bytes > merge_bytes ? ring_bytes : merge_bytes);
};

// Where the 16-byte piece c of row r of a step lies.
__device__ __forceinline__ int k_piece(int r, int c) { return c ^ ((r & 1) << 2); }
__device__ __forceinline__ int v_piece(int r, int c) { return c ^ ((r >> 1 & 3) << 1); }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// B operand of product s along a head from a lane's K loads.
template <typename S>
__device__ __forceinline__ void k_operand(const uint4 (&k)[S::KV], int s, uint32_t (&b)[S::KP][2]) {
  if constexpr (S::p32) {
    uint32_t w[3];
    split_pair<3>(__uint_as_float(k[s].x), __uint_as_float(k[s].y), w);
#pragma unroll
    for (int i = 0; i < 3; ++i) b[i][0] = w[i];
    split_pair<3>(__uint_as_float(k[s].z), __uint_as_float(k[s].w), w);
#pragma unroll
    for (int i = 0; i < 3; ++i) b[i][1] = w[i];
  } else {
    const uint4& u = k[s >> 1];
    b[0][0] = (s & 1) ? u.z : u.x;
    b[0][1] = (s & 1) ? u.w : u.y;
  }
}

// sum += A B over the parts of both, smallest products first; with kApart added up by
// themselves.
template <bool kApart, int NA, int NB>
__device__ __forceinline__ void add_products(float (&sum)[4], const uint4 (&a)[NA], const uint32_t (&b)[NB][2]) {
  float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int order = 2; order >= 0; --order)
#pragma unroll
    for (int i = 0; i < NA; ++i)
      if (order - i >= 0 && order - i < NB) mma_16816(kApart ? d : sum, a[i], b[order - i][0], b[order - i][1]);
  if (kApart) {
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[i] += d[i];
  }
}

__device__ __forceinline__ uint32_t word(const uint4& u, int i) {
  return i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w;
}

// B operand of accumulator block c from a lane's V loads of its four keys.
template <typename S>
__device__ __forceinline__ void v_operand(const uint4 (&v)[4][S::VV], int c, uint32_t (&b)[S::KP][2]) {
  if constexpr (S::p32) {
    const int p = c / 4, e = c % 4;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t w[3];
      split_pair<3>(__uint_as_float(word(v[2 * j][p], e)), __uint_as_float(word(v[2 * j + 1][p], e)), w);
#pragma unroll
      for (int i = 0; i < 3; ++i) b[i][j] = w[i];
    }
  } else {
    const int p = c / 8, e = c % 8;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t x = word(v[2 * j][p], e / 2), y = word(v[2 * j + 1][p], e / 2);
      b[0][j] = (e & 1) ? high_halves(x, y) : low_halves(x, y);
    }
  }
}

template <typename TQ, typename TP, int kDh, bool kWide, int kMt>
__global__ void __launch_bounds__(Shape<TQ, TP, kDh, kWide, kMt>::threads, Shape<TQ, TP, kDh, kWide, kMt>::blocks)
    paged_rows_kernel(const __grid_constant__ RowsParams p) {
  using S = Shape<TQ, TP, kDh, kWide, kMt>;
  constexpr int kWarps = S::warps, kThreads = S::threads, kTile = S::rows;
  extern __shared__ __align__(1024) uint8_t smem[];   // rows of the rings fill whole bank lines
  __shared__ WorkScratch s_work;
  __shared__ int s_last;
  uint4* s_q = reinterpret_cast<uint4*>(smem);                             // [kMt][QP][KS][32 lanes]
  // the warps' rings, and once they have run dry the merge of the warps' states
  const uint32_t ring = smem_u32(smem) + S::q_bytes + (threadIdx.x >> 5) * (S::stages * 2 * S::half_bytes);
  float* s_o = reinterpret_cast<float*>(smem + S::q_bytes);                // [kWarps][rows][PE]
  float* s_m = s_o + kWarps * kTile * S::PE;                               // [kWarps][rows]
  float* s_l = s_m + kWarps * kTile;
  float* s_w = s_o;                                                        // [2][kMaxParts][rows], in a merge

  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const PagedBatch& bt = p.batch;
  const int Hkv = p.layer.Hkv, shift = p.layer.page_shift, G = p.shape.G;
  WorkRange range;
  WorkCursor cur;
  WorkShape shape = p.shape;
  if (!work_locate<kThreads, true>(bt, shape, Hkv, &s_work, &range, &cur, p.status)) return;

  for (;;) {
    // ---- the part of the item in this block's range
    const int end = min(range.g1, cur.first + cur.nc);
    const int c0 = cur.c, c1 = end - cur.first;
    const PagedSeq seq = cur.seq;
    const int row0 = cur.rt * kTile;
    const int rows = min(kTile, work_rows(seq, shape) - row0);
    const int keys = tile_keys(seq, shape, cur.rt);

    // ---- the first steps on their way
    const int* table_row = bt.table + static_cast<size_t>(cur.b) * bt.width;
    const uint8_t* Kb = static_cast<const uint8_t*>(p.layer.K);
    const uint8_t* Vb = static_cast<const uint8_t*>(p.layer.V);
    const int steps = tile_steps(seq, shape, cur.rt);      // of all warps, kWarps * kStep keys
    const int s0 = chunk_step(shape, c0, cur.nc, steps) * kWarps;
    const int s1 = min(chunk_step(shape, c1, cur.nc, steps) * kWarps, (keys + kStep - 1) / kStep);
    auto step_page = [&](int s) {
      if (s >= s1) return 0;
      const int page = paged_lookup(table_row, bt.width, shift, p.layer.num_pages, s * kStep);
      if (page < 0 && lane == 0) atomicOr(p.status, kStatusBadPage);
      return page;
    };
    // Stream step s into stage st: rows that no query sees are not read and become zero (a
    // key that no row sees weighs 0, and its V may hold anything).
    auto fetch = [&](int s, int page, int st) {
      constexpr int PR = S::row_bytes / 16;            // pieces a row
      if (s < s1) {
        const bool there = page >= 0;
        // a step lies in one page
        const size_t at = (((static_cast<size_t>(there ? page : 0) * Hkv + cur.h) << shift) +
                           ((s * kStep) & ((1 << shift) - 1))) * S::row_bytes;
        const uint32_t dst = ring + st * (2 * S::half_bytes);
#pragma unroll
        for (int i = 0; i < kStep * PR / 32; ++i) {
          const int r = (i * 32 + lane) / PR, c = lane % PR;
          const bool real = there && s * kStep + r < keys;
          const size_t from = real ? at + r * S::row_bytes + c * 16 : 0;
          cp_async16(dst + r * S::row_bytes + k_piece(r, c) * 16, Kb + from, real);
          cp_async16(dst + S::half_bytes + r * S::row_bytes + v_piece(r, c) * 16, Vb + from, real);
        }
      }
      cp_commit();
    };

    int s = s0 + warp;
    int pages[S::stages];                              // looked up together, ahead of their use
#pragma unroll
    for (int i = 0; i < S::stages; ++i) pages[i] = step_page(s + i * kWarps);
    uint32_t gone = 0;                                 // steps under way whose page is bad, the newest at bit 0
#pragma unroll
    for (int i = 0; i < S::stages - 1; ++i) {
      fetch(s + i * kWarps, pages[i], i);
      gone = gone << 1 | (pages[i] < 0 ? 1u : 0u);
    }
    int page = pages[S::stages - 1];

    // ---- the queries as A operands: lane (g, t) holds rows g and g + 8, channels to match
    // the K loads
    for (int i = tid; i < kMt * S::KS * 32; i += kThreads) {
      const int mt = i / (S::KS * 32), s = (i >> 5) % S::KS, ql = i & 31, qg = ql >> 2, qt = ql & 3;
      const int ch = S::p32 ? 16 * s + 4 * qt : 32 * (s >> 1) + 8 * qt + 4 * (s & 1);
      uint32_t w[2][2][S::QP];     // [row][pair of channels]
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = mt * kRows + qg + 8 * r;
        const bool ok = row < rows;
        const int tok = (row0 + row) / G, hd = cur.h * G + (row0 + row) % G;
        const TQ* src = static_cast<const TQ*>(p.q) + (ok ? (seq.q0 + tok) * p.q_stride + hd * kDh + ch : 0);
        if constexpr (S::q32) {
          const float4 f = ok ? *reinterpret_cast<const float4*>(src) : make_float4(0.f, 0.f, 0.f, 0.f);
          split_pair<S::QP>(f.x, f.y, w[r][0]);
          split_pair<S::QP>(f.z, f.w, w[r][1]);
        } else {
          const uint2 u = ok ? *reinterpret_cast<const uint2*>(src) : make_uint2(0u, 0u);
          w[r][0][0] = u.x;
          w[r][1][0] = u.y;
        }
      }
#pragma unroll
      for (int j = 0; j < S::QP; ++j) s_q[(mt * S::QP + j) * S::KS * 32 + i % (S::KS * 32)] = make_uint4(w[0][0][j], w[1][0][j], w[0][1][j], w[1][1][j]);
    }
    // keys that this lane's rows (two a product) may see
    int see[2 * kMt];
#pragma unroll
    for (int r = 0; r < 2 * kMt; ++r) {
      const int row = g + 8 * r;
      see[r] = row < rows ? visible_keys(seq, (row0 + row) / G, shape.cap) : 0;
    }
    const int see_all = visible_keys(seq, row0 / G, shape.cap);   // keys that every row may see
    __syncthreads();

    float m[2 * kMt], l[2 * kMt], o[kMt][S::NB][4];
#pragma unroll
    for (int r = 0; r < 2 * kMt; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
    }
#pragma unroll
    for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
      for (int c = 0; c < S::NB; ++c) o[mt][c][0] = o[mt][c][1] = o[mt][c][2] = o[mt][c][3] = 0.f;

    int st = 0;
    for (; s < s1; s += kWarps) {
      cp_wait<S::stages - 2>();
      __syncwarp();          // the step has come for every lane, and the last one's stage is free
      fetch(s + (S::stages - 1) * kWarps, page, st == 0 ? S::stages - 1 : st - 1);
      gone = gone << 1 | (page < 0 ? 1u : 0u);
      page = step_page(s + S::stages * kWarps);
      const uint8_t* kt = smem + S::q_bytes + (warp * S::stages + st) * (2 * S::half_bytes);
      const uint8_t* vt = kt + S::half_bytes;
      st = st + 1 == S::stages ? 0 : st + 1;
      if (gone >> (S::stages - 1) & 1u) continue;      // a bad page: its keys are left out

      // ---- scores
      float sc[kMt][2][4];
#pragma unroll
      for (int nb = 0; nb < 2; ++nb) {
        uint4 k[S::KV];
#pragma unroll
        for (int v = 0; v < S::KV; ++v)
          k[v] = *reinterpret_cast<const uint4*>(kt + (8 * nb + g) * S::row_bytes + k_piece(8 * nb + g, 4 * v + t) * 16);
#pragma unroll
        for (int mt = 0; mt < kMt; ++mt) sc[mt][nb][0] = sc[mt][nb][1] = sc[mt][nb][2] = sc[mt][nb][3] = 0.f;
#pragma unroll
        for (int ks = 0; ks < S::KS; ++ks) {
          uint32_t b[S::KP][2];
          k_operand<S>(k, ks, b);
#pragma unroll
          for (int mt = 0; mt < kMt; ++mt) {
            uint4 a[S::QP];
#pragma unroll
            for (int i = 0; i < S::QP; ++i) a[i] = s_q[((mt * S::QP + i) * S::KS + ks) * 32 + lane];
            add_products<S::q32, S::QP, S::KP>(sc[mt][nb], a, b);
          }
        }
      }
      const bool masked = s * kStep + kStep > see_all;
#pragma unroll
      for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
        for (int nb = 0; nb < 2; ++nb)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            sc[mt][nb][i] *= p.qscale;
            if (masked && s * kStep + 8 * nb + 2 * t + (i & 1) >= see[2 * mt + (i >> 1)]) sc[mt][nb][i] = -INFINITY;
          }

      // ---- running reference: moved for the whole tile when some row passes the margin
      auto largest = [&](int r) {
        const float(&x)[2][4] = sc[r / 2];
        const int i = 2 * (r & 1);
        return fmaxf(fmaxf(x[0][i], x[0][i + 1]), fmaxf(x[1][i], x[1][i + 1]));
      };
      bool move = false;
#pragma unroll
      for (int r = 0; r < 2 * kMt; ++r) move |= largest(r) > m[r] + kMoveLog2;
      if (__any_sync(0xffffffffu, move)) {
#pragma unroll
        for (int r = 0; r < 2 * kMt; ++r) {
          float mx = largest(r);
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          mx = fmaxf(mx, m[r]);
          const float corr = m[r] == -INFINITY ? 0.f : ex2(m[r] - mx);
          m[r] = mx;
          l[r] *= corr;
#pragma unroll
          for (int c = 0; c < S::NB; ++c) {
            o[r / 2][c][2 * (r & 1)] *= corr;
            o[r / 2][c][2 * (r & 1) + 1] *= corr;
          }
        }
      }
      uint4 pa[kMt][S::PP];
#pragma unroll
      for (int mt = 0; mt < kMt; ++mt) {
        float pr[2][4];
#pragma unroll
        for (int nb = 0; nb < 2; ++nb)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = 2 * mt + (i >> 1);
            const float ref = m[r] == -INFINITY ? 0.f : m[r];             // nothing visible yet
            pr[nb][i] = ex2(sc[mt][nb][i] - ref);
            l[r] += pr[nb][i];
          }
        uint32_t w[4][S::PP];
        split_pair<S::PP>(pr[0][0], pr[0][1], w[0]);
        split_pair<S::PP>(pr[0][2], pr[0][3], w[1]);
        split_pair<S::PP>(pr[1][0], pr[1][1], w[2]);
        split_pair<S::PP>(pr[1][2], pr[1][3], w[3]);
#pragma unroll
        for (int i = 0; i < S::PP; ++i) pa[mt][i] = make_uint4(w[0][i], w[1][i], w[2][i], w[3][i]);
      }

      // ---- values. A row's weight for a key it may not see is 0, but 0 * inf is not: if a
      // masked step holds such a value, each token's rows are taken by themselves.
      uint4 v[4][S::VV];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = 8 * (j >> 1) + 2 * t + (j & 1);
#pragma unroll
        for (int i = 0; i < S::VV; ++i)
          v[j][i] = *reinterpret_cast<const uint4*>(vt + r * S::row_bytes + v_piece(r, 8 * i + g) * 16);
      }
      bool wild = false;
      if (masked) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < S::VV; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) wild |= nonfinite(word(v[j][i], e), !S::p32);
        wild = __any_sync(0xffffffffu, wild);
      }
      if (!wild) {
#pragma unroll
        for (int c = 0; c < S::NB; ++c) {
          uint32_t b[S::KP][2];
          v_operand<S>(v, c, b);
#pragma unroll
          for (int mt = 0; mt < kMt; ++mt) add_products<S::q32, S::PP, S::KP>(o[mt][c], pa[mt], b);
        }
      } else {
        for (int tok = row0 / G; tok <= (row0 + rows - 1) / G; ++tok) {
          const int lim = visible_keys(seq, tok, shape.cap);
          uint4 vm[4][S::VV];
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < S::VV; ++i)
              vm[j][i] = s * kStep + 8 * (j >> 1) + 2 * t + (j & 1) < lim ? v[j][i] : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int c = 0; c < S::NB; ++c) {
            uint32_t b[S::KP][2];
            v_operand<S>(vm, c, b);
#pragma unroll
            for (int mt = 0; mt < kMt; ++mt) {
              float d[4] = {0.f, 0.f, 0.f, 0.f};
              add_products<false, S::PP, S::KP>(d, pa[mt], b);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if ((row0 + mt * kRows + g + 8 * (i >> 1)) / G == tok) o[mt][c][i] += d[i];
            }
          }
        }
      }
    }

    // ---- the warps' states become one, in the rings' place
    cp_wait<0>();
    __syncthreads();
#pragma unroll
    for (int r = 0; r < 2 * kMt; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      if (t == 0) {
        s_m[warp * kTile + g + 8 * r] = m[r];
        s_l[warp * kTile + g + 8 * r] = l[r];
      }
    }
#pragma unroll
    for (int c = 0; c < kMt * S::NB; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = 2 * t + (i & 1);     // the block's column: which lanes' 16 bytes
        const int mt = c / S::NB, cc = c % S::NB;
        const int ch = S::p32 ? 32 * (cc / 4) + 4 * n + cc % 4 : 64 * (cc / 8) + 8 * n + cc % 8;
        s_o[(warp * kTile + mt * kRows + g + 8 * (i >> 1)) * S::PE + ch] = o[mt][cc][i];
      }
    __syncthreads();
    const bool whole = c0 == 0 && c1 == cur.nc;
    const int owner0 = cur.first / range.per;              // blocks that hold a part of the item
    const int parts = (cur.first + cur.nc - 1) / range.per - owner0 + 1;
    float* slot = p.part + (2 * static_cast<size_t>(blockIdx.x) + (c0 == 0 ? 1 : 0)) * kTile * (kDh + 2);

    auto write_out = [&](int r, int ch, float4 v, float sum) {
      const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
      const int tok = (row0 + r) / G, hd = cur.h * G + (row0 + r) % G;
      TQ* dst = static_cast<TQ*>(p.out) + (seq.q0 + tok) * p.o_stride + hd * kDh + ch;
      v = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
      if constexpr (S::q32) {
        *reinterpret_cast<float4*>(dst) = v;
      } else {
        __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
        *reinterpret_cast<uint2*>(dst) = make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
      }
    };
    for (int i = tid; i < rows * (kDh / 4); i += kThreads) {
      const int r = i / (kDh / 4), ch = 4 * (i % (kDh / 4));
      float M = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w * kTile + r]);
      const float ref = M == -INFINITY ? 0.f : M;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = ex2(s_m[w * kTile + r] - ref);
        const float4 x = *reinterpret_cast<const float4*>(s_o + (w * kTile + r) * S::PE + ch);
        sum += f * s_l[w * kTile + r];
        acc.x += f * x.x;
        acc.y += f * x.y;
        acc.z += f * x.z;
        acc.w += f * x.w;
      }
      if (whole) {
        write_out(r, ch, acc, sum);
      } else {
        *reinterpret_cast<float4*>(slot + r * kDh + ch) = acc;
        if (ch == 0) {
          slot[kTile * kDh + r] = M;
          slot[kTile * (kDh + 1) + r] = sum;
        }
      }
    }
    if (!whole) {
      // ---- merge: groups of kGroup parts first, then the groups, each by its last arriver
      auto slot_of = [&](int k) {
        return p.part + (2 * static_cast<size_t>(owner0 + k) + (k == 0 ? 1 : 0)) * kTile * (kDh + 2);
      };
      // Parts first, first + step, ... (n of them) into one state: the result, or part `first`.
      auto merge = [&](int first, int step, int n, bool final) {
        for (int i = tid; i < n * kTile; i += kThreads) {
          const float* sl = slot_of(first + i / kTile * step) + kTile * kDh;
          const int r = i % kTile;
          s_w[i] = r < rows ? __ldcg(sl + r) : -INFINITY;
          s_w[kMaxParts * kTile + i] = r < rows ? __ldcg(sl + kTile + r) : 0.f;
        }
        __syncthreads();
        for (int i = tid; i < rows * (kDh / 4); i += kThreads) {
          const int r = i / (kDh / 4), ch = 4 * (i % (kDh / 4));
          float M = -INFINITY, sum = 0.f;
          for (int k = 0; k < n; ++k) M = fmaxf(M, s_w[k * kTile + r]);
          const float ref = M == -INFINITY ? 0.f : M;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int k0 = 0; k0 < n; k0 += 8) {
            float4 x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
              x[j] = __ldcg(reinterpret_cast<const float4*>(slot_of(first + min(k0 + j, n - 1) * step) + r * kDh + ch));
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              if (k0 + j >= n) break;
              const float w = ex2(s_w[(k0 + j) * kTile + r] - ref);
              sum = fmaf(w, s_w[(kMaxParts + k0 + j) * kTile + r], sum);
              acc.x = fmaf(w, x[j].x, acc.x);
              acc.y = fmaf(w, x[j].y, acc.y);
              acc.z = fmaf(w, x[j].z, acc.z);
              acc.w = fmaf(w, x[j].w, acc.w);
            }
          }
          if (final) {
            write_out(r, ch, acc, sum);
          } else {
            float* to = slot_of(first);
            *reinterpret_cast<float4*>(to + r * kDh + ch) = acc;
            if (ch == 0) {
              to[kTile * kDh + r] = M;
              to[kTile * (kDh + 1) + r] = sum;
            }
          }
        }
      };
      // Whether this block is the last of n to come to a counter, which is then zero again.
      auto last_of = [&](unsigned int* counter, int n) {
        __syncthreads();      // what the block has to show is written
        if (tid == 0) {
          const bool last = atomic_add_acq_rel_gpu(counter, 1u) == static_cast<unsigned int>(n - 1);
          if (last) *counter = 0u;
          s_last = last;
        }
        __syncthreads();
        return s_last != 0;
      };
      const int me = static_cast<int>(blockIdx.x) - owner0, group = me / kGroup, leader = group * kGroup;
      const int groups = (parts + kGroup - 1) / kGroup, n = min(kGroup, parts - leader);
      // a block may lead a group of the item that ends in it and one of the item that begins in it
      unsigned int* counter = p.counters + 3 * static_cast<size_t>(owner0 + leader);
      if (last_of(counter + (group == 0 ? 0 : 1), n)) {
        merge(leader, 1, n, groups == 1);
        if (groups > 1 && last_of(p.counters + 3 * static_cast<size_t>(owner0) + 2, groups)) merge(0, kGroup, groups, true);
      }
    }
    if (end >= range.g1) break;
    work_next(bt, shape, Hkv, &cur);
    __syncthreads();        // the queries and states of this item are done with
  }
}

template <typename TQ, typename TP, int kDh, bool kWide, int kMt>
cudaError_t launch_shape(const PagedAttnLaunch& a, RowsParams prm, const DeviceInfo& dev, cudaStream_t stream) {
  using S = Shape<TQ, TP, kDh, kWide, kMt>;
  constexpr int smem = S::smem;
  const auto kernel = paged_rows_kernel<TQ, TP, kDh, kWide, kMt>;
  static SmemOnce once;
  cudaError_t e = allow_smem(kernel, smem, dev.device, &once);
  if (e != cudaSuccess) return e;
  prm.shape.chunk_shift = S::chunk_shift;
  prm.shape.rows = S::rows;
  cudaLaunchConfig_t cfg = {};
  int grid = dev.num_sms * S::blocks;
  if (grid > kMaxBlocks / kMt) grid = kMaxBlocks / kMt;      // the workspace's rows
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(S::threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kernel, prm);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

// One wide block an SM where there are fewer items (K/V heads of sequences) than SMs, several
// narrow ones otherwise. One item over 262144 keys of 4 heads: wide 59 us, narrow 62; 320 items
// (16 sequences, 20 heads, fp32): narrow 39 us, wide 54.
template <typename TQ, typename TP, int kDh>
cudaError_t launch(const PagedAttnLaunch& a, const RowsParams& prm, const DeviceInfo& dev, cudaStream_t stream) {
  // fp32 queries, more than 16 rows: tiles of 32 share what it costs to read and split K and V
  // (512 tokens over 2048 keys of 20 heads: 99 us against 118 with tiles of 16, 63 against 67
  // with a bf16 pool). Not at 512-byte rows, where the registers do not hold them (323 us
  // against 274).
  if constexpr (sizeof(TQ) == 4 && kDh * sizeof(TP) <= 256)
    if (static_cast<long long>(a.max_new) * prm.shape.G > kRows)
      return launch_shape<TQ, TP, kDh, false, 2>(a, prm, dev, stream);
  const long long tiles = a.batch.B + static_cast<long long>(a.batch.n_tokens) * prm.shape.G / kRows;   // at most, a head
  if constexpr (Shape<TQ, TP, kDh, true, 1>::warps != Shape<TQ, TP, kDh, false, 1>::warps)
    if (tiles * a.layer.Hkv < kWideItems * dev.num_sms) return launch_shape<TQ, TP, kDh, true, 1>(a, prm, dev, stream);
  return launch_shape<TQ, TP, kDh, false, 1>(a, prm, dev, stream);
}

template <int kDh>
cudaError_t launch_dh(const PagedAttnLaunch& a, const RowsParams& prm, const DeviceInfo& dev, cudaStream_t stream) {
  using bf = __nv_bfloat16;
  if (a.act_bf16) return launch<bf, bf, kDh>(a, prm, dev, stream);
  return a.pool_bf16 ? launch<float, bf, kDh>(a, prm, dev, stream) : launch<float, float, kDh>(a, prm, dev, stream);
}

}  // namespace

size_t paged_rows_part_bytes(int dh) { return static_cast<size_t>(2 * kMaxBlocks) * kRows * (dh + 2) * 4; }

bool paged_rows_countable(const PagedAttnLaunch& a, int max_rows) {
  PagedBatch bt = a.batch;
  if (max_rows <= kRows) bt.n_tokens = 0;      // a tile a sequence and head, whatever the others bring
  return work_bound(bt, a.layer.page_shift, a.layer.Hkv, a.Hq / a.layer.Hkv, kRows, 6) < kCountLimit;
}

cudaError_t launch_paged_rows(const PagedAttnLaunch& a, int max_rows, const DeviceInfo& dev, cudaStream_t stream) {
  RowsParams prm;
  prm.q = a.q;
  prm.out = a.out;
  prm.q_stride = a.q_stride;
  prm.o_stride = a.o_stride;
  prm.qscale = a.scale * 1.4426950408889634f;
  prm.counters = static_cast<unsigned int*>(a.workspace);
  prm.part = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + kPagedCounterBytes);
  prm.status = dev.status_word;
  prm.batch = a.batch;
  prm.layer = a.layer;
  prm.shape.G = a.Hq / a.layer.Hkv;
  prm.shape.coarse = false;
  prm.shape.cap = a.batch.width << a.layer.page_shift;
  prm.shape.min_rows = 0;
  prm.shape.max_rows = max_rows;
  return a.dh == 64 ? launch_dh<64>(a, prm, dev, stream) : launch_dh<128>(a, prm, dev, stream);
}

}  // namespace cxa
