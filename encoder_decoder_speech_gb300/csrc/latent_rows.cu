// Attention over a latent cache's pages in fp32, on the CUDA cores:
//
//   out[r] = sum_j p_rj c_j / sum_j p_rj,  p_rj = 2^(s_rj - m_r),  s_rj = scale log2(e) q_r . [c_j | r_j]
//
// for 16 query rows (tokens times heads) of a sequence at a time, each key's row read once for all of
// them, in one pass with the running reference m_r. (Products of three bf16 parts on the tensor cores, as the
// few-rows kernel of the K/V pages has them, have not been tried here.) On the CUDA cores the 16 rows of 2 latent +
// rope products a key are what binds: 17,400 of them for 512 + 64 channels, 136 clocks of an SM, against 98 for reading the key's 2304 bytes. 5 tokens in each of 16 sequences of up to 1500
// keys, 8 heads, 128 + 32 channels: 32 us with the merge, of which the products alone take 4: a block has at most four
// steps, each a chain of three barriers, and 46 % of the issue slots are taken (fragments, exchanges and masks beside
// the products). 16 tokens of 20 heads over up to 4000 keys of 512 + 64: 100 us, 14.8 TFLOP/s.
//
// A step is 32 keys, copied into shared memory a step ahead (cp.async). Scores: a warp has four keys
// in registers, a 32nd of the channels in each lane, and takes a row of q after the other from shared
// memory; the lanes' sums of 8 rows x 4 keys are added up by halving exchanges, after which every
// lane has one of them. Values: a thread has two channels of all rows (or of a part of them), and
// the weights of a key's rows come as one broadcast.
#include <cmath>

#include "latent_parts.cuh"
#include "paged_work.cuh"
#include "ptx.cuh"

namespace cxa {
namespace {

constexpr int kThreads = 256, kWarps = 8;
constexpr int kRows = kLatentRowsF32;
constexpr int kKeys = 32, kChunkShift = 5;
constexpr int kTail = 64;              // channels of the rotated part, rope of them not zero

struct RowsParams {
  const float* q;
  float* out;
  long long q_stride, o_stride;
  float qscale;
  LatentCut* cut;
  float* part;
  unsigned int* status;
  PagedBatch batch;
  LatentLayer layer;
  WorkShape shape;
};

template <int kQuads>     // latent / 128
struct Shape {
  static constexpr int dc = kQuads * 128, row = dc + kTail;
  static constexpr int groups = kQuads == 3 ? 1 : 4 / kQuads;      // of rows, in P.V
  static constexpr int rows = kRows / groups;                      // of a thread
  static constexpr int smem = (2 * kKeys + kRows) * row * 4;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}

template <int kQuads>
__global__ void __launch_bounds__(kThreads, latent_rows_blocks(kQuads * 128)) latent_rows_kernel(const __grid_constant__ RowsParams p) {
  using S = Shape<kQuads>;
  extern __shared__ __align__(16) float smem[];
  float* const s_k = smem;                               // [2][kKeys][row]
  float* const s_q = smem + 2 * kKeys * S::row;          // [kRows][row]
  __shared__ WorkScratch s_work;
  __shared__ __align__(16) float s_s[kRows][kKeys + 1];  // scores
  __shared__ __align__(16) float s_p[kKeys][kRows];      // weights
  __shared__ float s_corr[kRows], s_m[kRows], s_l[kRows];
  __shared__ long long s_row[kRows];      // where the rows' results begin
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const PagedBatch& bt = p.batch;
  const int H = p.shape.G, rope = p.layer.rope, width = S::dc + rope, shift = p.layer.page_shift;
  WorkRange range;
  WorkCursor cur;
  WorkShape shape = p.shape;
  LatentCut cut = {0, 0, 0, 0};
  if (!work_locate<kThreads, false, true>(bt, shape, 1, &s_work, &range, &cur, p.status)) {
    if (tid == 0) p.cut[blockIdx.x] = cut;
    return;
  }
  // the tails' channels that no copy writes
  for (int i = tid; i < (2 * kKeys + kRows) * kTail; i += kThreads)
    smem[static_cast<size_t>(i / kTail) * S::row + S::dc + i % kTail] = 0.f;
  __syncthreads();

  for (;;) {
    const int end = min(range.g1, cur.first + cur.nc);
    const int c0 = cur.c, c1 = end - cur.first;
    const PagedSeq seq = cur.seq;
    const int row0 = cur.rt * kRows, rows = min(kRows, work_rows(seq, shape) - row0);
    const int keys = tile_keys(seq, shape, cur.rt), steps = tile_steps(seq, shape, cur.rt);
    const int s0 = chunk_step(shape, c0, cur.nc, steps), s1 = chunk_step(shape, c1, cur.nc, steps);
    const int* table_row = bt.table + static_cast<size_t>(cur.b) * bt.width;
    const float* pool = static_cast<const float*>(p.layer.C);
    // the pages of a step's groups of 16 keys, in lanes 0 and 1 (-1: none, or outside the pool); asked for a
    // step before they are used
    auto look = [&](int s) {
      const int key = s * kKeys + lane * 16;
      int page = -1;
      if (lane < kKeys / 16 && s < s1 && key < keys) {
        page = paged_lookup(table_row, bt.width, shift, p.layer.num_pages, key);
        if (page < 0 && warp == 0) atomicOr(p.status, kStatusBadPage);
      }
      return page;
    };
    // rows that no query sees, and of bad pages, become zero
    auto fetch = [&](int s, int pages) {
      const int pieces = width / 4;
      float* buf = s_k + (s & 1) * (kKeys * S::row);
#pragma unroll
      for (int i = 0; i < kKeys / kWarps; ++i) {
        const int k = warp + i * kWarps, key = s * kKeys + k;
        const int page = __shfl_sync(0xffffffffu, pages, k >> 4);
        const bool real = page >= 0 && key < keys;
        const float* src =
            pool + ((static_cast<size_t>(max(page, 0)) << shift) + (key & ((1 << shift) - 1))) * static_cast<size_t>(width);
        for (int c = lane; c < pieces; c += 32)
          cp_async16(smem_u32(buf + k * S::row + c * 4), real ? src + c * 4 : pool, real);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int pages = look(s0), next = look(s0 + 1);
    // the queries, with the first keys (by loads and stores, one after the other, an item began 3 us later)
    for (int i = warp; i < kRows; i += kWarps) {
      const int at = row0 + i;
      const float* src = i < rows ? p.q + (seq.q0 + at / H) * p.q_stride + static_cast<long long>(at % H) * width : p.q;
      for (int c = lane; c < width / 4; c += 32)
        cp_async16(smem_u32(s_q + i * S::row + c * 4), src + (i < rows ? c * 4 : 0), i < rows);
    }
    fetch(s0, pages);
    if (tid < kRows) {
      const int at = row0 + tid;
      s_row[tid] = (seq.q0 + at / H) * p.o_stride + static_cast<long long>(at % H) * S::dc;
    }
    // softmax: warp w has rows 2w and 2w + 1, a key a lane
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    int see[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 2 * warp + i;
      see[i] = r < rows ? visible_keys(seq, (row0 + r) / H, shape.cap) : 0;
    }
    const int see_all = visible_keys(seq, row0 / H, shape.cap);
    // values: this thread's channels and rows
    const int ch = 2 * (tid % (S::dc / 2)), rg = tid / (S::dc / 2);
    const bool pv = rg < S::groups;
    float o[S::rows][2];
#pragma unroll
    for (int i = 0; i < S::rows; ++i) o[i][0] = o[i][1] = 0.f;

    for (int s = s0; s < s1; ++s) {
      const int now = pages;
      if (s + 1 < s1) {
        fetch(s + 1, next);
        pages = next;
        next = look(s + 2);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
      } else {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
      }
      __syncthreads();
      const float* buf = s_k + (s & 1) * (kKeys * S::row);
      const int key0 = s * kKeys;
      // ---- scores of keys 4 warp .. 4 warp + 3
      {
        float4 k[4][kQuads];
        float2 kt[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float* row = buf + (4 * warp + j) * S::row;
#pragma unroll
          for (int c = 0; c < kQuads; ++c) k[j][c] = *reinterpret_cast<const float4*>(row + c * 128 + lane * 4);
          kt[j] = *reinterpret_cast<const float2*>(row + S::dc + lane * 2);
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float v[32];
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            const float* row = s_q + (half * 8 + r) * S::row;
            const float2 qt = *reinterpret_cast<const float2*>(row + S::dc + lane * 2);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[r * 4 + j] = kt[j].x * qt.x + kt[j].y * qt.y;
#pragma unroll
            for (int c = 0; c < kQuads; ++c) {
              const float4 q = *reinterpret_cast<const float4*>(row + c * 128 + lane * 4);
#pragma unroll
              for (int j = 0; j < 4; ++j)
                v[r * 4 + j] = fmaf(k[j][c].w, q.w, fmaf(k[j][c].z, q.z, fmaf(k[j][c].y, q.y, fmaf(k[j][c].x, q.x, v[r * 4 + j]))));
            }
          }
          // lane i ends up with the whole warp's v[i]: each exchange halves what a lane keeps
#pragma unroll
          for (int w = 16; w >= 1; w >>= 1) {
            const bool up = (lane & w) != 0;
#pragma unroll
            for (int i = 0; i < w; ++i) {
              const float keep = up ? v[i + w] : v[i], give = up ? v[i] : v[i + w];
              v[i] = keep + __shfl_xor_sync(0xffffffffu, give, w);
            }
          }
          s_s[half * 8 + (lane >> 2)][4 * warp + (lane & 3)] = v[0];
        }
      }
      __syncthreads();
      // ---- softmax
      {
        const int key = key0 + lane;
        const bool there = __shfl_sync(0xffffffffu, now, lane >> 4) >= 0 && key < keys;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = 2 * warp + i;
          const float x = there && key < see[i] ? s_s[r][lane] * p.qscale : -INFINITY;
          float top = x;
#pragma unroll
          for (int off = 16; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
          const float to = fmaxf(m[i], top);
          const float corr = m[i] == -INFINITY ? 0.f : ex2(m[i] - to);
          const float w = x == -INFINITY ? 0.f : ex2(x - to);
          m[i] = to;
          l[i] = l[i] * corr + w;
          s_p[lane][r] = w;
          if (lane == 0) s_corr[r] = corr;
        }
      }
      __syncthreads();
      // ---- values
      if (pv) {
#pragma unroll
        for (int i = 0; i < S::rows; ++i) {
          const float c = s_corr[rg * S::rows + i];
          o[i][0] *= c;
          o[i][1] *= c;
        }
        const int n = min(kKeys, keys - key0);
        // keys that all rows see, and then those that some do not (a hidden key's row may hold anything)
        const int plain = max(0, min(n, see_all - key0));
#pragma unroll 4
        for (int k = 0; k < plain; ++k) {
          const float2 v = *reinterpret_cast<const float2*>(buf + k * S::row + ch);
#pragma unroll
          for (int i = 0; i < S::rows; i += 4) {
            const float4 w = *reinterpret_cast<const float4*>(&s_p[k][rg * S::rows + i]);
            const float ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              o[i + e][0] = fmaf(ws[e], v.x, o[i + e][0]);
              o[i + e][1] = fmaf(ws[e], v.y, o[i + e][1]);
            }
          }
        }
#pragma unroll 1
        for (int k = plain; k < n; ++k) {
          const float2 v = *reinterpret_cast<const float2*>(buf + k * S::row + ch);
#pragma unroll
          for (int i = 0; i < S::rows; ++i) {
            const float w = s_p[k][rg * S::rows + i];
            if (w != 0.f) {
              o[i][0] = fmaf(w, v.x, o[i][0]);
              o[i][1] = fmaf(w, v.y, o[i][1]);
            }
          }
        }
      }
      __syncthreads();      // the buffer, the scores and the weights are free
    }
    // ---- the part in this range: written out, or left for the merge
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], off);
      if (lane == 0) {
        s_m[2 * warp + i] = m[i];
        s_l[2 * warp + i] = l[i];
      }
    }
    __syncthreads();
    const bool whole = c0 == 0 && c1 == cur.nc;
    float* slot = p.part + (2 * static_cast<size_t>(blockIdx.x) + (c0 == 0 ? 1 : 0)) * latent_slot(kRows, S::dc);
    if (pv) {
      // (places and factors before the first store: one row after the other took 430 clocks each)
      float* to[S::rows];
      float by[S::rows];
#pragma unroll
      for (int i = 0; i < S::rows; ++i) {
        const int r = rg * S::rows + i;
        const float sum = s_l[r];
        by[i] = !whole ? 1.f : sum > 0.f || sum != sum ? 1.f / sum : 0.f;
        to[i] = (whole ? p.out + s_row[r] : slot + static_cast<size_t>(r) * S::dc) + ch;
      }
#pragma unroll
      for (int i = 0; i < S::rows; ++i)
        if (rg * S::rows + i < rows) *reinterpret_cast<float2*>(to[i]) = make_float2(o[i][0] * by[i], o[i][1] * by[i]);
    }
    if (!whole && tid < rows) {
      slot[kRows * S::dc + tid] = s_m[tid];
      slot[kRows * S::dc + kRows + tid] = s_l[tid];
    }
    if (c0 == 0 && c1 < cur.nc)
      cut = {seq.q0, cur.rt, (cur.first + cur.nc - 1) / range.per - cur.first / range.per + 1, rows};
    if (end >= range.g1) break;
    work_next(bt, shape, 1, &cur);
    __syncthreads();
  }
  if (tid == 0) p.cut[blockIdx.x] = cut;
}

template <int kQuads>
cudaError_t launch(const LatentAttnLaunch& a, const DeviceInfo& dev, cudaStream_t stream) {
  RowsParams p;
  p.q = static_cast<const float*>(a.q);
  p.out = static_cast<float*>(a.out);
  p.q_stride = a.q_stride;
  p.o_stride = a.o_stride;
  p.qscale = a.scale * 1.4426950408889634f;
  p.cut = latent_cuts(a.workspace);
  p.part = latent_part(a.workspace);
  p.status = dev.status_word;
  p.batch = a.batch;
  p.layer = a.layer;
  p.shape.G = a.H;
  p.shape.rows = kRows;
  p.shape.chunk_shift = kChunkShift;
  p.shape.coarse = false;
  p.shape.cap = a.batch.width << a.layer.page_shift;
  p.shape.min_rows = 0;
  p.shape.max_rows = 0x7FFFFFFF;
  static SmemOnce once;
  cudaError_t e = allow_smem(latent_rows_kernel<kQuads>, Shape<kQuads>::smem, dev.device, &once);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  constexpr int per_sm = latent_rows_blocks(kQuads * 128);
  const int most = latent_max_blocks(per_sm), grid = dev.num_sms * per_sm < most ? dev.num_sms * per_sm : most;
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Shape<kQuads>::smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, latent_rows_kernel<kQuads>, p);
  if (e != cudaSuccess) return e;
  count_launches(1);
  return launch_latent_merge(a, kRows, grid, dev, stream);
}

}  // namespace

cudaError_t launch_latent_rows(const LatentAttnLaunch& a, const DeviceInfo& dev, cudaStream_t stream) {
  switch (a.layer.latent / 128) {
    case 1: return launch<1>(a, dev, stream);
    case 2: return launch<2>(a, dev, stream);
    case 3: return launch<3>(a, dev, stream);
    default: return launch<4>(a, dev, stream);
  }
}

}  // namespace cxa
