// Attention of many new tokens per sequence over the paged cache on the CUDA cores (fp32).
//
// Per query tile (tokens x query heads of one KV head, 64 rows) and 64 slots, with a
// running reference m (log2 units):
//   S = Q K^T, x = log2(e) temp cap(sm_scale S), P = 2^(x - m), l += sum P, O += P V.
// fp32 stays on the CUDA cores: a TF32 product keeps 11 bits of q and k (three of split operands
// would keep them all; not tried).  256 threads, 4 x 4
// scores each (rows 4 ty .., keys tx + 16 z: 64 products for eight vectors of shared memory
// along D, whose padded rows spread over the banks) and 4 x D / 16 outputs, all in pairs of
// fp32 products: of the even and odd columns of a score, of two rows' outputs.  The next
// step's keys and values come in by cp.async meanwhile, their pages looked up a step before
// that.  Bound by shared memory's and the products' latencies (short scoreboard 2.2, wait 1.5
// stalls an issue; issue slots 44 %, 16 warps an SM at D = 64, eight at 128), and at small
// sizes by the first loads and the finish.  Four prompts of up to 1500 tokens, 16 heads x 64:
// 271 us (305 with products one at a time, 348 with loads through registers); x 128: 494
// (538, 647); four prompts of 61 to 333 tokens behind up to 700 others, 4 / 2 heads x 64: 39
// (42.5, 45).  Loops over D unrolled by 4, 8, 16: 289, 282, 271 and 524, 510, 506.
#include "cache_math.cuh"
#include "cap_math.cuh"
#include "paged_out.cuh"

namespace capattn {
namespace {

constexpr int BM = kAttendSimtRows;
constexpr int TK = 64;
constexpr int kThreads = 256;

template <int D>
struct SimtSmem {
  static constexpr int ROW = D + 4;  // a row's stride
  float q[BM][ROW];
  union {
    float k[TK][ROW];
    float p[TK * BM];  // once the scores are there: key-major; a key's rows in blocks of 4, rotated by key
  } k[2];
  float v[2][TK][D];
  RowMask mask[BM];
  float temp[BM];
  int row[BM];         // of o and lse, from the tile's first; -1: none
  uint32_t live[BM][TK / 32];
  Piece piece;
  ScheduleMem sched;
};

__device__ __forceinline__ void copy16(void* dst, const void* src, bool live) {  // zeros where !live
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int D, int METHOD>
__global__ void __launch_bounds__(kThreads, D == 64 ? 2 : 1)
paged_simt_kernel(PagedParams p) {
  extern __shared__ __align__(16) uint8_t raw[];
  using S = SimtSmem<D>;
  S& s = *reinterpret_cast<S*>(raw);
  constexpr int OC = D / 16;                   // output columns of a thread: 4 tx + 64 w
  constexpr int CH = D / 4;                    // 16-byte chunks of a row
  constexpr int NI = TK * CH / kThreads;       // of K (and of V) a thread copies a step
  constexpr int kNoRow = INT_MIN;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int chunk = threadIdx.x % CH * 4, row0 = threadIdx.x / CH;  // rows row0 + it * kThreads / CH
  pdl_trigger();
  pdl_wait();
  const bool few = p.c.B <= kWarpSeqs;
  if (!few) schedule_by_cta<TK>(p, kThreads, s.sched);
  PieceWalk<TK> walk(p, few ? schedule_by_warp<TK>(p, lane) : s.sched.out, lane);  // (used by warp 0)
  const CacheParams& c = p.c;
  const float* kc = static_cast<const float*>(c.k);
  const float* vc = static_cast<const float*>(c.v);
  bool shared = false;
  for (;;) {
    if (warp == 0) {
      const Piece x = walk.next(p);
      if (lane == 0) s.piece = x;
      if (x.steps > 0 && !x.whole && x.c0 == (int)blockIdx.x) {
        if (lane == 0) leave_record(p, x);
        shared = true;
      }
      if (x.steps < 0 && !shared && lane == 0) leave_no_record(p);
    }
    __syncthreads();
    const Piece x = s.piece;
    if (x.steps < 0) break;
    const int g = x.part / p.parts, h0 = (x.part - g * p.parts) * p.heads;
    const int heads = min(p.heads, c.G - h0);
    const int head0 = g * c.G + h0;
    // the pages of this thread's rows of a step, as read
    const int32_t* table = c.table + (size_t)x.b * c.max_pages;
    int pages[NI];
    auto look_up = [&](int step) {
#pragma unroll
      for (int it = 0; it < NI; ++it) {
        const int j = (x.tile0 + step) * TK + row0 + it * (kThreads / CH);
        pages[it] = step < x.steps && j >= x.first && j < x.len ? table[j >> c.page_shift] : kNoRow;
      }
    };
    auto copy = [&](int step) {
      const int st = step & 1;
#pragma unroll
      for (int it = 0; it < NI; ++it) {
        const int r = row0 + it * (kThreads / CH), j = (x.tile0 + step) * TK + r;
        const bool live = pages[it] != kNoRow;
        int page = pages[it];
        if (live && (page < 0 || page >= c.num_pages)) {  // flagged, and read as page 0
          atomicOr(c.status, kStatusBadPageBit);
          page = 0;
        }
        const size_t at = live ? ((((size_t)page * c.Hkv + g) << c.page_shift) + (j & (c.page_size - 1))) * D + chunk : 0;
        copy16(&s.k[st].k[r][chunk], kc + at, live);
        copy16(&s.v[st][r][chunk], vc + at, live);
      }
      copy_commit();
    };
    look_up(0);
    copy(0);
    look_up(1);
    if (threadIdx.x < BM) {
      const int r = threadIdx.x, t = r / p.heads;
      const SeqShape sh = {x.row0, x.n, x.len, x.base};
      const bool valid = t < x.count && r - t * p.heads < heads;
      s.mask[r] = valid ? row_mask(p, x.b, g, sh, x.i0 + t) : dead_row();
      s.temp[r] = (valid && c.temp ? c.temp[x.row0 + x.i0 + t] : 1.f) * kL2E;
      s.row[r] = valid ? t * c.Hq + r - t * p.heads : -1;
    }
    for (int i = threadIdx.x; i < BM * CH; i += kThreads) {
      const int r = i / CH, d = i % CH * 4, t = r / p.heads;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
      if (t < x.count && r - t * p.heads < heads)
        a = *reinterpret_cast<const float4*>(static_cast<const float*>(c.q) + (size_t)(x.row0 + x.i0 + t) * c.q_stride +
                                             (size_t)(head0 + r - t * p.heads) * D + d);
      *reinterpret_cast<float4*>(&s.q[r][d]) = a;
    }
    float m[4], l[4];
    F2 o2[2][OC];  // rows 4 ty + 2 x and the next
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      m[a] = -INFINITY;
      l[a] = 0.f;
    }
#pragma unroll
    for (int e = 0; e < OC; ++e) o2[0][e] = o2[1][e] = f2(0.f, 0.f);
    for (int step = 0; step < x.steps; ++step) {
      const int j0 = (x.tile0 + step) * TK, st = step & 1;
      __syncthreads();  // the last step's products (their stage is filled again), the row masks
      if (step + 1 < x.steps) {
        copy(step + 1);
        look_up(step + 2);
        copy_wait<1>();
      } else {
        copy_wait<0>();
      }
      if (threadIdx.x < 2 * BM) {
        const int r = threadIdx.x >> 1, half = threadIdx.x & 1, c0 = j0 + 32 * half;
        s.live[r][half] = all_live(s.mask[r], c0, 32) ? 0xFFFFFFFFu : live_slots(p, s.mask[r], c0);
      }
      __syncthreads();
      F2 sums[4][4];  // over the even and the odd columns
#pragma unroll
      for (int y = 0; y < 4; ++y)
#pragma unroll
        for (int z = 0; z < 4; ++z) sums[y][z] = f2(0.f, 0.f);
#pragma unroll 16
      for (int d = 0; d < D; d += 4) {
        float4 a[4], b[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) a[y] = *reinterpret_cast<const float4*>(&s.q[4 * ty + y][d]);
#pragma unroll
        for (int z = 0; z < 4; ++z) b[z] = *reinterpret_cast<const float4*>(&s.k[st].k[tx + 16 * z][d]);
#pragma unroll
        for (int y = 0; y < 4; ++y)
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            sums[y][z] = f2_fma(f2(a[y].x, a[y].y), f2(b[z].x, b[z].y), sums[y][z]);
            sums[y][z] = f2_fma(f2(a[y].z, a[y].w), f2(b[z].z, b[z].w), sums[y][z]);
          }
      }
      float acc[4][4];
#pragma unroll
      for (int y = 0; y < 4; ++y)
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          float even, odd;
          f2_split(sums[y][z], even, odd);
          acc[y][z] = even + odd;
        }
      float scales[4];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const float temp = s.temp[4 * ty + y];
        float top = -INFINITY;
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          const bool live = (s.live[4 * ty + y][z >> 1] >> (tx + 16 * (z & 1))) & 1u;
          acc[y][z] = live ? any_cap<METHOD>(acc[y][z], c.cap) * temp : -INFINITY;
          top = fmaxf(top, acc[y][z]);
        }
#pragma unroll
        for (int w = 1; w < 16; w <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, w));
        top = fmaxf(top, m[y]);
        const float scale = top == -INFINITY ? 1.f : ex2_approx(m[y] - top), ref = top == -INFINITY ? 0.f : top;
        m[y] = top;
        l[y] *= scale;
        scales[y] = scale;
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          acc[y][z] = ex2_approx(acc[y][z] - ref);
          l[y] += acc[y][z];
        }
      }
#pragma unroll
      for (int x2 = 0; x2 < 2; ++x2)
#pragma unroll
        for (int e = 0; e < OC; ++e) o2[x2][e] = f2_mul(o2[x2][e], f2(scales[2 * x2], scales[2 * x2 + 1]));
      __syncthreads();  // P takes the place of K
#pragma unroll
      for (int z = 0; z < 4; ++z)
        *reinterpret_cast<float4*>(&s.k[st].p[(tx + 16 * z) * BM + 4 * ((ty + tx) & 15)]) =
            make_float4(acc[0][z], acc[1][z], acc[2][z], acc[3][z]);
      __syncthreads();
#pragma unroll (D / 16)
      for (int j = 0; j < TK; ++j) {
        const float4 a = *reinterpret_cast<const float4*>(&s.k[st].p[j * BM + 4 * ((ty + j) & 15)]);
        const F2 a01 = f2(a.x, a.y), a23 = f2(a.z, a.w);
#pragma unroll
        for (int w = 0; w < OC / 4; ++w) {
          const float4 b = *reinterpret_cast<const float4*>(&s.v[st][j][64 * w + 4 * tx]);
          const float bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const F2 b2 = f2(bv[e], bv[e]);
            o2[0][4 * w + e] = f2_fma(a01, b2, o2[0][4 * w + e]);
            o2[1][4 * w + e] = f2_fma(a23, b2, o2[1][4 * w + e]);
          }
        }
      }
    }
    // ---------------------------------------------------------- end of a piece
    float o[4][OC];
#pragma unroll
    for (int e = 0; e < OC; ++e) {
      f2_split(o2[0][e], o[0][e], o[1][e]);
      f2_split(o2[1][e], o[2][e], o[3][e]);
    }
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const int r = 4 * ty + y;
      float zero = 0.f;  // NaN once an output is not finite
#pragma unroll
      for (int e = 0; e < OC; ++e) zero = fmaf(o[y][e], 0.f, zero);
#pragma unroll
      for (int w = 1; w < 16; w <<= 1) {
        l[y] += __shfl_xor_sync(0xFFFFFFFFu, l[y], w);
        zero += __shfl_xor_sync(0xFFFFFFFFu, zero, w);
      }
      // a row without live slots in this piece has l = 0 (and 0 times anything in O)
      const bool none = m[y] == -INFINITY && l[y] == 0.f, bad = !none && (zero != 0.f || !(l[y] < INFINITY));
      if (s.row[r] < 0) continue;
      const size_t row = (size_t)(x.row0 + x.i0) * c.Hq + head0 + s.row[r];
      if (x.whole) {
        const float inv = none ? 0.f : 1.f / l[y];
#pragma unroll
        for (int w = 0; w < OC / 4; ++w) {
          *reinterpret_cast<float4*>(static_cast<float*>(c.o) + row * D + 64 * w + 4 * tx) =
              none ? make_float4(0.f, 0.f, 0.f, 0.f)
                   : make_float4(o[y][4 * w] * inv, o[y][4 * w + 1] * inv, o[y][4 * w + 2] * inv, o[y][4 * w + 3] * inv);
        }
        if (tx == 0) {
          if (bad) ask_redo(p);
          c.lse[row] = bad ? kNaN32 : none ? -INFINITY : (m[y] + log2f(l[y])) * kLn2;
        }
      } else {
#pragma unroll
        for (int w = 0; w < OC / 4; ++w) {
          const int col = 64 * w + 4 * tx;
          reinterpret_cast<float4*>(p.part_o)[part_at<D, BM>(x.slot, r, col / (D / 4), col % (D / 4) / 4)] =
              make_float4(o[y][4 * w], o[y][4 * w + 1], o[y][4 * w + 2], o[y][4 * w + 3]);
        }
        if (tx == 0) {
          const size_t at = (size_t)x.slot * BM + r;
          p.part_ml[at] = make_float2(m[y], none ? 0.f : l[y]);
          p.part_bad[at] = bad ? 1u : 0u;
          if (x.c0 == (int)blockIdx.x) c.lse[row] = 0.f;  // whatever it held asks for nothing
        }
      }
    }
    __syncthreads();  // the next piece's rows
  }
}

template <int D, int METHOD>
cudaError_t launch(const PagedParams& p, cudaStream_t s) {
  auto* k = paged_simt_kernel<D, METHOD>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), sizeof(SimtSmem<D>), done);
  if (e != cudaSuccess) return e;
  return launch_pdl(k, dim3(p.ctas), dim3(kThreads), sizeof(SimtSmem<D>), s, p);
}

template <int METHOD>
struct PagedSimtLaunch {
  static cudaError_t run(const PagedParams& p, cudaStream_t s) {
    return p.c.D == 64 ? launch<64, METHOD>(p, s) : launch<128, METHOD>(p, s);
  }
};

}  // namespace

cudaError_t launch_paged_attend_simt(const PagedParams& p, cudaStream_t s) {
  return dispatch_cap<PagedSimtLaunch>(p.c.method, p, s);
}

}  // namespace capattn
