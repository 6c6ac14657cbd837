// One Muon step (or orthogonalisation) of many small blocks, every block on its own, in one launch:
//
//   M <- beta M + G;  U = G + beta M;  X = U / (||U||_F + eps);  k times
//   A = X X^T, B = a I + b A + c A A, X <- B X;  W <- (1 - lr wd) W - lr s(block) X
//
// A block (short side m <= 128, long side n) lives in the shared memory of one CTA, or of the CTAs of
// a cluster that cut its long side into slices, from the first product to the last; HBM sees G, M
// and W only.  The three products of an iteration run on the tensor cores from that one copy:
//
//   Gram    A (m x m)       = X X^T        contraction over the CTA's slice (cluster: partial sums)
//   square  A A (m x m)     -> B = a I + b A + c A A, written over A (fp32: a X is added to the update)
//   update  X'^T (n x m)    = X^T B        128 long-side elements a tile, written over X
//
// Forming the update transposed keeps all 128 TMEM lanes busy for every m.  X is held as the block
// lies in memory (rows of 128 bytes, 128-byte swizzle): wide blocks m x n, tall ones n x m; the
// operand descriptors take either as K-major or MN-major.
//
// Iterates are fp16, times a power of two: every value of the iteration is bounded by the coefficient
// table (singular values start at most 1), so fp16's range suffices and its 11 significant bits are
// eight times finer than bf16's at the same MMA rate.  fp32 blocks hold a second plane with the
// rounding error of the first (22 bits) and accumulate the three leading plane products.
//
// A cluster sums its Gram partials over distributed shared memory: each CTA stores the pieces of its
// partial (on and above the diagonal) at the CTAs that sum them, which add up in rank order and store the
// rounded sums to all; the tiles below the diagonal are copied from those above.  Results do not depend on
// timing.  Remote stores, not loads (those stall: 2.0 us for what stores and a barrier do in 1.6), and 64
// bytes of a row of A at a time (32 bytes took 1.4 us instead of 1.0): 1767 us for 24 matrices of 2048 x 4096
// in blocks of 2048 x 128, 1848 with 32-byte rows, 1880 with whole rows pulled from every CTA.
// Every mbarrier wait is bounded; after one has run out nothing is applied to W.
//
// What bounds it (measured; 5 quintic iterations).  576 blocks of 64 x 768 in bf16: 149 us against 61 for the
// 14 bytes an element.  Two CTAs an SM, two rounds; in each 28 us of loads and momentum stores for all SMs at
// once (5.6 TB/s), 5 us of norm and rescaling, 30 us of products (their operands' shared-memory reads, then the
// drains between them), 8 us of apply.  One order for the two CTAs of an SM, so that one loads while the other
// multiplies, did not shorten it.  768 blocks of 2048 x 128: 1767 us against 432; clusters of four, 33 at once;
// 13 to 19 us of loads, then per iteration 3.5 us of exchange, 1.4 of square, 3.4 of update and Gram, 7 of apply.
// 54 fp32 blocks of 128 x 768: 166 us against 16: two rounds of 33 clusters of four, each 77 us, three
// products for one.
#include <cuda_fp16.h>

#include <atomic>
#include <type_traits>

#include "blocks.h"
#include "device_utils.cuh"

namespace muon {

namespace {

constexpr int MAX_THREADS = 512;

__host__ __device__ constexpr int round16(int x) { return (x + 15) & ~15; }
__host__ __device__ constexpr int round64(int x) { return (x + 63) & ~63; }

// Byte sizes of one plane of X and of A.  X: chunks of 64 columns, 128-byte rows.
__host__ __device__ constexpr uint32_t x_plane_bytes(int m, int slice, bool tall) {
  return tall ? static_cast<uint32_t>((round64(round16(m)) / 64) * slice * 128)
              : static_cast<uint32_t>((slice / 64) * round16(m) * 128);
}
__host__ __device__ constexpr uint32_t a_plane_bytes(int m) {
  return static_cast<uint32_t>((round64(round16(m)) / 64) * round16(m) * 128);
}
// Operand reads run past the end of matrices with fewer than 128 (or 64) rows, into lanes nothing reads:
// those of X, whose last tile misses at most 64 rows, end in A and this, those of A in this.
__host__ __device__ constexpr uint32_t overrun_bytes(int m) { return static_cast<uint32_t>(128 - round16(m)) * 128u; }
// A cluster's Gram partials: every CTA sums a share of the 16 x 32 fp32 pieces (2 KB) of the 32 x 32 tiles on
// and above the diagonal, and has a place for each of them from each CTA.
__host__ __device__ constexpr int side_tiles(int m) { return (round16(m) + 31) / 32; }
__host__ __device__ constexpr int gram_pieces(int m) { return side_tiles(m) * (side_tiles(m) + 1); }
__host__ __device__ constexpr int piece_share(int m, int cluster) { return (gram_pieces(m) + cluster - 1) / cluster; }
// Where shared memory does not hold them beside A, they lie where A will be, and in what that lacks.
__host__ __device__ constexpr uint32_t part_bytes(int m, int cluster, int planes, bool alias) {
  const uint32_t have = alias ? planes * a_plane_bytes(m) + overrun_bytes(m) : 0u;
  const uint32_t need = cluster > 1 ? static_cast<uint32_t>(cluster * piece_share(m, cluster)) * 2048u : 0u;
  return need > have ? need - have : 0u;
}

constexpr int MAX_SLOTS = 4;  // update tiles in TMEM at a time, at most
// fp32 blocks: tiles of 128 long-side elements that one accumulator of the Gram matrix sums.  The tensor core
// cuts its partial sums towards zero, so that a long one shrinks: error of O after five quintic iterations for
// 24 x 2048, 16 x 3000, 64 x 760: 9.5e-6, 1.9e-5, 6.1e-6 with one accumulator, 1.2e-6, 1.1e-6, 3.6e-6 with one for
// two tiles (54 blocks of 128 x 768: 161 -> 166 us), 1.3e-6, 0.8e-6, 3.4e-6 with one each (167 us).
constexpr int GRAM_TILES = 2;

// Small shared state behind the buffers.
struct Vars {
  unsigned long long bar, drain, slot[MAX_SLOTS];
  double red[MAX_THREADS / 32];
  double sum;
  int abort;
  uint32_t tmem;
};

__device__ __forceinline__ uint32_t instr_desc_f16(int mrows, int n, bool a_mn, bool b_mn) {
  return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(mrows >> 4) << 24);
}

// The barrier's arrival is for converged warps.
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  cluster_sync_all();
}
__device__ __forceinline__ double ld_cluster_f64(uint32_t addr) {
  double v;
  asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float ld_cluster_f(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster_v4(uint32_t addr, uint4 v) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
__device__ __forceinline__ void fence_proxy_async_cluster() {
  asm volatile("fence.proxy.async.shared::cluster;" ::: "memory");
}

__device__ __forceinline__ void st_shared_v4u(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4u(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}

// Element (row, col) of a swizzled matrix: 64-column chunks of `rows` 128-byte rows; `col` in 8s.
__device__ __forceinline__ uint32_t piece_at(uint32_t base, int rows, int row, int col) {
  return base + static_cast<uint32_t>((col >> 6) * rows + row) * 128u +
         ((((static_cast<uint32_t>(col) >> 3) & 7u) ^ (static_cast<uint32_t>(row) & 7u)) << 4);
}

__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_half2(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }

// Eight values as one 16-byte piece per plane: plane 1 holds what plane 0 rounded away.
template <int PLANES>
__device__ __forceinline__ void split8(const float (&v)[8], uint4 (&out)[PLANES]) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = pack_half2(v[2 * j], v[2 * j + 1]);
  out[0] = make_uint4(w[0], w[1], w[2], w[3]);
  if (PLANES == 2) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 h = unpack_half2(w[j]);
      w[j] = pack_half2(v[2 * j] - h.x, v[2 * j + 1] - h.y);
    }
    out[PLANES - 1] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

template <int PLANES>
__device__ __forceinline__ void join8(uint32_t addr, uint32_t plane, float (&v)[8]) {
  const uint4 a = ld_shared_v4u(addr);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = unpack_half2(w[j]);
    v[2 * j] = f.x;
    v[2 * j + 1] = f.y;
  }
  if (PLANES == 2) {
    const uint4 b = ld_shared_v4u(addr + plane);
    const uint32_t l[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = unpack_half2(l[j]);
      v[2 * j] += f.x;
      v[2 * j + 1] += f.y;
    }
  }
}

// 32 bytes a thread in one access, so that a warp's fp32 pieces are whole lines (two 16-byte accesses
// would each touch every sector).
__device__ __forceinline__ void ld_global_v8(const float* p, uint32_t (&w)[8]) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p));
}
__device__ __forceinline__ void st_global_v8(float* p, const float (&v)[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// Eight consecutive elements of a row of which nv exist, as raw words (VEC: one aligned access, nv is
// eight or nothing).  Loading and unpacking are apart so that a thread's loads are all under way
// before it waits for the first.
template <bool F32, bool VEC>
struct Raw8 {
  uint32_t w[F32 ? 8 : 4];
  __device__ __forceinline__ void load(const void* p, long long at, int nv) {
    if (VEC) {
      if (nv > 0) {
        if constexpr (F32) {
          ld_global_v8(static_cast<const float*>(p) + at, w);
        } else {
          const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
          w[0] = a.x;
          w[1] = a.y;
          w[2] = a.z;
          w[3] = a.w;
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < (F32 ? 8 : 4); ++j) {
        if (F32) {
          w[j] = j < nv ? static_cast<const uint32_t*>(p)[at + j] : 0u;
        } else {
          const uint16_t* q = static_cast<const uint16_t*>(p) + at;
          const uint32_t lo = 2 * j < nv ? q[2 * j] : 0u, hi = 2 * j + 1 < nv ? q[2 * j + 1] : 0u;
          w[j] = lo | (hi << 16);
        }
      }
    }
  }
  __device__ __forceinline__ void get(float (&v)[8], int nv) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = F32 ? __uint_as_float(w[F32 ? j : 0])
                 : __uint_as_float((j & 1) ? w[F32 ? 0 : j / 2] & 0xFFFF0000u : w[F32 ? 0 : j / 2] << 16);
      if (VEC && nv <= 0) v[j] = 0.f;
    }
  }
};

template <bool F32, bool VEC>
__device__ __forceinline__ void store8(void* p, long long at, int nv, const float (&v)[8]) {
  if (VEC) {
    if (nv <= 0) return;
    if (F32) {
      st_global_v8(static_cast<float*>(p) + at, v);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&h);
      }
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < nv) {
        if (F32) static_cast<float*>(p)[at + j] = v[j];
        else static_cast<uint16_t*>(p)[at + j] = float_to_bf16_bits(v[j]);
      }
  }
}

// Powers of two as floats; exponents below the normal range give zero.
__device__ __forceinline__ float exp2i(int e) { return e < -126 ? 0.f : __int_as_float((e + 127) << 23); }

// A piece's values are scaled so that their largest lies in [2^TOP_EXP, 2^(TOP_EXP + 1)): inside
// fp16's range with all of its bits.  Pieces of zeros or of values below 2^-100 count as 2^-100.
constexpr int TOP_EXP = 14, EXP_BIAS = 110;
__device__ __forceinline__ int piece_exponent(float top) {
  const int e = (__float_as_int(top) >> 23) - 127;
  return min(max(e, -100), 127);
}

// (row, piece) of every blockDim.x-th piece of a row-major walk, without a division a step.
struct PieceWalk {
  int r, c, dr, dc, pieces;
  __device__ __forceinline__ PieceWalk(int first, int n) : pieces(max(n, 1)) {
    r = first / pieces;
    c = first - r * pieces;
    dr = blockDim.x / pieces;
    dc = blockDim.x - dr * pieces;
  }
  __device__ __forceinline__ void next() {
    r += dr;
    c += dc;
    if (c >= pieces) {
      c -= pieces;
      ++r;
    }
  }
};

// Asks L2 for the 128-byte lines of a region (aligned rows).
template <int BYTES>
__device__ __forceinline__ void prefetch_region(const void* p, long long ld, long long row0, long long col0, int rows,
                                                int cols) {
  const int lines = (cols * BYTES + 127) / 128;
  for (int i = threadIdx.x; i < rows * lines; i += blockDim.x) {
    const int r = i / lines;
    prefetch_l2(static_cast<const char*>(p) + ((row0 + r) * ld + col0) * BYTES + (i - r * lines) * 128);
  }
}

// The CTA's part of a block as it lies in memory and in shared memory.
struct Region {
  int rows, cols;      // elements that exist
  int rows_p, pieces;  // padded rows, 8-column pieces per padded row
  long long row0, col0;
  uint32_t xs, x_plane;
  int x_rows;
};

// M <- beta M + G, U into shared memory, each piece at its own power of two (exponents in `exps`).
// Returns this thread's part of sum U^2, the pieces' sums (of the scaled values) put together in 64 bits, so
// that it neither overflows nor vanishes for any fp32 values.  STEP false: U = G.
template <bool F32, bool STEP, bool VEC>
__device__ __forceinline__ double momentum_pass(const BlockParams& P, const Region& R, const void* gp, float* mp,
                                               uint8_t* exps) {
  constexpr int PLANES = F32 ? 2 : 1, BATCH = F32 ? 2 : 4;  // pieces a thread loads before it uses the first
  const int n = R.rows_p * R.pieces;
  double total = 0.0;
  PieceWalk walk(threadIdx.x, R.pieces);
  const int nt = blockDim.x;
  for (int i0 = threadIdx.x; i0 < n; i0 += BATCH * nt) {
    Raw8<F32, VEC> g[BATCH];
    Raw8<true, VEC> m[BATCH];
    int row[BATCH], col[BATCH];
#pragma unroll
    for (int q = 0; q < BATCH; ++q) {
      row[q] = walk.r;
      col[q] = walk.c * 8;
      walk.next();
      const int nv = row[q] < R.rows ? R.cols - col[q] : 0;
      g[q].load(gp, (R.row0 + row[q]) * P.ldg + R.col0 + col[q], nv);
      if (STEP) m[q].load(mp, (R.row0 + row[q]) * P.ldm + R.col0 + col[q], nv);
    }
#pragma unroll
    for (int q = 0; q < BATCH; ++q) {
      if (i0 + q * nt < n) {
        const int nv = row[q] < R.rows ? R.cols - col[q] : 0;
        float u[8];
        g[q].get(u, nv);
        if (STEP) {
          float v[8];
          m[q].get(v, nv);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float gs = P.gscale * u[j];
            v[j] = fmaf(P.beta, v[j], gs);
            u[j] = P.nesterov ? fmaf(P.beta, v[j], gs) : v[j];
          }
          store8<true, VEC>(mp, (R.row0 + row[q]) * P.ldm + R.col0 + col[q], nv, v);
        }
        float top = 0.f, sq = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(u[j]));
        const int e = piece_exponent(top);
        const float up = exp2i(TOP_EXP - e);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          u[j] *= up;
          sq = fmaf(u[j], u[j], sq);
        }
        total = fma(static_cast<double>(sq), __hiloint2double((1023 + 2 * (e - TOP_EXP)) << 20, 0), total);
        uint4 o[PLANES];
        split8<PLANES>(u, o);
        const uint32_t at = piece_at(R.xs, R.x_rows, row[q], col[q]);
#pragma unroll
        for (int t = 0; t < PLANES; ++t) st_shared_v4u(at + t * R.x_plane, o[t]);
        exps[i0 + q * nt] = static_cast<uint8_t>(e + EXP_BIAS);
      }
    }
  }
  return total;
}

// W <- decay W - lrs X (X held at 1 / inv_s), or W <- X.
template <bool F32, bool STEP, bool VEC>
__device__ __forceinline__ void apply_pass(const BlockParams& P, const Region& R, void* wp, float lrs, float inv_s) {
  constexpr int PLANES = F32 ? 2 : 1, BATCH = F32 ? 4 : 8;
  PieceWalk walk(threadIdx.x, R.pieces);
  for (int i0 = threadIdx.x; i0 < R.rows * R.pieces; i0 += BATCH * blockDim.x) {
    Raw8<F32, VEC> w[BATCH];
    int row[BATCH], col[BATCH];
#pragma unroll
    for (int q = 0; q < BATCH; ++q) {
      row[q] = walk.r;
      col[q] = walk.c * 8;
      walk.next();
      if (STEP) w[q].load(wp, (R.row0 + row[q]) * P.ldw + R.col0 + col[q], row[q] < R.rows ? R.cols - col[q] : 0);
    }
#pragma unroll
    for (int q = 0; q < BATCH; ++q) {
      if (row[q] < R.rows) {
        const int nv = R.cols - col[q];
        float o[8], v[8];
        join8<PLANES>(piece_at(R.xs, R.x_rows, row[q], col[q]), R.x_plane, o);
        if (STEP) w[q].get(v, nv);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = STEP ? fmaf(P.decay, v[j], -lrs * (inv_s * o[j])) : inv_s * o[j];
        store8<F32, VEC>(wp, (R.row0 + row[q]) * P.ldw + R.col0 + col[q], nv, o);
      }
    }
  }
}

// `steps` products of 16 contraction elements: the operands advance by SA / SB (16-byte units) a step and
// by chunk_a / chunk_b after four (a 64-element chunk).  One thread issues them, and its instructions,
// not the tensor core, bound small products: four steps are unrolled with constant offsets.
template <int SA, int SB>
__device__ __forceinline__ void mma_steps(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, int steps,
                                          uint32_t chunk_a, uint32_t chunk_b, bool accumulate) {
  uint32_t acc = accumulate ? 1u : 0u;
  for (; steps >= 4; steps -= 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) tc_mma_f16_elect(d, a + SA * i, b + SB * i, idesc, i == 0 ? acc : 1u);
    acc = 1u;
    a += chunk_a;
    b += chunk_b;
  }
  for (int i = 0; i < steps; ++i) {
    tc_mma_f16_elect(d, a, b, idesc, acc);
    acc = 1u;
    a += SA;
    b += SB;
  }
}

// A finished update tile goes back into X: `tmem` is this warp's lane quarter of it, j its first
// long-side element.  The `parts` warps of a lane quarter share out the 32 x 32 pieces.  fp32 blocks add
// `keep` X here, in registers: as a term of B it would pass through the tensor core's sums, which cut every
// partial sum (a model of them with 24 bits: 1.8e-6 of O instead of 0.9e-6 after five quintic iterations).
template <bool TALL, bool F32>
__device__ __forceinline__ void drain_update(uint32_t tmem, int j, int part, int parts,
                                             uint32_t xs, int x_rows, uint32_t x_plane, int mp, int np,
                                             float upd_s, float keep) {
  constexpr int PLANES = F32 ? 2 : 1;
  const int lane = threadIdx.x & 31;
  if (j >= np) return;
  for (int c = 32 * part; c < mp; c += 32 * parts) {
    const uint32_t at = tmem + c;
    uint32_t a[16], b[16];
    if (TALL) {  // lane = long-side element, registers = its short-side ones
      tmem_load_32x16(at, a);
      tmem_load_32x16(at + 16, b);
    } else {  // fragments of 16 long-side elements
      tmem_load_16x32(at, a);
      tmem_load_16x32(at + (16u << 16), b);
    }
    tmem_load_wait();
    tmem_loaded(a);
    tmem_loaded(b);
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      float x[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) x[q] = upd_s * __uint_as_float(g < 2 ? a[8 * (g & 1) + q] : b[8 * (g & 1) + q]);
      uint4 o[PLANES];
      if (TALL) {
        const uint32_t dst = piece_at(xs, x_rows, j + lane, c + 8 * g);
        if (j + lane < np && c + 8 * g < mp) {
          if (F32) {
            float old[8];
            join8<PLANES>(dst, x_plane, old);
#pragma unroll
            for (int q = 0; q < 8; ++q) x[q] = fmaf(keep, old[q], x[q]);
          }
          split8<PLANES>(x, o);
#pragma unroll
          for (int q = 0; q < PLANES; ++q) st_shared_v4u(dst + q * x_plane, o[q]);
        }
      } else {
        // 16 long-side elements x 16 rows; lane 8q + i addresses row i of matrix q
        const int js = j + 16 * (g >> 1), cs = c + 16 * (g & 1);
        const uint32_t dst = piece_at(xs, x_rows, cs + 8 * (lane >> 4) + (lane & 7), js + 8 * ((lane >> 3) & 1));
        if (js < np && cs < mp) {
          if (F32) {
#pragma unroll
            for (int p = 0; p < PLANES; ++p) {
              uint32_t old[4];
              ldmatrix_x4_trans(dst + p * x_plane, old);
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const float2 f = unpack_half2(old[q]);
                x[2 * q] = fmaf(keep, f.x, x[2 * q]);
                x[2 * q + 1] = fmaf(keep, f.y, x[2 * q + 1]);
              }
            }
          }
          split8<PLANES>(x, o);
#pragma unroll
          for (int q = 0; q < PLANES; ++q) stmatrix_x4_trans(dst + q * x_plane, o[q].x, o[q].y, o[q].z, o[q].w);
        }
      }
    }
  }
}

// 32 columns of a Gram matrix held as the sum of `sets` accumulators, mp columns apart.
template <bool F32>
__device__ __forceinline__ void load_gram(uint32_t taddr, int mp, int sets, uint32_t (&r)[32]) {
  tmem_load_32cols(taddr, r);
  tmem_load_wait();
  if (F32) {
    tmem_loaded(r);
    for (int s = 1; s < sets; ++s) {
      uint32_t more[32];
      tmem_load_32cols(taddr + s * mp, more);
      tmem_load_wait();
      tmem_loaded(more);
#pragma unroll
      for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) + __uint_as_float(more[i]));
    }
  }
}

// An item of a cluster's exchange: columns 8 group .. 8 group + 7 of a row of a 16 x 32 piece of the Gram matrix.
// A warp has eight rows (of each eight columns in turn, so that it reads no bank twice) and so writes 64
// bytes of each row of A.
struct Item {
  int slot, row, group;  // slot: which of the CTA's pieces
  __device__ __forceinline__ explicit Item(int i) : slot(i >> 6), row((i & 7) + 8 * ((i >> 5) & 1)), group((i >> 3) & 3) {}
};

// An item's sum over the CTAs' partials, in rank order.
__device__ __forceinline__ void sum_item(uint32_t buf, int share, const Item& I, int C, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.f;
  for (int r = 0; r < C; ++r) {
    const uint32_t at = buf + (r * share + I.slot) * 2048 + I.group * 512 + I.row * 16;
    const uint4 a = ld_shared_v4u(at), b = ld_shared_v4u(at + 256);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += __uint_as_float(w[i]);
  }
}

// Sends an item's rounded values to every CTA's A.
template <int PLANES>
__device__ __forceinline__ void send_item(uint32_t as, int a_rows, uint32_t a_plane, const Item& I, int rank, int side,
                                          int mp, int C, float gram_s, float (&v)[8]) {
  const int k = I.slot * C + rank;  // piece of the matrix
  int left = k >> 1, tr = 0;
  while (tr < side && left >= side - tr) left -= side - tr++;
  const int row = 32 * tr + 16 * (k & 1) + I.row, col = 32 * (tr + left) + 8 * I.group;
  if (row >= mp || col >= mp) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] *= gram_s;
  uint4 o[PLANES];
  split8<PLANES>(v, o);
  const uint32_t dst = piece_at(as, a_rows, row, col);
  for (int r = 0; r < C; ++r) {
    const uint32_t to = map_shared_rank(dst, r);
#pragma unroll
    for (int q = 0; q < PLANES; ++q) st_cluster_v4(to + q * a_plane, o[q]);
  }
}

// The 32 x 32 tiles of A below the diagonal from those above it, 16 x 16 values a warp at a time.
template <int PLANES>
__device__ __forceinline__ void mirror_a(uint32_t as, int a_rows, uint32_t a_plane, int side, int mp, int warp, int warps) {
  const int lane = threadIdx.x & 31, n = (side * (side - 1) / 2) * 4 * PLANES;
  for (int w = warp; w < n; w += warps) {
    const int q = PLANES == 2 ? w & 1 : 0, sub = (PLANES == 2 ? w >> 1 : w) & 3;
    int left = (PLANES == 2 ? w >> 1 : w) >> 2, tr = 0;
    while (left >= side - 1 - tr) left -= side - 1 - tr++;
    const int row = 32 * tr + 16 * (sub & 1), col = 32 * (tr + 1 + left) + 16 * (sub >> 1);
    if (col >= mp) continue;
    // lane 8 i + r addresses row r of 8 x 8 matrix i: (i & 1) is its half of the rows, (i >> 1) of the columns
    const int h = (lane >> 3) & 1, k = lane >> 4, r = lane & 7;
    uint32_t v[4];
    ldmatrix_x4(piece_at(as, a_rows, row + 8 * h + r, col + 8 * k) + q * a_plane, v);
    stmatrix_x4_trans(piece_at(as, a_rows, col + 8 * k + r, row + 8 * h) + q * a_plane, v[0], v[1], v[2], v[3]);
  }
}

// 256 threads where two CTAs share an SM, 512 where one has it alone: 128 registers a thread in both.
template <bool TALL, bool F32, bool CLUSTER>
__global__ void __launch_bounds__(MAX_THREADS, 1) block_kernel(const __grid_constant__ BlockParams P) {
  constexpr int PLANES = F32 ? 2 : 1;
  extern __shared__ __align__(1024) uint8_t smem_raw[];

  const int tid = threadIdx.x, nt = blockDim.x, warp = tid >> 5, lane = tid & 31;
  const int C = CLUSTER ? P.cluster : 1;
  const uint32_t rank = CLUSTER ? cluster_cta_rank() : 0u;
  const int b = static_cast<int>(blockIdx.x) / C;
  const int l = b / P.per_matrix, in_mat = b - l * P.per_matrix;
  const int bi = in_mat / P.grid_cols, bj = in_mat - bi * P.grid_cols;
  const int row0 = bi * P.block_rows, col0 = bj * P.block_cols;
  const int br = min(P.block_rows, P.rows - row0), bc = min(P.block_cols, P.cols - col0);

  // the CTA's slice: rows_t x cols_t at (srow, scol) of the matrix, as it lies in memory
  const int nominal_m = TALL ? P.block_cols : P.block_rows;
  const int m = TALL ? bc : br, n = TALL ? br : bc;
  const int mp = round16(m);
  const int s0 = static_cast<int>(rank) * P.slice;
  const int ns = max(0, min(P.slice, n - s0));  // long-side elements here
  const int np = round16(ns);
  const int rows_t = TALL ? ns : m, cols_t = TALL ? m : ns;
  const int rows_p = TALL ? np : mp, cols_p = TALL ? mp : np;
  const int srow = row0 + (TALL ? s0 : 0), scol = col0 + (TALL ? 0 : s0);

  // shared memory: X planes, A planes, overrun, Gram partials
  const uint32_t xs = smem_addr(smem_raw);
  const int x_rows = TALL ? P.slice : round16(nominal_m);  // rows of a 64-column chunk
  const int a_rows = round16(nominal_m);
  const uint32_t x_plane = x_plane_bytes(nominal_m, P.slice, TALL);
  const uint32_t a_plane = a_plane_bytes(nominal_m);
  const uint32_t as = xs + PLANES * x_plane;
  const uint32_t behind = as + PLANES * a_plane + overrun_bytes(nominal_m);
  const uint32_t buf = P.alias ? as : behind, rest = behind + part_bytes(nominal_m, C, PLANES, P.alias != 0);
  Vars& V = *reinterpret_cast<Vars*>(smem_raw + (rest - xs));
  volatile int* abort_flag = &V.abort;
  const uint32_t bar = smem_addr(&V.bar);

  if (xs & 1023u) {  // the swizzled layouts need it; nothing has been touched yet
    if (tid == 0) atomicOr(P.status, kStatusTimeout);
    return;
  }
  if (tid == 0) {
    mbar_init(bar, 1);
    mbar_init(smem_addr(&V.drain), 2);
    for (int i = 0; i < MAX_SLOTS; ++i) mbar_init(smem_addr(&V.slot[i]), 1);
    V.abort = 0;
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc(smem_addr(&V.tmem), static_cast<uint32_t>(P.tmem_cols));
    tmem_relinquish();
  }

  wait_for_previous_kernel();
  let_next_kernel_start();

  // ------------------------------------------------------------ momentum and norm
  // U is kept in shared memory while its norm is not known: fp16 pieces of eight, each scaled by its
  // own power of two (one exponent byte a piece, held where A will be), exact but for the rounding to
  // the planes' bits.  Once the norm is known the pieces are brought to one power of two.
  const Region R{rows_t, cols_t, rows_p, cols_p >> 3, srow, scol, xs, x_plane, x_rows};
  const bool vec = P.vec != 0 && cols_t % 8 == 0;
  const int npieces = R.rows_p * R.pieces;
  uint8_t* const exps = smem_raw + (as - xs);
  double sq;
  if (P.step) {
    if (vec) {
      // the apply pass reads W after the products: bring it to L2 meanwhile
      prefetch_region<F32 ? 4 : 2>(P.w[l], P.ldw, srow, scol, rows_t, cols_t);
      sq = momentum_pass<F32, true, true>(P, R, P.g[l], P.m[l], exps);
    } else {
      sq = momentum_pass<F32, true, false>(P, R, P.g[l], P.m[l], exps);
    }
  } else {
    sq = vec ? momentum_pass<F32, false, true>(P, R, P.g[l], nullptr, exps)
             : momentum_pass<F32, false, false>(P, R, P.g[l], nullptr, exps);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, d);
  if (lane == 0) V.red[warp] = sq;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = V.tmem;
  double total = 0.0;
  for (int w = 0; w < nt / 32; ++w) total += V.red[w];
  if (CLUSTER) {
    if (tid == 0) V.sum = total;
    cluster_sync();
    total = 0.0;
    for (int r = 0; r < C; ++r) total += ld_cluster_f64(map_shared_rank(smem_addr(&V.sum), r));
  }
  const float nu = static_cast<float>(sqrt(total));
  const float inv = 1.f / (nu + P.eps);
  const bool fine = isfinite(nu) && isfinite(inv);
  if (tid == 0 && rank == 0) {
    P.nu[b] = nu;
    P.flags[b] = fine ? 0 : MUON_FLAG_NONFINITE;
    if (!fine) atomicOr(P.status, kStatusNonfinite);
  }

  if (fine) {  // the same in every CTA of the cluster
    // ---------------------------------------------------------- X = U / (nu + eps), held at store_scale
    // as first * X: the pieces only move by powers of two, `first` in [1, 2) is applied to the first
    // iteration's products.
    const float S = P.store_scale, inv_s = 1.f / S;
    int block_e;
    const float first = frexpf(inv, &block_e) * 2.f;  // inv = first * 2^(block_e - 1)
    block_e += ilogbf(S) - 1;
    PieceWalk w2(tid, R.pieces);
    for (int i = tid; i < npieces; i += nt, w2.next()) {
      const uint32_t at = piece_at(xs, x_rows, w2.r, w2.c * 8);
      // piece value = stored * 2^(e - TOP_EXP); at the block's scale: times 2^block_e
      const float up = exp2i(min(static_cast<int>(exps[i]) - EXP_BIAS - TOP_EXP + block_e, 127));
#pragma unroll
      for (int t = 0; t < PLANES; ++t) {
        const uint4 p = ld_shared_v4u(at + t * x_plane);
        uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = unpack_half2(w[j]);
          w[j] = pack_half2(up * f.x, up * f.y);
        }
        st_shared_v4u(at + t * x_plane, make_uint4(w[0], w[1], w[2], w[3]));
      }
    }
    fence_proxy_async_smem();
    __syncthreads();

    // While this block is multiplied, memory is idle: bring the block that follows on the SM to L2.
    if (b + P.ahead < P.blocks && P.ahead > 0 && vec) {
      const int b2 = b + P.ahead, l2 = b2 / P.per_matrix, in2 = b2 - l2 * P.per_matrix;
      const int i2 = in2 / P.grid_cols, j2 = in2 - i2 * P.grid_cols;
      const int r2 = i2 * P.block_rows + (TALL ? s0 : 0), c2 = j2 * P.block_cols + (TALL ? 0 : s0);
      const int nr = min(rows_t, P.rows - r2), nc = min(cols_t, P.cols - c2);
      prefetch_region<F32 ? 4 : 2>(P.g[l2], P.ldg, r2, c2, nr, nc);
      if (P.step) prefetch_region<4>(P.m[l2], P.ldm, r2, c2, nr, nc);
    }

    // ---------------------------------------------------------- Newton-Schulz
    uint32_t parity = 0;
    const int uwarp = __shfl_sync(0xffffffffu, warp, 0);  // known to be uniform: its branches issue products
    const int quarter = warp & 3, sub = warp >> 2, parts = nt >> 7;  // warps of a lane quarter
    const uint32_t lane_off = static_cast<uint32_t>(32 * quarter) << 16;
    // plane pairs, smallest products first: hi lo, lo hi, hi hi
    constexpr int NPAIR = PLANES == 2 ? 3 : 1;
    auto pair_a = [](int q) { return NPAIR == 1 ? 0 : q == 1 ? 1 : 0; };
    auto pair_b = [](int q) { return NPAIR == 1 ? 0 : q == 0 ? 1 : 0; };
    const uint32_t x_chunk = static_cast<uint32_t>(x_rows) * 128u, a_chunk = static_cast<uint32_t>(a_rows) * 128u;
    auto wait_mma = [&]() {
      mbar_wait_bounded(bar, parity, abort_flag, P.status);
      parity ^= 1u;
      tc_fence_after();
    };
    // Products with A's rows in the lanes: 64 of them do for short sides up to 64 (rows 16 q .. 16 q + 15 in
    // lanes 32 q ..), for which the operands cost the shared memory 32 instead of 48 clocks an instruction
    // (blocks of 64 x 768: 149 instead of 153 us for 576 of them, 16.2 instead of 16.7 us for one 48 x 100).
    const int am = mp <= 64 ? 64 : 128;
    const int arow = am / 4 * quarter + lane;                       // this lane's row
    const bool ahere = am / 4 * quarter < mp, amine = lane < am / 4 && arow < mp;  // the warp has rows, the lane one
    // TMEM: the Gram matrix (and its square) from column 0 on, then the update's slots (reads take 32 columns)
    const int tiles = (ns + 127) / 128;
    const int sets = F32 ? max(1, (tiles + GRAM_TILES - 1) / GRAM_TILES) : 1;
    const int slots = min(MAX_SLOTS, (P.tmem_cols - sets * mp - (((mp + 31) & ~31) - mp)) / mp);
    const uint32_t slot0 = tmem + sets * mp;
    uint32_t slot_parity = 0;
    // Gram part of long-side elements 128 t .. 128 t + 127
    auto issue_gram = [&](int t) {
      const uint32_t idesc = instr_desc_f16(am, mp, TALL, TALL);
      const uint32_t lbo = TALL ? x_chunk : 16u;
      const int first_t = F32 ? t % GRAM_TILES : t;
      const uint32_t d = tmem + (F32 ? t / GRAM_TILES * mp : 0);
      const uint32_t at = TALL ? t * (128u * 128u) : 2 * t * x_chunk, chunk = (TALL ? 64u * 128u : x_chunk) >> 4;
#pragma unroll
      for (int q = 0; q < NPAIR; ++q)
        mma_steps<TALL ? 128 : 2, TALL ? 128 : 2>(d, smem_desc_sw128(xs + pair_a(q) * x_plane + at, lbo, 1024u),
                                                  smem_desc_sw128(xs + pair_b(q) * x_plane + at, lbo, 1024u), idesc,
                                                  min(8, np / 16 - 8 * t), chunk, chunk, (q | first_t) != 0);
    };
    // update tile t into a slot
    auto issue_update = [&](int t, int slot) {
      const uint32_t idesc = instr_desc_f16(128, mp, !TALL, false);
      const uint32_t tile_off = static_cast<uint32_t>(t) * (TALL ? 128u * 128u : 2u * x_chunk);
#pragma unroll
      for (int q = 0; q < NPAIR; ++q)
        mma_steps<TALL ? 2 : 128, 2>(slot0 + slot * mp,
                                     smem_desc_sw128(xs + pair_a(q) * x_plane + tile_off, TALL ? 16u : x_chunk, 1024u),
                                     smem_desc_sw128(as + pair_b(q) * a_plane, 16u, 1024u), idesc, mp / 16,
                                     TALL ? x_chunk >> 4 : 512u, a_chunk >> 4, q != 0);
      tc_commit_elect(smem_addr(&V.slot[slot]));
    };
    for (int it = 0; it < P.k; ++it) {
      const float ca = P.abc[3 * it], cb = P.abc[3 * it + 1], cc = P.abc[3 * it + 2];
      // the first iteration's X is first * (what is stored)
      const float gram_s = it == 0 ? inv_s * first * first : inv_s, upd_s = it == 0 ? inv_s * first : inv_s;
      if (it == 0 && uwarp == 1) {
        for (int t = 0; t < tiles; ++t) issue_gram(t);
        tc_commit_elect(bar);
      }
      wait_mma();
      if (!CLUSTER) {
        const int i = arow;
        if (ahere) {
          for (int c = 32 * sub; c < mp; c += 32 * parts) {
            uint32_t r[32];
            __syncwarp();
            load_gram<F32>(tmem + lane_off + c, mp, sets, r);
            if (amine) {
#pragma unroll
              for (int h = 0; h < 4; ++h) {
                if (c + 8 * h < mp) {
                  float v[8];
#pragma unroll
                  for (int j = 0; j < 8; ++j) v[j] = gram_s * __uint_as_float(r[8 * h + j]);
                  uint4 o[PLANES];
                  split8<PLANES>(v, o);
#pragma unroll
                  for (int q = 0; q < PLANES; ++q) st_shared_v4u(piece_at(as, a_rows, i, c + 8 * h) + q * a_plane, o[q]);
                }
              }
            }
          }
        }
      } else {
        // this CTA's partial goes to the CTAs that sum its pieces
        const int side = side_tiles(mp), tr = am / 4 * quarter / 32, share = piece_share(mp, C);
        if (P.alias) cluster_sync();  // no CTA's A is in use
        if (ahere) {
          for (int tc = tr + sub; tc < side; tc += parts) {
            uint32_t r[32];
            __syncwarp();
            load_gram<F32>(tmem + lane_off + 32 * tc, mp, sets, r);
            if (amine) {
              const int k = 2 * (tr * side - tr * (tr - 1) / 2 + tc - tr) + ((arow >> 4) & 1), slot = k / C;
              const uint32_t to = map_shared_rank(buf + (rank * share + slot) * 2048 + (arow & 15) * 16, k - slot * C);
#pragma unroll
              for (int h = 0; h < 8; ++h)
                st_cluster_v4(to + 256 * h, np > 0 ? make_uint4(r[4 * h], r[4 * h + 1], r[4 * h + 2], r[4 * h + 3])
                                                   : make_uint4(0, 0, 0, 0));
            }
          }
        }
        cluster_sync();
        // sum this CTA's pieces and send them to every CTA's A
        const Item item0(tid), item1(tid + nt);
        float v0[8], v1[8];
        if (item0.slot < share) sum_item(buf, share, item0, C, v0);
        if (item1.slot < share) sum_item(buf, share, item1, C, v1);
        if (P.alias) cluster_sync();  // all have read
        if (item0.slot < share) send_item<PLANES>(as, a_rows, a_plane, item0, rank, side, mp, C, gram_s, v0);
        if (item1.slot < share) send_item<PLANES>(as, a_rows, a_plane, item1, rank, side, mp, C, gram_s, v1);
        cluster_sync();
        mirror_a<PLANES>(as, a_rows, a_plane, side, mp, uwarp, nt / 32);
        fence_proxy_async_cluster();
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncthreads();
      // square of A, then B = a I + b A + c A A over A (fp32: without a I)
      if (cc != 0.f) {
        if (uwarp == 0) {
          tc_fence_after();
          const uint32_t idesc = instr_desc_f16(am, mp, false, false);
#pragma unroll
          for (int q = 0; q < NPAIR; ++q)
            mma_steps<2, 2>(tmem, smem_desc_sw128(as + pair_a(q) * a_plane, 16u, 1024u),
                            smem_desc_sw128(as + pair_b(q) * a_plane, 16u, 1024u), idesc, mp / 16, a_chunk >> 4,
                            a_chunk >> 4, q != 0);
          tc_commit_elect(bar);
        }
        wait_mma();
      }
      {
        const int i = arow;
        if (ahere) {
          for (int c = 32 * sub; c < mp; c += 32 * parts) {
            uint32_t r[32];
            if (cc != 0.f) {
              __syncwarp();
              tmem_load_32cols(tmem + lane_off + c, r);
              tmem_load_wait();
            }
            if (amine) {
#pragma unroll
              for (int h = 0; h < 4; ++h) {
                if (c + 8 * h < mp) {
                  const uint32_t at = piece_at(as, a_rows, i, c + 8 * h);
                  float v[8];
                  join8<PLANES>(at, a_plane, v);
#pragma unroll
                  for (int j = 0; j < 8; ++j) {
                    v[j] = cb * v[j] + (!F32 && i == c + 8 * h + j ? ca * S : 0.f);
                    if (cc != 0.f) v[j] = fmaf(cc * inv_s, __uint_as_float(r[8 * h + j]), v[j]);
                  }
                  uint4 o[PLANES];
                  split8<PLANES>(v, o);
#pragma unroll
                  for (int q = 0; q < PLANES; ++q) st_shared_v4u(at + q * a_plane, o[q]);
                }
              }
            }
          }
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncthreads();
      // Update and the next Gram matrix, tile by tile of 128 long-side elements: while a tile is drained,
      // the tensor core multiplies the following tiles and the Gram part of the drained ones.
      if (uwarp == 0) {
        tc_fence_after();
        for (int t = 0; t < min(slots, tiles); ++t) issue_update(t, t);
      }
      for (int t = 0, slot = 0; t < tiles; ++t) {
        mbar_wait_bounded(smem_addr(&V.slot[slot]), (slot_parity >> slot) & 1u, abort_flag, P.status);
        slot_parity ^= 1u << slot;
        tc_fence_after();
        drain_update<TALL, F32>(slot0 + slot * mp + lane_off, t * 128 + 32 * quarter, sub, parts, xs, x_rows, x_plane,
                                mp, np, upd_s, it == 0 ? ca * first : ca);
        fence_proxy_async_smem();
        tc_fence_before();
        __syncthreads();
        if (uwarp == 0) {
          tc_fence_after();
          if (t + slots < tiles) issue_update(t + slots, slot);
        } else if (uwarp == 1 && it + 1 < P.k) {
          tc_fence_after();
          issue_gram(t);
        }
        if (++slot == slots) slot = 0;
      }
      if (uwarp == 1 && it + 1 < P.k) tc_commit_elect(bar);
    }

    // ---------------------------------------------------------- apply
    bool good = *abort_flag == 0;
    if (CLUSTER) {
      cluster_sync();
      for (int r = 0; r < C; ++r) good = good && __float_as_int(ld_cluster_f(map_shared_rank(smem_addr(&V.abort), r))) == 0;
    }
    if (good) {
      float lrs = P.lr;
      if (P.scale_mode == MUON_SCALE_SQRT_RATIO) lrs *= sqrtf(fmaxf(1.f, static_cast<float>(br) / static_cast<float>(bc)));
      else if (P.scale_mode == MUON_SCALE_RMS_MATCH) lrs *= 0.2f * sqrtf(static_cast<float>(max(br, bc)));
      void* wp = P.w[l];
      if (P.step) {
        if (vec) apply_pass<F32, true, true>(P, R, wp, lrs, inv_s);
        else apply_pass<F32, true, false>(P, R, wp, lrs, inv_s);
      } else {
        if (vec) apply_pass<F32, false, true>(P, R, wp, lrs, inv_s);
        else apply_pass<F32, false, false>(P, R, wp, lrs, inv_s);
      }
    }
  }

  if (*abort_flag && warp < 2) {  // let the products these warps issued finish, within a limit
    tc_commit_elect(smem_addr(&V.drain));
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(smem_addr(&V.drain), 0) && global_timer_ns() - t0 < 200000000ull) {
    }
  }
  if (CLUSTER) cluster_sync();  // nobody leaves while its shared memory may be read
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, static_cast<uint32_t>(P.tmem_cols));
  }
}

template <bool TALL, bool F32, bool CLUSTER>
cudaError_t launch_variant(const BlockParams& p, int blocks, size_t smem, cudaStream_t stream) {
  constexpr int kMaxDevices = 64;
  static std::atomic<bool> configured[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDevices || !configured[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(block_kernel<TALL, F32, CLUSTER>, cudaFuncAttributeMaxDynamicSharedMemorySize, 226 * 1024);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDevices) configured[dev].store(true, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks) * p.cluster);
  cfg.blockDim = dim3(static_cast<unsigned>(p.threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, block_kernel<TALL, F32, CLUSTER>, p);
}

}  // namespace

size_t block_smem_bytes(int shorter, int slice, bool tall, bool f32, int cluster, bool alias) {
  const size_t planes = f32 ? 2 : 1;
  // the exponent bytes of X's pieces share A's place
  if (static_cast<size_t>(round16(shorter)) * slice / 8 > planes * a_plane_bytes(shorter) + overrun_bytes(shorter))
    return SIZE_MAX;
  return planes * (x_plane_bytes(shorter, slice, tall) + a_plane_bytes(shorter)) + overrun_bytes(shorter) +
         part_bytes(shorter, cluster, static_cast<int>(planes), alias) + sizeof(Vars);
}

cudaError_t launch_blocks(const BlockParams& p, int blocks, bool tall, bool f32, size_t smem, cudaStream_t stream) {
  const bool cl = p.cluster > 1;
  auto go = [&](auto t, auto f) {
    return cl ? launch_variant<t.value, f.value, true>(p, blocks, smem, stream)
              : launch_variant<t.value, f.value, false>(p, blocks, smem, stream);
  };
  using Yes = std::true_type;
  using No = std::false_type;
  return tall ? (f32 ? go(Yes(), Yes()) : go(Yes(), No())) : (f32 ? go(No(), Yes()) : go(No(), No()));
}

}  // namespace muon
