// Products of sorted token rows with the weights of the experts they belong to, and the weight
// gradients, on the tensor cores of sm_100a.  Rows offsets[e] .. offsets[e+1] belong to expert e:
//
//   forward    Y[t, :]  = W_e X[t, :]          out columns = N, contraction K
//   backward   dX[t, :] = W_e^T dY[t, :]       out columns = K, contraction N
//   gradient   G_e      = beta G_e + scale dY_e^T X_e   out N x K per expert, contraction over tokens
//
// All three form the TRANSPOSE of their output tile: the 128 TMEM lanes hold 128 output columns
// ("features", the side whose size is the same for every expert) and the accumulator's columns hold
// up to 256 output rows.  The tensor core's N is a multiple of 16 where its M is 128, so the ragged
// side costs at most 15 idle rows per segment instead of 127, few tokens cost few MMA cycles, and
// consecutive lanes hold consecutive output columns, so plain coalesced stores end a segment at any row.
//
//   forward    A = W_e  K-major   (features n)     B = X   K-major  (rows t)
//   backward   A = W_e  MN-major  (features k)     B = dY  K-major  (rows t)
//   gradient   A = X    MN-major  (features k)     B = dY  MN-major (rows n), contraction t
//
// The segments are read on the device (no host synchronisation): every CTA scans the offsets,
// derives the same tile list and walks it round-robin.  Warp 0 issues TMA loads into a ring of stages
// (64 deep), warp 1 the MMAs into two 256-column accumulators, warps 2..9 drain them.  The last
// token step of a segment's gradient holds rows of the next segment: warp 1 zeroes them in shared
// memory (both operands, up to the next multiple of 16) before its MMAs read them.
// fp32 operands are split into three bf16 planes and multiplied as six plane products, as in the
// Newton-Schulz kernel: by a packing pass before this kernel, or, where an expert has few tokens and so
// reads its weights once, by eight warps of this kernel, which store the planes where a TMA would have.
//
// Measured (GPU time; floor: the bytes at the copy rate of 6.53 TB/s or the operations at the library's
// 1.62 PFLOP/s) and what bounds it:
//   32 experts of 4096 x 2048, 32768 tokens   430 us (339: operations)  tensor pipe, 77 % busy; 5.8 GB through L2
//     (up to a hundred in a row, at 1965 MHz; a thousand run at 1.36 GHz under the power cap and take 482)
//   8 of 1536 x 768, 8192 tokens              22.8 us (11.9: operations)  210 pair tiles or more for 74 pairs: three
//     rounds, 14 us of products, and the start of the first and the draining of the last
//   64 of 1536 x 768, 24 tokens               14.0 us (8.7: bytes)  set-up 2.4 us, first loads 1.8, last stores 2
//   input gradient, 16 of them, 8191 tokens   25.0 us (11.9)  about 132 pair tiles: two rounds, the second 80 % full
//   gradient into fp32, 16 of them            48.5 us (28.9: bytes)  additions in the memory system, 2 TB/s of them
// A launch sets up while the one before it drains (programmatic serialisation): 14.0 instead of 14.5 us for
// the fourth, 22.8 instead of 23.7 us for the second.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <climits>

#include "device_utils.cuh"
#include "experts.h"
#include "../../include/muon.h"

namespace muon {

namespace {

constexpr int FM = 128;   // features per tile
constexpr int RN = 256;   // rows per tile, at most
constexpr int BK = 64;
// Operand and output types: bf16 both; bf16 operands with an fp32 output (gradients); fp32 both.  fp32
// operands bring all three planes of a contraction tile at once and make their six products from them;
// the same split by this kernel's own warps.
enum Kind { BF16_BF16 = 0, BF16_F32 = 1, F32_F32 = 2, F32_SPLIT = 3 };

// The ring holds as many stages as fit for the launch's widest tile: four of 256 rows, ten of a few.
// (With four stages in flight a narrow tile's stage takes a quarter of a load's latency, however small.)
__host__ __device__ constexpr uint32_t ring_bytes(int kind) {
  return (kind == BF16_F32 || kind == F32_F32 ? 176u : 192u) * 1024u;
}
constexpr int MAX_STAGES = 10;
constexpr uint32_t A_BYTES = FM * BK * 2;
constexpr uint32_t CHUNK_BYTES = 64 * BK * 2;  // MN-major: 64 columns x 64 contraction rows
// fp32 outputs: contraction tiles a TMEM accumulator sums before registers take over
__host__ __device__ constexpr int part_tiles(int kind) { return kind >= F32_F32 ? 2 : 8; }
// bf16 gradients: the same, for segments that are longer than this (32768 tokens), and the rows a tile of a launch
// with such segments has at most, so that the sums fit the registers.  Sums of 8192 tokens would narrow the tiles
// of ordinary launches (4 experts of 1536 x 768, 16384 tokens each: 155 us, 122 as it is); sums of 256 rows would
// spill registers in all of them (64 of 512 x 512, 64 tokens each: 24.0 us, 21.3 as it is).
constexpr int LONG_PART = 512, LONG_ROWS = 128;
__host__ __device__ constexpr int epi_warps(int kind) { return kind == F32_SPLIT ? 4 : 8; }
constexpr int SPLIT_WARPS = 8, SPLIT_ROWS = 64;  // F32_SPLIT: its warps, and rows of its tiles at most
// Staging per epilogue warp: 32 rows x 32 bf16, or two boxes of 16 rows x 32 fp32.
__host__ __device__ constexpr uint32_t staging_bytes(int kind) { return kind == BF16_BF16 ? 2048u : 4096u; }
// Fourteen warps with the split: four a scheduler leave each thread 128 registers (with 18, loads under way were
// spilled, which waits for each: 63 instead of 42 us for 64 experts of 1536 x 768 and 24 tokens).
__host__ __device__ constexpr int threads_of(int kind) {
  return 64 + 32 * epi_warps(kind) + (kind == F32_SPLIT ? 32 * SPLIT_WARPS : 0);
}
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t ACC_COLS = 256;
constexpr int NUM_BARS = 3 * MAX_STAGES + 5;
constexpr uint32_t BAR_BYTES = 8 * NUM_BARS + 24;
constexpr uint64_t kDrainLimitNs = 200000000ull;

// Tile widths to choose from: 256, 224, .., 32 rows; the launch takes the one whose rounds of tiles cost least.
// Wide tiles load less per product, narrow ones fill the last round: 16 experts of 2048 x 2048, 512 tokens
// 28.8 us chosen, 31.6 with 256, 29.1 with 128; 8 of 1536 x 768, 8192 tokens 22.8 chosen and with 256, 33.8
// with 128, 53.2 with 64; gradients of 16 of them 48.5 chosen and with 256, 55.0 with 128.
constexpr int kWidths = 8;
constexpr int kTileOverhead = 640;   // a tile's fixed cost, in operand rows loaded
constexpr int kMaxOrdered = 256;

struct Tile {
  int e;       // expert
  int f0;      // first output column
  int r0, nr;  // first output row (token row, or row of G_e) and how many the tile holds
  int nw;      // accumulator columns: nr rounded up to 16 (pair: 32)
  int k0, kn;  // gradient: first token and tokens of the segment
};

// Per-expert table in shared memory: first tile and first token row.
struct Segments {
  const int* base;  // [experts + 1] first tile, in `order`
  const int* off;   // [experts + 1] first token row
  const int* order; // [experts] experts as the tiles take them, or null: as they are
  int width;        // rows of a tile, at most
};

// PAIR: two CTAs of a cluster share a tile of 256 features: each holds 128 of them and half of the rows
// operand, so the pair loads a third less per product than two single tiles.  The instruction's N is a
// multiple of 32 there.
template <bool PAIR>
__device__ __forceinline__ int round_rows(int x) { return PAIR ? (x + 31) & ~31 : (x + 15) & ~15; }
template <bool PAIR>
__device__ __forceinline__ int feature_tiles(const ExpertParams& P) {
  return (P.features + (PAIR ? 2 : 1) * FM - 1) / ((PAIR ? 2 : 1) * FM);
}

// A segment's rows are cut evenly into tiles of at most `width` rows.
__device__ __forceinline__ int row_tiles(int rows, int width) { return (rows + width - 1) / width; }

template <int MODE, bool PAIR>
__device__ __forceinline__ int expert_tiles(const ExpertParams& P, int tokens, int width) {
  const int nf = feature_tiles<PAIR>(P);
  if (MODE == EXPERT_WGRAD) return tokens == 0 && P.beta == 1.f ? 0 : nf * row_tiles(P.rows, width);
  return nf * row_tiles(tokens, width);
}

// Tile t as CTA `rank` of its pair sees it: its own 128 features, all rows.
template <int MODE, bool PAIR>
__device__ __forceinline__ Tile decode_tile(const ExpertParams& P, const Segments& S, int t, int rank) {
  int lo = 0, hi = P.experts - 1;  // last expert whose first tile is <= t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (S.base[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  Tile ti;
  ti.e = S.order != nullptr ? S.order[lo] : lo;
  const int begin = S.off[ti.e], tokens = S.off[ti.e + 1] - begin;
  const int local = t - S.base[lo];
  const int nf = feature_tiles<PAIR>(P);
  const int rt = local / nf;
  ti.f0 = (local - rt * nf) * (PAIR ? 2 * FM : FM) + FM * rank;
  const int total = MODE == EXPERT_WGRAD ? P.rows : tokens;
  const int parts = row_tiles(total, S.width);
  const int width = round_rows<PAIR>((total + parts - 1) / parts);
  const int r = rt * width;
  ti.nr = min(width, total - r);
  ti.nw = round_rows<PAIR>(ti.nr);
  ti.r0 = MODE == EXPERT_WGRAD ? r : begin + r;
  ti.k0 = begin;
  ti.kn = tokens;
  return ti;
}

// Smallest token box (16 << box rows) that holds `rows` rows.
__device__ __forceinline__ int box_of(int rows) { return rows <= 16 ? 0 : 28 - __clz(rows - 1); }

// Plane pairs of the split products, smallest first (plane 0 = hi, 1 = mid, 2 = lo):
// mid mid, hi lo, lo hi, hi mid, mid hi, hi hi.
__device__ __forceinline__ int plane_a(int seg) { return (0x10201 >> (4 * seg)) & 0xF; }
__device__ __forceinline__ int plane_b(int seg) { return (0x01021 >> (4 * seg)) & 0xF; }

// Shared memory of one plane of `rows` rows of the rows operand: chunks of 64 (MN-major), or a token box.
template <bool B_MN, bool SPLIT>
__device__ __forceinline__ uint32_t b_bytes(int rows) {
  return static_cast<uint32_t>(B_MN ? (rows + 63) / 64 * 64 : SPLIT ? rows : 16 << box_of(rows)) * BK * 2;
}

// Position in the ring: stage and the phase of its barriers.
struct Ring {
  int s = 0;
  uint32_t phase = 0, count = 0;
  __device__ __forceinline__ void next(int stages) {
    ++count;
    if (++s == stages) {
      s = 0;
      phase ^= 1u;
    }
  }
  // whether the stage has been filled before
  __device__ __forceinline__ bool filled(int stages) const { return count >= static_cast<uint32_t>(stages); }
};

__device__ __forceinline__ bool wait_drain(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (global_timer_ns() - t0 > kDrainLimitNs) return false;
  }
  return true;
}

__device__ __forceinline__ void st_shared_zero16(uint32_t addr) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(addr), "r"(0) : "memory");
}

// Zero contraction rows [first, last) of `chunks` MN-major chunks (128-byte rows; the swizzle
// permutes 16-byte pieces inside a row only).
__device__ __forceinline__ void zero_rows(uint32_t base, int chunks, int first, int last, int lane) {
  for (int c = 0; c < chunks; ++c)
    for (int r = first + (lane >> 3); r < last; r += 4) st_shared_zero16(base + c * CHUNK_BYTES + r * 128 + (lane & 7) * 16);
}

// Output rows first .. last - 1 (STACK: of the gradients, counted through the experts) become zero: a warp of the
// grid takes a row at a time.
template <bool STACK>
__device__ __forceinline__ void clear_rows(const ExpertParams& P, int first, int last, int warp, int warps, int lane) {
  const int bytes = P.out_f32 ? 4 : 2, row_bytes = P.features * bytes;
  for (int r = first + warp; r < last; r += warps) {
    const int e = STACK ? r / P.rows : 0;
    char* row = static_cast<char*>(P.out) + (STACK ? e * P.s_out + (r - e * P.rows) * P.ld_out : r * P.ld_out) * bytes;
    const int wide = P.vec ? row_bytes & ~15 : 0;
    for (int i = 16 * lane; i < wide; i += 512) *reinterpret_cast<uint4*>(row + i) = make_uint4(0, 0, 0, 0);
    for (int i = wide + 2 * lane; i < row_bytes; i += 64) *reinterpret_cast<uint16_t*>(row + i) = 0;
  }
}

// One lane's column f of 32 bf16 output rows, v[i] in row i, added to beta * G: at = element offset of
// (first row, f).
__device__ __forceinline__ void add_column(const ExpertParams& P, long long at, int f, int nv, const float (&v)[32]) {
  if (f >= P.features) return;
  uint16_t* o = static_cast<uint16_t*>(P.out) + at;
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (i < nv)
      o[i * P.ld_out] =
          float_to_bf16_bits(P.beta != 0.f ? fmaf(P.beta, bf16_bits_to_float(o[i * P.ld_out]), v[i]) : v[i]);
}

// fp32 output: 32 columns from fw on (one a lane) x nv <= 32 rows from `row` on, v[i] in row i; at =
// element offset of (row, fw).  Full boxes of 16 rows go through shared memory, from where one TMA
// copies them (beta = 0) or adds them to G (beta = 1): the addition is done by the memory system, once
// per element, so nothing is read back and the order is fixed (16 experts of 1536 x 768: 48.5 us, 91.6
// with loads and stores; one bulk copy a row cost ~17 cycles each, whatever its length).  `boxes` counts this
// warp's, for the two staging buffers.
__device__ __forceinline__ void store_rows(const ExpertParams& P, long long at, int row, int e, bool rows_end,
                                           uint32_t stage, int& boxes, int fw, int nv, int lane, const float (&v)[32]) {
  float* const out = static_cast<float*>(P.out) + at;
  const int nf = P.features - fw;  // columns that exist
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (16 * h >= nv) break;
    // The map ends where the output does; a box may only be cut short there.  A store cuts the columns at a
    // 16-byte boundary, behind which up to three elements of the caller's may begin: then the last columns go
    // out one by one.
    if (P.vec && (P.beta == 0.f || P.beta == 1.f) && (16 * h + 16 <= nv || rows_end) &&
        (nf >= 32 || P.features % 4 == 0)) {
      const uint32_t buf = stage + (boxes++ & 1) * 2048u;
      if (lane == 0) bulk_wait_group_read<1>();  // the box before the last one has left this buffer
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 16; ++i)
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(buf + 128u * i + 4u * lane), "f"(v[16 * h + i]) : "memory");
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (P.beta == 0.f) tma_store_3d(&P.tmOut, buf, fw, row + 16 * h, e);
        else tma_add_3d(&P.tmOut, buf, fw, row + 16 * h, e);
        bulk_commit_group();
      }
    } else {
      float old[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        old[i] = 0.f;
        if (P.beta != 0.f && lane < nf && 16 * h + i < nv) old[i] = out[(16 * h + i) * P.ld_out + lane];
      }
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (lane < nf && 16 * h + i < nv) out[(16 * h + i) * P.ld_out + lane] = fmaf(P.beta, old[i], v[16 * h + i]);
    }
  }
}

// 16-byte piece r of a staged 32-row x 64-byte tile: pieces are permuted so that neither the transposed
// stores (eight rows of one piece) nor the reads (rows of four pieces) hit a bank twice.
__device__ __forceinline__ uint32_t staged_piece(uint32_t base, int row, int piece) {
  return base + static_cast<uint32_t>(row * 64 + ((piece ^ ((row >> 1) & 3)) << 4));
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// bf16 output, nothing to add to: 32 lanes (features fw ..) x 32 columns (rows) of the accumulator at
// `taddr`, rounded, transposed through shared memory and stored 16 bytes a lane, four lanes a row.
__device__ __forceinline__ void store_staged(const ExpertParams& P, uint32_t taddr, uint32_t stage, long long at, int fw,
                                             int nv, float scale, int lane) {
  uint32_t r[2][16];
  tmem_load_16x32(taddr, r[0]);
  tmem_load_16x32(taddr + (16u << 16), r[1]);
  tmem_load_wait();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    tmem_loaded(r[h]);
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
      uint32_t w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        w[q] = pack_bf16(scale * __uint_as_float(r[h][4 * k + 2 * q]), scale * __uint_as_float(r[h][4 * k + 2 * q + 1]));
      // lane 8q + i addresses row i of matrix q: features 8 (q & 1) .. of output rows 8 (k + q / 2) ..
      stmatrix_x4_trans(staged_piece(stage, 8 * (k + (lane >> 4)) + (lane & 7), 2 * h + ((lane >> 3) & 1)), w[0], w[1],
                        w[2], w[3]);
    }
  }
  __syncwarp();
  const int piece = lane & 3, f = fw + 8 * piece;
  uint4 v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[i].x), "=r"(v[i].y), "=r"(v[i].z), "=r"(v[i].w)
                 : "r"(staged_piece(stage, 8 * i + (lane >> 2), piece)));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = 8 * i + (lane >> 2);
    if (row < nv && f < P.features) {
      uint16_t* o = static_cast<uint16_t*>(P.out) + at + row * P.ld_out + 8 * piece;
      if (P.vec && f + 8 <= P.features) {
        *reinterpret_cast<uint4*>(o) = v[i];
      } else {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (f + j < P.features) o[j] = static_cast<uint16_t>(w[j / 2] >> (16 * (j & 1)));
      }
    }
  }
  __syncwarp();  // the staging tile is free again
}

// An fp32 operand's part of a tile, as `units` rows of 64 shared-memory columns.  K-major: unit u is row
// first + u of the matrix, its columns contraction elements; MN-major: unit 64 c + r is 64-column chunk c
// of contraction row r.
struct Side {
  const float* p;  // the matrix
  long long ld;
  int first, end;  // rows (K-major) or columns (MN-major) that exist: [first, end)
  int units;
};

// Predicated loads, zeros where `here` is false: without a branch the loads of a warp are all under way at once.
__device__ __forceinline__ float2 load_pair(const float* p, bool here) {
  float2 v;
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %3, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\t"
               "@q ld.global.v2.f32 {%0, %1}, [%2];\n\t}"
               : "=&f"(v.x), "=&f"(v.y)
               : "l"(p), "r"(static_cast<int>(here)));
  return v;
}
__device__ __forceinline__ float load_one(const float* p, bool here) {
  float v;
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\tmov.b32 %0, 0;\n\t@q ld.global.f32 %0, [%1];\n\t}"
               : "=&f"(v)
               : "l"(p), "r"(static_cast<int>(here)));
  return v;
}

// A warp's eight of units 64 part .. 64 part + 63, from contraction element k on (of which k_end exist): two columns
// a lane, zeros where nothing is.
template <bool MN, bool PAIRS>
__device__ __forceinline__ void load_units(const Side& S, int part, int k, int k_end, int warp, int lane, float2 (&v)[8]) {
  const int row0 = (MN ? k : S.first + 64 * part) + warp, col = (MN ? S.first + 64 * part : k) + 2 * lane;
  const int rows = MN ? (64 * part < S.units ? k_end : 0) : S.end, cols = MN ? S.end : k_end;
  const float* p = S.p + row0 * S.ld + col;
#pragma unroll
  for (int i = 0; i < 8; ++i, p += SPLIT_WARPS * S.ld) {
    const bool here = row0 + SPLIT_WARPS * i < rows && col < cols;
    if (PAIRS) {
      v[i] = load_pair(p, here);
    } else {
      v[i].x = load_one(p, here);
      v[i].y = load_one(p + 1, here && col + 1 < cols);
    }
  }
}
template <bool MN>
__device__ __forceinline__ void load_side(const Side& S, int part, int k, int k_end, bool pairs, int warp, int lane,
                                          float2 (&v)[8]) {
  if (pairs) load_units<MN, true>(S, part, k, k_end, warp, lane, v);
  else load_units<MN, false>(S, part, k, k_end, warp, lane, v);
}

// The three planes of loaded units, swizzled as a TMA writes them.
__device__ __forceinline__ void store_side(uint32_t base, uint32_t plane, int units, int part, int warp, int lane,
                                           float2 (&v)[8]) {
  const uint32_t at = base + (64 * part + warp) * 128 + (((lane >> 2) ^ warp) << 4) + (lane & 3) * 4;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (64 * part + warp + SPLIT_WARPS * i < units) {
#pragma unroll
      for (int q = 0; q < 3; ++q) {
        const uint32_t w = pack_bf16(v[i].x, v[i].y);
        v[i].x -= __uint_as_float(w << 16);
        v[i].y -= __uint_as_float(w & 0xFFFF0000u);
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + SPLIT_WARPS * 128 * i + q * plane), "r"(w) : "memory");
      }
    }
  }
}

template <bool PAIR>
__device__ __forceinline__ void issue_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  if (PAIR) tc_mma_f16_pair_elect(d, a, b, idesc, acc);
  else tc_mma_f16_elect(d, a, b, idesc, acc);
}
template <bool PAIR>
__device__ __forceinline__ void issue_commit(uint32_t bar) {
  if (PAIR) tc_commit_pair_elect(bar);
  else tc_commit_elect(bar);
}

// The tensor core's own fp32 additions truncate: one of 16 products loses up to two units of 2^-23 of the sum,
// always towards zero.  So OUT_F32 empties the accumulator into registers every PART_TILES contraction tiles,
// and gradients in bf16 every LONG_PART, as many elements as a product contracts at most: up to 4.9e-4 of the summed
// magnitudes, against a rounding of up to 3.9e-3.  (One accumulator over 2^20 tokens of one sign lost 6.5e-3.)
template <int MODE, int KIND, bool PAIR>
__global__ void __launch_bounds__(threads_of(KIND), 1) expert_kernel(const __grid_constant__ ExpertParams P) {
  constexpr bool OUT_F32 = KIND != BF16_BF16;
  constexpr bool SPLIT = KIND == F32_SPLIT;
  static_assert(!(SPLIT && PAIR), "split tiles are of one CTA");
  constexpr int PLANES = KIND >= F32_F32 ? 3 : 1, SEGMENTS = KIND >= F32_F32 ? 6 : 1, PART_TILES = part_tiles(KIND);
  constexpr bool PARTED = OUT_F32 || MODE == EXPERT_WGRAD;  // accumulators may hold parts of a contraction
  constexpr int PART = OUT_F32 ? PART_TILES : LONG_PART;
  constexpr int THREADS = threads_of(KIND), EPI_WARPS = epi_warps(KIND);
  constexpr bool A_MN = MODE != EXPERT_FORWARD;
  constexpr bool B_MN = MODE == EXPERT_WGRAD;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t staging = base + ring_bytes(KIND);
  constexpr uint32_t BAR0 = ring_bytes(KIND) + EPI_WARPS * staging_bytes(KIND);
  const uint32_t bar0 = base + BAR0;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(gbase + BAR0 + 8 * NUM_BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* bad = reinterpret_cast<int*>(tmem_holder + 2);
  int* seg_base = reinterpret_cast<int*>(gbase + BAR0 + BAR_BYTES);
  int* seg_off = seg_base + P.experts + 1;
  __shared__ long long seg_cost[kWidths];
  __shared__ int seg_longest;
  __shared__ int seg_order[MODE == EXPERT_WGRAD ? kMaxOrdered : 1];

  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (MAX_STAGES + s); };
  auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * MAX_STAGES + a); };
  auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * MAX_STAGES + 2 + a); };
  const uint32_t drain_bar = bar0 + 8u * (2 * MAX_STAGES + 4);
  auto peer_bar = [&](int s) { return bar0 + 8u * (2 * MAX_STAGES + 5 + s); };  // leader: the peer's stage is full

  const int rank = PAIR ? static_cast<int>(cluster_cta_rank()) : 0;
  const int first_tile = PAIR ? blockIdx.x >> 1 : blockIdx.x, tile_step = PAIR ? gridDim.x >> 1 : gridDim.x;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < MAX_STAGES; ++s) {
      mbar_init(full_bar(s), SPLIT ? SPLIT_WARPS : 1);
      mbar_init(empty_bar(s), 1);
      mbar_init(peer_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), (PAIR ? 2 : 1) * EPI_WARPS);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    *bad = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
    if (!SPLIT) {
      tma_prefetch_map(&P.tmA);
      for (int i = 0; i < (B_MN ? 1 : kExpertBoxes); ++i) tma_prefetch_map(&P.tmB[i]);
    }
  }
  if (warp == 1) {
    if (PAIR) {
      tmem_alloc_pair(smem_addr(tmem_holder), TMEM_COLS);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_addr(tmem_holder), TMEM_COLS);
      tmem_relinquish();
    }
  }
  wait_for_previous_kernel();
  let_next_kernel_start();
  for (int e = threadIdx.x; e <= P.experts; e += THREADS) seg_off[e] = P.offsets[e];
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // Tile width: the fewest rounds of tiles over the CTAs, each as long as the operand rows it loads.
  // Offsets that leave the rows or decrease: nothing is computed, the status word says so.
  if (warp < kWidths) {
    const int w = RN - 32 * warp;
    int tiles = 0, longest = 0, live = 0;
    bool wrong = false;
    for (int e = lane; e < P.experts; e += 32) {
      const int a = seg_off[e], n = seg_off[e + 1] - a;
      wrong = wrong || a < 0 || n < 0 || seg_off[e + 1] > P.tokens;
      if (wrong) break;
      tiles += expert_tiles<MODE, PAIR>(P, n, w);
      longest = max(longest, n);
      live += n > 0;
    }
    __syncwarp();
    if (warp == 0 && __any_sync(0xffffffffu, wrong) && lane == 0) *bad = 1;
    tiles = __reduce_add_sync(0xffffffffu, tiles);
    longest = __reduce_max_sync(0xffffffffu, longest);
    live = __reduce_add_sync(0xffffffffu, live);
    if (lane == 0) {
      const int rows = min(w, round_rows<PAIR>(max(MODE == EXPERT_WGRAD ? P.rows : longest, 1)));
      const int nk = (SPLIT ? 1 : PLANES) * (MODE == EXPERT_WGRAD ? (P.tokens / max(live, 1) + BK - 1) / BK : P.k_tiles);
      const long long rounds = (tiles + tile_step - 1) / tile_step;
      const int mine = PAIR ? rows / 2 : rows;
      // two stages have to fit (the narrowest width's always do)
      const bool fits = 2u * PLANES * (A_BYTES + b_bytes<B_MN, SPLIT>(mine)) <= ring_bytes(KIND) &&
                        !(SPLIT && w > SPLIT_ROWS) &&
                        !(PARTED && !OUT_F32 && longest > LONG_PART * BK && w > LONG_ROWS);
      seg_cost[warp] = fits ? rounds * (static_cast<long long>(nk) * (FM + mine) + kTileOverhead) : LLONG_MAX;
      if (warp == 0) seg_longest = longest;
    }
  }
  __syncthreads();
  int best = 0;
#pragma unroll
  for (int i = 1; i < kWidths; ++i) best = seg_cost[i] < seg_cost[best] ? i : best;
  const int width = RN - 32 * best;
  const int widest = min(width, round_rows<PAIR>(max(MODE == EXPERT_WGRAD ? P.rows : seg_longest, 1)));
  const int b_rows = PAIR ? widest / 2 : widest;  // of the rows operand in this CTA
  const uint32_t b_plane = b_bytes<B_MN, SPLIT>(b_rows);
  const uint32_t stage_bytes = PLANES * (A_BYTES + b_plane);  // the planes of A, then those of B
  const int stages = min(MAX_STAGES, static_cast<int>(ring_bytes(KIND) / stage_bytes));
  // A gradient's tiles take as long as their segments: the longest go first, so that the rounds even out
  // (16 experts of 1536 x 768, 8191 tokens: 48.5 instead of 50.7 us, 61.1 instead of 63.8 with a more skewed
  // router; 0.5 us more for 48 small ones.  Counting every pair of experts costs about a microsecond at
  // kMaxOrdered; more of them average out).
  const bool ordered = MODE == EXPERT_WGRAD && P.experts <= kMaxOrdered;
  if (ordered) {
    for (int e = threadIdx.x; e < P.experts; e += THREADS) {
      const int n = seg_off[e + 1] - seg_off[e];
      int before = 0;
      for (int o = 0; o < P.experts; ++o) {
        const int m = seg_off[o + 1] - seg_off[o];
        before += m > n || (m == n && o < e);
      }
      seg_order[before] = e;
    }
    __syncthreads();
  }
  if (warp == 2) {
    int carry = 0;
    for (int e0 = 0; e0 < P.experts; e0 += 32) {
      const int e = e0 + lane;
      const int x = e < P.experts ? (ordered ? seg_order[e] : e) : 0;
      const int n = e < P.experts && !*bad ? expert_tiles<MODE, PAIR>(P, seg_off[x + 1] - seg_off[x], width) : 0;
      int sum = n;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += up;
      }
      if (e < P.experts) seg_base[e] = carry + sum - n;
      carry += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (lane == 0) {
      seg_base[P.experts] = carry;
      if (*bad && blockIdx.x == 0 && P.status) atomicOr(P.status, kStatusBadSegments);
    }
  }
  __syncthreads();
  if (PAIR) cluster_sync_all();  // the peer's barriers exist
  const uint32_t tmem_base = *tmem_holder;
  const int total_tiles = seg_base[P.experts];
  const Segments S{seg_base, seg_off, ordered ? seg_order : nullptr, width};

  if (SPLIT && warp >= 2 + EPI_WARPS) {
    // ------------------------------------------------ fp32 operands: load, split, store
    const int w = warp - 2 - EPI_WARPS;
    const float* const pa = static_cast<const float*>(P.a);
    const float* const pb = static_cast<const float*>(P.b);
    Ring ring;
    bool ok = true;
    for (int t = first_tile; ok && t < total_tiles; t += tile_step) {
      const Tile ti = decode_tile<MODE, PAIR>(P, S, t, rank);
      const int k0 = B_MN ? ti.k0 : 0, k_end = B_MN ? ti.k0 + ti.kn : P.contraction;
      const int k_tiles = (k_end - k0 + BK - 1) / BK;
      const Side A{pa + (B_MN ? 0ll : ti.e * P.s_a), P.ld_a, ti.f0, P.features, FM};
      const Side B{pb, P.ld_b, ti.r0, ti.r0 + ti.nr, B_MN ? SPLIT_ROWS : ti.nw};
      float2 v[3][8];  // while 64 units are split the next ones' loads are under way
      load_side<A_MN>(A, 0, k0, k_end, P.pairs_a, w, lane, v[0]);
      load_side<A_MN>(A, 1, k0, k_end, P.pairs_a, w, lane, v[1]);
      load_side<B_MN>(B, 0, k0, k_end, P.pairs_b, w, lane, v[2]);
      for (int kt = 0; kt < k_tiles; ++kt, ring.next(stages)) {
        ok = mbar_wait_bounded(empty_bar(ring.s), ring.phase ^ 1u, abort_flag, P.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t at = base + ring.s * stage_bytes;
        const int next = k0 + (kt + 1) * BK;  // past the end nothing is loaded
        store_side(at, A_BYTES, A.units, 0, w, lane, v[0]);
        load_side<A_MN>(A, 0, next, k_end, P.pairs_a, w, lane, v[0]);
        store_side(at, A_BYTES, A.units, 1, w, lane, v[1]);
        load_side<A_MN>(A, 1, next, k_end, P.pairs_a, w, lane, v[1]);
        store_side(at + PLANES * A_BYTES, b_plane, B.units, 0, w, lane, v[2]);
        load_side<B_MN>(B, 0, next, k_end, P.pairs_b, w, lane, v[2]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(full_bar(ring.s));
      }
    }
  } else if (SPLIT && warp == 0) {
    // nothing to copy
  } else if (warp == 0) {
    // ------------------------------------------------ TMA producer
    // Each lane owns one copy of a stage, so that they go out in one instruction: the (up to two) chunks
    // of A's planes first, then the (up to four) chunks of B's.
    Ring ring;
    bool ok = true;
    constexpr int A_COPIES = A_MN ? 2 : 1, B_COPIES = B_MN ? 4 : 1;
    const bool is_a = lane < A_COPIES * PLANES;
    const int mine = is_a ? lane : lane - A_COPIES * PLANES;
    const int plane = mine / (is_a ? A_COPIES : B_COPIES), chunk = mine - plane * (is_a ? A_COPIES : B_COPIES);
    const CUtensorMap* map = is_a ? &P.tmA : &P.tmB[0];
    const uint32_t dst = base + chunk * CHUNK_BYTES + (is_a ? plane * A_BYTES : PLANES * A_BYTES + plane * b_plane);
    for (int t = first_tile; ok && t < total_tiles; t += tile_step) {
      const Tile ti = decode_tile<MODE, PAIR>(P, S, t, rank);
      const int k_tiles = B_MN ? (ti.kn + BK - 1) / BK : P.k_tiles;
      const int b_mine = PAIR ? ti.nw / 2 : ti.nw;  // rows of the rows operand in this CTA
      const int a_chunks = A_MN ? max(0, (min(FM, P.features - ti.f0) + 63) / 64) : 1;
      const int b_chunks = B_MN ? (b_mine + 63) / 64 : 1;
      const int box = B_MN ? 0 : box_of(b_mine);
      const uint32_t bytes = PLANES * ((A_MN ? a_chunks * CHUNK_BYTES : A_BYTES) +
                                       (B_MN ? b_chunks * CHUNK_BYTES : (16u << box) * BK * 2));
      const bool copies = plane < PLANES && chunk < (is_a ? a_chunks : b_chunks);
      if (!B_MN && !is_a) map = &P.tmB[box];
      // contraction along the first coordinate (K-major) or the second; the other is fixed for the tile
      const bool k_first = is_a ? !A_MN : !B_MN;
      const int fixed = (is_a ? ti.f0 : ti.r0 + b_mine * rank) + 64 * chunk;
      const int k_base = B_MN ? ti.k0 : 0, mat = is_a && !B_MN ? ti.e : 0;
      for (int kt = 0; kt < k_tiles; ++kt, ring.next(stages)) {
        ok = mbar_wait_bounded(empty_bar(ring.s), ring.phase ^ 1u, abort_flag, P.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t bar = full_bar(ring.s);
        if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
        __syncwarp();
        const int k = k_base + kt * BK;
        if (copies) tma_load_4d(dst + ring.s * stage_bytes, map, bar, k_first ? k : fixed, k_first ? fixed : k, mat, plane);
      }
    }
    if (!ok) {
      // Let the copies this warp started land before the CTA exits.
      for (int i = 0; i < stages; ++i, ring.next(stages))
        if (ring.filled(stages)) wait_drain(full_bar(ring.s), ring.phase ^ 1u);
    }
  } else if (warp == 1) {
    // ------------------------------------------------ UMMA issuer (one lane; all lanes zero segment ends)
    Ring ring;
    int local = 0;
    bool ok = true;
    const uint64_t a_desc0 = smem_desc_sw128(base, A_MN ? CHUNK_BYTES : 16u, 1024u);
    const uint64_t b_desc0 = smem_desc_sw128(base + PLANES * A_BYTES, B_MN ? CHUNK_BYTES : 16u, 1024u);
    constexpr uint32_t a_step = (A_MN ? 2048u : 32u) >> 4, b_step = (B_MN ? 2048u : 32u) >> 4;
    for (int t = first_tile; ok && t < total_tiles; t += tile_step) {
      const Tile ti = decode_tile<MODE, PAIR>(P, S, t, rank);
      const uint32_t idesc = instr_desc_bf16_major(PAIR ? 2 * FM : FM, ti.nw, A_MN, B_MN);
      const int nk = B_MN ? (ti.kn + BK - 1) / BK : P.k_tiles;
      for (int kk = 0; ok && kk < nk; ++local) {
        const int acc = local & 1;
        if (rank == 0) {
          ok = mbar_wait_bounded(tempty_bar(acc), ((local >> 1) & 1) ^ 1u, abort_flag, P.status);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
        }
        const uint32_t d_tmem = tmem_base + acc * ACC_COLS;
        const int part_end = PARTED ? min(kk + PART, nk) : nk;
        for (uint32_t more = 0; kk < part_end; ++kk, ring.next(stages)) {
          const int s = ring.s;
          ok = mbar_wait_bounded(full_bar(s), ring.phase, abort_flag, P.status);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          int steps = BK / 16;
          bool zeroed = false;
          if (B_MN) {
            const int left = ti.kn - kk * BK;
            if (left < BK) {
              steps = (left + 15) / 16;
              if (!SPLIT && left < 16 * steps) {
                const uint32_t sa = base + s * stage_bytes;
                zero_rows(sa, PLANES * FM / 64, left, 16 * steps, lane);
                for (int q = 0; q < PLANES; ++q)
                  zero_rows(sa + PLANES * A_BYTES + q * b_plane, ((PAIR ? ti.nw / 2 : ti.nw) + 63) / 64, left, 16 * steps,
                            lane);
                fence_proxy_async_smem();
                __syncwarp();
                zeroed = true;
              }
            }
          }
          if (PAIR && rank != 0) {
            // the peer passes its full stages on; what it wrote itself (rare) needs cluster-wide order
            if (lane == 0) {
              if (zeroed) mbar_arrive_remote_release(map_shared_rank(peer_bar(s), 0));
              else mbar_arrive_remote(map_shared_rank(peer_bar(s), 0));
            }
            __syncwarp();
            continue;
          }
          if (PAIR) {
            ok = mbar_wait_bounded(peer_bar(s), ring.phase, abort_flag, P.status);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
          }
          const uint64_t ad = a_desc0 + static_cast<uint32_t>(s) * (stage_bytes >> 4);
          const uint64_t bd = b_desc0 + static_cast<uint32_t>(s) * (stage_bytes >> 4);
#pragma unroll
          for (int seg = 0; seg < SEGMENTS; ++seg) {
            const uint64_t as = ad + (PLANES == 3 ? plane_a(seg) * (A_BYTES >> 4) : 0u);
            const uint64_t bs = bd + (PLANES == 3 ? plane_b(seg) * (b_plane >> 4) : 0u);
            if (steps == BK / 16) {
#pragma unroll
              for (int k4 = 0; k4 < BK / 16; ++k4)
                issue_mma<PAIR>(d_tmem, as + a_step * k4, bs + b_step * k4, idesc, (seg | k4) == 0 ? more : 1u);
            } else {
              for (int k4 = 0; k4 < steps; ++k4)
                issue_mma<PAIR>(d_tmem, as + a_step * k4, bs + b_step * k4, idesc, (seg | k4) == 0 ? more : 1u);
            }
          }
          more = 1u;
          issue_commit<PAIR>(empty_bar(s));
        }
        if (ok && rank == 0) issue_commit<PAIR>(tfull_bar(acc));
      }
    }
    if (!ok && rank == 0) {
      issue_commit<PAIR>(drain_bar);
      wait_drain(drain_bar, 0);
    }
  } else {
    // ------------------------------------------------ epilogue (warps 2 .. 2+EPI_WARPS-1)
    // The (two, split: one) warps of a TMEM lane quarter take its 32-column chunks in turn.
    const int quarter = warp & 3;
    const int half = (warp - 2) >> 2;
    const uint32_t stage = staging + static_cast<uint32_t>(warp - 2) * staging_bytes(KIND);
    const uint32_t lane_off = static_cast<uint32_t>(32 * quarter) << 16;
    int local = 0, boxes = 0;
    bool ok = true;
    auto take = [&]() {  // the next accumulator, or false
      ok = mbar_wait_bounded(tfull_bar(local & 1), (local >> 1) & 1, abort_flag, P.status);
      tc_fence_after();
      return ok;
    };
    auto give_back = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (PAIR) mbar_arrive_remote(map_shared_rank(tempty_bar(local & 1), 0));
        else mbar_arrive(tempty_bar(local & 1));
      }
      ++local;
    };
    for (int t = first_tile; ok && t < total_tiles; t += tile_step) {
      const Tile ti = decode_tile<MODE, PAIR>(P, S, t, rank);
      const int fw = ti.f0 + 32 * quarter;  // this warp's first feature
      const int nk = B_MN ? (ti.kn + BK - 1) / BK : P.k_tiles;
      const long long at = (B_MN ? ti.e * P.s_out : 0ll) + static_cast<long long>(ti.r0) * P.ld_out + fw;
      const bool live = fw < P.features;
      if (OUT_F32 || (PARTED && nk > LONG_PART)) {
        constexpr int CHUNKS = SPLIT ? SPLIT_ROWS / 32 : OUT_F32 ? 4 : LONG_ROWS / 64, NEXT = 8 * EPI_WARPS;
        float sum[CHUNKS][32];  // running sums of this warp's chunks
#pragma unroll
        for (int j = 0; j < CHUNKS; ++j)
#pragma unroll
          for (int i = 0; i < 32; ++i) sum[j][i] = 0.f;
        for (int kk = 0; kk < nk; kk += PART) {
          if (!take()) break;
#pragma unroll
          for (int j = 0; j < CHUNKS; ++j) {
            const int c = 32 * half + NEXT * j;
            if (live && c < ti.nr) {
              uint32_t r[32];
              __syncwarp();
              tmem_load_32cols(tmem_base + (local & 1) * ACC_COLS + lane_off + c, r);
              tmem_load_wait();
              tmem_loaded(r);
#pragma unroll
              for (int i = 0; i < 32; ++i) sum[j][i] = fmaf(P.scale, __uint_as_float(r[i]), sum[j][i]);
            }
          }
          give_back();
        }
        if (!ok) break;
#pragma unroll
        for (int j = 0; j < CHUNKS; ++j) {
          const int c = 32 * half + NEXT * j;
          if (!live || c >= ti.nr) continue;
          if (!OUT_F32)
            add_column(P, at + lane + c * P.ld_out, fw + lane, min(32, ti.nr - c), sum[j]);
          else
            store_rows(P, at + c * P.ld_out, ti.r0 + c, B_MN ? ti.e : 0, B_MN && ti.r0 + ti.nr == P.rows, stage, boxes, fw,
                       min(32, ti.nr - c), lane, sum[j]);
        }
      } else {
        if (nk > 0 && !take()) break;
        if (live) {
          for (int c = 32 * half; c < ti.nr; c += 64) {
            const uint32_t taddr = tmem_base + (local & 1) * ACC_COLS + lane_off + c;
            const int nv = min(32, ti.nr - c);
            __syncwarp();
            if (nk > 0 && (MODE != EXPERT_WGRAD || P.beta == 0.f)) {
              store_staged(P, taddr, stage, at + c * P.ld_out, fw, nv, P.scale, lane);
            } else {  // adds to a bf16 G, or an expert without tokens
              uint32_t r[32];
              float v[32];
              if (nk > 0) {
                tmem_load_32cols(taddr, r);
                tmem_load_wait();
                tmem_loaded(r);
              }
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] = nk > 0 ? P.scale * __uint_as_float(r[i]) : 0.f;
              add_column(P, at + lane + c * P.ld_out, fw + lane, nv, v);
            }
          }
        }
        if (nk > 0) give_back();
      }
    }
    bulk_wait_group_all();
    if (P.clear_rest && (!B_MN || *bad)) {
      const int w = blockIdx.x * EPI_WARPS + warp - 2, warps = gridDim.x * EPI_WARPS;
      if (B_MN) {
        clear_rows<true>(P, 0, P.experts * P.rows, w, warps, lane);
      } else {  // with bad offsets no row is of any segment
        clear_rows<false>(P, 0, *bad ? P.tokens : seg_off[0], w, warps, lane);
        if (!*bad) clear_rows<false>(P, seg_off[P.experts], P.tokens, w, warps, lane);
      }
    }
  }

  __syncthreads();
  if (PAIR) cluster_sync_all();  // no product or arrival still reaches the other CTA
  if (warp == 1) {
    tc_fence_after();
    if (PAIR) tmem_dealloc_pair(tmem_base, TMEM_COLS);
    else tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

// ------------------------------------------------------------------ packing
// A warp takes 256 columns of a row at a time, a lane pairs of neighbouring ones 64 apart, so that its
// loads and stores are whole lines whatever the row's alignment.
template <bool F32, int PLANES>
__global__ void __launch_bounds__(256) pack_kernel(const __grid_constant__ PackParams P) {
  wait_for_previous_kernel();
  let_next_kernel_start();
  const bool second = P.count > 1 && static_cast<int>(blockIdx.x) >= P.item[1].block0;
  const PackItem& p = P.item[second ? 1 : 0];
  const int blocks = (!second && P.count > 1 ? P.item[1].block0 : static_cast<int>(gridDim.x)) - p.block0;
  const int lane = threadIdx.x & 31, per_row = (p.pitch + 255) / 256;
  const long long units = static_cast<long long>(p.mats) * p.rows * per_row, step = static_cast<long long>(blocks) * 8;
  for (long long u = static_cast<long long>(blockIdx.x - p.block0) * 8 + (threadIdx.x >> 5); u < units; u += step) {
    const long long row = u / per_row;
    const int mat = static_cast<int>(row / p.rows), r = static_cast<int>(row - static_cast<long long>(mat) * p.rows);
    if (p.offsets != nullptr && p.offsets[mat + 1] <= p.offsets[mat]) continue;  // an expert without tokens
    const int c0 = static_cast<int>(u - row * per_row) * 256 + 2 * lane;
    const long long at = mat * p.s + r * p.ld;
    float v[4][2];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = c0 + 64 * j + h;
        v[j][h] = 0.f;
        if (c < p.cols)
          v[j][h] = F32 ? static_cast<const float*>(p.src)[at + c]
                        : bf16_bits_to_float(static_cast<const uint16_t*>(p.src)[at + c]);
      }
    uint16_t* o = p.dst + mat * p.dst_mat + static_cast<long long>(r) * p.pitch + c0;
#pragma unroll
    for (int q = 0; q < PLANES; ++q)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t w = pack_bf16(v[j][0], v[j][1]);
        v[j][0] -= __uint_as_float(w << 16);
        v[j][1] -= __uint_as_float(w & 0xFFFF0000u);
        if (c0 + 64 * j < p.pitch) *reinterpret_cast<uint32_t*>(o + q * p.dst_plane + 64 * j) = w;
      }
  }
}

template <int MODE, int KIND, bool PAIR>
cudaError_t launch_mode(const ExpertParams& p, int ctas, cudaStream_t stream) {
  constexpr int kMaxDevices = 64;
  static std::atomic<bool> configured[kMaxDevices];
  const int smem = ring_bytes(KIND) + epi_warps(KIND) * staging_bytes(KIND) + BAR_BYTES +
                   2 * sizeof(int) * (MUON_MAX_EXPERTS + 1) + 1024;
  const auto kernel = expert_kernel<MODE, KIND, PAIR>;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDevices || !configured[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDevices) configured[dev].store(true, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(threads_of(KIND));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = PAIR ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int MODE, int KIND>
cudaError_t launch_kind(const ExpertParams& p, bool pair, int ctas, cudaStream_t stream) {
  return pair ? launch_mode<MODE, KIND, true>(p, ctas, stream) : launch_mode<MODE, KIND, false>(p, ctas, stream);
}

}  // namespace

cudaError_t launch_experts(const ExpertParams& p, ExpertMode mode, bool pair, int ctas, cudaStream_t stream) {
  switch (mode) {
    case EXPERT_FORWARD:
      if (p.split) return launch_mode<EXPERT_FORWARD, F32_SPLIT, false>(p, ctas, stream);
      return p.in_f32 ? launch_kind<EXPERT_FORWARD, F32_F32>(p, pair, ctas, stream)
                      : launch_kind<EXPERT_FORWARD, BF16_BF16>(p, pair, ctas, stream);
    case EXPERT_BACKWARD:
      if (p.split) return launch_mode<EXPERT_BACKWARD, F32_SPLIT, false>(p, ctas, stream);
      return p.in_f32 ? launch_kind<EXPERT_BACKWARD, F32_F32>(p, pair, ctas, stream)
                      : launch_kind<EXPERT_BACKWARD, BF16_BF16>(p, pair, ctas, stream);
    default:
      if (p.split) return launch_mode<EXPERT_WGRAD, F32_SPLIT, false>(p, ctas, stream);
      return p.in_f32    ? launch_kind<EXPERT_WGRAD, F32_F32>(p, pair, ctas, stream)
             : p.out_f32 ? launch_kind<EXPERT_WGRAD, BF16_F32>(p, pair, ctas, stream)
                         : launch_kind<EXPERT_WGRAD, BF16_BF16>(p, pair, ctas, stream);
  }
}

cudaError_t launch_pack(PackParams& p, bool src_f32, int sm_count, cudaStream_t stream) {
  long long blocks = 0;
  for (int i = 0; i < p.count; ++i) {
    PackItem& q = p.item[i];
    q.block0 = static_cast<int>(blocks);
    const long long units = static_cast<long long>(q.mats) * q.rows * ((q.pitch + 255) / 256);  // a warp's
    blocks += std::max(1ll, std::min<long long>((units + 7) / 8, 8ll * sm_count));
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return src_f32 ? cudaLaunchKernelEx(&cfg, pack_kernel<true, 3>, p) : cudaLaunchKernelEx(&cfg, pack_kernel<false, 1>, p);
}

}  // namespace muon
