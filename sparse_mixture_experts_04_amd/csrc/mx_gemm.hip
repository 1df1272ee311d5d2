// The experts' products on microscaled (MX) operands: e2m1 weights, e2m1 or
// e4m3 token rows, one e8m0 scale per 32 elements along K on both sides.
//
//   up:   H[r, :]  = MX(gelu(sum_k Xq[perm[r] / k, k] * W1q[e][:, k]))
//   down: Yp[r, :] = sum_f Hq[r, f] * W2q[e][:, f]
//
// for the rows r of expert e's segment [offsets[e], offsets[e+1]).  The
// matrix cores take the codes and the scales as they are stored
// (v_mfma_scale_f32_*_f8f6f4) and accumulate in fp32: nothing is widened in
// memory.  The up-projection's GELU and the quantisation of its result to the
// next product's operand run on the accumulators.
#include <atomic>
#include <type_traits>

#include "kernels.hpp"
#include "mx.hpp"

namespace moe {
namespace {

// Operand B of the scaled MFMA: its format code is 0 for e4m3, 4 for e2m1.
template <int kFmt> __device__ __forceinline__ constexpr int mx_code() { return kFmt == kMxFp4 ? 4 : 0; }

// 32 weight rows (operand A, e2m1) x 32 token rows (operand B) x 64 of K.
// Lane l holds, of weight row l%32, the 32 elements of K block l/32; of token
// row l%32 the same for e2m1, and for e4m3 the 16 elements l/32 of both
// blocks.  The scales come from lanes l/32 = block for either format.
// Byte kSel of ws and xs is the scale.
template <int kFmt, int kSel>
__device__ __forceinline__ f32x16_t mx_mfma32(i32x8_t w, i32x8_t x, f32x16_t c, int ws, int xs) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, x, c, 4, mx_code<kFmt>(), kSel, ws, kSel, xs);
}

__device__ __forceinline__ i32x8_t frag(u32x4_t lo, u32x4_t hi) {
  return i32x8_t{static_cast<int>(lo[0]), static_cast<int>(lo[1]), static_cast<int>(lo[2]), static_cast<int>(lo[3]),
                 static_cast<int>(hi[0]), static_cast<int>(hi[1]), static_cast<int>(hi[2]), static_cast<int>(hi[3])};
}

// Word 3 of a raw buffer resource on the gfx9 family: 32-bit data format, no
// swizzle; bounds are checked against num_records in bytes.
constexpr int kRsrcWord3 = 0x00020000;
constexpr int kOutside = static_cast<int>(0x80000000u);  // an offset beyond any resource here

__device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, static_cast<int>(bytes), kRsrcWord3);
}

// What a product does with its results: Out::Tile is bound to the rows [m0,
// m0 + rows) of the result, and takes 16 consecutive columns of one of them,
// of which this lane holds the half `half` of a block of 32 and lane ^ 32 the
// other half.  Stores go through buffer resources over the tile's rows: a row
// past them is dropped by the hardware, and so is a column past N, which gets
// an offset beyond the range. 
template <int kFmt> struct UpOut {
  uint8_t* hq;
  uint8_t* hs;
  // One value per lane, the block of 32 in 32 consecutive lanes: column n0 + c of row r.
  __device__ __forceinline__ void store_one(int64_t r, int N, int n0, int c, bool ok, float v) const {
    v = gelu_tanh_fast(v);
    uint32_t m = abs_bits(v);
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), x)));
    const uint32_t b = mx_scale_byte<kFmt>(m);
    v *= mx_inv_scale(b);
    const float next = __shfl_xor(v, 1);
    if (!ok) return;
    if constexpr (kFmt == kMxFp4) {
      const uint32_t code = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v, next, 1.0f, 0);
      if ((c & 1) == 0) hq[(r * N + n0 + c) / 2] = b == 255u ? 0 : static_cast<uint8_t>(code);
    } else {
      const int code = __builtin_amdgcn_cvt_pk_fp8_f32(clamp448(v), 0.f, 0, false);
      hq[r * N + n0 + c] = b == 255u ? 0 : static_cast<uint8_t>(code);
    }
    if (c == 0) hs[(r * N + n0) / kMxBlock] = static_cast<uint8_t>(b);
  }
  struct Tile {
    __amdgpu_buffer_rsrc_t codes, scales;
    int N;
    __device__ __forceinline__ Tile(const UpOut& o, int64_t m0, int rows, int n)
        : codes(resource(o.hq + m0 * Mx<kFmt>::bytes(n), rows * Mx<kFmt>::bytes(n))),
          scales(resource(o.hs + m0 * (n / kMxBlock), int64_t{1} * rows * (n / kMxBlock))),
          N(n) {}
    // returns the block's scale byte
    __device__ __forceinline__ uint32_t store(int row, int col, int half, float* v) const {
      uint32_t m = 0;
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        v[q] = gelu_tanh_fast(v[q]);
        m = max(m, abs_bits(v[q]));
      }
      m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 32)));
      const uint32_t b = mx_scale_byte<kFmt>(m);
      const float inv = mx_inv_scale(b);
      const bool bad = b == 255u;
      const int at = row * static_cast<int>(Mx<kFmt>::bytes(N)) + static_cast<int>(Mx<kFmt>::bytes(col + 16 * half));
      const int off = col < N ? at : kOutside;
      if constexpr (kFmt == kMxFp4)
        __builtin_amdgcn_raw_buffer_store_b64(u32x2_t{mx_encode8_fp4(v, inv, bad), mx_encode8_fp4(v + 8, inv, bad)},
                                              codes, off, 0, 0);
      else
        __builtin_amdgcn_raw_buffer_store_b128(u32x4_t{mx_encode4_fp8(v, inv, bad), mx_encode4_fp8(v + 4, inv, bad),
                                                       mx_encode4_fp8(v + 8, inv, bad),
                                                       mx_encode4_fp8(v + 12, inv, bad)},
                                               codes, off, 0, 0);
      return b;
    }
    // the scale bytes of one block, or of the two blocks of 64 columns
    __device__ __forceinline__ void store_scale(int row, int col, int half, uint32_t b) const {
      const int off = col < N && half == 0 ? row * (N / kMxBlock) + col / kMxBlock : kOutside;
      __builtin_amdgcn_raw_buffer_store_b8(static_cast<uint8_t>(b), scales, off, 0, 0);
    }
    __device__ __forceinline__ void store_scales(int row, int col, int half, uint32_t b0, uint32_t b1) const {
      const int off = col < N && half == 0 ? row * (N / kMxBlock) + col / kMxBlock : kOutside;
      __builtin_amdgcn_raw_buffer_store_b16(static_cast<uint16_t>(b0 | b1 << 8), scales, off, 0, 0);
    }
  };
};
template <typename T> struct DownOut {
  T* y;
  __device__ __forceinline__ void store_one(int64_t r, int N, int n0, int c, bool ok, float v) const {
    const float next = __shfl_xor(v, 1);
    if (!ok) return;
    if constexpr (sizeof(T) == 2) {
      if ((c & 1) == 0) *reinterpret_cast<uint32_t*>(y + r * N + n0 + c) = pack_bf16x2(v, next);
    } else {
      y[r * N + n0 + c] = v;
    }
  }
  struct Tile {
    __amdgpu_buffer_rsrc_t res;
    int N;
    __device__ __forceinline__ Tile(const DownOut& o, int64_t m0, int rows, int n)
        : res(resource(o.y + m0 * n, int64_t{rows} * n * static_cast<int>(sizeof(T)))), N(n) {}
    __device__ __forceinline__ uint32_t store(int row, int col, int half, float* v) const {
      const int at = (row * N + col + 16 * half) * static_cast<int>(sizeof(T));
      const int off = col < N ? at : kOutside;
      if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          u32x4_t r;
#pragma unroll
          for (int q = 0; q < 4; ++q) r[q] = pack_bf16x2(v[8 * h + 2 * q], v[8 * h + 2 * q + 1]);
          __builtin_amdgcn_raw_buffer_store_b128(r, res, off + 16 * h, 0, 0);
        }
      } else {
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          u32x4_t r;
#pragma unroll
          for (int q = 0; q < 4; ++q) r[q] = __float_as_uint(v[4 * h + q]);
          __builtin_amdgcn_raw_buffer_store_b128(r, res, off + 16 * h, 0, 0);
        }
      }
      return 0;
    }
    __device__ __forceinline__ void store_scale(int, int, int, uint32_t) const {}
    __device__ __forceinline__ void store_scales(int, int, int, uint32_t, uint32_t) const {}
  };
};

// ---------------------------------------------------------------------------
// Few rows per expert: bound by streaming each active expert's weights.  A
// block of four waves owns 32 weight rows (one MX block of the result) and a
// chunk of up to `chunk` of the expert's token rows; its waves take windows of K
// (1024, or 512 where K is short) in turn, and every wave asks for its whole
// window, 16 KB, before the first MFMA: with about 12 waves on a CU 192 KB of
// weights are on their way.  The chunks of one expert's weight rows are
// neighbours on one XCD, so its L2 serves the weights to all but the first.
// Measured on MI355X, both products (d = 3584, F = 2560, 64 experts, k = 2): one
// token, e4m3, 13.3 us (6.9 + 5.8, of which a launch alone takes about 3 each);
// 8 tokens, e2m1, 34.6 us: 140 MB at 4.05 TB/s.
//
// One 16x16x128 scaled MFMA takes 8 weight rows x 2 K-slices (operand A) and 8
// token rows x the same 2 slices (operand B); of its 16x16 results those of
// matching slices are wanted, and are added at the end.  So a weight
// load reads a whole 128-byte line of each of 8 rows: lane (row, slice s, group
// g) holds, at step t, block 8 t + 4 s + g of its window.  (For e4m3 rows an
// MFMA's K block b lies in lanes of groups 2 (b % 2) and + 1, halves b / 2;
// their addresses follow that.)  The scales of a row's window are 8 (or 4)
// dwords, loaded by its lanes, and handed round by lane exchanges.
// The token groups of 8 are taken in turn under the window's weights, and
// every wave keeps its partial sums, by slice, in its own part of LDS; at the
// end they are added in order.
constexpr int kFewWaves = 4;
constexpr int kFewRows = 32;

// The scales of blocks blk .. blk + 3 of a row of nblk (blk a multiple of 4).
// kDwords: nblk is a multiple of 4, so rows are whole dwords; else nblk is
// even.  Blocks past the row's end give 0.
template <bool kDwords>
__device__ __forceinline__ uint32_t scales4(const uint8_t* row, int blk, int nblk) {
  const int at = blk < nblk ? blk : 0;
  if constexpr (kDwords) {
    const uint32_t v = *reinterpret_cast<const uint32_t*>(row + at);
    return blk < nblk ? v : 0u;
  } else {
    const int at2 = blk + 2 < nblk ? blk + 2 : 0;
    const uint32_t lo = *reinterpret_cast<const uint16_t*>(row + at);
    const uint32_t hi = *reinterpret_cast<const uint16_t*>(row + at2);
    return (blk < nblk ? lo : 0u) | (blk + 2 < nblk ? hi << 16 : 0u);
  }
}

template <int kFmt, int kSel>
__device__ __forceinline__ f32x4_t mx_mfma16(u32x4_t w, u32x4_t x0, u32x4_t x1, f32x4_t c, uint32_t sw, uint32_t sx) {
  const u32x4_t zero = {0u, 0u, 0u, 0u};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(frag(w, zero), frag(x0, x1), c, 4, mx_code<kFmt>(), kSel,
                                                          static_cast<int>(sw), kSel, static_cast<int>(sx));
}

// kSt: MFMA steps of a window of 256 kSt of K.
template <int kFmt, bool kGather, bool kDwords, int kSt, typename Out>
__global__ __launch_bounds__(kFewWaves * kWave) void mx_product_few(MxOperands o, const int32_t* __restrict__ gidx,
                                                                   int gdiv, int src_rows, int chunk, Out out) {
  constexpr int kWindowBlocks = 8 * kSt;
  // partial sums: [wave][slice][token of the chunk][weight row]
  extern __shared__ __attribute__((aligned(16))) float part[];
  const int tid = threadIdx.x;
  const int lane = tid % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  int t_seg0 = 0, t_seg1 = 0;
  if (lane < o.E) {
    // offsets come from device memory: clamped, every access stays inside the buffers
    t_seg0 = min(max(o.offsets[lane], 0), o.max_rows);
    t_seg1 = min(max(o.offsets[lane + 1], t_seg0), o.max_rows);
  }
  // tiles: by expert, 32 weight rows, chunk (fastest); a run of them for each XCD
  const int t_chunks = (t_seg1 - t_seg0 + chunk - 1) / chunk;
  const int ntn = o.N / kFewRows;
  int t_incl = t_chunks;
#pragma unroll
  for (int m = 1; m < kWave; m <<= 1) {
    const int u = __shfl_up(t_incl, m);
    if (lane >= m) t_incl += u;
  }
  const int total = __builtin_amdgcn_readlane(t_incl, o.E - 1) * ntn;
  const int per_xcd = (total + 7) / 8;
  const int r8 = lane & 7;
  const int slice = (lane >> 3) & 1;
  const int g = lane >> 4;
  const int nblk = o.K / kMxBlock;
  const int nwin = (nblk + kWindowBlocks - 1) / kWindowBlocks;
  const int wstride = o.K / 2;
  const int64_t xstride = Mx<kFmt>::bytes(o.K);
  // The scales of this lane's blocks, step st's in byte st: byte g of the dword 2 st + s of its row.  Dword j is in
  // the lane of slice j / 4, group j % 4.
  auto step_scales = [&](uint32_t dwords) {
    uint32_t v = 0;
#pragma unroll
    for (int st = 0; st < kSt; ++st) {
      const int from = r8 + 8 * (st >> 1) + 16 * (2 * (st & 1) + slice);
      v |= (static_cast<uint32_t>(__shfl(static_cast<int>(dwords), from)) >> (8 * g) & 255u) << (8 * st);
    }
    return v;
  };
  // (the grid covers the tiles that the rows' bound allows; offsets beyond it take further turns)
  for (int at = blockIdx.x >> 3; at < per_xcd; at += gridDim.x >> 3) {
    const int tile = (blockIdx.x & 7) * per_xcd + at;
    if (tile >= total) break;
    const int e = __builtin_amdgcn_readfirstlane(
        static_cast<int>(__popcll(__ballot(lane < o.E && t_incl * ntn <= tile))));
    const int chunks_e = __builtin_amdgcn_readlane(t_chunks, e);
    const int local = tile - (__builtin_amdgcn_readlane(t_incl, e) - chunks_e) * ntn;
    const int n0 = __builtin_amdgcn_readfirstlane(local / chunks_e * kFewRows);
    const int seg1 = __builtin_amdgcn_readlane(t_seg1, e);
    const int row0 = __builtin_amdgcn_readfirstlane(__builtin_amdgcn_readlane(t_seg0, e) + local % chunks_e * chunk);
    const int ntok = min(seg1 - row0, chunk);

    const int64_t wrow0 = static_cast<int64_t>(e) * o.N + n0;
    const __amdgpu_buffer_rsrc_t wres = resource(o.wq + wrow0 * wstride, int64_t{kFewRows} * wstride);
    const uint8_t* const wsp = o.ws + (wrow0 + r8) * nblk;

    float* const mypart = part + (wave * 2 + slice) * chunk * kFewRows;
    // Expert row of this lane's token in the group from t0 (rows past the last
    // repeat it; never stored), and its pair, which is asked for ahead of the
    // weights: loads return in order.
    auto row_of = [&](int t0) { return row0 + min(t0 + r8, ntok - 1); };
    int pair = kGather ? gidx[row_of(0)] : 0;
    for (int win = wave; win < nwin; win += kFewWaves) {
      // the blocks whose scales this lane loads (the window's 2 kSt dwords; with fewer than 8 the rest repeat them)
      const int sblk = win * kWindowBlocks + (slice * 16 + g * 4) % kWindowBlocks;
      const int blk = win * kWindowBlocks + slice * 4 + g;       // this lane's block at step 0 (+ 8 a step)
      u32x4_t w[4][kSt];
      uint32_t sw[4];
#pragma unroll
      for (int rg = 0; rg < 4; ++rg)
        sw[rg] = scales4<kDwords>(wsp + static_cast<int64_t>(rg) * 8 * nblk, sblk, nblk);
      // (No branch for whole windows: past one the compiler no longer counts
      // the loads in flight and waits for all of them.)
#pragma unroll
      for (int rg = 0; rg < 4; ++rg)
#pragma unroll
        for (int st = 0; st < kSt; ++st)  // blocks past K load as zero codes (aux 2: non-temporal)
          w[rg][st] = __builtin_amdgcn_raw_buffer_load_b128(
              wres, blk + st * 8 < nblk ? r8 * wstride + (blk + st * 8) * 16 : kOutside, rg * 8 * wstride, 2);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int rg = 0; rg < 4; ++rg) sw[rg] = step_scales(sw[rg]);
      for (int t0 = 0; t0 < ntok; t0 += 8) {
        int64_t src = row_of(t0);
        if constexpr (kGather) {
          const unsigned u = static_cast<unsigned>(pair) / static_cast<unsigned>(gdiv);
          src = u < static_cast<unsigned>(src_rows) ? u : 0u;
          if (ntok > 8) pair = gidx[row_of(t0 + 8 < ntok ? t0 + 8 : 0)];  // of the next group, or the next window's first
        }
        u32x4_t x0[kSt], x1[kSt];
        const uint32_t sx = scales4<kDwords>(o.xs + src * nblk, sblk, nblk);
        const uint8_t* const xp = o.xq + src * xstride;
        // bytes of a block, and of this lane's (first) chunk in its step-0 block
        constexpr int kBlockBytes = static_cast<int>(Mx<kFmt>::bytes(kMxBlock));
        const int xblk = kFmt == kMxFp4 ? blk : win * kWindowBlocks + slice * 4 + (g >> 1);
        const uint8_t* const xl = xp + (kFmt == kMxFp4 ? 0 : (g & 1) * 16);
        // a block past K is replaced by the row's first: the weights there are zero
#pragma unroll
        for (int st = 0; st < kSt; ++st) {
          const int b0 = xblk + st * 8, b1 = b0 + 2;
          x0[st] = ld16(xl + (b0 < nblk ? b0 : 0) * kBlockBytes);
          if constexpr (kFmt == kMxFp8) x1[st] = ld16(xl + (b1 < nblk ? b1 : 0) * kBlockBytes);
          else x1[st] = u32x4_t{0u, 0u, 0u, 0u};
        }
        __builtin_amdgcn_sched_barrier(0);
        const uint32_t sxs = step_scales(sx);
        f32x4_t acc[4];
#pragma unroll
        for (int rg = 0; rg < 4; ++rg) {
          acc[rg] = f32x4_t{0.f, 0.f, 0.f, 0.f};
          acc[rg] = mx_mfma16<kFmt, 0>(w[rg][0], x0[0], x1[0], acc[rg], sw[rg], sxs);
          acc[rg] = mx_mfma16<kFmt, 1>(w[rg][1], x0[1], x1[1], acc[rg], sw[rg], sxs);
          if constexpr (kSt == 4) {
            acc[rg] = mx_mfma16<kFmt, 2>(w[rg][2], x0[2], x1[2], acc[rg], sw[rg], sxs);
            acc[rg] = mx_mfma16<kFmt, 3>(w[rg][3], x0[3], x1[3], acc[rg], sw[rg], sxs);
          }
        }
        // Pin the MFMAs here, where all lanes are active: the compiler would
        // move them, and with them their operands' last steps, under the branch.
#pragma unroll
        for (int rg = 0; rg < 4; ++rg) asm volatile("" : "+v"(acc[rg]));
        // acc[rg][q]: slice lane / 32 of weight row rg*8 + (lane/16 % 2)*4 + q,
        // token t0 + lane % 8 at its slice lane/8 % 2: kept where they match.
        if ((lane >> 5) == slice) {
          float* const p = mypart + (t0 + r8) * kFewRows + (g & 1) * 4;
#pragma unroll
          for (int rg = 0; rg < 4; ++rg) {
            f32x4_t* const at = reinterpret_cast<f32x4_t*>(p + rg * 8);
            if (win >= kFewWaves) acc[rg] += *at;  // not this wave's first window
            *at = acc[rg];
          }
        }
      }
    }
    __syncthreads();
    // thread -> weight row tid % 32 of token tid / 32 (+ 8 per turn)
    const int wr = tid % kFewRows;
    const int nw = min(nwin, kFewWaves) * 2;
    for (int tok = tid / kFewRows; (tok & ~7) < ntok; tok += kFewWaves * kWave / kFewRows) {
      float v = 0.f;
      for (int w = 0; w < nw; ++w) v += part[(w * chunk + tok) * kFewRows + wr];
      const int r = row0 + tok;
      if constexpr (kGather) {
        // an entry that names no token gives a zero row
        const unsigned u = tok < ntok ? static_cast<unsigned>(gidx[r]) / static_cast<unsigned>(gdiv) : 0u;
        if (u >= static_cast<unsigned>(src_rows)) v = 0.f;
      }
      out.store_one(r, o.N, n0, wr, tok < ntok, v);
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Tiled kernel on 32x32x64 scaled MFMAs, fed by direct buffer->LDS loads, in
// two shapes:
//   Big: 256 token rows x 256 weight rows, 8 waves of 128 x 64: the least
//     traffic per product.
//   Mid: 64 token rows x 128 weight rows (e2m1 rows: 64), 4 waves of 64 x 32,
//     for experts of some dozen rows: bound by the weight stream and its
//     latency, so more tiles and several blocks on a CU, with rings of 4 stages
//     (two blocks) or of 2 (three).
//
// * A stage is 128 bytes of every token row (256 of K in e2m1, 128 in e4m3)
//   and the same K of the weight rows.  LDS holds a ring of token units, a ring
//   of weight units and two chunks of scales: those of up to 1024 (Mid: 2048)
//   of K of all the tile's rows.  The scales come in runs of 32 bytes per row,
//   not per stage: a stage needs 4 or 8 bytes of a row, and fetching those
//   alone would move a cache line for each.
// * The streams of weight units, token units and scale chunks run on across
//   the persistent block's tiles, at most one tile ahead.
// * Loads go through buffer resources whose range covers only the tile's
//   valid rows: rows past an expert's segment or past N read as zero, and
//   per-lane offsets are 32-bit.
// * LDS layout: 16-byte chunk c of row r at chunk c ^ key(r), with keys that
//   spread the fragment reads of 16 lanes over all banks.
// * The weight rows are operand A, so a lane of the result holds one token
//   row, and they are read in the order pi(x) = 16*((x>>2)&1) + 4*(x>>3) +
//   (x&3): a lane's 16 results are 16 consecutive columns, and lane and lane ^
//   32 hold one block of 32, which the up-projection's epilogue quantises with
//   a single exchange.
// * Where K ends inside a stage, the token chunks past it are loaded as zero
//   and the scales past it are masked, so what the weight unit holds there
//   (e2m1 codes are all finite) adds nothing.
// Measured on MI355X, Big, both products: e4m3 rows, d = 2048, F = 5632, 32
// experts, k = 2: 0.46 ms at 8192 tokens (1.63 PFLOP/s; 2.5 tiles per CU in the
// down projection, so the last round of tiles runs half full), 1.48 ms at 32768
// (2.05); e2m1 rows, d = 4096, F = 14336, 64 experts, k = 2: 2.45 ms at 16384
// tokens (3.15).  A stage's MFMAs take about 60 % of its cycles; the waits for
// data 2 to 5 % (e2m1 up to 18), the barrier 16 % and the up-projection's
// epilogue 18 %.  Tried and slower: a block's tiles as one contiguous run of
// equal cost (8192 tokens: 0.50 ms; neighbouring tiles then no longer run at the
// same time and share the L2), scales in LDS with a swizzle against bank
// conflicts (2.74 ms), 128 x 192 tiles in two blocks per CU (1.54 ms at 32768).
constexpr int kXRow = 128;  // bytes of a token row per stage
constexpr int kRun = 32;    // bytes of a row's scales that one load covers
template <int kFmt> struct Stage {
  static constexpr int kK = kFmt == kMxFp4 ? 256 : 128;
  static constexpr int kSteps = kK / 64;             // k-steps of one MFMA depth
  static constexpr int kWRow = kK / 2;               // bytes of a weight row
  static constexpr int kScales = kK / kMxBlock;      // scale bytes of a row
};
// kBM x kBN tile of kWM x kWN waves; kXS, kWS: stages in the token and weight
// rings (kXS <= kWS); kRuns: runs of scales in a chunk.
template <int kFmt_> struct BigShape {
  static constexpr int kFmt = kFmt_, kBM = 256, kBN = 256, kWM = 2, kWN = 4, kXS = 2, kWS = kFmt_ == kMxFp4 ? 2 : 4,
                       kRuns = 1;
};
template <int kFmt_, int kRing> struct MidShape {
  static constexpr int kFmt = kFmt_, kBM = 64, kBN = kFmt_ == kMxFp4 ? 64 : 128, kWM = kFmt_ == kMxFp4 ? 2 : 1,
                       kWN = 4 / kWM, kXS = kRing, kWS = kRing, kRuns = kFmt_ == kMxFp4 ? 2 : 1;
};
// kOdd: K is an odd multiple of 64, so every second row of scales starts in the
// middle of a dword.
template <typename S, bool kOdd> struct Plan {
  using St = Stage<S::kFmt>;
  static constexpr int kWaves = S::kWM * S::kWN;
  static constexpr int kWUnit = S::kBN * St::kWRow;
  static constexpr int kXUnit = S::kBM * kXRow;
  static constexpr int kXAt = S::kWS * kWUnit;                 // LDS: weight ring, token ring, scale chunks
  static constexpr int kScaleAt = kXAt + S::kXS * kXUnit;
  static constexpr int kChunkW = S::kRuns * S::kBN * kRun;     // a chunk: the weights' runs, then the tokens'
  static constexpr int kChunk = kChunkW + S::kRuns * S::kBM * kRun;
  static constexpr size_t kLds = kScaleAt + 2 * kChunk;
  static constexpr int kPerCu = 160 * 1024 / kLds;             // blocks that fit a CU
  // (an odd row's scales lie 2 bytes into the first dword)
  static constexpr int kChunkStages = (S::kRuns * kRun - (kOdd ? 4 : 0)) / St::kScales;
  static constexpr int kRowsW = S::kBN / kWaves;               // rows of a unit that a wave fills
  static constexpr int kRowsX = S::kBM / kWaves;
  static constexpr int kLdW = kRowsW * St::kWRow / 1024;       // 16-byte loads per lane per unit
  static constexpr int kLdX = kRowsX * kXRow / 1024;
  static constexpr int kWF = S::kBN / (S::kWN * 32);           // 32-row fragments of a wave
  static constexpr int kNJ = S::kBM / (S::kWM * 32);
  // Loads that may be in flight when a stage begins: those issued after the
  // ones it needs (each stage issues its token unit, then its weight unit).
  static constexpr int kInFlightShort = (S::kXS - 2) * (kLdW + kLdX);  // the weight ring no longer than the token ring
  static constexpr int kInFlight = kInFlightShort + (S::kWS > S::kXS ? kLdW : 0);
  // A chunk of scales is issued in the first stage of the chunk before, at its
  // end, and has landed kXS - 2 stages later; it is read at the end of that
  // chunk's last stage.  More than one chunk split K into chunks of at least
  // (kChunkStages + 1) / 2 stages.
  static_assert((kChunkStages + 1) / 2 >= (S::kXS > 3 ? S::kXS - 1 : 2), "scale chunks too short for the rings");
  static_assert(kLds <= 160 * 1024 && kInFlight < 64, "does not fit");
};

typedef __attribute__((address_space(3))) void* lds_ptr_t;

// kBytes (4 or 16) per lane straight to LDS: lane l's go to dst + l * kBytes.
// (A device function: the host compilation does not know the 16-byte form.)
// `at` is the same for all lanes; offset + at counts in the bounds check.
template <int kBytes>
__device__ __forceinline__ void load_lds(__amdgpu_buffer_rsrc_t rsrc, unsigned char* dst, int offset, int at) {
  if constexpr (kBytes == 16)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_ptr_t)dst, 16, offset, at, 0, 0);
  else
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_ptr_t)dst, 4, offset, at, 0, 0);
}

template <int N> __device__ __forceinline__ void wait_vmcnt_lgkm0() {
  // gfx9 s_waitcnt: vmcnt[3:0] and [15:14], expcnt[6:4] (7 = no wait), lgkmcnt[11:8]
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
}

template <typename S, bool kGather, bool kOdd, typename Out>
__global__ __launch_bounds__((Plan<S, kOdd>::kWaves * kWave)) void mx_product_tiled(MxOperands o, const int32_t* __restrict__ gidx,
                                                                     int gdiv, int src_rows, Out out) {
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  using P = Plan<S, kOdd>;
  using St = typename P::St;
  constexpr int kFmt = S::kFmt, kSteps = St::kSteps, kWRow = St::kWRow, kBM = S::kBM, kBN = S::kBN, kLdW = P::kLdW,
                kLdX = P::kLdX, kLd = kLdX + kLdW, kWF = P::kWF;
  constexpr int kWLanes = kWRow / 16;  // lanes that fill one weight row

  const int tid = threadIdx.x;
  const int lane = tid % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int wm = wave / S::kWN;  // token part: fragments j * kWM + wm
  const int wn = wave % S::kWN;  // weight part

  // Expert table in registers: lane e has expert e's row segment (clamped:
  // offsets come from device memory) and the count of m-tiles through it.  An
  // expert's m-tiles have equal heights (rounded up to 32 rows).
  int t_seg0 = 0, t_seg1 = 0;
  if (lane < o.E) {
    t_seg0 = min(max(o.offsets[lane], 0), o.max_rows);
    t_seg1 = min(max(o.offsets[lane + 1], t_seg0), o.max_rows);
  }
  const int t_rows = t_seg1 - t_seg0;
  const int t_mt = (t_rows + kBM - 1) / kBM;
  const int t_h = t_mt > 0 ? ((t_rows + t_mt - 1) / t_mt + 31) & ~31 : kBM;
  int t_incl = t_mt;
#pragma unroll
  for (int m = 1; m < kWave; m <<= 1) {
    const int u = __shfl_up(t_incl, m);
    if (lane >= m) t_incl += u;
  }
  const int N = o.N, K = o.K, E = o.E;
  const int n_tiles_n = (N + kBN - 1) / kBN;
  const int total = __builtin_amdgcn_readlane(t_incl, E - 1) * n_tiles_n;
  const int G = gridDim.x;
  // Blocks are dealt round-robin to the 8 XCDs: each XCD gets a contiguous run
  // of every G tiles, or an eighth of them all if they are fewer.
  int tile = blockIdx.x;
  if ((G & 7) == 0) {
    const int run = total < G ? (total + 7) >> 3 : G >> 3;
    if (static_cast<int>(blockIdx.x >> 3) >= run) return;
    tile = (blockIdx.x & 7) * run + (blockIdx.x >> 3);
  }
  if (tile >= total) return;
  const int kstages = (K + St::kK - 1) / St::kK;
  // chunks of scales: as equal as can be, so that none is short
  const int nchunks = (kstages + P::kChunkStages - 1) / P::kChunkStages;
  const int chunk_base = kstages / nchunks, chunk_more = kstages % nchunks;
  const int wstride = K / 2;
  const int xstride = static_cast<int>(Mx<kFmt>::bytes(K));
  const int sstride = K / kMxBlock;

  struct TileCoord {
    int e, m0, n0, rows;  // rows = 0: no tile
  };
  // Within an expert, tiles run in groups of up to 8 m-tiles: all n-tiles of
  // the group, m-tile fastest, so one XCD's run of tiles reuses both operands
  // from its L2.
  auto coord = [&](int at) {
    constexpr int kGroupM = 8;
    const unsigned long long done = __ballot(lane < E && t_incl * n_tiles_n <= at);
    const int e = __builtin_amdgcn_readfirstlane(static_cast<int>(__popcll(done)));
    if (e >= E) return TileCoord{0, 0, 0, 0};
    const int mt_e = __builtin_amdgcn_readlane(t_mt, e);
    const int local = at - (__builtin_amdgcn_readlane(t_incl, e) - mt_e) * n_tiles_n;
    const int group = local / (kGroupM * n_tiles_n);
    const int first_m = group * kGroupM;
    const int gsize = min(kGroupM, mt_e - first_m);
    const int in = local - group * kGroupM * n_tiles_n;
    const int h = __builtin_amdgcn_readlane(t_h, e);
    const int m0 = __builtin_amdgcn_readlane(t_seg0, e) + (first_m + in % gsize) * h;
    return TileCoord{e, __builtin_amdgcn_readfirstlane(m0), __builtin_amdgcn_readfirstlane((in / gsize) * kBN),
                     __builtin_amdgcn_readfirstlane(min(h, __builtin_amdgcn_readlane(t_seg1, e) - m0))};
  };
  auto key_x = [](int r) { return (r >> 1) & 7; };
  // of a weight row, from the rows 16 lanes read together (pi of 16 consecutive)
  auto key_w = [](int r) {
    return kWRow == 128 ? ((r >> 1) & 3) | (((r >> 4) & 1) << 2) : ((r >> 2) & 1) | (((r >> 4) & 1) << 1);
  };

  // Offset of a row's scales, down to a whole dword.
  auto scale_offset = [&](int row) { return row * sstride - (kOdd ? (row & 1) * 2 : 0); };

  // ---- producers.  This wave fills kRowsW and kRowsX rows of every unit: a
  // load instruction moves 1 KB, 8 token rows (or 8 or 16 weight rows), or runs
  // of 8 rows' scales.
  constexpr int kTW = P::kRowsW / 8;  // scale loads of a run, weights
  const int srow = wave * P::kRowsX + (lane >> 3);  // token rows: + 8 i
  int vw[kLdW], vx[kLdX], vs[kLdX], vt[kTW];  // offsets of weight, token, token-scale and weight-scale loads
  bool past[kLdX];                            // this lane's token chunk lies past K in the last stage
  const int last_bytes = xstride - (kstages - 1) * kXRow;
#pragma unroll
  for (int i = 0; i < kLdW; ++i) {
    const int r = wave * P::kRowsW + i * (64 / kWLanes) + lane / kWLanes;
    vw[i] = r * wstride + (((lane % kWLanes) ^ key_w(r)) << 4);
  }
#pragma unroll
  for (int i = 0; i < kTW; ++i) vt[i] = scale_offset(wave * P::kRowsW + 8 * i + (lane >> 3)) + (lane & 7) * 4;
#pragma unroll
  for (int i = 0; i < kLdX; ++i) {
    const int r = srow + 8 * i;
    const int c = (lane & 7) ^ key_x(r);
    vx[i] = r * xstride + (c << 4);
    past[i] = (c << 4) >= last_bytes;
    vs[i] = scale_offset(r) + (lane & 7) * 4;
  }
  TileCoord cur = coord(tile), nxt = coord(tile + G);
  int gn[kLdX] = {};  // gathered: the pairs of rows srow + 8 i of the next tile
  auto load_gidx = [&](const TileCoord& t) {
    const __amdgpu_buffer_rsrc_t rsrc = resource(gidx + t.m0, t.rows * 4);
#pragma unroll
    for (int i = 0; i < kLdX; ++i) gn[i] = __builtin_amdgcn_raw_buffer_load_b32(rsrc, (srow + 8 * i) * 4, 0, 0);
  };
  // Source row of row srow + 8 i of tile t (whose pairs gn holds), or -1: past the tile, or no token.
  auto source = [&](const TileCoord& t, int i) {
    const unsigned src = static_cast<unsigned>(gn[i]) / static_cast<unsigned>(gdiv);
    return srow + 8 * i < t.rows && src < static_cast<unsigned>(src_rows) ? static_cast<int>(src) : -1;
  };
  __amdgpu_buffer_rsrc_t w_res, x_res;  // the streams' operand rows of their tile (none: loads give zero)
  const uint8_t *cw_base = nullptr, *cx_base = nullptr;
  int cw_rows = 0, cx_rows = 0;
  int w_ks = 0, x_ks = 0, c_chunk = 0, c_start = 0;  // next stage or chunk (and its first stage) of each stream's tile
  int w_slot = 0, x_slot = 0, c_slot = 0;
  auto to_w = [&](const TileCoord& t) {
    w_ks = 0;
    w_res = resource(o.wq + (static_cast<int64_t>(t.e) * N + t.n0) * wstride,
                     t.rows > 0 ? min(N - t.n0, kBN) * wstride : 0);
  };
  auto to_x = [&](const TileCoord& t) {
    x_ks = 0;
    if constexpr (kGather) {
      x_res = resource(o.xq, t.rows > 0 ? src_rows * xstride : 0);
#pragma unroll
      for (int i = 0; i < kLdX; ++i) {
        const int s = source(t, i);
        vx[i] = s < 0 ? kOutside : s * xstride + (((lane & 7) ^ key_x(srow + 8 * i)) << 4);
      }
    } else {
      x_res = resource(o.xq + static_cast<int64_t>(t.m0) * xstride, t.rows * xstride);
    }
  };
  auto to_scales = [&](const TileCoord& t) {
    c_chunk = c_start = 0;
    cw_base = o.ws + (static_cast<int64_t>(t.e) * N + t.n0) * sstride;
    cw_rows = t.rows > 0 ? min(N - t.n0, kBN) : 0;
    if constexpr (kGather) {
      cx_base = o.xs;
      cx_rows = t.rows > 0 ? src_rows : 0;
#pragma unroll
      for (int i = 0; i < kLdX; ++i) {
        const int s = source(t, i);
        vs[i] = s < 0 ? kOutside : scale_offset(s) + (lane & 7) * 4;
      }
    } else if constexpr (kOdd) {
      // from an even row on, so that its dwords are whole
      const int lead = t.m0 & 1;
      cx_base = o.xs + static_cast<int64_t>(t.m0 - lead) * sstride;
      cx_rows = t.rows > 0 ? t.rows + lead : 0;
#pragma unroll
      for (int i = 0; i < kLdX; ++i) vs[i] = scale_offset(srow + 8 * i + lead) + (lane & 7) * 4;
    } else {
      cx_base = o.xs + static_cast<int64_t>(t.m0) * sstride;
      cx_rows = t.rows;
    }
  };
  // Where a stage's loads go, where in K they start, and whether it is the tile's last.
  struct Refill {
    int xd, wd;  // LDS offsets
    int xk, wk;
    bool last;
  };
  auto refill = [&]() {
    return Refill{P::kXAt + x_slot * P::kXUnit + wave * P::kRowsX * kXRow, w_slot * P::kWUnit + wave * P::kRowsW * kWRow,
                  x_ks * kXRow, w_ks * kWRow, x_ks + 1 == kstages};
  };
  // Load i of a stage's kLd: the token unit first.
  auto issue = [&](const Refill& f, int i) {
    if (i < kLdX) load_lds<16>(x_res, smem + f.xd + i * 1024, f.last && past[i] ? kOutside : vx[i], f.xk);
    else load_lds<16>(w_res, smem + f.wd + (i - kLdX) * 1024, vw[i - kLdX], f.wk);
  };
  auto advance_w = [&]() {
    w_slot = w_slot + 1 == S::kWS ? 0 : w_slot + 1;
    ++w_ks;
  };
  auto advance_x = [&]() {
    x_slot = x_slot + 1 == S::kXS ? 0 : x_slot + 1;
    ++x_ks;
  };
  // Dword loads.  A row's bytes past its last scale are the next row's, or zero
  // past the range, which ends with a whole dword (an odd row's last one holds
  // 2 bytes of the row after it, or past the array's end: not used).
  auto issue_scales = [&]() {
    const __amdgpu_buffer_rsrc_t wr = resource(cw_base, (cw_rows * sstride + 3) / 4 * 4);
    const __amdgpu_buffer_rsrc_t xr = resource(cx_base, (cx_rows * sstride + 3) / 4 * 4);
    const int at = c_start * St::kScales;
    unsigned char* wd = smem + P::kScaleAt + c_slot * P::kChunk + wave * P::kRowsW * kRun;
    unsigned char* xd = smem + P::kScaleAt + c_slot * P::kChunk + P::kChunkW + wave * P::kRowsX * kRun;
#pragma unroll
    for (int run = 0; run < S::kRuns; ++run) {
#pragma unroll
      for (int i = 0; i < kTW; ++i) load_lds<4>(wr, wd + run * kBN * kRun + i * 256, vt[i], at + run * kRun);
#pragma unroll
      for (int i = 0; i < kLdX; ++i) load_lds<4>(xr, xd + run * kBM * kRun + i * 256, vs[i], at + run * kRun);
    }
    c_slot ^= 1;
    c_start += chunk_base + (c_chunk < chunk_more ? 1 : 0);
    ++c_chunk;
  };

  // ---- prologue: the first scale chunk, kXS token units, kWS weight units
  // (the host has seen to kstages >= kXS)
  if constexpr (kGather) load_gidx(cur);
  to_w(cur);
  to_x(cur);
  to_scales(cur);
  issue_scales();
#pragma unroll
  for (int u = 0; u < S::kWS; ++u) {
    if (u >= kstages) break;  // a tile shorter than the weight ring: the ring is kept as short
    const Refill f = refill();
#pragma unroll
    for (int i = 0; i < kLd; ++i)
      if (u < S::kXS || i >= kLdX) issue(f, i);
    if (u < S::kXS) advance_x();
    advance_w();
  }

  const int frow = lane & 31;
  const int half = lane >> 5;
  const int wrow = ((frow >> 2) & 1) * 16 + (frow >> 3) * 4 + (frow & 3);
  const int kx = key_x(frow);
  const int kw = key_w(wrow);
  int r_w = 0, r_x = 0, r_c = 0, r_cs = 0;  // slots the next fragments are read from; stage within the scale chunk
  int r_chunk = 0;                          // that chunk
  // bytes of the scale words that lie before K, in the last stage of a tile
  const int tail_steps = kSteps - (kstages * St::kK - K) / 64;
  const uint32_t tail_mask = kFmt == kMxFp4 ? 0xffffffffu >> (8 * (kSteps - tail_steps))
                                            : (tail_steps == kSteps ? 0x00ff00ffu : 0x000000ffu);

  u32x4_t wf[2][kWF], xlo[P::kNJ], xhi[P::kNJ];  // weight fragments double-buffered; token fragments replaced when used
  uint32_t sw[kWF], sx[P::kNJ];                  // this stage's scales: byte kk (e2m1) or 2 kk (e4m3) is k-step kk's
  const u32x4_t zero = {0u, 0u, 0u, 0u};
  const int w_at = (wn * kWF * 32 + wrow) * kWRow;
  const int x_at = P::kXAt + (wm * 32 + frow) * kXRow;
  auto read_w = [&](int kk, int i) {
    return *reinterpret_cast<const u32x4_t*>(smem + r_w * P::kWUnit + i * 32 * kWRow +
                                             (w_at + (((kk * 2 + half) ^ kw) << 4)));
  };
  auto read_x = [&](int kk, int j, int hi) {
    const int c = kFmt == kMxFp4 ? kk * 2 + half : kk * 4 + 2 * hi + half;
    return *reinterpret_cast<const u32x4_t*>(smem + r_x * P::kXUnit + j * S::kWM * 32 * kXRow + (x_at + ((c ^ kx) << 4)));
  };
  // The words of this stage's scales of a row, as they lie in LDS, and the
  // scales of this lane's K blocks from them (odd: they start 2 bytes into
  // their word).
  struct Words {
    uint32_t w[(kFmt == kMxFp4 ? 2 : 1) + (kOdd ? 1 : 0)];
  };
  int s_w = 0, s_x = 0;  // LDS offsets of the stage's scales: of row 0's, weights and tokens
  auto place_scales = [&]() {
    const int b = r_cs * St::kScales, run = S::kRuns == 1 ? 0 : b / kRun;
    s_w = P::kScaleAt + r_c * P::kChunk + b + run * (kBN - 1) * kRun;
    s_x = P::kScaleAt + P::kChunkW + r_c * P::kChunk + b + run * (kBM - 1) * kRun;
  };
  auto fetch_scale = [&](int at, int rows) {
    Words v;
    constexpr int kN = sizeof(v.w) / 4;
    if constexpr (!kOdd && kN == 2) {
      const uint2 u = *reinterpret_cast<const uint2*>(smem + at);
      v.w[0] = u.x;
      v.w[1] = u.y;
    } else {
#pragma unroll
      for (int n = 0; n < kN; ++n) {
        // with two runs a later word may be in the second
        const int over = S::kRuns > 1 && r_cs * St::kScales % kRun + 4 * n >= kRun ? (rows - 1) * kRun : 0;
        v.w[n] = *reinterpret_cast<const uint32_t*>(smem + at + 4 * n + over);
      }
    }
    return v;
  };
  auto scale_of = [&](const Words& v, uint32_t mask, int odd) {
    uint32_t lo = v.w[0], hi = 0;
    if constexpr (kOdd) lo = __builtin_amdgcn_alignbit(v.w[1], lo, 16 * odd);
    if constexpr (kFmt == kMxFp4) {
      hi = v.w[1];
      if constexpr (kOdd) hi = __builtin_amdgcn_alignbit(v.w[2], hi, 16 * odd);
      return __builtin_amdgcn_perm(hi, lo, half ? 0x07050301u : 0x06040200u) & mask;
    } else {
      return (lo >> (8 * half)) & mask;
    }
  };
  const int sw_at = (wn * kWF * 32 + wrow) * kRun;
  const int sx_at = (wm * 32 + frow) * kRun;
  int x_odd[P::kNJ] = {};  // kOdd: whether the lane's token rows are odd rows of xs
  Words ww[kWF], xw[P::kNJ];
  auto fetch_scales = [&](auto nj_c) {
#pragma unroll
    for (int i = 0; i < kWF; ++i) ww[i] = fetch_scale(s_w + sw_at + i * 32 * kRun, kBN);
#pragma unroll
    for (int j = 0; j < decltype(nj_c)::value; ++j) xw[j] = fetch_scale(s_x + sx_at + j * S::kWM * 32 * kRun, kBM);
  };
  auto finish_scales = [&](auto nj_c, bool last) {
    const uint32_t mask = last ? tail_mask : 0xffffffffu;
#pragma unroll
    for (int i = 0; i < kWF; ++i) sw[i] = scale_of(ww[i], mask, wrow & 1);
#pragma unroll
    for (int j = 0; j < decltype(nj_c)::value; ++j) sx[j] = scale_of(xw[j], mask, x_odd[j]);
  };
  auto barrier = [&]() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  wait_vmcnt_lgkm0<0>();
  barrier();

  auto run_tile = [&](auto nj_c) {
    constexpr int NJ = decltype(nj_c)::value;
    f32x16_t acc[kWF][NJ];
#pragma unroll
    for (int i = 0; i < kWF; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.f;
    if constexpr (kOdd) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int r = (j * S::kWM + wm) * 32 + frow;
        if constexpr (kGather) {
          const __amdgpu_buffer_rsrc_t rsrc = resource(gidx + cur.m0, cur.rows * 4);  // zero past the tile
          x_odd[j] = static_cast<unsigned>(__builtin_amdgcn_raw_buffer_load_b32(rsrc, r * 4, 0, 0)) /
                     static_cast<unsigned>(gdiv) & 1;
        } else {
          x_odd[j] = (cur.m0 + r) & 1;
        }
      }
    }
    // k-step 0 of the tile (the previous tile's last block read it with that tile's NJ)
#pragma unroll
    for (int i = 0; i < kWF; ++i) wf[0][i] = read_w(0, i);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      xlo[j] = read_x(0, j, 0);
      if constexpr (kFmt == kMxFp8) xhi[j] = read_x(0, j, 1);
    }
    place_scales();
    fetch_scales(nj_c);
    finish_scales(nj_c, false);

    // One k-step: its kWF NJ MFMAs, each token fragment replaced by that of
    // `next` once used, and (last) the loads that refill the freed slots.
    auto block = [&](auto kk_c, auto next_c, auto last_c, const Refill& f, u32x4_t (&wa)[kWF], u32x4_t (&wb)[kWF]) {
      constexpr int kk = decltype(kk_c)::value, next = decltype(next_c)::value;
      constexpr int kSel = kFmt == kMxFp4 ? kk : 2 * kk;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
#pragma unroll
        for (int i = 0; i < kWF; ++i) {
          acc[i][j] = mx_mfma32<kFmt, kSel>(frag(wa[i], zero), frag(xlo[j], kFmt == kMxFp8 ? xhi[j] : zero), acc[i][j],
                                            static_cast<int>(sw[i]), static_cast<int>(sx[j]));
          if (j == 0) wb[i] = read_w(next, i);
        }
        xlo[j] = read_x(next, j, 0);
        if constexpr (kFmt == kMxFp8) xhi[j] = read_x(next, j, 1);
        if constexpr (decltype(last_c)::value) {
#pragma unroll
          for (int l = j * kLd / NJ; l < (j + 1) * kLd / NJ; ++l) issue(f, l);
        }
      }
      // Pin the accumulators here: the compiler would else sink the MFMAs
      // past the stage's branches to its end, with every fragment live.
#pragma unroll
      for (int i = 0; i < kWF; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) asm volatile("" : "+a"(acc[i][j]));
    };
    for (int ks = 0; ks < kstages; ++ks) {
      using std::integral_constant;
      constexpr integral_constant<bool, false> no{};
      constexpr integral_constant<bool, true> yes{};
      // scalar work before the wait, in the MFMAs' shadow
      if (x_ks == kstages) to_x(nxt);
      if (w_ks == kstages) to_w(nxt);
      Refill f = refill();
      advance_x();
      advance_w();
      block(integral_constant<int, 0>{}, integral_constant<int, 1>{}, no, f, wf[0], wf[1]);
      if constexpr (kSteps == 4) {
        block(integral_constant<int, 1>{}, integral_constant<int, 2>{}, no, f, wf[1], wf[0]);
        block(integral_constant<int, 2>{}, integral_constant<int, 3>{}, no, f, wf[0], wf[1]);
      }
      // (and before the barrier: the asm statements keep the compiler from
      // putting it off until every wave waits for it)
      const bool chunk_begins = r_cs == 0;
      r_w = r_w + 1 == S::kWS ? 0 : r_w + 1;
      r_x = r_x + 1 == S::kXS ? 0 : r_x + 1;
      if (++r_cs == chunk_base + (r_chunk < chunk_more ? 1 : 0)) {
        r_cs = 0;
        r_c ^= 1;
        r_chunk = r_chunk + 1 == nchunks ? 0 : r_chunk + 1;
      }
      place_scales();
      asm volatile("" : "+s"(r_w), "+s"(r_x), "+s"(r_c), "+s"(r_cs), "+s"(s_w), "+s"(s_x));
      asm volatile("" : "+s"(f.xd), "+s"(f.wd), "+s"(f.xk), "+s"(f.wk));
      // The next stage must have landed.  lgkmcnt(0): this wave's reads of the
      // stage are complete, so after the barrier its units are free.
      if (S::kWS > S::kXS && kstages < S::kWS) wait_vmcnt_lgkm0<P::kInFlightShort>();
      else wait_vmcnt_lgkm0<P::kInFlight>();
      barrier();
      __builtin_amdgcn_sched_barrier(0);
      // The first stage of a scale chunk: the other chunk slot is free.
      if (chunk_begins) {
        if (c_chunk == nchunks) to_scales(nxt);
        issue_scales();
      }
      fetch_scales(nj_c);
      block(integral_constant<int, kSteps - 1>{}, integral_constant<int, 0>{}, yes, f, wf[1], wf[0]);
      finish_scales(nj_c, ks + 2 == kstages);
    }

    // acc[i][j][q]: tile row (j kWM + wm)*32 + frow, column (wn kWF + i)*32 + 16 half + q.
    const typename Out::Tile to(out, cur.m0, cur.rows, N);
    const int col = cur.n0 + wn * kWF * 32;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int row = (j * S::kWM + wm) * 32 + frow;
      uint32_t b[kWF];
#pragma unroll
      for (int i = 0; i < kWF; ++i) {
        // Redefine the group's accumulators here (an empty asm on their
        // registers): otherwise the compiler copies all of them out of the
        // accumulator registers at the loop exit.
        asm volatile("" : "+a"(acc[i][j])::"memory");
        float v[16];
#pragma unroll
        for (int q = 0; q < 16; ++q) v[q] = acc[i][j][q];
        b[i] = to.store(row, col + 32 * i, half, v);
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (kWF == 2) to.store_scales(row, col, half, b[0], b[1]);
      else to.store_scale(row, col, half, b[0]);
    }
  };

  for (;;) {
    if constexpr (kGather) load_gidx(nxt);
    const int nj = (((cur.rows + 31) >> 5) + S::kWM - 1) / S::kWM;  // 1..kNJ
    if constexpr (P::kNJ == 4) {
      if (nj >= 4) run_tile(std::integral_constant<int, 4>{});
      else if (nj == 3) run_tile(std::integral_constant<int, 3>{});
    }
    if constexpr (P::kNJ >= 2)
      if (nj == 2) run_tile(std::integral_constant<int, 2>{});
    if (nj <= 1) run_tile(std::integral_constant<int, 1>{});
    tile += G;
    if (tile >= total) break;
    cur = nxt;
    nxt = coord(tile + G);
  }
  wait_vmcnt_lgkm0<0>();
}

// The tiled kernels take K at least the token ring long and 32-bit buffer
// offsets: a tile's rows of K and of the result, and where rows are gathered
// all of them, below 2^31 bytes.
template <typename S> bool tiled_runs(const MxOperands& o, bool gather, int src_rows) {
  constexpr int64_t kLimit = int64_t{1} << 31;
  return o.K > (S::kXS - 1) * Stage<S::kFmt>::kK && int64_t{256} * o.K < kLimit &&
         int64_t{256} * 4 * o.N < kLimit && (!gather || Mx<S::kFmt>::bytes(o.K) * src_rows < kLimit);
}

template <typename S, bool kGather, bool kOdd, typename Out>
hipError_t launch_tiled(const MxOperands& o, const int32_t* gidx, int gdiv, int src_rows, const Out& out,
                        hipStream_t stream) {
  using P = Plan<S, kOdd>;
  // once per device (of the first 64; past them at every launch)
  static std::atomic<uint64_t> allowed{0};
  int device = 0;
  if (hipError_t e = hipGetDevice(&device); e != hipSuccess) return e;
  const uint64_t bit = device < 64 ? uint64_t{1} << device : 0;
  if (!(allowed.load(std::memory_order_relaxed) & bit)) {
    if (hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(&mx_product_tiled<S, kGather, kOdd, Out>),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(P::kLds));
        e != hipSuccess)
      return e;
    allowed.fetch_or(bit, std::memory_order_relaxed);
  }
  // at most this many tiles
  const int64_t tiles = (static_cast<int64_t>((o.max_rows + S::kBM - 1) / S::kBM) + o.E) * ((o.N + S::kBN - 1) / S::kBN);
  if (tiles > 0x7fffffff) return hipErrorInvalidValue;
  const int64_t most = int64_t{device_cu_count()} * P::kPerCu;
  hipLaunchKernelGGL((mx_product_tiled<S, kGather, kOdd, Out>), dim3(static_cast<unsigned>(tiles < most ? tiles : most)),
                     dim3(P::kWaves * kWave), P::kLds, stream, o, gidx, gdiv, src_rows, out);
  return hipGetLastError();
}

template <typename S, bool kGather, typename Out>
hipError_t launch_tiled(const MxOperands& o, const int32_t* gidx, int gdiv, int src_rows, const Out& out,
                        hipStream_t stream) {
  return o.K % 128 == 0 ? launch_tiled<S, kGather, false>(o, gidx, gdiv, src_rows, out, stream)
                        : launch_tiled<S, kGather, true>(o, gidx, gdiv, src_rows, out, stream);
}

// Token rows of a block: all that an expert can have, up to 32 (16 and 32 measured: 91 and 81 us at 42 rows per expert).
int few_chunk(const MxOperands& o) { return o.rows_bound <= 8 ? 8 : o.rows_bound <= 16 ? 16 : 32; }

template <int kFmt, bool kGather, bool kDwords, int kSt, typename Out>
hipError_t launch_few(const MxOperands& o, const int32_t* gidx, int gdiv, int src_rows, const Out& out,
                      hipStream_t stream) {
  const int chunk = few_chunk(o);
  // (expert, chunk) pairs: each expert with rows has at most one chunk that is not full
  const int64_t active = o.max_rows < o.E ? o.max_rows : o.E;
  const int64_t rows = int64_t{o.rows_bound} * o.E < o.max_rows ? int64_t{o.rows_bound} * o.E : o.max_rows;
  const int64_t chunks = o.rows_bound <= chunk ? active : rows / chunk + active;
  const int64_t blocks = (chunks * (o.N / kFewRows) + 7) / 8 * 8;
  if (blocks > 0x7fffffff || int64_t{kFewRows} * o.K / 2 >= (int64_t{1} << 31)) return hipErrorInvalidValue;
  hipLaunchKernelGGL((mx_product_few<kFmt, kGather, kDwords, kSt, Out>), dim3(static_cast<unsigned>(blocks)),
                     dim3(kFewWaves * kWave), sizeof(float) * 2 * kFewWaves * kFewRows * chunk, stream, o, gidx, gdiv,
                     src_rows, chunk, out);
  return hipGetLastError();
}

template <int kFmt, bool kGather, typename Out>
hipError_t launch_few(const MxOperands& o, const int32_t* gidx, int gdiv, int src_rows, const Out& out,
                      hipStream_t stream) {
  // four windows of 512 where they cover K, else of 1024
  if (o.K % 128 == 0)
    return o.K <= 2048 ? launch_few<kFmt, kGather, true, 2>(o, gidx, gdiv, src_rows, out, stream)
                       : launch_few<kFmt, kGather, true, 4>(o, gidx, gdiv, src_rows, out, stream);
  return o.K <= 2048 ? launch_few<kFmt, kGather, false, 2>(o, gidx, gdiv, src_rows, out, stream)
                     : launch_few<kFmt, kGather, false, 4>(o, gidx, gdiv, src_rows, out, stream);
}

// Which kernel runs.  rows, active: what the batch can bring in all, and the
// experts that can have any.  Measured on MI355X (both products, us; fp8: d =
// 2048, F = 1408, 32 experts, k = 4; fp4: d = 3584, F = 2560, 64 experts, k = 2):
//   rows per expert       4     8    12    25    42    62    88
//   fp8  few             32    38    46    62    82   107   134
//        Mid             31    35    36    38    42    49    53
//        Big             43    45    46    46    51    57    65
//   rows per expert       1     3     9    19    31    62
//   fp4  few             38   117   157   209   272   447
//        Mid             66   177   184   185   207   260
//        Big             59   178   183   184   189   213
// and for one expert (d = F = 2048):
//   rows                100   200   400  3000  4000  6000  8000
//   fp8  few             19    25    38   174
//        Mid             25    26    27    47    60    83   106
//        Big             42    65    65    71    72    74    80
//   fp4  Mid                               43    57    78    97
//        Big                               49    52    54    59
//   few: weights dominate, or all its blocks run at once;
//   Mid: its tiles (an expert's last one half full) are at most two rounds of
//   two blocks per CU, three for e2m1 rows, whose tiles are half as wide; with
//   the short rings, three blocks per CU, where that saves a round (one expert,
//   d = F = 2048: fp8, 3000 rows 57 -> 47 us, fp4 46 -> 43; 42 rows per expert as
//   above 45.6 -> 42.5), not where it does not (2000 tokens, 8 experts, F = 5632,
//   fp8: 68 with the deep rings, 80 with the short);
//   few also takes what the tiled kernels do not: K shorter than their rings, rows past 32-bit offsets.
template <int kFmt, bool kGather, typename Out>
hipError_t launch_product(const MxOperands& o, const int32_t* gidx, int gdiv, int src_rows, const Out& out,
                          hipStream_t stream) {
  const int64_t bound = int64_t{o.rows_bound} * o.E;
  const int64_t rows = bound < o.max_rows ? bound : o.max_rows;
  const int64_t active = rows < o.E ? rows : o.E;
  const int cus = device_cu_count();
  const bool few = rows <= (kFmt == kMxFp4 ? 12 : 6) * active ||
                   (rows / few_chunk(o) + active) * (o.N / kFewRows) <= 3 * cus;
  if (!few) {
    using Deep = MidShape<kFmt, 4>;
    using Short = MidShape<kFmt, 2>;
    constexpr int kDeepPerCu = Plan<Deep, false>::kPerCu, kShortPerCu = Plan<Short, false>::kPerCu;
    static_assert(kDeepPerCu == 2 && kShortPerCu == 3, "the rule below was measured with these");
    const int64_t mid = (rows / Deep::kBM + (active + 1) / 2) * ((o.N + Deep::kBN - 1) / Deep::kBN);
    if (mid <= (kFmt == kMxFp4 ? 6 : 4) * cus) {
      auto rounds = [&](int per_cu) { return (mid + per_cu * cus - 1) / (per_cu * cus); };
      if (rounds(kShortPerCu) < rounds(kDeepPerCu) && tiled_runs<Short>(o, kGather, src_rows))
        return launch_tiled<Short, kGather>(o, gidx, gdiv, src_rows, out, stream);
      if (tiled_runs<Deep>(o, kGather, src_rows))
        return launch_tiled<Deep, kGather>(o, gidx, gdiv, src_rows, out, stream);
    }
    if (tiled_runs<BigShape<kFmt>>(o, kGather, src_rows))
      return launch_tiled<BigShape<kFmt>, kGather>(o, gidx, gdiv, src_rows, out, stream);
  }
  return launch_few<kFmt, kGather>(o, gidx, gdiv, src_rows, out, stream);
}

}  // namespace

hipError_t launch_mx_up(int fmt, const MxOperands& o, const int32_t* gidx, int gdiv, int src_rows, uint8_t* hq,
                        uint8_t* hs, hipStream_t stream) {
  if (o.max_rows <= 0) return hipSuccess;
  if (fmt == kMxFp4)
    return launch_product<kMxFp4, true>(o, gidx, gdiv, src_rows, UpOut<kMxFp4>{hq, hs}, stream);
  return launch_product<kMxFp8, true>(o, gidx, gdiv, src_rows, UpOut<kMxFp8>{hq, hs}, stream);
}

hipError_t launch_mx_down(int dtype, int fmt, const MxOperands& o, void* y, hipStream_t stream) {
  if (o.max_rows <= 0) return hipSuccess;
  const int rows = o.max_rows;
  if (dtype == kDtypeBF16) {
    const DownOut<uint16_t> out{static_cast<uint16_t*>(y)};
    return fmt == kMxFp4 ? launch_product<kMxFp4, false>(o, nullptr, 1, rows, out, stream)
                         : launch_product<kMxFp8, false>(o, nullptr, 1, rows, out, stream);
  }
  const DownOut<float> out{static_cast<float*>(y)};
  return fmt == kMxFp4 ? launch_product<kMxFp4, false>(o, nullptr, 1, rows, out, stream)
                       : launch_product<kMxFp8, false>(o, nullptr, 1, rows, out, stream);
}

}  // namespace moe
