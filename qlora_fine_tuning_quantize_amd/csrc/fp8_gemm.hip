// fp8_gemm.hip -- out [M, N] = a b^T of two block-scaled 8-bit matrices.
//
// 16-bit outputs: the matrix cores multiply the codes and apply the scales
// themselves (a byte 2^(s - 127) for every 32 products; the four of a block of
// 128 are the same one), so the accumulators are the result and nothing but
// matrix instructions and their operands' movement is left.  Tiles of 256 x 256
// (one workgroup to a CU, 128 x 128 in the 256 accumulators a lane of each of 4
// waves has) move the fewest bytes for a product: of the 2048 cycles that a block
// of K takes the matrix cores, 1024 load it (64 bytes a cycle), and LDS (128 a
// cycle) takes 512 to write and 1024 to read it.  What that needs is an even
// stream of all three (4096 x 28672 x 8192):
//   whole lines: rows of 64 bytes a step fetched each line twice, 759 us, rows
//     of 128 710;
//   loads spread over the products: a wave is alone on its SIMD, and one that
//     waits for the load unit starves the matrix core: in the first quarter of
//     a half block 761 us, in all of it 710;
//   rows of LDS freed and loaded again in halves, so that loads go on all the
//     time and have two blocks' time to arrive: 660 us.
// (Best of five runs each, as they were built.)  In a long run it takes 682 to
// 707 us, 2.7 - 2.8 PFLOP/s, matrix cores busy 83 % of the time at the clock that
// their power leaves (on registers alone 3.6 - 4.1 PFLOP/s with such operands).
// Where 256 x 256 tiles leave CUs idle: 128 x 256 (2.3 PFLOP/s: LDS, with 1152 of
// 1024 cycles, bounds it), then 128 x 128, and slices of K.
//
// fp32 outputs: every 8-bit matrix instruction adds with fewer bits than fp32
// (error 1.4e-5 of the result, however it is chained), so the codes are made
// bf16 and multiplied as such; k_fp8_gemm_f32.
#include "fp8_gemm.h"

namespace qlora {

namespace {

// f(j) for the share of 0 .. COUNT - 1 that falls to slot I of SLOTS
template <int SLOTS, int COUNT, int I, typename F>
__device__ __forceinline__ void spread(F &&f) {
  constexpr int from = I * COUNT / SLOTS, to = (I + 1) * COUNT / SLOTS;
  for_each<to - from>([&](auto j) { f(std::integral_constant<int, from + decltype(j)::value>{}); });
}

// and for a share of the first three quarters of the slots
template <int SLOTS, int COUNT, int I, typename F>
__device__ __forceinline__ void spread_early(F &&f) {
  if constexpr (I < SLOTS * 3 / 4) spread<SLOTS * 3 / 4, COUNT, I>(f);
}

// 16 (or 4) bytes per lane from global memory straight into LDS: lane i's go
// to lds + 16 i (4 i).  The wave's lds is uniform.
__device__ __forceinline__ void load_to_lds16(const uint8_t *g, uint8_t *lds) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)g,
                                   (__attribute__((address_space(3))) void *)lds, 16, 0, 0);
}
__device__ __forceinline__ void load_to_lds4(const uint8_t *g, uint8_t *lds) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)g,
                                   (__attribute__((address_space(3))) void *)lds, 4, 0, 0);
}

// Slot s of a group of 32 T rows in LDS holds row T (s % 32) + s / 32 of the
// group: tile t (slots 32 t ..) has every T-th row, so that the T scales of
// rows T r .. T r + T - 1 are one aligned word, and the outputs of a lane are
// 4 T consecutive ones.  Rows are 128 bytes; chunk c of 16 bytes is stored at
// place c ^ (s / 2 % 8), which spreads the 16 lanes that read one chunk of
// consecutive slots over all banks.
__device__ __forceinline__ int place_key(int slot) { return (slot >> 1) & 7; }
template <int T>
__device__ __forceinline__ uint32_t row_offset(const Fp8In &x, int64_t first, int slot, int chunk) {
  const int row = slot / (32 * T) * (32 * T) + T * (slot & 31) + slot % (32 * T) / 32;
  const int64_t most = x.rows - 1 - first;  // rows past the end read the last one
  return (uint32_t)((row < most ? row : most) * x.ld + 16 * chunk);
}

// the T scales (bytes, the first in the lowest) at an address that T divides
template <int T>
__device__ __forceinline__ uint32_t read_scales(const uint8_t *p) {
  if constexpr (T == 4) return *reinterpret_cast<const uint32_t *>(p);
  return *reinterpret_cast<const uint16_t *>(p);
}

// waits until at most n loads of this wave are under way (they finish in order)
template <int n>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(n) : "memory");
}
// and until its reads of LDS are done
template <int n>
__device__ __forceinline__ void wait_reads_and_loads() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(n) : "memory");
}

// all waves of the workgroup; nothing that is read or written moves across
__device__ __forceinline__ void meet() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The tile of a workgroup.  Workgroups go round the 8 XCDs, so each XCD is
// given a run of consecutive tiles, in bands of up to 8 tiles of m that are
// walked along n: what runs on an XCD at one time shares rows of a and of b in
// its L2.
__device__ __forceinline__ void tile_of(unsigned id, unsigned tiles_m, unsigned tiles_n,
                                        unsigned &tm, unsigned &tn) {
  const unsigned total = tiles_m * tiles_n, per = total / 8, more = total % 8;
  const unsigned x = id % 8, i = id / 8;
  const unsigned t = x * per + (x < more ? x : more) + i;
  const unsigned band = t / (8 * tiles_n), in = t % (8 * tiles_n);
  const unsigned high = tiles_m - 8 * band < 8 ? tiles_m - 8 * band : 8;
  tm = 8 * band + in % high;
  tn = in / high;
}

// A lane's outputs: tile (i, j) has row TM r + i of a and, in value 4 q + e,
// row TN (8 q + 4 h + e) + j of b, so that a lane holds runs of 4 TN of a row.
template <int TM, int TN>
__device__ __forceinline__ void run_of(const f32x16 (&acc)[TM][TN], int i, int q,
                                       float (&v)[4 * TN]) {
#pragma unroll
  for (int e = 0; e < 4; ++e)
#pragma unroll
    for (int j = 0; j < TN; ++j) v[TN * e + j] = acc[i][j][4 * q + e];
}

template <bool F16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if constexpr (F16) return Half<_Float16>::pack2(lo, hi);
  else return pack_bf16x2(lo, hi);
}

// The stores below are straight code for one type and one way each.  With both
// types made at every pair of values and one chosen, 4096 x 4096 x 128 took
// 14.0 us in place of 13.6.

// Stores a wave's tiles, whose first row and column are m0 and n0, through the
// wave's own part of LDS, 32 rows at a time (kOutRow<TN, Out> bytes a row: 16
// more than the row, so that the lanes of a run fall on different banks).  They
// leave as whole lines, 4 outputs a lane (14336 x 4096 x 2000, fp32, added: 233
// us; without, 257).  What they are added to is read a turn ahead (1240 x 2242 x
// 263: 15.3 us when read in its own turn, so 11 to 12).  EVEN: N % 4 == 0;
// otherwise 4 outputs are at any multiple of an output's size, which loads and
// stores take (14336 x 4097 x 512 in bf16 68 us, by single outputs 93; added in
// fp32 167 and 186).
template <int TN, typename Out>
constexpr int kOutRow = 32 * TN * (int)sizeof(Out) + 16;

template <int TM, int TN, bool EVEN, bool F16, bool ADD, typename Out>
__device__ __forceinline__ void store_in_lines(const f32x16 (&acc)[TM][TN], int lane,
                                               uint8_t *part, Out *out, int64_t m0, int64_t n0,
                                               int64_t M, int64_t N) {
  typedef Out Piece __attribute__((ext_vector_type(4)));
  struct Loose {
    Out v[4];
  };
  constexpr int kAcross = 32 * TN / 4, kTurns = 32 * kAcross / 64;  // pieces of a row
  const int r = lane & 31, h = lane >> 5;
  Piece was[2][kTurns];
  auto load_was = [&](int i) {
    if constexpr (ADD)
#pragma unroll
      for (int x = 0; x < kTurns; ++x) {
        const int p = 64 * x + lane;
        const int64_t m = m0 + TM * (p / kAcross) + i, n = n0 + p % kAcross * 4;
        const Out *const o = out + m * N + n;
        if (m >= M) continue;
        if constexpr (EVEN) {
          if (n < N) was[i & 1][x] = *reinterpret_cast<const Piece *>(o);
        } else if (n + 4 <= N) {
          was[i & 1][x] = __builtin_bit_cast(Piece, *reinterpret_cast<const Loose *>(o));
        } else {
#pragma unroll
          for (int e = 0; e < 3; ++e)
            if (n + e < N) was[i & 1][x][e] = o[e];
        }
      }
  };
  load_was(0);
#pragma unroll
  for (int i = 0; i < TM; ++i) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float v[4 * TN];
      run_of(acc, i, q, v);
      Out *to = (Out *)(part + r * kOutRow<TN, Out>) + TN * (8 * q + 4 * h);
      if constexpr (sizeof(Out) == 4) {
#pragma unroll
        for (int w = 0; w < TN; ++w)
          *reinterpret_cast<f32x4 *>(to + 4 * w) =
              f32x4{v[4 * w], v[4 * w + 1], v[4 * w + 2], v[4 * w + 3]};
      } else {
#pragma unroll
        for (int w = 0; w < TN; ++w) {
          const u32x2 x = {pack16<F16>(v[4 * w], v[4 * w + 1]),
                           pack16<F16>(v[4 * w + 2], v[4 * w + 3])};
          *reinterpret_cast<u32x2 *>(to + 4 * w) = x;
        }
      }
    }
    if (i + 1 < TM) load_was(i + 1);
    // a wave's own accesses of LDS are done in the order they are written in
    asm volatile("" ::: "memory");
#pragma unroll
    for (int x = 0; x < kTurns; ++x) {
      const int p = 64 * x + lane, row = p / kAcross, col = p % kAcross * 4;
      Piece w = *reinterpret_cast<const Piece *>((const Out *)(part + row * kOutRow<TN, Out>) + col);
      if constexpr (ADD) w += was[i & 1][x];
      const int64_t m = m0 + TM * row + i, n = n0 + col;
      Out *const o = out + m * N + n;
      if (m >= M) continue;
      if constexpr (EVEN) {
        if (n < N) *reinterpret_cast<Piece *>(o) = w;
      } else if (n + 4 <= N) {
        *reinterpret_cast<Loose *>(o) = __builtin_bit_cast(Loose, w);
      } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
          if (n + e < N) o[e] = w[e];
      }
    }
    asm volatile("" ::: "memory");
  }
}

template <int TM, int TN, bool F16, bool ADD, typename Out>
__device__ __forceinline__ void store_tiles(const f32x16 (&acc)[TM][TN], int lane, uint8_t *part,
                                            Out *out, int64_t m0, int64_t n0, int64_t M,
                                            int64_t N) {
  if (N % 4 == 0) store_in_lines<TM, TN, true, F16, ADD>(acc, lane, part, out, m0, n0, M, N);
  else store_in_lines<TM, TN, false, F16, ADD>(acc, lane, part, out, m0, n0, M, N);
}

// In 16 bits where rows start at multiples of 16 bytes: straight from the
// registers, 16 bytes a lane.  (Through LDS they take as long: 4096 x 4096 x 1024
// 23.9 us against 22.7.)  FULL: all of the wave's tiles are inside.
template <int TM, int TN, bool F16, bool FULL>
__device__ __forceinline__ void store_tiles16(const f32x16 (&acc)[TM][TN], int lane, uint16_t *out,
                                              int64_t m0, int64_t n0, int64_t M, int64_t N) {
  const int64_t m = m0 + TM * (lane & 31), n = n0 + TN * 4 * (lane >> 5);
  uint16_t *const o = out + m * N + n;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    if (!FULL && m + i >= M) continue;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float v[4 * TN];
      run_of(acc, i, q, v);
#pragma unroll
      for (int x = 0; x < TN / 2; ++x) {
        u32x4 w;
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = pack16<F16>(v[8 * x + 2 * e], v[8 * x + 2 * e + 1]);
        if (FULL || n + 8 * TN * q + 8 * x < N)
          *reinterpret_cast<u32x4 *>(o + i * N + 8 * TN * q + 8 * x) = w;
      }
    }
  }
}
template <int TM, int TN, bool F16>
__device__ __forceinline__ void store_tiles16(const f32x16 (&acc)[TM][TN], int lane, uint16_t *out,
                                              int64_t m0, int64_t n0, int64_t M, int64_t N) {
  if (m0 + 32 * TM <= M && n0 + 32 * TN <= N)
    store_tiles16<TM, TN, F16, true>(acc, lane, out, m0, n0, M, N);
  else
    store_tiles16<TM, TN, F16, false>(acc, lane, out, m0, n0, M, N);
}

// Tiles of 64 TM (m) x 64 TN (n): 4 waves of 2 x 2, each TM x TN tiles of 32 x
// 32, over blocks of 128 of K, two of them in LDS.  16-bit outputs.
// SPLIT: K is cut into slices, and the workgroups of each (the tiles' number of
// them) leave fp32 sums in part [slice][M][N up to 4].
template <int TM, int TN, bool A_E5M2, bool SPLIT>
__global__ __launch_bounds__(256, 1) void k_fp8_gemm(Fp8In a, Fp8In b,
                                                     uint16_t *__restrict__ out, bool f16,
                                                     int64_t M, int64_t N, unsigned tiles_m,
                                                     unsigned tiles_n, int slice_blocks,
                                                     float *__restrict__ part) {
  constexpr int BM = 64 * TM, BN = 64 * TN, kBytesA = BM * 128, kBlock = (BM + BN) * 128;
  // a wave's tiles are used in two halves of HA (a) and HB (b), and a block's
  // rows are loaded in the same halves: LA and LB loads of 8 rows per wave
  constexpr int HA = TM / 2, HB = TN / 2, LA = BM / 64, LB = BN / 64;
  // a block's scales are four pieces of 256 bytes: wave w loads words kWords w
  // .. kWords (w + 1) - 1 of a's and then b's bytes
  constexpr int kWords = (BM + BN) / 16, kScales = 2 * kBlock;
  __shared__ __align__(1024) uint8_t lds[kScales + 2 * 1024];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 31, h = lane >> 5;
  const int wm = wave >> 1, wn = wave & 1;
  const unsigned slice = SPLIT ? blockIdx.x / (tiles_m * tiles_n) : 0;
  unsigned tm, tn;
  tile_of(SPLIT ? blockIdx.x % (tiles_m * tiles_n) : blockIdx.x, tiles_m, tiles_n, tm, tn);
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
  const int skip = SPLIT ? (int)slice * slice_blocks : 0, rest = (int)(a.ld / 128) - skip;
  const int blocks = SPLIT && slice_blocks < rest ? slice_blocks : rest;

  // Rows of half x in LDS: slots 32 T g + 16 T x .. + 16 T - 1 of groups g =
  // 0 and 1 (the waves' two); load j of a wave takes the 8 slots from
  // first_slot on.
  auto first_slot = [&](auto T, int x, int j) {
    constexpr int each = 2 * decltype(T)::value;  // loads of 8 slots in a group's half
    const int i = 4 * j + wave;
    return (i / each * 32 + x * 16) * decltype(T)::value + i % each * 8;
  };
  using TA = std::integral_constant<int, TM>;
  using TB = std::integral_constant<int, TN>;
  auto offset_of = [&](const Fp8In &x, int64_t first, auto T, int slot) {
    return row_offset<decltype(T)::value>(x, first, slot, (lane & 7) ^ place_key(slot));
  };
  uint32_t off_a[2][LA], off_b[2][LB];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
#pragma unroll
    for (int j = 0; j < LA; ++j)
      off_a[x][j] = offset_of(a, m0, TA{}, first_slot(TA{}, x, j) + (lane >> 3));
#pragma unroll
    for (int j = 0; j < LB; ++j)
      off_b[x][j] = offset_of(b, n0, TB{}, first_slot(TB{}, x, j) + (lane >> 3));
  }
  const uint8_t *ca = a.codes + m0 * a.ld + (int64_t)skip * 128;
  const uint8_t *cb = b.codes + n0 * b.ld + (int64_t)skip * 128;
  const int word = wave * kWords + (lane < kWords ? lane : kWords - 1);
  const bool of_a = 4 * word < BM;
  const int64_t rp = of_a ? a.rp : b.rp, first = of_a ? m0 + 4 * word : n0 + 4 * word - BM;
  const uint8_t *scale_from =
      (of_a ? a.scales : b.scales) + skip * rp + (first < rp - 4 ? first : rp - 4);
  auto fetch_scales = [&](int block, int buf) {
    load_to_lds4(scale_from + block * rp, lds + kScales + buf * 1024 + wave * 256);
  };
  auto fetch_a = [&](int block, int buf, auto xc, auto jc) {
    constexpr int x = decltype(xc)::value, j = decltype(jc)::value;
    load_to_lds16(ca + (int64_t)block * 128 + off_a[x][j],
                  lds + buf * kBlock + first_slot(TA{}, x, j) * 128);
  };
  auto fetch_b = [&](int block, int buf, auto xc, auto jc) {
    constexpr int x = decltype(xc)::value, j = decltype(jc)::value;
    load_to_lds16(cb + (int64_t)block * 128 + off_b[x][j],
                  lds + buf * kBlock + kBytesA + first_slot(TB{}, x, j) * 128);
  };
  auto scales_at = [&](int byte) { return kScales + byte / 4 / kWords * 256 + byte / 4 % kWords * 4 + byte % 4; };
  const int sa_at = scales_at(wm * 32 * TM + TM * r), sb_at = scales_at(BM + wn * 32 * TN + TN * r);

  f32x16 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  // Fragment u (of 2) of a tile: chunks 4 u + h and 4 u + h + 2 of row r
  // (which values of K a lane holds does not matter, as long as it is the same
  // for a and b and all are of one block).
  const int at = r * 128 + ((h ^ place_key(r)) << 4);
  i32x8 fa[TM][2], fb[TN][2];
  auto read_half = [&](i32x8 &to, int tile_at, auto uc, auto vc) {
    constexpr int u = decltype(uc)::value, v = decltype(vc)::value;
    const u32x4 x =
        *reinterpret_cast<const u32x4 *>(lds + tile_at + (at ^ (v << 5) ^ (u << 6)));
#pragma unroll
    for (int e = 0; e < 4; ++e) to[4 * v + e] = (int)x[e];
  };
  // read j of the 4 HA (4 HB) that fetch the fragments of half x: first all
  // of u = 0
  auto read_a = [&](int buf, auto xc, auto jc) {
    constexpr int j = decltype(jc)::value, u = j / (2 * HA), t = decltype(xc)::value * HA + j / 2 % HA;
    read_half(fa[t][u], buf * kBlock + (wm * TM + t) * 4096, std::integral_constant<int, u>{},
              std::integral_constant<int, j & 1>{});
  };
  auto read_b = [&](int buf, auto xc, auto jc) {
    constexpr int j = decltype(jc)::value, u = j / (2 * HB), t = decltype(xc)::value * HB + j / 2 % HB;
    read_half(fb[t][u], buf * kBlock + kBytesA + (wn * TN + t) * 4096,
              std::integral_constant<int, u>{}, std::integral_constant<int, j & 1>{});
  };
  struct Scales {
    uint32_t a, b;
  };
  auto read_scales_of = [&](int buf, Scales &sc) {
    sc.a = read_scales<TM>(lds + buf * 1024 + sa_at);
    sc.b = read_scales<TN>(lds + buf * 1024 + sb_at);
  };
  // The products of half xa of a's tiles and half xb of b's over one block,
  // with what is issued between them: aside(i) after product i of kProducts.
  constexpr int kProducts = HA * HB * 2;
  auto multiply = [&](auto xa, auto xb, const Scales &sc, auto &&aside) {
    constexpr int i0 = decltype(xa)::value * HA, j0 = decltype(xb)::value * HB;
    for_each<kProducts>([&](auto ic) {
      constexpr int u = decltype(ic)::value / (HA * HB), e = decltype(ic)::value % (HA * HB);
      constexpr int i = i0 + e / HB, j = j0 + e % HB;
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
          fb[j][u], fa[i][u], acc[i][j], 0, A_E5M2 ? 1 : 0, j, (int)sc.b, i, (int)sc.a);
      aside(ic);
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;

  // Block k is multiplied in four phases, (half of a, half of b) = (0, p), (0,
  // q), (1, q), (1, p), with p = k % 2 and q = 1 - p: from one phase to the
  // next, over the border of blocks too, one of the two halves stays, and the
  // other one's fragments are read in the phase before.  So block k's half 0
  // of a and p of b are read in the last two phases of block k - 1, and their
  // rows in LDS are free in its first two, which load block k + 2's there;
  // its half q of b and 1 of a are read in its first two phases and loaded in
  // its last two.  A barrier before each pair of phases holds both together:
  // every wave has waited for its own reads of the pair before, and for its
  // loads of the pair that was issued three pairs ago, which this pair reads.
  // Loads have two whole blocks' time, and are issued evenly.  Past the last
  // block that one is loaded again, into rows that nothing reads, so that the
  // number of loads under way is always the same.
  constexpr int kPair = LA + LB, kUnderWay = 2 * kPair + 1;  // + the scales
  auto clamp = [&](int block) { return block < blocks ? block : blocks - 1; };
  auto fetch_first = [&](int block, int buf, auto p) {
    for_each<LA>([&](auto j) { fetch_a(block, buf, I0{}, j); });
    for_each<LB>([&](auto j) { fetch_b(block, buf, p, j); });
  };
  auto fetch_second = [&](int block, int buf, auto q) {
    for_each<LB>([&](auto j) { fetch_b(block, buf, q, j); });
    for_each<LA>([&](auto j) { fetch_a(block, buf, I1{}, j); });
  };
  fetch_scales(0, 0);
  fetch_first(0, 0, I0{});
  fetch_second(0, 0, I1{});
  fetch_scales(clamp(1), 1);
  fetch_first(clamp(1), 1, I1{});
  fetch_second(clamp(1), 1, I0{});
  Scales sc;
  wait_loads<3 * kPair + 1>();
  meet();
  for_each<4 * HA>([&](auto j) { read_a(0, I0{}, j); });
  for_each<4 * HB>([&](auto j) { read_b(0, I0{}, j); });
  read_scales_of(0, sc);

  auto block = [&](int k, auto p, auto q) {
    constexpr int buf = decltype(p)::value;
    const int next = clamp(k + 2);
    wait_reads_and_loads<kUnderWay>();
    meet();
    __builtin_amdgcn_sched_barrier(0);
    multiply(I0{}, p, sc, [&](auto ic) {
      constexpr int i = decltype(ic)::value;
      if constexpr (i == 0) fetch_scales(next, buf);
      spread_early<kProducts, 4 * HB, i>([&](auto j) { read_b(buf, q, j); });
      spread<kProducts, LA, i>([&](auto j) { fetch_a(next, buf, I0{}, j); });
    });
    multiply(I0{}, q, sc, [&](auto ic) {
      constexpr int i = decltype(ic)::value;
      spread_early<kProducts, 4 * HA, i>([&](auto j) { read_a(buf, I1{}, j); });
      spread<kProducts, LB, i>([&](auto j) { fetch_b(next, buf, p, j); });
    });
    wait_reads_and_loads<kUnderWay>();
    meet();
    __builtin_amdgcn_sched_barrier(0);
    Scales sn;
    multiply(I1{}, q, sc, [&](auto ic) {
      constexpr int i = decltype(ic)::value;
      if constexpr (i == 0) read_scales_of(1 - buf, sn);
      spread_early<kProducts, 4 * HA, i>([&](auto j) { read_a(1 - buf, I0{}, j); });
      spread<kProducts, LB, i>([&](auto j) { fetch_b(next, buf, q, j); });
    });
    multiply(I1{}, p, sc, [&](auto ic) {
      constexpr int i = decltype(ic)::value;
      spread_early<kProducts, 4 * HB, i>([&](auto j) { read_b(1 - buf, q, j); });
      spread<kProducts, LA, i>([&](auto j) { fetch_a(next, buf, I1{}, j); });
    });
    sc = sn;
  };
  __builtin_amdgcn_sched_barrier(0);
  for (int k = 0; k + 1 < blocks; k += 2) {
    block(k, I0{}, I1{});
    block(k + 1, I1{}, I0{});
  }
  if (blocks & 1) block(blocks - 1, I0{}, I1{});
  wait_loads<0>();  // the loads past the last block
  meet();
  const int64_t m = m0 + wm * 32 * TM, n = n0 + wn * 32 * TN;
  if constexpr (SPLIT) {
    constexpr int kPart = 32 * kOutRow<TN, float>;
    static_assert(4 * kPart <= (int)sizeof(lds), "the outputs' rows fit LDS");
    const int64_t np = (N + 3) / 4 * 4;
    store_in_lines<TM, TN, true, false, false>(acc, lane, lds + wave * kPart, part + slice * M * np,
                                            m, n, M, np);
  } else if (N % 8 == 0) {
    if (f16) store_tiles16<TM, TN, true>(acc, lane, out, m, n, M, N);
    else store_tiles16<TM, TN, false>(acc, lane, out, m, n, M, N);
  } else {
    constexpr int kPart = 32 * kOutRow<TN, uint16_t>;
    static_assert(4 * kPart <= (int)sizeof(lds), "the outputs' rows fit LDS");
    uint8_t *const mine = lds + wave * kPart;
    if (f16) store_tiles<TM, TN, true, false>(acc, lane, mine, out, m, n, M, N);
    else store_tiles<TM, TN, false, false>(acc, lane, mine, out, m, n, M, N);
  }
}

// The same tiles for fp32 outputs: the codes, times their scale, are bf16
// values and are multiplied as such.  Steps of 64 over K, three of them in
// LDS.  A conversion (two codes) takes as long as a quarter of a product of 32
// x 32 x 16, so each code is converted once per wave, in slices of 16 of K,
// between the products of the slice before (converted again for each half of
// the tiles, 14336 x 4096 x 2000 took 265 us, so 257).  Two workgroups to a CU, so
// that one multiplies while the other writes: with tiles of 256 x 256, fewer
// conversions and one workgroup, it took 346 us instead of 233.  Bound by both at
// once: vector instructions 70 % of the time, matrix cores 61 %; long products
// come to 1.29 PFLOP/s (4096 x 4096 x 16384).
template <int TM, int TN, bool A_E5M2, bool SPLIT>
__global__ __launch_bounds__(256, 2) void k_fp8_gemm_f32(Fp8In a, Fp8In b,
                                                         float *__restrict__ out, bool accumulate,
                                                         int64_t M, int64_t N, unsigned tiles_m,
                                                         unsigned tiles_n, int slice_blocks) {
  constexpr int BM = 64 * TM, BN = 64 * TN, kBytesA = BM * 64, kStage = (BM + BN) * 64;
  constexpr int LA = BM / 64, LB = BN / 64;  // loads of 16 rows per wave and step
  constexpr int kWords = (BM + BN) / 16, kScales = 3 * kStage;  // as in k_fp8_gemm
  __shared__ __align__(1024) uint8_t lds[kScales + 2 * 1024];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 31, h = lane >> 5;
  const int wm = wave >> 1, wn = wave & 1;
  const unsigned slice = SPLIT ? blockIdx.x / (tiles_m * tiles_n) : 0;
  unsigned tm, tn;
  tile_of(SPLIT ? blockIdx.x % (tiles_m * tiles_n) : blockIdx.x, tiles_m, tiles_n, tm, tn);
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
  const int skip = SPLIT ? (int)slice * slice_blocks : 0, rest = (int)(a.ld / 128) - skip;
  const int steps = 2 * (SPLIT && slice_blocks < rest ? slice_blocks : rest);

  // rows of 64 bytes: chunk c of 16 is stored at place c ^ (slot / 4 % 4)
  uint32_t off_a[LA], off_b[LB];
#pragma unroll
  for (int j = 0; j < LA; ++j) {
    const int slot = (j * 4 + wave) * 16 + (lane >> 2);
    off_a[j] = row_offset<TM>(a, m0, slot, (lane & 3) ^ ((slot >> 2) & 3));
  }
#pragma unroll
  for (int j = 0; j < LB; ++j) {
    const int slot = (j * 4 + wave) * 16 + (lane >> 2);
    off_b[j] = row_offset<TN>(b, n0, slot, (lane & 3) ^ ((slot >> 2) & 3));
  }
  const uint8_t *ca = a.codes + m0 * a.ld + (int64_t)skip * 128;
  const uint8_t *cb = b.codes + n0 * b.ld + (int64_t)skip * 128;
  const int word = wave * kWords + (lane < kWords ? lane : kWords - 1);
  const bool of_a = 4 * word < BM;
  const int64_t rp = of_a ? a.rp : b.rp, first = of_a ? m0 + 4 * word : n0 + 4 * word - BM;
  const uint8_t *scale_from =
      (of_a ? a.scales : b.scales) + skip * rp + (first < rp - 4 ? first : rp - 4);
  const int last = steps - 1;
  auto fetch_scales = [&](int block) {
    load_to_lds4(scale_from + (block < steps / 2 ? block : steps / 2 - 1) * rp,
                 lds + kScales + (block & 1) * 1024 + wave * 256);
  };
  auto fetch_one = [&](int step, int buf, auto jc) {
    constexpr int j = decltype(jc)::value;
    const int64_t k = (int64_t)(step < last ? step : last) * 64;
    uint8_t *to = lds + buf * kStage;
    if constexpr (j < LA) load_to_lds16(ca + k + off_a[j], to + (j * 4 + wave) * 1024);
    else load_to_lds16(cb + k + off_b[j - LA], to + kBytesA + ((j - LA) * 4 + wave) * 1024);
  };
  auto scales_at = [&](int byte) { return kScales + byte / 4 / kWords * 256 + byte / 4 % kWords * 4 + byte % 4; };
  const int sa_at = scales_at(wm * 32 * TM + TM * r), sb_at = scales_at(BM + wn * 32 * TN + TN * r);

  f32x16 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  // T = TM + TN fragments, a's first.  Two slices of one are 16 codes a lane,
  // chunk 2 p + h of a row.
  constexpr int T = TM + TN;
  const int at = r * 64 + ((h ^ ((r >> 2) & 3)) << 4);
  u32x4 raw[2][T], half[2][T];
  float scale[T];
  auto read_one = [&](int buf, auto pc, auto tc) {
    constexpr int p = decltype(pc)::value, t = decltype(tc)::value;
    raw[p][t] = *reinterpret_cast<const u32x4 *>(
        lds + buf * kStage + (t < TM ? (wm * TM + t) * 2048 : kBytesA + (wn * TN + t - TM) * 2048) +
        (at ^ (p << 5)));
  };
  // conversion c of the 4 T of slice s
  auto convert_one = [&](auto sc, auto cc) {
    constexpr int s = decltype(sc)::value, t = decltype(cc)::value / 4, w = decltype(cc)::value % 4;
    half[s & 1][t][w] = codes_to_bf16<(t < TM) && A_E5M2, (w & 1) != 0>(
        raw[s / 2][t][2 * (s & 1) + w / 2], scale[t]);
  };
  auto multiply = [&](auto sc, auto &&aside) {
    constexpr int s = decltype(sc)::value;
    for_each<TM * TN>([&](auto ic) {
      constexpr int i = decltype(ic)::value / TN, j = decltype(ic)::value % TN;
      acc[i][j] = Half<uint16_t>::mfma32(half[s & 1][TM + j], half[s & 1][i], acc[i][j]);
      aside(ic);
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  uint32_t ba, bb;
  auto read_scales_of = [&](int block) {
    ba = read_scales<TM>(lds + (block & 1) * 1024 + sa_at);
    bb = read_scales<TN>(lds + (block & 1) * 1024 + sb_at);
  };
  auto widen_scales = [&]() {
#pragma unroll
    for (int t = 0; t < TM; ++t) scale[t] = scale_f32((ba >> (8 * t)) & 255u);
#pragma unroll
    for (int t = 0; t < TN; ++t) scale[TM + t] = scale_f32((bb >> (8 * t)) & 255u);
  };
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  using I2 = std::integral_constant<int, 2>;
  using I3 = std::integral_constant<int, 3>;
  constexpr int kTiles = TM * TN;

  fetch_scales(0);
  fetch_scales(1);
  for (int s = 0; s < 3; ++s) for_each<LA + LB>([&](auto j) { fetch_one(s, s, j); });
  wait_loads<2 * (LA + LB)>();
  meet();
  for_each<T>([&](auto t) { read_one(0, I0{}, t); });
  read_scales_of(0);
  widen_scales();
  for_each<4 * T>([&](auto c) { convert_one(I0{}, c); });
  __builtin_amdgcn_sched_barrier(0);
  // Step k in four slices.  While slice s is multiplied, s + 1 is converted;
  // the second two's codes are read in the first slice, the next step's first
  // two's in the third.  Before that a barrier: behind it every wave has read
  // all of step k, whose rows step k + 3 is loaded into, and has waited for
  // its loads of step k + 1 (those of step k + 2 may be under way).  A block's
  // scales are loaded four steps ahead.
  int buf = 0;
  auto step = [&](int k, auto odd) {
    const int from = buf < 2 ? buf + 1 : 0;
    multiply(I0{}, [&](auto ic) {
      constexpr int i = decltype(ic)::value;
      spread_early<kTiles, T, i>([&](auto t) { read_one(buf, I1{}, t); });
      spread<kTiles, 4 * T, i>([&](auto c) { convert_one(I1{}, c); });
    });
    multiply(I1{}, [&](auto ic) {
      spread<kTiles, 4 * T, decltype(ic)::value>([&](auto c) { convert_one(I2{}, c); });
    });
    wait_reads_and_loads<LA + LB>();
    meet();
    __builtin_amdgcn_sched_barrier(0);
    multiply(I2{}, [&](auto ic) {
      constexpr int i = decltype(ic)::value;
      if constexpr (i == 0) {
        if constexpr (decltype(odd)::value) read_scales_of(k / 2 + 1);
        else fetch_scales(k / 2 + 2);
      }
      spread_early<kTiles, T, i>([&](auto t) { read_one(from, I0{}, t); });
      spread<kTiles, 4 * T, i>([&](auto c) { convert_one(I3{}, c); });
    });
    if constexpr (decltype(odd)::value) widen_scales();
    multiply(I3{}, [&](auto ic) {
      constexpr int i = decltype(ic)::value;
      spread<kTiles, LA + LB, i>([&](auto j) { fetch_one(k + 3, buf, j); });
      spread<kTiles, 4 * T, i>([&](auto c) { convert_one(I0{}, c); });
    });
    buf = from;
  };
  for (int k = 0; k < steps; k += 2) {
    step(k, std::false_type{});
    step(k + 1, std::true_type{});
  }
  wait_loads<0>();  // the loads past the last step
  meet();
  constexpr int kPart = 32 * kOutRow<TN, float>;
  static_assert(4 * kPart <= (int)sizeof(lds), "the outputs' rows fit LDS");
  const int64_t m = m0 + wm * 32 * TM, n = n0 + wn * 32 * TN, np = (N + 3) / 4 * 4;
  uint8_t *const mine = lds + wave * kPart;
  if constexpr (SPLIT)
    store_in_lines<TM, TN, true, false, false>(acc, lane, mine, out + slice * M * np, m, n, M, np);
  else if (accumulate)
    store_tiles<TM, TN, false, true>(acc, lane, mine, out, m, n, M, N);
  else
    store_tiles<TM, TN, false, false>(acc, lane, mine, out, m, n, M, N);
}

// out = the sum of S slices of part in order (or that added to out)
template <typename Out>
__global__ __launch_bounds__(256) void k_fp8_sum(const float *__restrict__ part, int S, int64_t M,
                                                 int64_t N, Out *__restrict__ out, bool f16,
                                                 bool accumulate) {
  const int64_t np = (N + 3) / 4 * 4, quads = np / 4;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= M * quads) return;
  f32x4 v = reinterpret_cast<const f32x4 *>(part)[i];
#pragma unroll 4
  for (int s = 1; s < S; ++s) v += reinterpret_cast<const f32x4 *>(part + s * M * np)[i];
  const int64_t n = i % quads * 4;
  store4(out + i / quads * N + n, v, n, N, sizeof(Out) == 4 ? accumulate : f16);
}

// How a product is cut: tiles of 64 TM x 64 TN, K in slices of slice_blocks
// blocks.
struct Plan {
  int tm, tn, slices, slice_blocks;
};
Plan plan_of(int64_t M, int64_t N, int64_t K, bool f32) {
  const auto tiles = [&](int bm, int bn) { return ((M + bm - 1) / bm) * ((N + bn - 1) / bn); };
  const int blocks = (int)((K + 127) / 128);
  // the largest tiles that still give most of the 256 CUs one
  if (!f32 && tiles(256, 256) >= 192) return {4, 4, 1, blocks};
  if (tiles(128, 256) >= 192) return {2, 4, 1, blocks};
  // Few tiles: as many slices as make a product the fastest, at most one
  // workgroup to a CU.  In us, a block of K takes a workgroup 0.37 (0.85 for
  // fp32 outputs), the launch that adds the slices 2.2, and writing and reading
  // them 8 bytes an output at 4.1 TB/s: 128 x 4096 x 14336 19.0 with 6 slices (43.7
  // with one, 20.1 with 8), 77 x 1000 x 1111 7.1 with one (8.7 with three), 512 x
  // 4096 x 4096 16.5 with one (17.9 with two).
  const int64_t most = 256 / tiles(128, 128);
  int best = blocks;
  double least = 1e30;
  for (int s = 1; s == 1 || (s <= most && s <= blocks); ++s) {
    const int each = (blocks + s - 1) / s;
    const double us = each * (f32 ? 0.85 : 0.37) +
                      (s > 1 ? 2.2 + (double)s * (double)M * (double)N * 8 / 4.1e6 : 0.0);
    if (us < least) least = us, best = each;
  }
  return {2, 2, (blocks + best - 1) / best, best};
}

// Few rows of a: the stream kernel, while its workgroups' reading all of a for
// every 16 rows of b costs less than the tiles' second launch.  (24 rows against
// 14336 x 4096: 24.0 us, in tiles 14.2; against 4096 x 4096 8.4 and 9.5; 64 rows
// against 1000 x 1000: 6.0 and 6.7, against 4096 x 14336 34.6 and 16.6.)
bool stream_preferred(int64_t M, int64_t N, int64_t K) {
  if (N >= 1 << 26) return false;  // 1024 threads for 32 rows of b: a grid's limit is 2^32
  return M <= 16 || (M <= 32 && N * K <= 1 << 24) || (M <= kStreamRows && N * K <= 1 << 22);
}

}  // namespace

size_t fp8_matmul_partial_floats(int64_t M, int64_t N, int64_t K) {
  if (stream_preferred(M, N, K)) return 0;
  int most = 1;
  for (const bool f32 : {false, true}) {
    const int s = plan_of(M, N, K, f32).slices;
    most = s > most ? s : most;
  }
  return most > 1 ? (size_t)most * (size_t)M * (size_t)((N + 3) / 4 * 4) : 0;
}

int launch_fp8_matmul(const ql_fp8 *a, const ql_fp8 *b, void *out, int out_dtype, bool accumulate,
                      float *part, hipStream_t stream) {
  const int64_t M = a->rows, N = b->rows;
  if (stream_preferred(M, N, a->cols)) {
    launch_fp8_stream(a, b, out, out_dtype, accumulate, stream);
    QL_HIP_CHECK_LAUNCH();
    return QL_OK;
  }
  const Plan p = plan_of(M, N, a->cols, out_dtype == QL_F32);
  auto go = [&](auto tmc, auto tnc, auto e5, auto split) {
    constexpr int TM = decltype(tmc)::value, TN = decltype(tnc)::value;
    constexpr bool E5 = decltype(e5)::value, SPLIT = decltype(split)::value;
    const int64_t tm = (M + 64 * TM - 1) / (64 * TM), tn = (N + 64 * TN - 1) / (64 * TN);
    const dim3 grid((unsigned)(tm * tn * p.slices)), block(256);
    if constexpr (TM * TN < 16) {
      if (out_dtype == QL_F32) {
        hipLaunchKernelGGL((k_fp8_gemm_f32<TM, TN, E5, SPLIT>), grid, block, 0, stream, fp8_in(a),
                           fp8_in(b), SPLIT ? part : (float *)out, accumulate, M, N, (unsigned)tm,
                           (unsigned)tn, p.slice_blocks);
        return;
      }
    }
    hipLaunchKernelGGL((k_fp8_gemm<TM, TN, E5, SPLIT>), grid, block, 0, stream, fp8_in(a),
                       fp8_in(b), (uint16_t *)out, out_dtype == QL_F16, M, N, (unsigned)tm,
                       (unsigned)tn, p.slice_blocks, part);
  };
  auto sized = [&](auto e5) {
    using Two = std::integral_constant<int, 2>;
    using Four = std::integral_constant<int, 4>;
    if (p.tm == 4) go(Four{}, Four{}, e5, std::false_type{});
    else if (p.tn == 4) go(Two{}, Four{}, e5, std::false_type{});
    else if (p.slices == 1) go(Two{}, Two{}, e5, std::false_type{});
    else go(Two{}, Two{}, e5, std::true_type{});
  };
  if (a->format == QL_E5M2) sized(std::true_type{});
  else sized(std::false_type{});
  QL_HIP_CHECK_LAUNCH();
  if (p.slices > 1) {
    const dim3 grid((unsigned)((M * ((N + 3) / 4) + 255) / 256)), block(256);
    if (out_dtype == QL_F32)
      hipLaunchKernelGGL((k_fp8_sum<float>), grid, block, 0, stream, part, p.slices, M, N,
                         (float *)out, false, accumulate);
    else
      hipLaunchKernelGGL((k_fp8_sum<uint16_t>), grid, block, 0, stream, part, p.slices, M, N,
                         (uint16_t *)out, out_dtype == QL_F16, false);
    QL_HIP_CHECK_LAUNCH();
  }
  return QL_OK;
}

}  // namespace qlora
