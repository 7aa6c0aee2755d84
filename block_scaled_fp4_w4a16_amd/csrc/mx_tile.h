// The tiles of MXFP4 products on the scaled matrix instruction, shared by the kernels that run them: geometry, the loads of codes and
// scales into LDS, the operand reads and the matrix instructions of a stage. mx_gemm.hip describes how they play together.
#pragma once
#include "mx.h"
#include "mx_plan.h"

namespace mx {

constexpr int GM_STAGE_BLOCKS = 8, GM_ROW_BYTES = 128;

// A BM x BN tile by WM x WN waves with NBUF stages in LDS, 2 or 4 (a stage is loaded NBUF stages ahead). The scales of SG
// groups of two stages, 16 SG bytes per row, are loaded at once: with one group every lane of the load takes a line of its
// own, which keeps the address unit as long as four loads of codes; two groups where LDS has the room (NBUF 4).
template <int BM_, int BN_, int WM_, int WN_, int NBUF_, int SG_>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NBUF = NBUF_, SG = SG_;
  static constexpr int WAVES = WM * WN, THREADS = 64 * WAVES;
  static constexpr int TM = BM / 16 / WM, TN = BN / 16 / WN;  // 16-row tiles per wave
  static constexpr int ROWS = BM + BN;                        // rows of both operands, A's first
  static constexpr int CODES = ROWS * GM_ROW_BYTES;           // bytes per stage
  static constexpr int SCALES = ROWS * 16 * SG;               // bytes per SG groups
  static constexpr int SBUF = SG == 2 ? 2 : NBUF / 2;         // buffers of them
  static constexpr int RING = NBUF * CODES + SBUF * SCALES;
  static constexpr int STAGE = 16 * (TN * 32 + 16);           // per wave: 16 rows of 16-bit outputs on their way out
  static constexpr int LDS = RING + WAVES * STAGE;
  static constexpr int SLOTS = CODES / 16 / THREADS;          // 16-byte direct loads per thread and stage
  static constexpr int SSLOTS = (ROWS * SG + THREADS - 1) / THREADS;  // the same of the scales, per SG groups
  static constexpr int OPS = TM + TN;                         // operands of a chunk, B's first
  static constexpr int READ_ROWS = TM > 2 ? TM * 3 / 4 : 1;   // row tiles of a chunk during which the next one's are read
  // direct loads of a thread that may be on their way when a stage has to be there: those of the NBUF - 2 stages
  // behind the next one (with SG 1 half of them bring scales too)
  static constexpr int BEHIND = (NBUF - 2) * SLOTS + (SG == 2 ? 0 : (NBUF / 2 - 1) * SSLOTS);
  static_assert((SG == 1 || (SG == 2 && NBUF == 4)) && (NBUF == 2 || NBUF == 4) && BEHIND + SLOTS < 64 && BM % (8 * WAVES) == 0 && ROWS % 64 == 0 && (NBUF == 2 || ROWS * SG % THREADS == 0), "");
};

__device__ __forceinline__ int swizzle(int row) { return row & 7; }

// Every LDS read of this wave is done, and every direct load but the last N, and so are every wave's of the workgroup.
template <int N>
__device__ __forceinline__ void wait_and_meet() {
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
  asm volatile("s_barrier" ::: "memory");
}

struct Sources {
  __amdgpu_buffer_rsrc_t aq, as, bq, bs;
  int ldqa, ldqb, ldsa, ldsb;
};

// Direct load I of one stage's codes: instruction I of wave w brings rows 8 (WAVES I + w) .. + 7, eight lanes a row.
// `from` (128 times the stage) is part of the range-checked offset: past the operand's last byte nothing is read.
// NOTHING lies past every operand's last byte (an operand's tile has at most 2^30 bytes).
constexpr uint32_t NOTHING = 1u << 31;

template <class G, int I>
__device__ __forceinline__ void issue_codes_part(const Sources& src, uint8_t* buf, uint32_t from, int wave, int lane) {
  const int first = (G::WAVES * I + wave) * 8;
  const int row = first + (lane >> 3);
  const uint32_t at = from + ((lane & 7) ^ swizzle(row)) * 16;
  auto* to = (__attribute__((address_space(3))) void*)(buf + first * GM_ROW_BYTES);
  if constexpr (8 * G::WAVES * I < G::BM)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(src.aq, to, 16, (uint32_t)(row * src.ldqa) + at, 0, 0, 0);
  else
    __builtin_amdgcn_raw_ptr_buffer_load_lds(src.bq, to, 16, (uint32_t)((row - G::BM) * src.ldqb) + at, 0, 0, 0);
}

template <class G, int I0, int I1>
__device__ __forceinline__ void issue_codes(const Sources& src, uint8_t* buf, uint32_t from, int wave, int lane) {
  if constexpr (I0 < I1) {
    issue_codes_part<G, I0>(src, buf, from, wave, lane);
    issue_codes<G, I0 + 1, I1>(src, buf, from, wave, lane);
  }
}

// The direct loads of SG groups' scales (`from`: 16 times the first group): 64 / SG rows per instruction, dealt to the waves.
// With two groups per row, their order is swapped in rows 8 .. 15 of 16, which keeps the reads of one group off each
// other's banks.
template <class G>
__device__ __forceinline__ void issue_scales(const Sources& src, uint8_t* buf, uint32_t from, int wave, int lane) {
#pragma unroll
  for (int i = 0; i < G::SSLOTS; ++i) {
    const int first = (G::WAVES * i + wave) * (64 / G::SG);
    if (G::ROWS * G::SG % G::THREADS && first >= G::ROWS) break;  // the last waves have none (NBUF 2: no wait counts them)
    const int row = first + lane / G::SG;
    const uint32_t at = from + (G::SG == 2 ? ((lane ^ row >> 3) & 1) * 16 : 0);
    auto* to = (__attribute__((address_space(3))) void*)(buf + first * 16 * G::SG);
    if (first < G::BM) __builtin_amdgcn_raw_ptr_buffer_load_lds(src.as, to, 16, (uint32_t)(row * src.ldsa) + at, 0, 0, 0);
    else __builtin_amdgcn_raw_ptr_buffer_load_lds(src.bs, to, 16, (uint32_t)((row - G::BM) * src.ldsb) + at, 0, 0, 0);
  }
}

// acc += A B^T with scale byte C of both scale registers, as mfma() but written out so that the sum stays in the
// accumulation registers that it came from: with the compiler's builtin, whose result is a new register, a tile of
// 256 sums per lane is copied and spilled in the loop. A vector instruction that writes an operand needs two wait
// states before the MFMA that reads it, which the compiler does not see here: FIRST, the first MFMA behind a scheduling
// barrier, waits for them, and no operand of the MFMAs that follow it up to the next barrier is written in between.
template <int C, bool FIRST>
__device__ __forceinline__ void mfma_acc(f32x4& acc, const u32x4& a, uint32_t sa, const u32x4& b, uint32_t sb) {
#define MX_MFMA_(WAIT, SEL)                                                                              \
  asm volatile(WAIT "v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 " SEL " cbsz:4 blgp:4"     \
               : "+a"(acc)                                                                               \
               : "v"(a), "v"(b), "v"(sa), "v"(sb))
#define MX_MFMA(SEL)                                 \
  if constexpr (FIRST) MX_MFMA_("s_nop 1\n\t", SEL); \
  else MX_MFMA_("", SEL)
  if constexpr (C == 0) { MX_MFMA("op_sel:[0,0,0] op_sel_hi:[0,0,0]"); }
  else if constexpr (C == 1) { MX_MFMA("op_sel:[1,1,0] op_sel_hi:[0,0,0]"); }
  else if constexpr (C == 2) { MX_MFMA("op_sel:[0,0,0] op_sel_hi:[1,1,0]"); }
  else { MX_MFMA("op_sel:[1,1,0] op_sel_hi:[1,1,0]"); }
#undef MX_MFMA
#undef MX_MFMA_
}

// Sum number I from the end.
template <class G, int I>
__device__ __forceinline__ f32x4& sum_from_end(f32x4 (&acc)[G::TM][G::TN]) {
  constexpr int at = G::TM * G::TN - 1 - I;
  return acc[at / G::TN][at % G::TN];
}
template <class G>
__device__ __forceinline__ void wait_for_sums(f32x4 (&acc)[G::TM][G::TN]) {
#define MX_SUM(I) "+a"(sum_from_end<G, I>(acc))
  if constexpr (G::TM * G::TN == 4)
    asm volatile("s_nop 15\n\ts_nop 1" : MX_SUM(0), MX_SUM(1), MX_SUM(2), MX_SUM(3));
  else
    asm volatile("s_nop 15\n\ts_nop 1"
                 : MX_SUM(0), MX_SUM(1), MX_SUM(2), MX_SUM(3), MX_SUM(4), MX_SUM(5), MX_SUM(6), MX_SUM(7));
#undef MX_SUM
}

// Four dwords of a row's scales (four chunks of four blocks) -> byte c is block g of chunk c.
__device__ __forceinline__ uint32_t pick_scales(const u32x4& w, int g) {
  const uint32_t sel = (uint32_t)g | (uint32_t)(4 + g) << 8;
  const uint32_t lo = __builtin_amdgcn_perm(w[1], w[0], sel);
  const uint32_t hi = __builtin_amdgcn_perm(w[3], w[2], sel);
  return __builtin_amdgcn_perm(hi, lo, 0x05040100u);
}

// Workgroup -> (tile row, tile column, part of K). Workgroups go round-robin over the 8 XCDs, each of which has its
// own L2: XCD x takes a contiguous run of the tiles, walked in columns of `BAND` tile rows so that the tiles in
// flight on one XCD share rows of both operands.
__device__ __forceinline__ void place(int id, int total, int tiles_m, int tiles_n, int& tm, int& tn, int& part) {
  const int xcds = 8, x = id % xcds, i = id / xcds;
  const int q = total / xcds, r = total % xcds;
  int t = x * q + min(x, r) + i;  // bijective for any total
  const int tiles = tiles_m * tiles_n;
  part = t / tiles;
  t -= part * tiles;
  constexpr int BAND = 4;
  const int per = BAND * tiles_n, band = t / per, in = t - band * per;
  const int h = min(BAND, tiles_m - band * BAND);
  tn = in / h;
  tm = band * BAND + in - tn * h;
}

// A wave's state.
template <class G>
struct Wave {
  f32x4 acc[G::TM][G::TN];
  u32x4 op[2][G::OPS];                  // operands (B's, then A's) of even and of odd chunks
  u32x4 raw[G::OPS];                    // scales as read: four dwords of a row
  uint32_t sc[2][G::OPS];               // scales of this and the next group: byte c is this lane's block of chunk c
  Sources src;
  uint8_t* lds;
  int wave, lane;
  uint32_t frag_a, frag_b;    // LDS offsets of this lane's block of chunk 0, row tile 0; ^ 64 leads to chunk 1
  uint32_t scale_a, scale_b;  // LDS offsets of this lane's row of scales, row tile 0
  int last_group;
  uint32_t tail;              // mask of the last group's scales

  // Stage st of group st / 2 is in buffer st % NBUF: with `ring` = group % (NBUF / 2), buffer 2 ring + st % 2.
  __device__ __forceinline__ uint8_t* codes(int ring, int half) const { return lds + (2 * ring + half) * G::CODES; }
  // The scales of a group are in buffer group / SG % SBUF.
  __device__ __forceinline__ uint8_t* scales(int group) const {
    return lds + G::NBUF * G::CODES + (G::SBUF == 1 ? 0 : group / G::SG % G::SBUF) * G::SCALES;
  }
  static __device__ __forceinline__ int ring_of(int group) { return G::NBUF == 2 ? 0 : group & (G::NBUF / 2 - 1); }
  __device__ __forceinline__ u32x4 read_codes(uint32_t at, int ring, int half, int chunk, int t) const {
    return *reinterpret_cast<const u32x4*>(codes(ring, half) + (chunk ? at ^ 64u : at) + t * 16 * GM_ROW_BYTES);
  }
  __device__ __forceinline__ u32x4 read_op(int ring, int half, int chunk, int i) const {
    return i < G::TN ? read_codes(frag_b, ring, half, chunk, i) : read_codes(frag_a, ring, half, chunk, i - G::TN);
  }
  __device__ __forceinline__ u32x4 read_raw(int group, int i) const {
    const uint32_t half = G::SG == 2 ? (group & 1) * 16 : 0;
    const uint32_t at = i < G::TN ? (scale_b ^ half) + 256 * G::SG * i : (scale_a ^ half) + 256 * G::SG * (i - G::TN);
    return *reinterpret_cast<const u32x4*>(scales(group) + at);
  }
  __device__ __forceinline__ uint32_t pick(int i, int group) const {
    return pick_scales(raw[i], lane >> 4) & (group == last_group ? tail : ~0u);
  }

  // What is done between the MFMAs of row tile I of chunk C: direct loads (second chunk of a stage), reads of the next
  // chunk's operands, reads of the next group's scales (the group's last chunk), in this order; operation X of them.
  template <int C, int I>
  struct Between {
    static constexpr bool reads = I < G::READ_ROWS;
    static constexpr int l0 = C & 1 ? G::SLOTS * I / G::TM : 0, l1 = C & 1 ? G::SLOTS * (I + 1) / G::TM : 0;
    static constexpr int r0 = reads ? G::OPS * I / G::READ_ROWS : 0, r1 = reads ? G::OPS * (I + 1) / G::READ_ROWS : 0;
    static constexpr int s0 = C == 3 ? r0 : 0, s1 = C == 3 ? r1 : 0;
    static constexpr int loads = l1 - l0, ops = r1 - r0, scales = s1 - s0, all = loads + ops + scales;
  };
  template <int C, int I, int X, int END>
  __device__ __forceinline__ void between(int group, int next, uint32_t codes_from) {
    if constexpr (X < END) {
      using B = Between<C, I>;
      if constexpr (X < B::loads) {
        issue_codes_part<G, B::l0 + X>(src, codes(ring_of(group), C >> 1), codes_from, wave, lane);
      } else if constexpr (X < B::loads + B::ops) {
        constexpr int i = B::r0 + X - B::loads, NC = (C + 1) & 1, NH = ((C + 1) >> 1) & 1;
        op[NC][i] = read_op(ring_of(C == 3 ? next : group), NH, NC, i);
      } else {
        constexpr int i = B::s0 + X - B::loads - B::ops;
        raw[i] = read_raw(next, i);
      }
      between<C, I, X + 1, END>(group, next, codes_from);
    }
  }

  // Chunk C of `group` (`next` is the group after it) from its MFMA (I, J) on, a share of the other work behind each.
  // A stage's second chunk ends the stage behind its first MFMA (every LDS read of the stage was issued in the chunk
  // before) and issues the loads of the stage NBUF behind it (from byte `codes_from` of the codes and `scales_from` of
  // the scales), whose buffer is free.
  template <int C, int I, int J>
  __device__ __forceinline__ void chunk(int group, int next, uint32_t codes_from, uint32_t scales_from) {
    if constexpr (I < G::TM) {
      mfma_acc<C, J == 0>(acc[I][J], op[C & 1][J], sc[0][J], op[C & 1][G::TN + I], sc[0][G::TN + I]);
      if constexpr ((C & 1) && I == 0 && J == 0) wait_and_meet<G::BEHIND>();
      using B = Between<C, I>;
      if constexpr (C == 3 && J == 0 && I > 0) {  // the scales read behind the row tile before
        using P = Between<C, I - 1>;
#pragma unroll
        for (int i = P::s0; i < P::s1; ++i) sc[1][i] = pick(i, next);
      }
      between<C, I, B::all * J / G::TN, B::all*(J + 1) / G::TN>(group, next, codes_from);
      if constexpr (C == 1 && I == G::TM - 1 && J == G::TN - 1) {  // two groups' scales with the even one
        if (G::SG == 1 || !(group & 1)) issue_scales<G>(src, scales(group + G::NBUF / 2), scales_from, wave, lane);
      }
      __builtin_amdgcn_sched_barrier(0);
      chunk<C, J + 1 < G::TN ? I : I + 1, J + 1 < G::TN ? J + 1 : 0>(group, next, codes_from, scales_from);
    }
  }
};

// ------------------------------------------------------------------------------------------------ host side

struct LinearSpace {
  int64_t q, s, planes;  // bytes, each a multiple of 256
};
static inline int64_t round256(int64_t b) { return (b + 255) / 256 * 256; }
static inline LinearSpace linear_space(const Plan& p, int64_t M, int64_t K) {
  const int64_t nb = blocks_of(K);
  return {round256(M * nb * 16), round256(M * ((nb + 3) / 4 * 4)), plane_bytes(p, M)};
}

}  // namespace mx
