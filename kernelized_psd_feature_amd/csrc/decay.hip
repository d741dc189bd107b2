// Linear attention with one decay per head, gfx950: chunked form and recurrent form.
//
//   S_t = g S_{t-1} + k_t v_t^T,   o_t = scale q_t S_t,   g = exp(log_decay[h])
//
// Chunk of 64 tokens with entry state E (the state before it, decayed to its first token), tokens
// i, j = 0..63 of the chunk:
//   o_i = scale ( g^i q_i E + sum_{j<=i} g^(i-j) (q_i . k_j) v_j )
//   E  <- g^64 E + sum_j g^(64-j) k_j v_j^T
// so the three products are MFMA work and every power of g is a constant of the workgroup.
// A sequence is cut into segments of L chunks: a first pass sums each segment (but the last),
// decay_scan_kernel turns the sums into entry states (with few segments the walk adds them up
// itself), and the walk runs the chunks of each segment from its entry state.  With enough
// sequences, heads and value blocks a sequence is one segment and the walk runs alone.
//
// Bound.  State pass: HBM (k and v, which the walk reads again).  Walk: a chunk's chain of products, LDS
// exchanges and barriers more than memory.  A token takes as long at 8 x 4096, whether the operands
// are in the Infinity Cache (54 us) or not (59), as at 131072 (242); the waves stand ready and do not
// issue for 42% of their cycles, wait for memory, LDS or a barrier for 30%, and the MFMA units are
// busy for 13%.  The gradients likewise (their roles read 9 tensors where 4 are distinct, through the
// caches).  Measured by kernel over three sets of inputs in turn, 16 bf16 heads: 131072 tokens of
// width 64, state pass 101 to 110 us (5.1 TB/s), scan 8, walk 242 to 246 (4.4); 4 x 16384 of width 128,
// 145 to 149 (3.7), 9, 258 to 264 (4.1); 8 x 4096 of width 64, 28 and 59 (with the inputs in the
// cache 20 and 54), backward 178 to 182 (805 MB, 470 MB distinct); 32 x 2048, the walk alone, 118.
//
// Layout (four waves, or eight for value blocks of 128 columns; tiles are 16 x 16, K steps 32 wide;
// fragment conventions as in mfma_util.h).  Both operands of a product enumerate its K step in one
// order, of two: "straight" (slot r of lane group g is index 8 g + r) or "split" (slots 0..3 are
// 4 g + r, slots 4..7 are 16 + 4 g + r - 4, the order in which two accumulator tiles hold their rows).
//   - scores (straight over dk): wave w computes rows 16 (w % 4) .. of P (of eight waves each pair
//     halves the keys), transposed, K as the first operand, so that a lane ends with four
//     neighbouring keys of one row, weights them, and leaves them in LDS;
//   - the value columns are split over the waves, 16 each: a wave keeps the whole state of its
//     columns in registers, and the state's accumulators are the operand of the readout (split
//     over dk) without any exchange;
//   - products over keys are split: the transposing reads of V and K^T then take rows 0..7 of 16
//     at a time, which the row strides below spread over the banks;
//   - outputs are computed transposed (columns x rows), so a lane stores four neighbouring ones;
//     they are stored while the next chunk is staged, so that the wait for its loads does not
//     wait for stores just issued;
//   - a chunk is straight code: the chunk that may end early is a second copy of it, every wave
//     computes all its score tiles, masked ones too, and the state is read out and added to before
//     the wait for the other waves' weights, so the products' reads overlap.
// fp32 problems run the same code with eight fp32 MFMAs (K = 4) for one K step.
#include <type_traits>

#include "decay.h"
#include "decay_slots.h"
#include "device.h"
#include "mfma_util.h"
#include "tiles.h"

namespace kata {
namespace {

constexpr int kThreads = 256;             // of the scan and decode kernels

// ---- powers of the decay -----------------------------------------------------------------
// A decay of zero (log -inf) is taken as exp(-1e30): g^0 = 1 and every other power 0, where
// 0 * -inf would be nan.
__device__ __forceinline__ double log2_decay(float log_decay) {
  return (log_decay < -1e30f ? -1e30 : (double)log_decay) * 1.4426950408889634;
}
// g^n, the exponent held in 64 bits: its fp32 rounding would cost |n log2 g| 2^-24.
__device__ __forceinline__ float decay_power(double lg, int n) {
  const double x = lg * n;
  const float hi = (float)x;
  return exp2f(hi) * (1.f + 0.69314718f * (float)(x - hi));
}

// ---- segments ------------------------------------------------------------------------------
// Batch form: slot = sequence * n_seg + segment.  Packed form: decay_slots.h; the rows behind the
// last sequence are the segments of one more.  Offsets are clamped to [0, T], so that no content
// of cu reaches outside the tensors or the slots.
struct Segment {
  int seq, b, start, len, seg;
};

__device__ __forceinline__ int cu_at(const DecayArgs& A, int i) {
  return min(max(A.cu[i], 0), A.T);
}

// False where the slot holds no segment; sh: one int of LDS.  Every thread calls it.
__device__ __forceinline__ bool find_segment(const DecayArgs& A, int slot, int* sh, Segment& s) {
  if (!A.packed) {
    s = Segment{slot / A.n_seg, slot / A.n_seg, 0, A.T, slot % A.n_seg};
    return true;
  }
  const int SL = kC * A.L;
  if (threadIdx.x == 0) *sh = -1;
  __syncthreads();
  for (int i = threadIdx.x; i <= A.n_seq; i += blockDim.x) {
    const int lo = decay_first_slot(cu_at(A, i), i, SL);
    const int hi = i < A.n_seq ? decay_first_slot(cu_at(A, i + 1), i + 1, SL) : A.n_slots;
    if (lo <= slot && slot < hi) *sh = i;
  }
  __syncthreads();
  const int i = *sh;
  if (i < 0) return false;
  const int first = cu_at(A, i), end = i < A.n_seq ? cu_at(A, i + 1) : A.T;
  s = Segment{i, 0, first, max(end - first, 0), slot - decay_first_slot(first, i, SL)};
  return true;
}

// Row strides of the LDS tiles, in elements.  bf16 (64 banks of 4 bytes, s the stride in words): a
// read of one 16-byte vector of 16 rows is free of conflicts for s = 4 odd mod 64, the transposing
// reads of 16 bytes of 8 rows for s = 8 odd.  K is read both ways.  At 64 columns s = 36, for the
// former: conflicts are 31% of the LDS cycles of the state pass, which reads K transposed only, and
// 42% of the walk's.  At 128, where the padding to 36 mod 64 would not fit, s = 72, for the more
// frequent transposed reads: none in the state pass, 34% in the walk.
template <typename T, int DK, int W>
struct Tiles {
  static constexpr bool kBf = sizeof(T) == 2;
  static constexpr int DV = 16 * W;                 // value columns of a block
  static constexpr int LQ = DK + 16 / sizeof(T), LK = kBf && DK == 128 ? DK + 16 : LQ;
  static constexpr int LV = DV + (kBf ? 16 : 4), LP = kC + 16 / sizeof(T);
  // Two buffers of the operands' tiles where eight waves a CU still fit: the next chunk is staged
  // while this one is computed, for one barrier and one exposed LDS write less a chunk.
  static constexpr int kBuffers = kBf && (DK <= 64 || W == 8) ? 2 : 1;
  static constexpr int stage(bool state_pass) { return kC * (LK + LV + (state_pass ? 0 : LQ)); }
  static constexpr int kHead = 288;                 // an int, then the powers g^0 .. g^64
  // Terms of a score weight.  The rounding of one weight moves a whole row of outputs alike, and a row
  // with few weights does not average that out.  A row's rms error over its own rounding, by the weights
  // that it has in effect, n = sum g^2(t-s) <= 1 / (1 - g^2) (64 columns, computed in 64 bits with the
  // operands rounded): 1.4 in the mean whatever n is, but in one row of 100
  //     n = 1: 2.6   1.6: 2.5   2.5: 2.2   4 to 17: 2.0 to 2.2   above 100: 1.9
  // A second term, of what the rounding left, makes it 1.0 in the first chunk; behind it the entry
  // state's rounding joins: 1.0 below n = 4, 1.2 at 34, 1.35 above 100, where it hardly helps any more.
  // So two terms for the first rows of a sequence, which costs nothing measurable, and for all rows of
  // a head of n < 4, g^2 < 3/4; one such head of 16 costs the walk 3% (8 x 4096 forward and backward:
  // 265 us, 272; 4 x 4096 of width 128: 272, 282), since all wait for its workgroups.
  static constexpr int kTerms = kBf ? 2 : 1, kFineRows = 512;
  static constexpr float kFineDecay = -0.1438f;         // log(3/4) / 2
  static constexpr int bytes(bool state_pass) {
    return kHead + (kBuffers * stage(state_pass) + (state_pass ? 0 : kTerms * kC * LP)) * (int)sizeof(T);
  }
  // waves a SIMD that the registers are held to (the launch bound counts workgroups a CU)
  static constexpr int occupancy(bool state_pass) {
    return (!kBf ? (DK == 128 ? 1 : 2) : !state_pass ? 2 : W == 8 ? 4 : DK == 128 ? 3 : 4) * 4 / W;
  }
};

// Value weights of the state's update, x = w v, as SPLIT bf16 terms that add up to it: two (2^-17 of
// x: one rounded term puts the outputs 1.7 times as far off the exact ones as their own
// rounding), or three, the whole fp32 product, for a state that the caller keeps; fp32 as it is.
// An infinity among the values makes the later terms, and the state's entries, nan.
template <int SPLIT>
__device__ __forceinline__ void weigh(const bf16x8& v, const float (&w)[8], bf16x8 (&out)[SPLIT]) {
  const uint4 u = __builtin_bit_cast(uint4, v);
  const uint32_t in[4] = {u.x, u.y, u.z, u.w};
  uint32_t o[SPLIT][4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    float x = w[2 * r] * bf_lo(in[r]), y = w[2 * r + 1] * bf_hi(in[r]);
#pragma unroll
    for (int k = 0; k < SPLIT; ++k) {
      o[k][r] = pack_bf16x2(x, y);
      x -= bf_lo(o[k][r]);
      y -= bf_hi(o[k][r]);
    }
  }
#pragma unroll
  for (int k = 0; k < SPLIT; ++k)
    out[k] = __builtin_bit_cast(bf16x8, uint4{o[k][0], o[k][1], o[k][2], o[k][3]});
}
template <int SPLIT>
__device__ __forceinline__ void weigh(const f32x8& v, const float (&w)[8], f32x8 (&out)[SPLIT]) {
#pragma unroll
  for (int r = 0; r < 8; ++r) out[0][r] = w[r] * v[r];
}

template <typename T, int DK, int W, int SPLIT, bool kStatePass>
__global__ __launch_bounds__(64 * W, (Tiles<T, DK, W>::occupancy(kStatePass))) void decay_chunks_kernel(
    DecayArgs A) {
  using TL = Tiles<T, DK, W>;
  constexpr int kThr = 64 * W;
  using frag = typename Elem<T>::frag;
  constexpr int DV = TL::DV, M = DK / 32, NS = DK / 16, LQ = TL::LQ, LK = TL::LK, LV = TL::LV, LP = TL::LP;
  extern __shared__ __align__(16) char lds[];
  int* const sh = reinterpret_cast<int*>(lds);
  float* const pw = reinterpret_cast<float*>(lds) + 4;
  constexpr bool kTwo = TL::kBuffers == 2;
  constexpr int kStage = TL::stage(kStatePass);
  T* const sP = reinterpret_cast<T*>(lds + TL::kHead);             // walk only
  T* sK = sP + (kStatePass ? 0 : TL::kTerms * kC * LP);
  T* sV = sK + kC * LK;
  T* sQ = sV + kC * LV;                             // walk only
  int other = kStage;                               // from this chunk's tiles to the next one's

  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, l16 = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  // The value blocks and roles of one (slot, head) read the same rows, and its other segments write
  // the sums that it adds up: their workgroups get ids congruent mod 8, one XCD.  Over the sequences
  // the heads go round: with 16 heads an XCD would otherwise have two of them all along, whose rows
  // lie 2 KB apart and meet few of its L2's channels (8 x 4096 backward: 173 us for 185, 4 x 16384
  // walk: 113 for 121; round over the segments too: 173 and 124, and 2048 tokens 22.3 for 19.7).
  const unsigned x = block_number(), per = A.blocks, y = x / 8 / per, unit = 8 * y + x % 8;
  int sub = int(x / 8 - y * per), role = 0;
  if (unit >= (unsigned)A.n_slots * (unsigned)A.H) return;
  const int slot = int(unit / (unsigned)A.H);
  const unsigned turn = A.packed ? 0u : (unsigned)slot / (unsigned)A.n_seg;
  const int h = int((unit - (unsigned)slot * (unsigned)A.H + turn) % (unsigned)A.H);
  // The roles' blocks one after the other, none without columns: a workgroup that only leaves still
  // takes its turn in the order in which they are dealt out (2 x 1001 fp32, 3 heads of 72 and 40:
  // backward 68 us with one such of six).
  if (A.n_roles > 1) {
    const int n0 = (A.role[0].dv + DV - 1) / DV, n1 = n0 + (A.role[1].dv + DV - 1) / DV;
    role = (sub >= n0) + (sub >= n1);
    sub -= sub >= n1 ? n1 : sub >= n0 ? n0 : 0;
  }
  const DecayRole& R = A.role[role];
  const int c0 = sub * DV;                          // first value column

  Segment s;
  if (!find_segment(A, slot, sh, s)) return;
  const int L = A.L;
  T* const out = reinterpret_cast<T*>(R.out) + s.b * R.so[0] + h * R.so[2] + c0;
  const int per_row = min(DV, R.dv - c0) / 4;
  auto clear = [&](int from, int rows) {            // the block's columns of `rows` output rows
    for (long long i = tid; i < (long long)rows * per_row; i += kThr)
      store4(out + (from + i / per_row) * R.so[1] + i % per_row * 4, zero4());
  };
  if (s.seq == A.n_seq) {                           // rows behind the last sequence
    if (!kStatePass && A.zero_tail) clear(s.start + kC * L * s.seg, min(kC * L, s.len - kC * L * s.seg));
    return;
  }
  if (!kStatePass && A.packed && A.zero_tail && s.seq == 0 && s.seg == 0) clear(0, s.start);   // before the first
  const int n_chunks = (s.len + kC - 1) / kC, n_seg = (n_chunks + L - 1) / L;
  const long long SE = (long long)R.dk * R.dv, st_off = ((long long)s.seq * A.H + h) * SE;
  const int rs = R.init_trans ? 1 : R.dv, cs = R.init_trans ? R.dk : 1;   // strides of init
  if (s.seg >= n_seg) {
    if (!kStatePass && (!A.scan || A.join) && s.len == 0 && s.seg == 0 && R.fin)          // an empty sequence
      for (int i = tid; i < R.dk * DV; i += kThr) {
        const int r = i / DV, c = c0 + i % DV;
        if (c < R.dv)
          R.fin[st_off + (long long)r * R.dv + c] =
              R.init ? R.init[st_off + (long long)r * rs + (long long)c * cs] : 0.f;
      }
    return;
  }
  const bool last_seg = s.seg == n_seg - 1;
  if (kStatePass && last_seg && !R.fin) return;     // enters no entry state
  const int first = s.seg * L, behind = min(first + L, n_chunks);
  const int fine_before = A.log_decay[h] < TL::kFineDecay ? n_chunks : TL::kFineRows / kC;   // chunks

  // rows in the role's time order: row i of the sequence is start + i, or its mirror image
  const int dir = R.rev ? -1 : 1, dk = R.dk, dv = R.dv;
  const long long t0 = (R.rev ? s.start + s.len - 1 : s.start) + (long long)dir * kC * first;
  const long long sta = dir * R.sa[1], stb = dir * R.sb[1], stc = dir * R.sc[1], sto = dir * R.so[1];
  Stage<T, DK, kThr> ra(reinterpret_cast<const T*>(R.a) + s.b * R.sa[0] + t0 * R.sa[1] + h * R.sa[2], sta, dk, true);
  Stage<T, DK, kThr> rb(reinterpret_cast<const T*>(R.b) + s.b * R.sb[0] + t0 * R.sb[1] + h * R.sb[2], stb, dk, false);
  Stage<T, DV, kThr> rc(reinterpret_cast<const T*>(R.c) + s.b * R.sc[0] + t0 * R.sc[1] + h * R.sc[2] + c0, stc, dv - c0, false);
  const int wc = 16 * w;                            // the wave's columns in the block
  const bool live_col = c0 + wc + 4 * g < dv;
  T* po = out + (t0 + (long long)dir * l16) * R.so[1] + wc + 4 * g;   // the lane's first output

  auto fetch = [&](int n) {
    if (n < kC) {                                   // uniform
      if constexpr (!kStatePass) ra.fetch(sta, n);
      rb.fetch(stb, n);
      rc.fetch(stc, n);
    } else if (A.stream) {
      // (the empty asm keeps the compiler from joining the two branches' loads, as plain ones)
      asm volatile("" ::: "memory");
      if constexpr (!kStatePass) ra.template fetch<true>(sta);
      rb.template fetch<true>(stb);
      rc.template fetch<true>(stc);
      asm volatile("" ::: "memory");
    } else {
      if constexpr (!kStatePass) ra.template fetch<false>(sta);
      rb.template fetch<false>(stb);
      rc.template fetch<false>(stc);
    }
  };
  const int n_last = min(kC, s.len - kC * (behind - 1));   // rows of the segment's last chunk
  fetch(behind - first > 1 ? kC : n_last);

  // state tiles: S[i] lane holds rows 16 i + 4 g + r of column wc + l16
  f32x4 S[NS];
  // The scan has left every entry state in its slot, and may have put the final state of a sequence of one
  // segment where its initial one was.
  const bool from_scan = A.scan && !A.join && (n_seg > 1 || (R.init && R.fin));
  const bool has_state = !kStatePass && (from_scan || R.init);
  {
    const float* src = from_scan ? R.states + ((long long)slot * A.H + h) * SE : R.init + st_off;
    const int r1 = from_scan ? dv : rs, q1 = from_scan ? 1 : cs, col = c0 + wc + l16;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      S[i] = zero4();
      const int row = 16 * i + 4 * g;
      if (has_state && col < dv)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (row + r < dk) S[i][r] = src[(long long)(row + r) * r1 + (long long)col * q1];
    }
  }
  // (after the loads above are on their way)
  if (dk < DK || dv - c0 < DV) {                    // columns that no operand has: zeros all along
    uint4* const z = reinterpret_cast<uint4*>(sK);
    for (int i = tid; i < TL::kBuffers * kStage * (int)sizeof(T) / 16; i += kThr) z[i] = uint4{0u, 0u, 0u, 0u};
  }
  if (tid <= kC) pw[tid] = decay_power(log2_decay(A.log_decay[h]), tid);
  __syncthreads();
  if (has_state && !from_scan && !R.rev)            // a given state is decayed to the first token
#pragma unroll
    for (int i = 0; i < NS; ++i) S[i] *= pw[1];
  if constexpr (!kStatePass)
    if (A.join && dv > c0 + wc) {
      // The entry state from the sums of the segments before, as the scan adds them; with the own sum
      // it becomes the final state.
      constexpr int JB = NS > 4 ? 2 : 4;            // sums in flight
      const double lg = log2_decay(A.log_decay[h]);
      const float f = decay_power(lg, kC * L);
      const float f_last = decay_power(lg, s.len - (n_seg - 1) * kC * L - (R.rev ? 0 : 1));
      const int sums = s.seg + (last_seg && R.fin ? 1 : 0), col = c0 + wc + l16;
      const bool live = col < dv;
      const float* src = R.states + ((long long)(slot - s.seg) * A.H + h) * SE + 4 * g * dv + (live ? col : 0);
      for (int j = 0; j < sums; j += JB) {
        f32x4 u[JB][NS];
#pragma unroll
        for (int b = 0; b < JB; ++b) {
          const float* at = src + (long long)min(j + b, sums - 1) * A.H * SE;
#pragma unroll
          for (int i = 0; i < NS; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) u[b][i][r] = 16 * i + 4 * g + r < dk ? at[(16 * i + r) * dv] : 0.f;
        }
#pragma unroll
        for (int b = 0; b < JB; ++b) {
          if (j + b < s.seg) {
#pragma unroll
            for (int i = 0; i < NS; ++i)
#pragma unroll
              for (int r = 0; r < 4; ++r) S[i][r] = fmaf(f, S[i][r], u[b][i][r]);
          } else if (j + b < sums && live) {
            float* dst = R.fin + st_off + 4 * g * dv + col;
#pragma unroll
            for (int i = 0; i < NS; ++i)
#pragma unroll
              for (int r = 0; r < 4; ++r)
                if (16 * i + 4 * g + r < dk) dst[(16 * i + r) * dv] = fmaf(f_last, S[i][r], u[b][i][r]);
          }
        }
      }
    }

  // scores: the wave's row tile, and its J key tiles from j0 on
  constexpr int J = 16 / W;
  const int rt = w & 3, j0 = J * (w >> 2);
  // powers: dec[j][r] of (row, key) = (16 rt + l16, 16 (j0 + j) + 4 g + r), row0 of row l16 (the other
  // readout rows are steps of g^16 from it), vw[m][r] of the key in slot r of the m-th 32
  const float g16 = pw[16];
  float dec[J][4], row0 = 0.f, vw[2][8];
  if constexpr (!kStatePass) {
    row0 = pw[l16] * R.out_scale;
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        dec[j][r] = pw[max(16 * (rt - j0 - j) + l16 - 4 * g - r, 0)] * (R.out_scale * R.kv_scale);
  }
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int r = 0; r < 8; ++r) vw[m][r] = pw[kC - 32 * m - 16 * (r / 4) - 4 * g - r % 4] * R.kv_scale;
  float whole = pw[kC];

  Quad<T> O[4];                                     // outputs of the last chunk
  auto store = [&](int rows) {
    if (live_col)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (16 * i + l16 < rows) *reinterpret_cast<Quad<T>*>(po + 16 * i * sto) = O[i];
    po += kC * sto;
  };

  auto stage = [&](int to) {
    rb.template put<LK>(sK + to);
    rc.template put<LV>(sV + to);
    if constexpr (!kStatePass) ra.template put_split<LQ>(sQ + to);
  };
  if constexpr (kTwo) {
    stage(0);
    if (behind - first > 1) fetch(behind - first > 2 ? kC : n_last);
  }

  // one chunk, its rows on their way (or, with two buffers, staged and the next one's on their
  // way); kLast: the segment's last one, n_last rows
  auto chunk = [&](int c, auto last) {
    constexpr bool kLast = decltype(last)::value;
    const bool fine = c < fine_before;              // uniform
    // rows of the chunk after the next one to be staged
    const int n_next = c + (kTwo ? 3 : 2) < behind ? kC : n_last;
    __syncthreads();                                // the last chunk's tiles have been read
    if constexpr (!kTwo) {
      stage(0);
      if constexpr (!kStatePass)
        if (c > first) store(kC);
      if constexpr (kStatePass && !kLast) fetch(n_next);
      __syncthreads();
    } else if constexpr (!kStatePass) {
      if (c > first) store(kC);
    }

    f32x4 o[4];
    if constexpr (!kStatePass) {
      // Reads are issued in batches, ahead of the work that hides them (reads_above): left alone, the
      // compiler waits for nearly every read before its product, 4400 cycles a chunk for one
      // workgroup a CU.
      frag qf[M], kr[M][J], qr[4];
      f32x4 p[J];
#pragma unroll
      for (int m = 0; m < M; ++m) {
        qf[m] = straight_frag(sQ + (16 * rt + l16) * LQ + 32 * m, g);
#pragma unroll
        for (int j = 0; j < J; ++j) kr[m][j] = row_frag(sK + (16 * (j0 + j) + l16) * LK + 32 * m + 8 * g);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) qr[i] = row_frag(sQ + (16 * i + l16) * LQ + 8 * g);
      reads_above<T>();
#pragma unroll
      for (int j = 0; j < J; ++j) p[j] = zero4();
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int j = 0; j < J; ++j) p[j] = mma(kr[m][j], qf[m], p[j]);
      // readout of the entry state (bf16: rounded as an operand, the sum itself stays fp32)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = zero4();
#pragma unroll
      for (int m = 0; m < M; ++m) {
        frag next[4];
        if (m + 1 < M)
#pragma unroll
          for (int i = 0; i < 4; ++i) next[i] = row_frag(sQ + (16 * i + l16) * LQ + 32 * (m + 1) + 8 * g);
        reads_above<T>();
        if (m == 0) {
          // weights, zero by selection where the key is later (bf16: rounded, an operand; fine: and
          // what that left, as a second one)
#pragma unroll
          for (int j = 0; j < J; ++j) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
              p[j][r] = 16 * (j0 + j) + 4 * g + r > 16 * rt + l16 ? 0.f : p[j][r] * dec[j][r];
            T* const at = sP + (16 * rt + l16) * LP + split_place(16 * (j0 + j) + 4 * g);
            const Quad<T> hi = quad(p[j], T());
            *reinterpret_cast<Quad<T>*>(at) = hi;
            if constexpr (TL::kTerms == 2)
              if (fine) store4(at + kC * LP, p[j] - unquad(hi));
          }
        }
        const frag sf = pack_frag(S[2 * m], S[2 * m + 1], T());
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = mma(sf, qr[i], o[i]);
        if (m + 1 < M)
#pragma unroll
          for (int i = 0; i < 4; ++i) qr[i] = next[i];
      }
    }
    frag vf[2], kf[NS];                             // the wave's values, 32 keys each; K^T of 32 keys
#pragma unroll
    for (int m = 0; m < 2; ++m) vf[m] = column_frag<LV>(sV + 32 * m * LV + wc, lane);
#pragma unroll
    for (int i = 0; i < NS; ++i) kf[i] = column_frag<LK>(sK + 16 * i, lane);
    reads_above<T>();
    if constexpr (!kStatePass) {
      float f = row0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        o[i] *= f;
        f *= g16;
      }
    }

    if constexpr (kTwo && !kLast) {                 // the next chunk into the other buffer
      stage(other);
      if (c + 2 < behind) fetch(n_next);
    }

    if (kLast && last_seg) {
      // The state behind the last token, n_last - 1 (reversed: its product with g, the gradient of
      // the initial state).  Keys behind it are zero rows.
      const int e = n_last - (R.rev ? 0 : 1);
      whole = pw[e];
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int r = 0; r < 8; ++r)
          vw[m][r] = pw[max(e - 32 * m - 16 * (r / 4) - 4 * g - r % 4, 0)] * R.kv_scale;
    }
#pragma unroll
    for (int i = 0; i < NS; ++i) S[i] *= whole;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      frag vx[SPLIT], next[NS];
      if (m == 0)
#pragma unroll
        for (int i = 0; i < NS; ++i) next[i] = column_frag<LK>(sK + 32 * LK + 16 * i, lane);
      reads_above<T>();
      weigh<SPLIT>(vf[m], vw[m], vx);
#pragma unroll
      for (int k = 0; k < SPLIT; ++k)
#pragma unroll
        for (int i = 0; i < NS; ++i) S[i] = mma(kf[i], vx[k], S[i]);
      if (m == 0)
#pragma unroll
        for (int i = 0; i < NS; ++i) kf[i] = next[i];
    }

    if constexpr (!kStatePass) {
      const float sick = poison(vf[1], poison(vf[0], 0.f));
      // The loads are issued late: early ones, a whole chunk ahead of their use, measured slower
      // (131k tokens: 276 us for 252), as many in flight as there are then cost more than they hide.
      if constexpr (!kLast && !kTwo) fetch(n_next);
      const bool bad = __any(sick != sick);
      __syncthreads();                              // the weights are there
      auto weighted = [&](const T* sp) {              // o += weights at sp x values
        frag pf[2][4];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int i = 2 * m; i < 4; ++i) pf[m][i] = row_frag(sp + (16 * i + l16) * LP + 32 * m + 8 * g);
        reads_above<T>();
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int i = 2 * m; i < 4; ++i) o[i] = mma(vf[m], pf[m][i], o[i]);
      };
      if (!bad) {
        weighted(sP);
        if (TL::kTerms == 2 && fine) weighted(sP + kC * LP);
      } else {
        // An infinity or nan among the values: in the product above a masked weight of zero
        // would still meet it and leave nan in earlier rows, so the pairs are added one by one.
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll 1
          for (int key = 0; key < 16 * i + 16; ++key) {
            if (key > 16 * i + l16) continue;
            const int at = (16 * i + l16) * LP + split_place(key);
            float p = to_f32(sP[at]);
            if (TL::kTerms == 2 && fine) p += to_f32(sP[kC * LP + at]);
#pragma unroll
            for (int r = 0; r < 4; ++r) o[i][r] += p * to_f32(sV[key * LV + wc + 4 * g + r]);
          }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) O[i] = quad(o[i], T());
    }
    if constexpr (kTwo && !kLast) {
      sK += other;
      sV += other;
      sQ += other;
      other = -other;
    }
  };
  for (int c = first; c < behind - 1; ++c) chunk(c, std::false_type());
  chunk(behind - 1, std::true_type());
  if constexpr (!kStatePass) store(n_last);

  float* dst = kStatePass ? R.states + ((long long)slot * A.H + h) * SE
               : last_seg && R.fin && !A.scan ? R.fin + st_off : nullptr;
  const int col = c0 + wc + l16;
  if (!dst || col >= dv) return;
#pragma unroll
  for (int i = 0; i < NS; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (16 * i + 4 * g + r < dk) dst[(long long)(16 * i + 4 * g + r) * dv + col] = S[i][r];
}

// ---- scan ------------------------------------------------------------------------------------
// Per (sequence, head, role) and element, over the segments in order: the sum U_j of segment j is
// replaced by the entry state E_j, E_{j+1} = g^SL E_j + U_j; the last sum, over the n tokens that the
// segment has, completes the final state, g^(n-1) E + U (reversed: g^n E + U).  One thread has four
// neighbouring elements; the loads of 16 segments are in flight together.  Bound: the latency of
// those loads, from the cache that the state pass has just written: 32 segments of 16 heads of 64 x
// 64, 8.4 MB in and out, 7.4 us (9.3 with four loads in flight).
__global__ __launch_bounds__(kThreads) void decay_scan_kernel(DecayArgs A) {
  const int SE = A.role[0].dk * A.role[0].dv, nb = (SE / 4 + kThreads - 1) / kThreads;
  unsigned x = blockIdx.x;                         // sequences: blockIdx.y, at most 65535
  const int e4 = 4 * (int(x % (unsigned)nb) * kThreads + threadIdx.x);
  x /= (unsigned)nb;
  const int h = int(x % (unsigned)A.H);
  x /= (unsigned)A.H;
  const DecayRole& R = A.role[x];
  const int seq = blockIdx.y, SL = kC * A.L;
  int slot = seq * A.n_seg, len = A.T;
  if (A.packed) {
    const int first = cu_at(A, seq);
    slot = decay_first_slot(first, seq, SL);
    len = max(cu_at(A, seq + 1) - first, 0);
  }
  const int n = (len + SL - 1) / SL;
  if ((n < 2 && !R.fin) || e4 >= SE) return;
  const double lg = log2_decay(A.log_decay[h]);
  const float f = decay_power(lg, SL);
  const long long st_off = ((long long)seq * A.H + h) * SE;
  float4 e = {0.f, 0.f, 0.f, 0.f};
  if (R.init) {
    const float f0 = R.rev || len == 0 ? 1.f : decay_power(lg, 1);
    float y[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int i = (e4 + r) / R.dv, j = (e4 + r) % R.dv;
      y[r] = f0 * R.init[st_off + (R.init_trans ? j * R.dk + i : e4 + r)];
    }
    e = float4{y[0], y[1], y[2], y[3]};
  }
  float* p = R.states + ((long long)slot * A.H + h) * SE + e4;
  const long long step = (long long)A.H * SE;
  const int sums = R.fin ? n : n - 1;
  constexpr int F = 16;                            // loads in flight
  for (int j = 0; j < n; j += F) {
    float4 u[F];
#pragma unroll
    for (int r = 0; r < F; ++r) {
      u[r] = float4{0.f, 0.f, 0.f, 0.f};
      if (j + r < sums) u[r] = *reinterpret_cast<const float4*>(p + (j + r) * step);
    }
#pragma unroll
    for (int r = 0; r < F; ++r) {
      if (j + r >= n) break;
      *reinterpret_cast<float4*>(p + (j + r) * step) = e;
      const float fj = j + r < n - 1 ? f : decay_power(lg, len - (n - 1) * SL - (R.rev ? 0 : 1));
      e.x = fmaf(fj, e.x, u[r].x); e.y = fmaf(fj, e.y, u[r].y);
      e.z = fmaf(fj, e.z, u[r].z); e.w = fmaf(fj, e.w, u[r].w);
    }
  }
  if (R.fin) *reinterpret_cast<float4*>(R.fin + st_off + e4) = e;
}

// ---- recurrent form ------------------------------------------------------------------------
// One workgroup per (column block, head, sequence) keeps its part of the state in registers over
// the call's tokens: thread (row group, lane group) has 4 neighbouring columns of the rows
// row group + RG i.  LC lanes share a row: 4 LC columns of a block.
// Bound: HBM, the state's one read and one write: 512 sequences of 16 heads of 64 x 64, 276 MB in 54
// us, 5.1 TB/s.  One sequence: 4.0 us on the card, 8 us with the launch and the binding.
struct DecodeArgs {
  int T, H, dk, dv;
  long long sq[3], sk[3], sv[3], so[3];
  float scale;
};

template <typename T>
__device__ __forceinline__ f32x4 load4(const T* p);
template <>
__device__ __forceinline__ f32x4 load4<float>(const float* p) {
  return *reinterpret_cast<const f32x4*>(p);
}
template <>
__device__ __forceinline__ f32x4 load4<__bf16>(const __bf16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return unquad(u);
}

template <typename T, int LC, int RI>
__global__ __launch_bounds__(kThreads) void decay_decode_kernel(
    DecodeArgs A, const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
    const float* __restrict__ log_decay, float* __restrict__ state, T* __restrict__ o) {
  constexpr int RG = kThreads / LC;
  __shared__ f32x4 part[4][LC];
  const int tid = threadIdx.x, rg = tid / LC, col = 4 * (blockIdx.x * LC + tid % LC);
  const int h = blockIdx.y, b = blockIdx.z, w = tid >> 6;
  const bool live = col < A.dv;
  float* st = state + ((long long)b * A.H + h) * A.dk * A.dv + col;
  f32x4 S[RI];
#pragma unroll
  for (int i = 0; i < RI; ++i) {
    const int row = rg + RG * i;
    S[i] = zero4();
    if (live && row < A.dk) S[i] = *reinterpret_cast<const f32x4*>(st + row * A.dv);
  }
  const float gamma = expf(log_decay[h]);
  for (int t = 0; t < A.T; ++t) {
    const T* qt = q + row_off(A.sq, b, t, h);
    const T* kt = k + row_off(A.sk, b, t, h);
    const f32x4 vt = live ? load4<T>(v + row_off(A.sv, b, t, h) + col) : zero4();
    f32x4 acc = zero4();
#pragma unroll
    for (int i = 0; i < RI; ++i) {
      const int row = rg + RG * i;
      if (row < A.dk) {
        const float kr = to_f32(kt[row]), qr = to_f32(qt[row]);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          S[i][r] = fmaf(kr, vt[r], gamma * S[i][r]);
          acc[r] = fmaf(qr, S[i][r], acc[r]);
        }
      }
    }
#pragma unroll
    for (int m = LC; m < 64; m <<= 1)
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[r] += __shfl_xor(acc[r], m);
    if ((tid & 63) < LC) part[w][tid % LC] = acc;
    __syncthreads();
    if (tid < LC && live) {
      f32x4 y = part[0][tid] + part[1][tid] + part[2][tid] + part[3][tid];
      y *= A.scale;
      store4(o + row_off(A.so, b, t, h) + col, y);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < RI; ++i) {
    const int row = rg + RG * i;
    if (live && row < A.dk) *reinterpret_cast<f32x4*>(st + row * A.dv) = S[i];
  }
}

template <typename T, int DK, int W, int SPLIT>
hipError_t launch_chunks_t(const DecayArgs& a, bool state_pass, hipStream_t st) {
  const long long units = (long long)a.n_slots * a.H;
  const long long blocks = (units + 7) / 8 * 8 * a.blocks;
  auto run = [&](auto kernel, int bytes) {
    hipError_t e = ensure_dynamic_lds(reinterpret_cast<const void*>(kernel), bytes);
    if (e != hipSuccess) return e;
    launch_kernel(kernel, grid_rows(blocks), 64 * W, bytes, st, a);
    return hipGetLastError();
  };
  using TL = Tiles<T, DK, W>;
  return state_pass ? run(decay_chunks_kernel<T, DK, W, SPLIT, true>, TL::bytes(true))
                    : run(decay_chunks_kernel<T, DK, W, SPLIT, false>, TL::bytes(false));
}

template <typename T, int W, int SPLIT>
hipError_t launch_chunks_d(const DecayArgs& a, int dk, bool state_pass, hipStream_t st) {
  if constexpr (W == 4)                             // eight waves stage rows of 64 columns at least
    if (dk <= 32) return launch_chunks_t<T, 32, W, SPLIT>(a, state_pass, st);
  if (dk <= 64) return launch_chunks_t<T, 64, W, SPLIT>(a, state_pass, st);
  if (dk <= 128) return launch_chunks_t<T, 128, W, SPLIT>(a, state_pass, st);
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_decay_chunks(DecayArgs& a, bool bf16, bool exact_state, bool state_pass,
                               hipStream_t st) {
  int dk = 0, dv = 0;
  for (int r = 0; r < a.n_roles; ++r) {
    dk = dk > a.role[r].dk ? dk : a.role[r].dk;
    dv = dv > a.role[r].dv ? dv : a.role[r].dv;
  }
  const int cols = decay_columns(bf16, dv);
  a.blocks = 0;
  for (int r = 0; r < a.n_roles; ++r) a.blocks += (a.role[r].dv + cols - 1) / cols;
  if (!bf16) return launch_chunks_d<float, 4, 1>(a, dk, state_pass, st);
  // a state that the caller keeps gets the exact terms, in the pass that computes it
  const bool exact = exact_state && state_pass == (a.scan != 0);
  if (cols == 128)
    return exact ? launch_chunks_d<__bf16, 8, 3>(a, dk, state_pass, st)
                 : launch_chunks_d<__bf16, 8, 2>(a, dk, state_pass, st);
  return exact ? launch_chunks_d<__bf16, 4, 3>(a, dk, state_pass, st)
               : launch_chunks_d<__bf16, 4, 2>(a, dk, state_pass, st);
}

hipError_t launch_decay_scan(const DecayArgs& a, hipStream_t st) {
  const int SE = a.role[0].dk * a.role[0].dv, nb = (SE / 4 + kThreads - 1) / kThreads;
  launch_kernel(decay_scan_kernel, dim3(nb * a.H * a.n_roles, a.n_seq), kThreads, 0, st, a);
  return hipGetLastError();
}

hipError_t launch_decay_decode(bool bf16, int B, int T, int H, int dk, int dv,
                               const long long sq[3], const long long sk[3],
                               const long long sv[3], const long long so[3], const void* q,
                               const void* k, const void* v, const float* log_decay,
                               float scale, float* state, void* o, hipStream_t st) {
  DecodeArgs a;
  a.T = T; a.H = H; a.dk = dk; a.dv = dv; a.scale = scale;
  for (int i = 0; i < 3; ++i) {
    a.sq[i] = sq[i]; a.sk[i] = sk[i]; a.sv[i] = sv[i]; a.so[i] = so[i];
  }
  constexpr int LC = 16, kMost = 65535;             // sequences that a grid axis holds
  auto run = [&](auto t, auto ri) {
    using T_ = decltype(t);
    hipError_t e = hipSuccess;
    for (long long b = 0; b < B && e == hipSuccess; b += kMost) {
      const dim3 grid((dv + 4 * LC - 1) / (4 * LC), H, (unsigned)(B - b < kMost ? B - b : kMost));
      launch_kernel(decay_decode_kernel<T_, LC, decltype(ri)::value>, grid, kThreads, 0, st, a,
                    (const T_*)q + b * sq[0], (const T_*)k + b * sk[0], (const T_*)v + b * sv[0], log_decay,
                    state + b * H * dk * dv, (T_*)o + b * so[0]);
      e = hipGetLastError();
    }
    return e;
  };
  auto rows = [&](auto t) {
    if (dk <= 32) return run(t, std::integral_constant<int, 2>());
    if (dk <= 64) return run(t, std::integral_constant<int, 4>());
    return run(t, std::integral_constant<int, 8>());
  };
  return bf16 ? rows(__bf16()) : rows(float());
}

}  // namespace kata
