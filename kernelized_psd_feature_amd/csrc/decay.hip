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
// decay_scan_kernel turns the sums into entry states, and the walk runs the chunks of each
// segment from its entry state.  With enough sequences, heads and value blocks a sequence is
// one segment and the walk runs alone.
//
// Layout (256 threads, four waves; tiles are 16 x 16, K steps 32 wide; fragment conventions as in
// mfma_util.h with K slot r of lane group g being index 8 g + r of the step):
//   - scores: wave w computes rows 16 w .. of P (transposed, K as the first operand, so that a
//     lane ends with four neighbouring keys of one row), weights them, and leaves them in LDS;
//   - the value columns are split over the waves, 16 NT each: a wave keeps the whole state of
//     its columns in registers, and the state's accumulators are the operand of the readout
//     without any exchange.  For that, row 4 g + b of state tile 2 m + a is dk index
//     32 m + 8 g + 4 a + b: slots 0..7 of lane group g are then indices 8 g .. 8 g + 7 of step m,
//     the order of a plain 16-byte read of a q row;
//   - outputs are computed transposed (columns x rows), so a lane stores four neighbouring ones.
// fp32 problems run the same code with eight fp32 MFMAs (K = 4) for one K step.
#include <type_traits>

#include "decay.h"
#include "decay_slots.h"
#include "device.h"
#include "mfma_util.h"

namespace kata {
namespace {

constexpr int kC = 64;                    // tokens of a chunk
constexpr int kThreads = 256;

typedef __attribute__((__vector_size__(8 * sizeof(float)))) float f32x8;

template <typename T>
struct Elem;
template <>
struct Elem<__bf16> {
  using frag = bf16x8;
  static constexpr int V = 8;             // elements of a 16-byte vector
};
template <>
struct Elem<float> {
  using frag = f32x8;
  static constexpr int V = 4;
};

__device__ __forceinline__ f32x4 mma(const bf16x8& a, const bf16x8& b, const f32x4& c) {
  return mfma32(a, b, c);
}
__device__ __forceinline__ f32x4 mma(const f32x8& a, const f32x8& b, f32x4 c) {
#pragma unroll
  for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
  return c;
}

// Slots 0..7 from eight neighbouring elements.
__device__ __forceinline__ bf16x8 row_frag(const __bf16* p) {
  return __builtin_bit_cast(bf16x8, ld16(p));
}
__device__ __forceinline__ f32x8 row_frag(const float* p) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
  return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

// Slots 0..7 from eight rows of one column: lane i of a 16-lane group g gets rows 8 g .. 8 g + 7
// of column cs (i / 4) + i % 4, p pointing at row 0 of column 0 (LD: elements of a row).
template <int LD, int CS>
__device__ __forceinline__ bf16x8 column_frag(const __bf16* p, int lane) {
  const int g = lane >> 4, j = lane & 15;
  const __bf16* at = p + (8 * g + (j >> 2)) * LD + CS * (j & 3);
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at));
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 4 * LD));
  const uint2 ul = __builtin_bit_cast(uint2, lo), uh = __builtin_bit_cast(uint2, hi);
  return __builtin_bit_cast(bf16x8, uint4{ul.x, ul.y, uh.x, uh.y});
}
template <int LD, int CS>
__device__ __forceinline__ f32x8 column_frag(const float* p, int lane) {
  const int g = lane >> 4, i = lane & 15;
  const float* at = p + 8 * g * LD + CS * (i >> 2) + (i & 3);
  f32x8 x;
#pragma unroll
  for (int r = 0; r < 8; ++r) x[r] = at[r * LD];
  return x;
}

__device__ __forceinline__ bf16x8 pack_frag(const f32x4& a, const f32x4& b, __bf16) {
  return __builtin_bit_cast(bf16x8, uint4{pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]),
                                          pack_bf16x2(b[0], b[1]), pack_bf16x2(b[2], b[3])});
}
__device__ __forceinline__ f32x8 pack_frag(const f32x4& a, const f32x4& b, float) {
  return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

__device__ __forceinline__ bool has_nonfinite(const bf16x8& x) {
  return nonfinite_bf16x8(__builtin_bit_cast(uint4, x)) != 0u;
}
__device__ __forceinline__ bool has_nonfinite(const f32x8& x) {
  bool bad = false;
#pragma unroll
  for (int r = 0; r < 8; ++r) bad |= !(fabsf(x[r]) < __builtin_inff());
  return bad;
}

__device__ __forceinline__ void store4(__bf16* p, const f32x4& x) {
  *reinterpret_cast<uint2*>(p) = uint2{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
}
__device__ __forceinline__ void store4(float* p, const f32x4& x) {
  *reinterpret_cast<f32x4*>(p) = x;
}

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

// ---- staging -------------------------------------------------------------------------------
// A chunk of one operand: 64 rows of W columns (those behind `width` and the rows behind n zero),
// W / (4 V) 16-byte vectors a thread.
template <typename T, int W>
struct Stage {
  static constexpr int V = Elem<T>::V, PER = W / V, N = kC * PER / kThreads;
  static_assert(N >= 1, "a vector a thread");
  uint4 x[N];
  // row 0 at p, rows st elements apart (negative in reversed time)
  __device__ __forceinline__ void load(const T* p, long long st, int n, int width) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int idx = threadIdx.x + kThreads * i, row = idx / PER, col = (idx % PER) * V;
      x[i] = uint4{0u, 0u, 0u, 0u};
      if (row < n && col < width) x[i] = *reinterpret_cast<const uint4*>(p + row * st + col);
    }
  }
  template <int LD>
  __device__ __forceinline__ void put(T* tile) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int idx = threadIdx.x + kThreads * i, row = idx / PER, col = (idx % PER) * V;
      *reinterpret_cast<uint4*>(tile + row * LD + col) = x[i];
    }
  }
};

template <typename T, int DK, int NT>
struct Tiles {
  static constexpr int V = Elem<T>::V;
  static constexpr int DV = 64 * NT;                // value columns of a block
  static constexpr int LK = DK + V, LV = DV + V, LP = kC + V;   // row strides: one vector of padding
  static constexpr int kState = kC * (LK + LV), kWalk = kState + kC * (LK + LP);
  static constexpr int kHead = 288;                 // an int, then the powers g^0 .. g^64
  static constexpr int bytes(bool state_pass) {
    return kHead + (state_pass ? kState : kWalk) * (int)sizeof(T);
  }
};

// Value weights of the state's update, x = w v, as SPLIT bf16 terms that add up to it: two (2^-17 of
// x: one rounded term puts the outputs 1.7 times as far off the exact ones as their own
// rounding), or three, the whole fp32 product, for a state that the caller keeps; fp32 as it is.
template <int SPLIT>
__device__ __forceinline__ void weigh(const bf16x8& v, const float (&w)[8], bf16x8 (&out)[SPLIT]) {
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    float x = w[r] * (float)v[r];
#pragma unroll
    for (int k = 0; k < SPLIT; ++k) {
      const __bf16 y = (__bf16)x;
      out[k][r] = y;
      x = fabsf((float)y) < __builtin_inff() ? x - (float)y : 0.f;   // inf and nan: once
    }
  }
}
template <int SPLIT>
__device__ __forceinline__ void weigh(const f32x8& v, const float (&w)[8], f32x8 (&out)[SPLIT]) {
#pragma unroll
  for (int r = 0; r < 8; ++r) out[0][r] = w[r] * v[r];
}

template <typename T, int DK, int NT, int SPLIT, bool kStatePass>
__global__ __launch_bounds__(kThreads) void decay_chunks_kernel(DecayArgs A) {
  using TL = Tiles<T, DK, NT>;
  using frag = typename Elem<T>::frag;
  constexpr int LK = TL::LK, LV = TL::LV, LP = TL::LP, DV = TL::DV, M = DK / 32, NS = DK / 16;
  extern __shared__ __align__(16) char lds[];
  int* const sh = reinterpret_cast<int*>(lds);
  float* const pw = reinterpret_cast<float*>(lds) + 4;
  T* const sK = reinterpret_cast<T*>(lds + TL::kHead);
  T* const sV = sK + kC * LK;
  T* const sQ = sV + kC * LV;                       // walk only
  T* const sP = sQ + kC * LK;

  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, g = lane >> 4, l16 = lane & 15;
  // The value blocks and roles of one (slot, head) read the same rows: their workgroups get ids
  // congruent mod 8, one XCD.
  const long long x = blockIdx.x;
  const int per = A.nvb * A.n_roles;
  const long long unit = x / (8LL * per) * 8 + x % 8;
  const int sub = int(x / 8 % per);
  if (unit >= (long long)A.n_slots * A.H) return;
  const int slot = int(unit / A.H), h = int(unit % A.H);
  const DecayRole& R = A.role[sub % A.n_roles];
  const int c0 = sub / A.n_roles * DV;              // first value column
  if (c0 >= R.dv) return;

  Segment s;
  if (!find_segment(A, slot, sh, s)) return;
  const int L = A.L;
  T* const out = reinterpret_cast<T*>(R.out) + s.b * R.so[0] + h * R.so[2] + c0;
  if (s.seq == A.n_seq) {                           // rows behind the last sequence
    if (kStatePass || !A.zero_tail) return;
    const int per_row = min(DV, R.dv - c0) / 4, r0 = kC * L * s.seg;
    const long long todo = (long long)min(kC * L, s.len - r0) * per_row;
    for (long long i = tid; i < todo; i += kThreads)
      store4(out + (s.start + r0 + i / per_row) * R.so[1] + i % per_row * 4, zero4());
    return;
  }
  const int n_chunks = (s.len + kC - 1) / kC, n_seg = (n_chunks + L - 1) / L;
  const long long SE = (long long)R.dk * R.dv, st_off = ((long long)s.seq * A.H + h) * SE;
  const int rs = R.init_trans ? 1 : R.dv, cs = R.init_trans ? R.dk : 1;   // strides of init
  if (s.seg >= n_seg) {
    if (!kStatePass && s.len == 0 && s.seg == 0 && R.fin)          // an empty sequence
      for (int i = tid; i < R.dk * DV; i += kThreads) {
        const int r = i / DV, c = c0 + i % DV;
        if (c < R.dv)
          R.fin[st_off + (long long)r * R.dv + c] =
              R.init ? R.init[st_off + (long long)r * rs + (long long)c * cs] : 0.f;
      }
    return;
  }
  const bool last_seg = s.seg == n_seg - 1;
  if (kStatePass && last_seg) return;
  const int first = s.seg * L, behind = min(first + L, n_chunks);

  if (tid <= kC) pw[tid] = decay_power(log2_decay(A.log_decay[h]), tid);
  __syncthreads();
  const int wc = 16 * NT * w;                       // the wave's columns in the block

  // rows in the role's time order: row i of the sequence is start + i, or its mirror image
  const int dir = R.rev ? -1 : 1, t0 = R.rev ? s.start + s.len - 1 : s.start;
  const long long sta = dir * R.sa[1], stb = dir * R.sb[1], stc = dir * R.sc[1], sto = dir * R.so[1];
  const T* const pa = reinterpret_cast<const T*>(R.a) + s.b * R.sa[0] + t0 * R.sa[1] + h * R.sa[2];
  const T* const pb = reinterpret_cast<const T*>(R.b) + s.b * R.sb[0] + t0 * R.sb[1] + h * R.sb[2];
  const T* const pc = reinterpret_cast<const T*>(R.c) + s.b * R.sc[0] + t0 * R.sc[1] + h * R.sc[2] + c0;
  T* const po = out + t0 * R.so[1];

  // state tiles: S[i][n] lane holds row 32 (i / 2) + 8 g + 4 (i % 2) + r, column wc + 16 n + l16
  f32x4 S[NS][NT];
  const bool from_scan = n_seg > 1;
  bool has_state = !kStatePass && (from_scan || R.init);
  {
    const float* src = from_scan ? R.states + ((long long)slot * A.H + h) * SE : R.init + st_off;
    const int r1 = from_scan ? R.dv : rs, q1 = from_scan ? 1 : cs;
    const float f = from_scan || R.rev ? 1.f : pw[1];
#pragma unroll
    for (int i = 0; i < NS; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        S[i][n] = zero4();
        const int row = 32 * (i / 2) + 8 * g + 4 * (i % 2), col = c0 + wc + 16 * n + l16;
        if (has_state && col < R.dv)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (row + r < R.dk) S[i][n][r] = f * src[(long long)(row + r) * r1 + (long long)col * q1];
      }
  }

  // powers: dec[j][r] of (row, key) = (16 w + l16, 16 j + 4 g + r), rowp[i] of row 16 i + l16,
  // vw[m][r] of key 32 m + 8 g + r
  float dec[4][4], rowp[4], vw[2][8];
  if constexpr (!kStatePass) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      rowp[j] = pw[16 * j + l16] * R.out_scale;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        dec[j][r] = pw[max(16 * (w - j) + l16 - 4 * g - r, 0)] * (R.out_scale * R.kv_scale);
    }
    // keys of the K step that no score tile of this wave covers
    if (!(w & 1)) store4(sP + (16 * w + l16) * LP + 16 * (w + 1) + 4 * g, zero4());
  }
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int r = 0; r < 8; ++r) vw[m][r] = pw[kC - 32 * m - 8 * g - r] * R.kv_scale;
  float whole = pw[kC];

  Stage<T, DK> ra, rb;
  Stage<T, DV> rc;
  auto fetch = [&](int c) {
    const int n = min(kC, s.len - kC * c);
    if constexpr (!kStatePass) ra.load(pa + (long long)kC * c * sta, sta, n, R.dk);
    rb.load(pb + (long long)kC * c * stb, stb, n, R.dk);
    rc.load(pc + (long long)kC * c * stc, stc, n, R.dv - c0);
  };
  fetch(first);
  for (int c = first; c < behind; ++c) {
    const int n = min(kC, s.len - kC * c);
    __syncthreads();                                // the last chunk's tiles have been read
    rb.template put<LK>(sK);
    rc.template put<LV>(sV);
    if constexpr (!kStatePass) ra.template put<LK>(sQ);
    if (c + 1 < behind) fetch(c + 1);
    __syncthreads();

    f32x4 O[4][NT];
    if constexpr (!kStatePass) {
      frag qf[M];
#pragma unroll
      for (int m = 0; m < M; ++m) qf[m] = row_frag(sQ + (16 * w + l16) * LK + 32 * m + 8 * g);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j > w) continue;                        // uniform in the wave
        f32x4 p = zero4();
#pragma unroll
        for (int m = 0; m < M; ++m)
          p = mma(row_frag(sK + (16 * j + l16) * LK + 32 * m + 8 * g), qf[m], p);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          p[r] *= dec[j][r];
          if (j == w && 4 * g + r > l16) p[r] = 0.f;   // select, never multiply
        }
        // bf16: the weights are an operand of the next product
        store4(sP + (16 * w + l16) * LP + 16 * j + 4 * g, p);
      }
      // readout of the entry state (bf16: rounded as an operand, the sum itself stays fp32)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) O[i][nt] = zero4();
      if (has_state) {
#pragma unroll
        for (int m = 0; m < M; ++m) {
          frag sf[NT];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) sf[nt] = pack_frag(S[2 * m][nt], S[2 * m + 1][nt], T());
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const frag qr = row_frag(sQ + (16 * i + l16) * LK + 32 * m + 8 * g);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) O[i][nt] = mma(sf[nt], qr, O[i][nt]);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) O[i][nt] *= rowp[i];
      }
      __syncthreads();                              // the weights are there
    }

    const bool ends = last_seg && c + 1 == behind;
    const bool update = kStatePass || c + 1 < behind || (ends && R.fin);
    if (ends && update) {
      // the state behind token n - 1 (reversed: its product with g, the gradient of the initial
      // state); keys behind n are zero rows
      const int e = n - (R.rev ? 0 : 1);
      whole = pw[e];
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int r = 0; r < 8; ++r)
          vw[m][r] = pw[max(e - 32 * m - 8 * g - r, 0)] * R.kv_scale;
    }
    if (update)
#pragma unroll
      for (int i = 0; i < NS; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) S[i][nt] *= whole;

#pragma unroll
    for (int m = 0; m < 2; ++m) {                   // 32 keys
      frag vf[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) vf[nt] = column_frag<LV, 4>(sV + 32 * m * LV + wc + 16 * nt, lane);
      if constexpr (!kStatePass) {
        bool bad = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) bad |= has_nonfinite(vf[nt]);
        if (!__any(bad)) {
#pragma unroll
          for (int i = 2 * m; i < 4; ++i) {
            const frag pf = row_frag(sP + (16 * i + l16) * LP + 32 * m + 8 * g);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) O[i][nt] = mma(vf[nt], pf, O[i][nt]);
          }
        } else {
          // An infinity or nan among the values: in the product above a masked weight of zero
          // would still meet it and leave nan in earlier rows, so the pairs are added one by one.
#pragma unroll
          for (int i = 2 * m; i < 4; ++i)
#pragma unroll 1
            for (int key = 32 * m; key < min(32 * m + 32, 16 * i + 16); ++key) {
              if (key > 16 * i + l16) continue;
              const float p = to_f32(sP[(16 * i + l16) * LP + key]);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                  O[i][nt][r] += p * to_f32(sV[key * LV + wc + 16 * nt + 4 * g + r]);
            }
        }
      }
      if (update) {
        frag vx[NT][SPLIT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) weigh<SPLIT>(vf[nt], vw[m], vx[nt]);
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          const frag kf = column_frag<LK, 8>(sK + 32 * m * LK + 32 * (i / 2) + 4 * (i % 2), lane);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < SPLIT; ++k) S[i][nt] = mma(kf, vx[nt][k], S[i][nt]);
        }
      }
    }
    has_state = true;

    if constexpr (!kStatePass) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int row = 16 * i + l16, col = wc + 16 * nt + 4 * g;
          if (row < n && c0 + col < R.dv) store4(po + (long long)(kC * c + row) * sto + col, O[i][nt]);
        }
    }
  }

  float* dst = kStatePass ? R.states + ((long long)slot * A.H + h) * SE
               : last_seg && R.fin ? R.fin + st_off : nullptr;
  if (!dst) return;
#pragma unroll
  for (int i = 0; i < NS; ++i)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = 32 * (i / 2) + 8 * g + 4 * (i % 2), col = c0 + wc + 16 * nt + l16;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (row + r < R.dk && col < R.dv) dst[(long long)(row + r) * R.dv + col] = S[i][nt][r];
    }
}

// ---- scan ------------------------------------------------------------------------------------
// Per (sequence, head, role) and element, over the segments in order: the sum U_j of segment j is
// replaced by the entry state E_j, E_{j+1} = g^SL E_j + U_j.  One thread has four neighbouring
// elements; the loads of four segments are in flight together.  Bound: HBM (or the Infinity Cache
// that the state pass has just written), one read and one write of the segment states.
__global__ __launch_bounds__(kThreads) void decay_scan_kernel(DecayArgs A) {
  const int SE = A.role[0].dk * A.role[0].dv, nb = (SE / 4 + kThreads - 1) / kThreads;
  long long x = blockIdx.x;
  const int e4 = 4 * (int(x % nb) * kThreads + threadIdx.x);
  x /= nb;
  const int h = int(x % A.H);
  x /= A.H;
  const DecayRole& R = A.role[x % A.n_roles];
  const int seq = int(x / A.n_roles), SL = kC * A.L;
  int slot = seq * A.n_seg, len = A.T;
  if (A.packed) {
    const int first = cu_at(A, seq);
    slot = decay_first_slot(first, seq, SL);
    len = max(cu_at(A, seq + 1) - first, 0);
  }
  const int n = (len + SL - 1) / SL;
  if (n < 2 || e4 >= SE) return;
  const double lg = log2_decay(A.log_decay[h]);
  const float f = decay_power(lg, SL);
  float4 e = {0.f, 0.f, 0.f, 0.f};
  if (R.init) {
    const float* p = R.init + ((long long)seq * A.H + h) * SE;
    const float f0 = R.rev ? 1.f : decay_power(lg, 1);
    float y[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int i = (e4 + r) / R.dv, j = (e4 + r) % R.dv;
      y[r] = f0 * p[R.init_trans ? j * R.dk + i : e4 + r];
    }
    e = float4{y[0], y[1], y[2], y[3]};
  }
  float* p = R.states + ((long long)slot * A.H + h) * SE + e4;
  const long long step = (long long)A.H * SE;
  for (int j = 0; j < n; j += 4) {
    float4 u[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      u[r] = float4{0.f, 0.f, 0.f, 0.f};
      if (j + r < n - 1) u[r] = *reinterpret_cast<const float4*>(p + (j + r) * step);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if (j + r < n) *reinterpret_cast<float4*>(p + (j + r) * step) = e;
      e.x = fmaf(f, e.x, u[r].x); e.y = fmaf(f, e.y, u[r].y);
      e.z = fmaf(f, e.z, u[r].z); e.w = fmaf(f, e.w, u[r].w);
    }
  }
}

// ---- recurrent form ------------------------------------------------------------------------
// One workgroup per (column block, head, sequence) keeps its part of the state in registers over
// the call's tokens: thread (row group, lane group) has 4 neighbouring columns of the rows
// row group + RG i.  Bound by the state's one read and one write.  LC lanes share a row:
// 4 LC columns of a block.
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
  return f32x4{bf_lo(u.x), bf_hi(u.x), bf_lo(u.y), bf_hi(u.y)};
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

template <typename T, int DK, int NT, int SPLIT>
hipError_t launch_chunks_t(const DecayArgs& a, bool state_pass, hipStream_t st) {
  const long long units = (long long)a.n_slots * a.H;
  const long long blocks = (units + 7) / 8 * 8 * a.nvb * a.n_roles;
  auto run = [&](auto kernel, int bytes) {
    hipError_t e = ensure_dynamic_lds(reinterpret_cast<const void*>(kernel), bytes);
    if (e != hipSuccess) return e;
    launch_kernel(kernel, dim3((unsigned)blocks), kThreads, bytes, st, a);
    return hipGetLastError();
  };
  using TL = Tiles<T, DK, NT>;
  return state_pass ? run(decay_chunks_kernel<T, DK, NT, SPLIT, true>, TL::bytes(true))
                    : run(decay_chunks_kernel<T, DK, NT, SPLIT, false>, TL::bytes(false));
}

template <typename T, int NT, int SPLIT>
hipError_t launch_chunks_d(const DecayArgs& a, int dk, bool state_pass, hipStream_t st) {
  if (dk <= 32) return launch_chunks_t<T, 32, NT, SPLIT>(a, state_pass, st);
  if (dk <= 64) return launch_chunks_t<T, 64, NT, SPLIT>(a, state_pass, st);
  if (dk <= 128) return launch_chunks_t<T, 128, NT, SPLIT>(a, state_pass, st);
  return hipErrorInvalidValue;
}

}  // namespace

int decay_block_columns(bool bf16, int dk, int dv) { return bf16 && dv > 64 ? 128 : 64; }

hipError_t launch_decay_chunks(DecayArgs& a, bool bf16, bool exact_state, bool state_pass,
                               hipStream_t st) {
  int dk = 0, dv = 0;
  for (int r = 0; r < a.n_roles; ++r) {
    dk = dk > a.role[r].dk ? dk : a.role[r].dk;
    dv = dv > a.role[r].dv ? dv : a.role[r].dv;
  }
  const int cols = decay_block_columns(bf16, dk, dv);
  a.nvb = (dv + cols - 1) / cols;
  if (!bf16) return launch_chunks_d<float, 1, 1>(a, dk, state_pass, st);
  if (cols == 128)
    return exact_state ? launch_chunks_d<__bf16, 2, 3>(a, dk, state_pass, st)
                       : launch_chunks_d<__bf16, 2, 2>(a, dk, state_pass, st);
  return exact_state ? launch_chunks_d<__bf16, 1, 3>(a, dk, state_pass, st)
                     : launch_chunks_d<__bf16, 1, 2>(a, dk, state_pass, st);
}

hipError_t launch_decay_scan(const DecayArgs& a, hipStream_t st) {
  const int SE = a.role[0].dk * a.role[0].dv, nb = (SE / 4 + kThreads - 1) / kThreads;
  const long long blocks = (long long)nb * a.H * a.n_roles * a.n_seq;
  launch_kernel(decay_scan_kernel, dim3((unsigned)blocks), kThreads, 0, st, a);
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
  constexpr int LC = 16;
  const dim3 grid((dv + 4 * LC - 1) / (4 * LC), H, B);
  auto run = [&](auto t, auto ri) {
    using T_ = decltype(t);
    launch_kernel(decay_decode_kernel<T_, LC, decltype(ri)::value>, grid, kThreads, 0, st, a,
                  (const T_*)q, (const T_*)k, (const T_*)v, log_decay, state, (T_*)o);
    return hipGetLastError();
  };
  auto rows = [&](auto t) {
    if (dk <= 32) return run(t, std::integral_constant<int, 2>());
    if (dk <= 64) return run(t, std::integral_constant<int, 4>());
    return run(t, std::integral_constant<int, 8>());
  };
  return bf16 ? rows(__bf16()) : rows(float());
}

}  // namespace kata
