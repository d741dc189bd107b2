// The walk over the chunks of a segment of the gated delta rule (delta.hip), as a device function: the forward
// pass's kernels and the backward pass's call it.
#pragma once

#include <type_traits>

#include "delta.h"
#include "delta_tiles.h"
#include "device.h"
#include "mfma_util.h"

namespace kata {

// ---- the walk ----------------------------------------------------------------------------------
enum class Walk { output, states, sums };

template <typename T, int DK, int W, int NT, bool kOut>
struct WalkTiles {
  static constexpr bool kBf = sizeof(T) == 2;
  static constexpr int DV = 16 * W;
  static constexpr int LK = DK + 16 / (int)sizeof(T), LV = DV + (kBf ? 16 : 4), LP = kC + 16 / (int)sizeof(T);
  static constexpr int kHead = 16 + kDeltaVec * 4;
  static constexpr int kTiles = kC * (LK * (kOut ? 2 : 1) + LV);
  static constexpr int kPO = kBf ? 2 : 1;           // terms of the outputs' operands
  static constexpr int NI = kBf ? (NT == 3 ? 3 : 2) : 1;               // terms of the inverse
  static constexpr int bytes = kHead + (kTiles + (NI + (kOut ? kPO : 0)) * kC * LP) * (int)sizeof(T);
  // waves a SIMD that the registers are held to (the launch bound counts workgroups a CU)
  static constexpr int occupancy = !kBf && DK == 128 ? 1 : kBf && !kOut && W == 8 && DK == 64 ? 4 : 8 / W;
};

// A wave has 16 columns of the values (or of the transition), and a part of P; W waves share K, Q and the inverse in LDS.
// With outputs a chunk takes 7.5 us where two workgroups share a CU (131072 tokens, width 64), without them and
// alone on its CU 2.5.
// kWhat: outputs and the final state; or (backward) the states before the chunks; or, of the segments,
// sums and transitions (blocks of columns behind those of the values).  NT: terms of the recurrence's operands.
// unit, sub: the segment and head, and which block of 16 W columns.
template <typename T, int DK, int W, int NT, Walk kWhat>
__device__ __forceinline__ void delta_walk(const DeltaArgs& A, unsigned unit, int sub, int backward, char* lds) {
  constexpr bool kOut = kWhat == Walk::output, kSums = kWhat == Walk::sums;
  using TL = WalkTiles<T, DK, W, NT, kOut>;
  using frag = typename Elem<T>::frag;
  constexpr int kThr = 64 * W, DV = TL::DV, M = DK / 32, NS = DK / 16, LK = TL::LK, LV = TL::LV, LP = TL::LP;
  constexpr int NI = TL::NI, PO = TL::kPO, J = 16 / W;            // J: key tiles of a wave's part of P
  constexpr bool kAlways = kWhat == Walk::states;   // fetch_rows
  // Sums of bf16 heads of up to 64: values and transition are eight waves, two workgroups a CU if they keep to 128
  // registers: LDS is read where it is used, without batches (131072 tokens: 407 us; four waves each for values
  // and transition, with batches, 475).
  constexpr bool kLean = sizeof(T) == 2 && kSums && W == 8 && DK == 64;
  // Products of several tiles in turn, or a tile's one after the other.  In turn 4 x 16384 tokens of width 128 take
  // 1284 us for 1332; outputs at width 64 and the sums above lack the registers (131072 tokens: 1075 for 1031).
  constexpr bool kTurns = !kLean && (!kOut || M > 2);
  constexpr int P = kTurns ? 2 : 1;                 // tiles of outputs
  int* const sh = reinterpret_cast<int*>(lds);
  float* const vec = reinterpret_cast<float*>(lds + 16);
  T* const sK = reinterpret_cast<T*>(lds + TL::kHead);
  T* const sV = sK + kC * LK;
  T* const sQ = sV + kC * LV;
  T* const sT = sK + TL::kTiles;
  T* const sP = sT + NI * kC * LP;

  const DeltaMap& m = A.m;
  const float scale = A.scale;
  const int tid = threadIdx.x;
  int lane = tid & 63, g = lane >> 4, l16 = lane & 15;
  // Wide heads: the places in LDS that a phase uses are computed there; kept from chunk to chunk they would cost
  // registers that are not there (a reload from scratch waits for the loads on their way, too).
  auto forget = [&]() __attribute__((always_inline)) {
    if constexpr ((kOut && M > 2) || kLean) {
      asm volatile("" : "+v"(lane));
      g = lane >> 4;
      l16 = lane & 15;
    }
  };
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  if (unit >= (unsigned)m.n_slots * (unsigned)m.H) return;
  const int slot = int(unit / (unsigned)m.H), h = int(unit - (unsigned)slot * (unsigned)m.H);
  const int ct = (m.dv + 15) / 16, c0 = sub * DV;
  const bool values = c0 < m.dv;                    // uniform
  // Sums: behind the tiles of the values' columns are those of the transition's, which start from the unit matrix
  // and have no values.
  const bool unit_matrix = kSums && sub * W + w >= ct;

  DeltaPart s;
  if (!find_part(m, slot, m.L, m.n_seg, m.n_slots, sh, kThr, s)) return;
  const int L = m.L;
  T* const out = kOut ? reinterpret_cast<T*>(A.o) + s.b * A.so[0] + h * A.so[2] + c0 : nullptr;
  if constexpr (kOut) {
    const int per_row = min(DV, m.dv - c0) / 4;
    auto clear = [&](int from, int rows) __attribute__((always_inline)) {          // the block's columns of `rows` output rows
      for (long long i = tid; i < (long long)rows * per_row; i += kThr)
        store4(out + (from + i / per_row) * A.so[1] + i % per_row * 4, zero4());
    };
    if (s.seq == m.n_seq) {                         // rows behind the last sequence
      if (A.zero_tail) clear(s.start + kC * L * s.part, min(kC * L, s.len - kC * L * s.part));
      return;
    }
    if (m.packed && A.zero_tail && s.seq == 0 && s.part == 0) clear(0, s.start);   // before the first
  }
  if (s.seq == m.n_seq) return;
  const int n_chunks = (s.len + kC - 1) / kC, n_seg = (n_chunks + L - 1) / L;
  const long long SE = (long long)m.dk * m.dv, st_off = ((long long)s.seq * m.H + h) * SE;
  if (s.part >= n_seg) {
    if (kOut && s.len == 0 && s.part == 0 && A.fin)  // an empty sequence
      for (int i = tid; i < m.dk * DV; i += kThr) {
        const int r = i / DV, c = c0 + i % DV;
        if (c < m.dv) A.fin[st_off + (long long)r * m.dv + c] = A.init ? A.init[st_off + (long long)r * m.dv + c] : 0.f;
      }
    return;
  }
  const bool last_seg = s.part == n_seg - 1;
  if constexpr (kSums) {
    // the sum of the last segment enters no entry state; a transition is used where a state comes in
    // from before, or in reversed time from behind
    const bool from_before = !last_seg && (s.part > 0 || A.init);
    const bool from_behind = backward && s.part > 0 && (!last_seg || A.dfin);
    if ((!values || last_seg) && (sub * W + W <= ct || (!from_before && !from_behind))) return;
  }
  const int first = s.part * L, behind = min(first + L, n_chunks);
  const long long row0 = s.start + (long long)kC * first;
  const int hk = h / (m.H / m.Hk);
  Stage<T, DK, kThr> rk(reinterpret_cast<const T*>(A.k) + s.b * A.sk[0] + row0 * A.sk[1] + hk * A.sk[2], A.sk[1], m.dk, true);
  Stage<T, DK, kThr> rq(reinterpret_cast<const T*>(kOut ? A.q : A.k) + s.b * A.sq[0] + row0 * A.sq[1] + hk * A.sq[2], A.sq[1], m.dk, true);
  Stage<T, DV, kThr> rv(reinterpret_cast<const T*>(A.v) + s.b * A.sv[0] + row0 * A.sv[1] + h * A.sv[2] + (values ? c0 : 0),
                        A.sv[1], m.dv - (values ? c0 : 0), false);
  StageInv<T, NI, LP, kThr> ri;
  const int n_last = min(kC, s.len - kC * (behind - 1));
  uint4 vec_next;
  const long long chunk0 = (long long)(s.c_slot + first) * m.H + h;    // [c_slots][H]
  const float* p_inv = A.inv + chunk0 * kInvFloats;
  const float* p_vec = A.vec + chunk0 * kDeltaVec;
  auto fetch = [&](int c) __attribute__((always_inline)) {
    const int n = c == behind - 1 ? n_last : kC;
    fetch_rows<kAlways>(rk, A.sk[1], n);
    if constexpr (kOut) fetch_rows<kAlways>(rq, A.sq[1], n);
    if (!kSums || values) fetch_rows<kAlways>(rv, A.sv[1], n);
    ri.template fetch<kAlways>(p_inv);
    if constexpr (kAlways) vec_next = fetch_vec(p_vec);
    else if (tid < kDeltaVec / 4) vec_next = reinterpret_cast<const uint4*>(p_vec)[tid];
    p_inv += (long long)m.H * kInvFloats;
    p_vec += (long long)m.H * kDeltaVec;
  };
  fetch(first);

  // state tiles: S[i] lane holds rows 16 i + 4 g + r of column c0 + wc + l16
  const int wc = 16 * w, col = c0 + wc + l16 - (unit_matrix ? 16 * ct : 0), cols = unit_matrix ? m.dk : m.dv;
  f32x4 S[NS];
  {
    const float* given = kSums ? nullptr : s.part > 0 ? A.sums + ((long long)slot * m.H + h) * SE : A.init ? A.init + st_off : nullptr;
#pragma unroll
    for (int i = 0; i < NS; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) S[i][r] = kSums && unit_matrix && 16 * i + 4 * g + r == col ? 1.f : 0.f;
    if (given) load_state(S, given, m.dk, m.dv, col, g);               // uniform
  }
  if (m.dk < DK || m.dv - c0 < DV) {                // columns that no operand has: zeros all along
    uint4* const z = reinterpret_cast<uint4*>(sK);
    for (int i = tid; i < TL::kTiles * (int)sizeof(T) / 16; i += kThr) z[i] = uint4{0u, 0u, 0u, 0u};
  }
  ri.zeros(sT);
  const int rt = w & 3, j0 = J * (w >> 2);          // the wave's rows and first key tile of P
  const bool live_col = c0 + wc + 4 * g < m.dv;
  T* po = kOut ? out + (row0 + l16) * A.so[1] + wc + 4 * g : nullptr;
  float *p_state = nullptr, *p_u = nullptr;
  if (kWhat == Walk::states && c0 / 16 + w < ct) {
    p_state = A.cstates + (chunk0 * ct + c0 / 16 + w) * (DK * 16) + lane * 4;
    p_u = A.u + (chunk0 * ct + c0 / 16 + w) * 1024 + lane * 4;
  }

  Quad<T> O[4];                                     // outputs of the last chunk
  auto store = [&](int rows) __attribute__((always_inline)) {
    if (kOut && live_col)
#pragma unroll
      for (int it = 0; it < 4; ++it)
        if (16 * it + l16 < rows) *reinterpret_cast<Quad<T>*>(po + 16 * it * A.so[1]) = O[it];
    po += kC * A.so[1];
  };
  f32x4 U[4];
  auto store_u = [&]() __attribute__((always_inline)) {                              // of the last chunk
#pragma unroll
    for (int it = 0; it < 4; ++it) *reinterpret_cast<f32x4*>(p_u + it * 256) = U[it];
    p_u += (long long)m.H * ct * 1024;
  };
#pragma unroll 1
  for (int c = first; c < behind; ++c) {
    __syncthreads();                                // the last chunk's tiles have been read
    if constexpr (kAlways) {
      const int n = c == behind - 1 ? n_last : kC;
      keep_rows(rk, n);
      keep_rows(rv, n);
    }
    rk.template put_split<LK>(sK);
    if constexpr (kOut) rq.template put_split<LK>(sQ);
    if (!kSums || values) rv.template put<LV>(sV);
    ri.put(sT);
    put_vec(vec, vec_next);
    // (stores before the next loads: the wait for these then does not wait for stores just issued)
    if (kWhat == Walk::states && p_state) {         // uniform
      if (c > first) store_u();
#pragma unroll
      for (int i = 0; i < NS; ++i) *reinterpret_cast<f32x4*>(p_state + i * 256) = S[i];
      p_state += (long long)m.H * ct * (DK * 16);
    }
    if (kOut && c > first) store(kC);
    if (c + 1 < behind) fetch(c + 1);
    __syncthreads();

    // LDS reads are issued in batches, ahead of the work that hides them (reads_above): left alone, the compiler
    // waits for nearly every read before its product.
    f32x4 X[4], o[4];
    Op<T, NI> inv[6];                               // (row tile, K step): (0, 0), (1, 0), (2, 0), (2, 1), (3, 0), (3, 1)
    auto read_inv = [&]() __attribute__((always_inline)) {
#pragma unroll
      for (int f = 0; f < 6; ++f)
        inv[f] = row_op<NI>(sT + (16 * (f < 2 ? f : 1 + f / 2) + l16) * LP + (f < 2 ? 0 : 32 * (f & 1)) + 8 * g, kC * LP);
    };
    frag vf[2];
    forget();
    if constexpr (kOut) {
      Op<T, NT> sf[M];
#pragma unroll
      for (int i = 0; i < M; ++i) split_terms(S[2 * i], S[2 * i + 1], sf[i]);
      // bf16: with two terms of the state, of P and of U an output has no error but its own rounding
#pragma unroll
      for (int i0 = 0; i0 < 4; i0 += P) {
#pragma unroll
        for (int p = 0; p < P; ++p) X[i0 + p] = o[i0 + p] = zero4();
#pragma unroll
        for (int i = 0; i < M; ++i) {
          frag kr[P], qr[P];
#pragma unroll
          for (int p = 0; p < P; ++p) {
            kr[p] = row_frag(sK + (16 * (i0 + p) + l16) * LK + 32 * i + 8 * g);
            qr[p] = row_frag(sQ + (16 * (i0 + p) + l16) * LK + 32 * i + 8 * g);
          }
#pragma unroll
          for (int t = NT - 1; t >= 0; --t)
#pragma unroll
            for (int p = 0; p < P; ++p) {
              X[i0 + p] = mma(kr[p], sf[i].t[t], X[i0 + p]);
              if (t < PO) o[i0 + p] = mma(sf[i].t[t], qr[p], o[i0 + p]);
            }
        }
#pragma unroll
        for (int p = 0; p < P; ++p) o[i0 + p] *= vec[16 * (i0 + p) + l16] * scale;
      }
      reads_above<T>();
      forget();
      put_scores<T, DK, LK, LP, J, PO>(sP, sQ, sK, vec + 3 * kC, rt, j0, lane, scale);
      reads_above<T>();
#pragma unroll
      for (int i = 0; i < 2; ++i) vf[i] = column_frag<LV>(sV + 32 * i * LV + wc, lane);
    } else {
      frag kr[4][M];
      if constexpr (!kLean) {
#pragma unroll
        for (int it = 0; it < 4; ++it)
#pragma unroll
          for (int i = 0; i < M; ++i) kr[it][i] = row_frag(sK + (16 * it + l16) * LK + 32 * i + 8 * g);
        reads_above<T>();
      }
      Op<T, NT> sf[M];
#pragma unroll
      for (int i = 0; i < M; ++i) split_terms(S[2 * i], S[2 * i + 1], sf[i]);
#pragma unroll
      for (int i = 0; i < 2; ++i) vf[i] = column_frag<LV>(sV + 32 * i * LV + wc, lane);
      if constexpr (M <= 2 && !kLean) read_inv();
      reads_above<T>();
#pragma unroll
      for (int it = 0; it < 4; ++it) X[it] = zero4();
#pragma unroll
      for (int i = 0; i < M; ++i)
        if constexpr (kLean) {
#pragma unroll
          for (int it = 0; it < 4; ++it) X[it] = mul(row_frag(sK + (16 * it + l16) * LK + 32 * i + 8 * g), sf[i], X[it]);
          reads_above<T>();
        } else {
#pragma unroll
          for (int t = NT - 1; t >= 0; --t)
#pragma unroll
            for (int it = 0; it < 4; ++it) X[it] = mma(kr[it][i], sf[i].t[t], X[it]);
        }
    }
    forget();
    if constexpr (M > 2 || kOut) read_inv();
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const f32x4 yv = *reinterpret_cast<const f32x4*>(vec + 16 * it + 4 * g);
      const f32x4 bv = *reinterpret_cast<const f32x4*>(vec + 2 * kC + 16 * it + 4 * g);
      X[it] = bv * (half_of(vf[it >> 1], it & 1) - yv * X[it]);
    }
    frag kt[2][NS];                                 // K transposed, 32 keys each
    auto read_kt = [&](int j) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < NS; ++i) kt[j][i] = split_column_frag<LK>(sK + 32 * j * LK, i, lane);
    };
    if constexpr (M <= 2 && !kOut && !kLean) read_kt(0);
    reads_above<T>();
    auto correct = [&]() __attribute__((always_inline)) {
      Op<T, NT> xf[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) split_terms(X[2 * i], X[2 * i + 1], xf[i]);
      if constexpr (kLean) {
#pragma unroll
        for (int it = 0; it < 4; ++it) {
          U[it] = zero4();
#pragma unroll
          for (int i = 0; i <= it >> 1; ++i)
            U[it] = mul(row_op<NI>(sT + (16 * it + l16) * LP + 32 * i + 8 * g, kC * LP), xf[i], U[it]);
          reads_above<T>();
        }
      } else if constexpr (!kTurns) {
        U[0] = mul(inv[0], xf[0], zero4());
        U[1] = mul(inv[1], xf[0], zero4());
        U[2] = mul(inv[2], xf[0], zero4());
        U[3] = mul(inv[4], xf[0], zero4());
        U[2] = mul(inv[3], xf[1], U[2]);
        U[3] = mul(inv[5], xf[1], U[3]);
      } else {
#pragma unroll
        for (int it = 0; it < 4; ++it) U[it] = zero4();
        each_term<NI, NT>([&](int n, int k) __attribute__((always_inline)) {
#pragma unroll
          for (int it = 0; it < 4; ++it) U[it] = mma(inv[it < 2 ? it : 2 * it - 2].t[n], xf[0].t[k], U[it]);
        });
        each_term<NI, NT>([&](int n, int k) __attribute__((always_inline)) {
          U[2] = mma(inv[3].t[n], xf[1].t[k], U[2]);
          U[3] = mma(inv[5].t[n], xf[1].t[k], U[3]);
        });
      }
      float sick = 0.f;
#pragma unroll
      for (int it = 0; it < 4; ++it)
#pragma unroll
        for (int r = 0; r < 4; ++r) sick = fmaf(U[it][r], 0.f, sick);
      return sick != 0.f;
    };
    // An infinity or nan in row j: in products a zero of a later column would still meet it and leave nan in
    // earlier rows.  From row j on the column's outputs and its state are nan; the rows before it are
    // computed without.
    int ill = kC;                                   // the column's first such row
    const bool any_ill = __any(correct());
    if (any_ill) {
      auto look = [&](f32x4 (&x)[4]) {
#pragma unroll
        for (int it = 0; it < 4; ++it)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (!(fabsf(x[it][r]) < __builtin_huge_valf())) ill = min(ill, 16 * it + 4 * g + r);
        ill = min(ill, __shfl_xor(ill, 16));
        ill = min(ill, __shfl_xor(ill, 32));
#pragma unroll
        for (int it = 0; it < 4; ++it)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (16 * it + 4 * g + r >= ill) x[it][r] = 0.f;
      };
      look(X);
      if constexpr (!kLean) read_inv();
      correct();
      look(U);
    }
    {
      const float whole = vec[kC - 1];
      f32x4 u[4];
#pragma unroll
      for (int it = 0; it < 4; ++it) u[it] = U[it] * *reinterpret_cast<const f32x4*>(vec + kC + 16 * it + 4 * g);
      if constexpr (!kLean) {
        if constexpr (M > 2 || kOut) read_kt(0);
        read_kt(1);
        reads_above<T>();
      }
      forget();
      Op<T, NT> uf[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) split_terms(u[2 * i], u[2 * i + 1], uf[i]);
#pragma unroll
      for (int i = 0; i < NS; ++i) S[i] *= whole;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if constexpr (kLean) read_kt(j);
        if constexpr (kTurns) {
#pragma unroll
          for (int t = NT - 1; t >= 0; --t)
#pragma unroll
            for (int i = 0; i < NS; ++i) S[i] = mma(kt[j][i], uf[j].t[t], S[i]);
        } else {
#pragma unroll
          for (int i = 0; i < NS; ++i) S[i] = mul(kt[j][i], uf[j], S[i]);
        }
        if constexpr (kLean) reads_above<T>();
      }
      if (any_ill && ill < kC)
#pragma unroll
        for (int i = 0; i < NS; ++i) S[i] = f32x4{1.f, 1.f, 1.f, 1.f} * __builtin_nanf("");
    }
    if constexpr (kOut) {
      __syncthreads();                              // P is there
      forget();
      Op<T, PO> uf[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) split_terms(U[2 * i], U[2 * i + 1], uf[i]);
#pragma unroll
      for (int i0 = 0; i0 < 4; i0 += P)
#pragma unroll
        for (int i = 0; i <= i0 >> 1; ++i) {
          Op<T, PO> pf[P];
#pragma unroll
          for (int p = 0; p < P; ++p) pf[p] = row_op<PO>(sP + (16 * (i0 + p) + l16) * LP + 32 * i + 8 * g, kC * LP);
          each_term<PO, PO>([&](int n, int k) __attribute__((always_inline)) {
#pragma unroll
            for (int p = 0; p < P; ++p) o[i0 + p] = mma(uf[i].t[n], pf[p].t[k], o[i0 + p]);
          });
        }
      if (any_ill)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int at = __shfl(ill, 4 * g + r);
#pragma unroll
          for (int it = 0; it < 4; ++it)
            if (16 * it + l16 >= at) o[it][r] = __builtin_nanf("");
        }
#pragma unroll
      for (int it = 0; it < 4; ++it) O[it] = quad(o[it], T());
    }
  }

  if constexpr (kOut) store(n_last);
  if (kWhat == Walk::states && p_state) store_u();

  if (kWhat == Walk::states && last_seg && A.fstates && p_state) {     // the state behind the last chunk
    float* at = A.fstates + (((long long)s.seq * m.H + h) * ct + c0 / 16 + w) * (DK * 16) + lane * 4;
#pragma unroll
    for (int i = 0; i < NS; ++i) *reinterpret_cast<f32x4*>(at + i * 256) = S[i];
  }

  float* dst = kSums ? (unit_matrix ? A.trans + ((long long)slot * m.H + h) * m.dk * m.dk
                                    : A.sums + ((long long)slot * m.H + h) * SE)
               : kOut && last_seg && A.fin ? A.fin + st_off : nullptr;
  if (!dst || col >= cols) return;
#pragma unroll
  for (int i = 0; i < NS; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (16 * i + 4 * g + r < m.dk) dst[(16 * i + 4 * g + r) * cols + col] = S[i][r];
}

}  // namespace kata
