// What the gated delta rule's forward and backward kernels share: the chunks of
// packed sequences, operands as sums of bf16 terms in shared memory, and their
// products on the tensor cores.
//
// Within a chunk of 64 positions, with c the running sum of ln f and D_ti =
// exp(c_t - c_i) for i <= t:
//   A = beta D (K K^T) below the diagonal,   M = (I + A)^-1 beta
//   U = M (V - e^c K S),                      the writes of all its positions
//   Y = scale e^c Q S + P U,                  P = scale D (Q K^T)
//   S <- e^c_last S + K^T (e^(c_last - c) U)
// M and P do not depend on the state: prepare_kernel makes them for all chunks at
// once, and the kernels that follow the chunks one after another take them from
// there.
//
// Precision.  The states and sums are fp32.  A product's operands are sums of bf16
// terms (8 bits each): an input of type bf16 is one term and exact; what is
// computed on the way is three (24 bits, as fp32 has) wherever it reaches a state,
// and two (16 bits) where it only reaches outputs of type bf16: 2^-17 of the terms
// that an output is made of, far below bf16's own rounding unless these cancel.  (A
// decay's gradient is where they do: see delta_grad.cu.)  Of the terms' products those
// are taken that are not below the last bit that is kept.  (mma.sync's bf16 form does
// 1024 multiply-adds a clock and SM here and its tf32 form 512, measured: three bf16
// terms of one operand cost less than two tf32 ones.)  The tcgen05 form is three times
// as fast (1920 TFLOP/s against 590) and has not been tried.  With the value columns as
// its 128 rows it would be one block a head; with a chunk's rows of K over those of Q,
// and the key columns, as its rows, the value columns could be spread over blocks as
// they are here.  Every value would come from tensor memory to registers between any two
// products, to be scaled and split; here that is where they are.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "engram_internal.h"
#include "train_device.cuh"

namespace engram {
namespace delta {

constexpr int kC = ENGRAM_DELTA_CHUNK;  // 64 positions
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxDim = ENGRAM_DELTA_MAX_DIM;
// Lower triangles of 64 x 64 are kept as ten blocks of 16 x 16, a term's 512 bytes
// each, the 16-byte halves of a block's rows 4 to 7 and 12 to 15 exchanged (eight
// rows then lie in different banks).
constexpr int kBlocks = 10, kTerm = kBlocks * 512;
constexpr int kStateTerms = 3;  // of M, and of everything that reaches a state

template <class E>
constexpr int kIn = E::kBytes == 2 ? 1 : 3;  // terms of an input
template <class E>
constexpr int kOut = E::kBytes == 2 ? 2 : 3;  // of what only reaches outputs

// Per (chunk, head) in the workspace.
constexpr int kTriBytes = kTerm * 2 * kStateTerms;  // M, P
struct Gates {
  float into[kC], last[kC], hi[kC], lo[kC], beta[kC];  // e^c, e^(c_last - c), c in two parts, beta (0: masked)
};

template <class E>
struct Args {
  using T = typename E::T;
  const T *q, *k, *v, *g, *b, *dy;
  T *y, *dq, *dk_out, *dv_out, *dg, *db;
  int64_t q_stride, k_stride, v_stride, g_stride, b_stride, y_stride, dy_stride;
  int64_t dq_stride, dk_stride, dv_stride, dg_stride, db_stride;
  const int64_t* cu;
  const int32_t* slots;
  const uint8_t* mask;
  const float* state;
  float *state_out, *carry;
  int64_t n_slots;
  int32_t n_tokens, n_seqs, max_chunks, keys, heads, dk, dv;
  float scale;
  bool vec;        // rows of q, k, v and dy in 16-byte pieces
  bool pairs;      // rows of y or dv in pairs of elements
  bool key_pairs;  // rows of dq and dk, likewise
  bool has_state;  // slots are checked against n_slots
  // workspace
  int32_t* first;  // [n_seqs + 1] number of a sequence's first chunk
  int64_t* line;   // [n_seqs + 2] what the sequences before s take of a head's line; the blocks' share (see Item)
  uint32_t* given;  // [blocks] whether a block's first state has been handed on
  float* between;   // the states that are handed on, kHandedOn floats a block
  int32_t blocks, slices;  // of the kernels that follow the sequences; slices of a head's value columns
  unsigned char* tri;
  Gates* gates;
  // backward: states' gradients behind the chunks, as `carry` has the states in front of them; the second and the third
  // terms of the values' gradients (bf16), one array behind the other; sums over heads that share a key
  float* after;
  uint16_t* writes;
  float* shared;
  int32_t* status;
  // (0; see engram_selftest_delta_wait)
  uint32_t absent;  // bytes that every stage's copies are expected to have beyond theirs
  bool withheld;    // states are handed on without a word
};

// ------------------------------------------------------------------- chunks

struct Chunk {
  int start, len;  // positions
  int seq;
  bool live;
};

template <class E>
__device__ __forceinline__ void bounds(const Args<E>& a, int s, int& lo, int& hi) {
  const int64_t n = a.n_tokens, x = a.cu[s], y = a.cu[s + 1];
  lo = static_cast<int>(x < 0 ? 0 : x > n ? n : x);
  hi = static_cast<int>(y < lo ? lo : y > n ? n : y);
}

// Whether the sequence, of n chunks from c0 on, has a state slot of its own, or needs none.
// A sequence that the forward pass took for padding has left nothing but kPadding in its
// chunks' gates: it is padding in the backward pass too, which need not have the states.
constexpr float kPadding = -1.f;  // in place of e^c
template <class E>
__device__ __forceinline__ bool live_slot(const Args<E>& a, int s, int c0, int n, int64_t& slot) {
  slot = a.slots != nullptr ? a.slots[s] : s;
  if (slot < 0 || (a.has_state && slot >= a.n_slots)) return false;
  return a.y != nullptr || n == 0 || a.gates[static_cast<size_t>(c0) * a.heads].into[0] != kPadding;
}

// Chunk number c, or false where there are fewer.
template <class E>
__device__ __forceinline__ bool chunk_at(const Args<E>& a, int c, Chunk& ch) {
  if (c >= a.first[a.n_seqs]) return false;
  int lo = 0, hi = a.n_seqs - 1;  // the last sequence that begins at or before c, of which the others are empty
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.first[mid] <= c) lo = mid;
    else hi = mid - 1;
  }
  int from, to;
  bounds(a, lo, from, to);
  ch.seq = lo;
  ch.start = from + (c - a.first[lo]) * kC;
  ch.len = to - ch.start < kC ? to - ch.start : kC;
  int64_t slot;
  ch.live = live_slot(a, lo, a.first[lo], 1, slot);
  return ch.len > 0;
}

// ------------------------------------------------------------ shared memory

__device__ __forceinline__ void st32(uint32_t at, uint32_t v) { asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory"); }
__device__ __forceinline__ uint32_t ld32(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at));
  return v;
}
__device__ __forceinline__ float lo_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_of(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// Two values as N terms, `term` bytes apart.
template <int N>
__device__ __forceinline__ void put(uint32_t at, int term, float x0, float x1) {
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const uint32_t w = pack(x0, x1);
    st32(at + n * term, w);
    x0 -= lo_of(w);
    x1 -= hi_of(w);
  }
}
// and back
template <int N>
__device__ __forceinline__ void get(uint32_t at, int term, float& x0, float& x1) {
  x0 = x1 = 0.f;
#pragma unroll
  for (int n = N - 1; n >= 0; --n) {
    const uint32_t w = ld32(at + n * term);
    x0 += lo_of(w);
    x1 += hi_of(w);
  }
}

__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_begun() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_group 0;" ::: "memory"); }

// A matrix of bf16 terms: rows `pitch` bytes apart (16 bytes more than a multiple of
// 128 or 64: eight rows lie in different banks), terms `term` bytes apart.
struct Mat {
  uint32_t base;
  int pitch, term;
};
__host__ __device__ constexpr int mat_bytes(int rows, int cols) { return rows * (cols + 8) * 2; }
template <int kRows, int kCols>
__device__ __forceinline__ Mat mat(uint32_t base) { return Mat{base, (kCols + 8) * 2, mat_bytes(kRows, kCols)}; }

// kC rows of kCols columns (the first `cols` of them), zeros past the chunk's end and at
// masked positions.  `src` is the first row's first element.
template <class E, int kCols, int kT = kThreads>
__device__ __forceinline__ void load_rows(const Mat& m, const typename E::T* src, int64_t stride, int len, int cols,
                                          const uint8_t* mask, bool vec, int tid = threadIdx.x) {
  if (E::kBytes == 2 && vec) {
#pragma unroll
    for (int i0 = 0; i0 < kC * (kCols / 8); i0 += kT) {
      const int i = i0 + tid;
      if (kC * (kCols / 8) % kT != 0 && i >= kC * (kCols / 8)) break;
      const int r = i / (kCols / 8), c = i % (kCols / 8) * 8;
      const bool on = r < len && c < cols && !(mask != nullptr && mask[r]);
      copy16(m.base + r * m.pitch + c * 2, on ? src + r * stride + c : src, on);
    }
  } else {
    constexpr int kAhead = 4;  // pairs on their way at once
    for (int i0 = tid; i0 < kC * (kCols / 2); i0 += kAhead * kT) {
      float x[kAhead][2];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = i0 + u * kT, r = i / (kCols / 2), c = i % (kCols / 2) * 2;
        const bool on = r < len && !(mask != nullptr && mask[r]);
        x[u][0] = on && c < cols ? E::load(src + r * stride + c) : 0.f;
        x[u][1] = on && c + 1 < cols ? E::load(src + r * stride + c + 1) : 0.f;
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = i0 + u * kT, r = i / (kCols / 2), c = i % (kCols / 2) * 2;
        if (i < kC * (kCols / 2)) put<kIn<E>>(m.base + r * m.pitch + c * 2, m.term, x[u][0], x[u][1]);
      }
    }
  }
}

// ----------------------------------------------------------------- products

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ld4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void ld4t(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}

// 16 x 16 pieces of an operand A(m, k), as stored or transposed, of a term
struct Rows {  // A(m, k) = X[m][k]
  Mat x;
  __device__ __forceinline__ void operator()(uint32_t (&r)[4], int m, int k, int n) const {
    const int l = lane_id();
    ld4(r, x.base + n * x.term + (m + (l & 15)) * x.pitch + (k + (l >> 4) * 8) * 2);
  }
};
struct Cols {  // A(m, k) = X[k][m]
  Mat x;
  __device__ __forceinline__ void operator()(uint32_t (&r)[4], int m, int k, int n) const {
    const int l = lane_id();
    ld4t(r, x.base + n * x.term + (k + (l & 7) + (l >> 4) * 8) * x.pitch + (m + ((l >> 3) & 1) * 8) * 2);
  }
};
__device__ __forceinline__ uint32_t tri_at(int row, int half) { return row * 32 + ((half ^ ((row >> 2) & 1)) << 4); }
// 16 x 8 N pieces of an operand B(k, n)
struct Down {  // B(k, n) = X[k][n]
  Mat x;
  template <int N>
  __device__ __forceinline__ void get(uint32_t (&r)[N][2], int k, int n, int t) const {
    const int l = lane_id();
    const uint32_t at = x.base + t * x.term + (k + (l & 15)) * x.pitch + n * 2;
    static_assert(N % 2 == 0, "pairs of tiles");
#pragma unroll
    for (int j = 0; j < N; j += 2) {
      uint32_t w[4];
      ld4t(w, at + (j * 8 + (l >> 4) * 8) * 2);
      r[j][0] = w[0]; r[j][1] = w[1]; r[j + 1][0] = w[2]; r[j + 1][1] = w[3];
    }
  }
};
struct Across {  // B(k, n) = X[n][k]
  Mat x;
  template <int N>
  __device__ __forceinline__ void get(uint32_t (&r)[N][2], int k, int n, int t) const {
    const int l = lane_id();
    const uint32_t at = x.base + t * x.term + k * 2 + ((l >> 3) & 1) * 16;
    static_assert(N % 2 == 0, "pairs of tiles");
#pragma unroll
    for (int j = 0; j < N; j += 2) {
      uint32_t w[4];
      ld4(w, at + (n + j * 8 + (l & 7) + (l >> 4) * 8) * x.pitch);
      r[j][0] = w[0]; r[j][1] = w[1]; r[j + 1][0] = w[2]; r[j + 1][1] = w[3];
    }
  }
};

// c += A(m.., k0 ..k1) B(k0 ..k1, n..), a 16 x 8 N tile, of TA and TB terms: the
// products of terms i and j with i + j < kLimit.  The tensor cores cut each sum of an
// instruction off at the accumulator's last bit: where 24 bits are to be kept, the
// small terms' products have an accumulator of their own, so that the large ones' is
// cut once for every 16 of k and not six times (fp32: 1.8e-6 against 5e-7 of the result).
template <int TA, int TB, int kLimit, int N, class A, class B>
__device__ __forceinline__ void product(float (&c)[N][4], const A& a, const B& b, int m, int n, int k0, int k1) {
  constexpr bool kApart = kLimit > 2;
  float small[kApart ? N : 1][4] = {};
#pragma unroll 2
  for (int k = k0; k < k1; k += 16) {
    uint32_t fa[TA][4];
#pragma unroll
    for (int i = 0; i < TA; ++i) a(fa[i], m, k, i);
#pragma unroll
    for (int j = 0; j < TB; ++j) {
      uint32_t fb[N][2];
      b.template get<N>(fb, k, n, j);
#pragma unroll
      for (int i = 0; i < TA; ++i)
        if (i + j < kLimit) {
#pragma unroll
          for (int t = 0; t < N; ++t) mma(kApart && i + j > 0 ? small[kApart ? t : 0] : c[t], fa[i], fb[t][0], fb[t][1]);
        }
    }
  }
  if constexpr (kApart) {
#pragma unroll
    for (int t = 0; t < N; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) c[t][j] += small[t][j];
  }
}

// 16 x 16 pieces of a triangle as an operand B(k, n)
struct TriAcross {  // B(k, n) = X[n][k]
  uint32_t base;
  __device__ __forceinline__ void get(uint32_t (&r)[2][2], int kb, int nb, int t) const {
    const int l = lane_id();
    uint32_t w[4];
    ld4(w, base + t * kTerm + (nb * (nb + 1) / 2 + kb) * 512 + tri_at((l & 7) + (l >> 4) * 8, (l >> 3) & 1));
    r[0][0] = w[0]; r[0][1] = w[1]; r[1][0] = w[2]; r[1][1] = w[3];
  }
};
struct TriDown {  // B(k, n) = X[k][n]
  uint32_t base;
  __device__ __forceinline__ void get(uint32_t (&r)[2][2], int kb, int nb, int t) const {
    const int l = lane_id();
    uint32_t w[4];
    ld4t(w, base + t * kTerm + (kb * (kb + 1) / 2 + nb) * 512 + tri_at(l & 15, l >> 4));
    r[0][0] = w[0]; r[0][1] = w[1]; r[1][0] = w[2]; r[1][1] = w[3];
  }
};

// Two neighbouring 16 x 8 accumulators as an operand A, 16 x 16, of N terms: the
// places of the one are those of the other, so nothing goes through shared memory.
template <int N>
__device__ __forceinline__ void as_operand(uint32_t (&f)[N][4], const float (&lo)[4], const float (&hi)[4]) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    float x0 = p < 2 ? lo[2 * p] : hi[2 * p - 4], x1 = p < 2 ? lo[2 * p + 1] : hi[2 * p - 3];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      f[n][p] = pack(x0, x1);
      x0 -= lo_of(f[n][p]);
      x1 -= hi_of(f[n][p]);
    }
  }
}
// An 8 x 8 matrix of 16-bit values, a row's pair a lane, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// States that are kept for the backward pass: fp32 as they are, transposed, [dv][dk]; for
// inputs of type bf16 two terms in blocks of 16 columns and 16 rows, 1 KB each: for
// either term four 8 x 8 matrices, S^T's (columns, rows) 0 0, 8 0, 0 8 and 8 8.  A warp
// writes a matrix as its lanes hold it, 128 bytes, and reads it as an operand from where
// it was copied to.
constexpr int kBlockBytes = 1024;
template <class E>
__host__ __device__ size_t saved_floats(int dk, int dv) {  // of a chunk's state
  if (E::kBytes == 4) return static_cast<size_t>(dk) * dv;
  return static_cast<size_t>((dk + 15) / 16) * ((dv + 15) / 16) * (kBlockBytes / 4);
}
__device__ __forceinline__ uint32_t* block_of(float* base, int dk, int vb, int kb) {
  return reinterpret_cast<uint32_t*>(base) + (static_cast<size_t>(vb) * ((dk + 15) / 16) + kb) * (kBlockBytes / 4);
}
// a lane's part of a block: the first two terms of an operand
__device__ __forceinline__ void save_block(uint32_t* block, const uint32_t (&f)[kStateTerms][4]) {
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j) block[n * 128 + j * 32 + lane_id()] = f[n][j];
}
// the same of fp32: 16 columns from vw and 16 rows from k0 of [dv][dk]
__device__ __forceinline__ void save_rows(float* to, int dk, int dv, int vw, int k0, const float (&lo)[4], const float (&hi)[4]) {
  const int g = lane_id() >> 2, t2 = (lane_id() & 3) * 2;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int v = vw + g + ((j >> 1) & 1) * 8, k = k0 + (j >> 2) * 8 + t2 + (j & 1);
    if (v < dv && k < dk) to[static_cast<size_t>(v) * dk + k] = j < 4 ? lo[j & 3] : hi[j & 3];
  }
}
// S^T's blocks in shared memory as an operand B(k, n), 16 x 16 pieces
struct BlocksDown {  // k: columns, n: rows
  uint32_t base;
  int across;
  template <int N>
  __device__ __forceinline__ void get(uint32_t (&r)[N][2], int k, int n, int t) const {
    static_assert(N % 2 == 0, "blocks of 16 rows");
    const int l = lane_id();
#pragma unroll
    for (int j = 0; j < N; j += 2) {
      uint32_t w[4];
      ld4t(w, base + ((k >> 4) * across + (n >> 4) + j / 2) * kBlockBytes + t * 512 + l * 16);
      r[j][0] = w[0]; r[j][1] = w[1]; r[j + 1][0] = w[2]; r[j + 1][1] = w[3];
    }
  }
};

template <int N>
__device__ __forceinline__ void clear(float (&c)[N][4]) {
#pragma unroll
  for (int t = 0; t < N; ++t)
#pragma unroll
    for (int j = 0; j < 4; ++j) c[t][j] = 0.f;
}

// The chunk's triangles and gates, 16 bytes a copy.  kP: terms of P.
template <int kP, int kT = kThreads>
__device__ __forceinline__ void load_tri(uint32_t m, uint32_t p, const unsigned char* from, int tid = threadIdx.x) {
  for (int i = tid; i < kStateTerms * kTerm / 16; i += kT) copy16(m + i * 16, from + i * 16, true);
  for (int i = tid; i < kP * kTerm / 16; i += kT) copy16(p + i * 16, from + kStateTerms * kTerm + i * 16, true);
}
template <int kT = kThreads>
__device__ __forceinline__ void load_gates(uint32_t to, const Gates* from, int tid = threadIdx.x) {
  for (int i = tid; i < static_cast<int>(sizeof(Gates)) / 16; i += kT)
    copy16(to + i * 16, reinterpret_cast<const unsigned char*>(from) + i * 16, true);
}

// The kernels that follow the sequences have a block on each SM.  What there is to do, a
// sequence in a slice of a head's columns after the other, lies on a line, a sequence's
// chunks and one more for its state; each block has an equal share of it, T, or as much as
// the longest sequence takes.  Where the end of a share cuts a sequence, the next block
// takes its first chunks, as the first thing that it does, and hands the state on; this block
// takes the others as its last.  The two do not overlap as no sequence is longer than T.
// Shares are given from the line's end on, so that a block waits only for one that was
// launched before it, and what it waits for waits for nothing.  (16,384 positions of 40
// heads in four sequences of 114, 91, 50 and 3 chunks, forwards: 1049 us with a block for
// each sequence and slice, longest first, 768 this way; where the longest sequence alone
// takes as long, 201 of 259 chunks, 1121 and 1116.)
constexpr int kMaxBlocks = 256, kHandedOn = 512 * 16;
struct Item {
  int64_t at, end;        // on the line, and the share's end
  int64_t begin, behind;  // the sequence's part of the line, and what it takes in each slice
  int cost;
  int seq, h, v0;
  int lo, hi, c0, n;      // positions, chunks
  int from, to;           // the chunks that are done here, in the order of the kernel
  bool any, take, give;
};
// The same value in every lane, known as such: what is worked out from it is worked out once a warp.
__device__ __forceinline__ int uniform(int x) { return __reduce_max_sync(0xffffffffu, x); }
template <class E>
__device__ __forceinline__ int chunks_of(const Args<E>& a, int s, int& lo, int& hi) {
  bounds(a, s, lo, hi);
  return min((hi - lo + kC - 1) / kC, a.max_chunks - a.first[s]);
}
// The block's next item, by one thread; the first one if `it.seq` is negative.
template <class E>
__device__ __forceinline__ void next_item(const Args<E>& a, Item& it, int across) {
  const int64_t per = static_cast<int64_t>(a.heads) * a.slices, share = gridDim.x - 1 - blockIdx.x;
  auto enter = [&](int s) {
    it.seq = s;
    it.begin = a.line[s] * per;
    it.behind = a.line[s + 1] * per;
    it.cost = static_cast<int>(a.line[s + 1] - a.line[s]);
    it.n = chunks_of(a, s, it.lo, it.hi);
    it.c0 = a.first[s];
  };
  if (it.seq < 0) {
    const int64_t T = a.line[a.n_seqs + 1];
    it.at = share * T;
    it.end = min(it.at + T, a.line[a.n_seqs] * per);
    int lo = 0, hi = a.n_seqs - 1;  // the last sequence that begins at or before the share
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.line[mid] * per <= it.at) lo = mid;
      else hi = mid - 1;
    }
    enter(lo);
  } else if (it.give) {  // (its writers have made it visible before the barrier in front of this)
    __threadfence();
    if (!a.withheld) atomicExch(a.given + share, 1u);
  }
  it.take = it.give = false;
  for (;;) {
    it.any = it.at < it.end;
    if (!it.any) return;
    if (it.at >= it.behind) enter(it.seq + 1);  // (each of them takes something)
    const int rest = static_cast<int>((it.at - it.begin) % it.cost), task = static_cast<int>((it.at - it.begin) / it.cost);
    const int64_t behind = it.at - rest + it.cost;
    it.from = 0;
    it.to = it.cost - 1;
    if (rest > 0) {  // another block has its last chunks
      it.to = it.cost - rest - 1;
      it.at = behind;
      if (it.to == 0) continue;  // all of them
      it.give = true;
    } else if (behind > it.end) {
      it.from = static_cast<int>(behind - it.end) - 1;
      it.take = it.from > 0;
      it.at = it.end;
    } else {
      it.at = behind;
    }
    it.h = task / a.slices;
    it.v0 = task % a.slices * across;
    break;
  }
  if (!it.take) return;
  const long long begun = clock64();
  for (;;) {
    uint32_t there;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(there) : "l"(a.given + share + 1) : "memory");
    if (there) return;
    if (clock64() - begun > kWaitBudgetCycles) {
      if (a.status != nullptr) atomicOr(a.status, ENGRAM_ST_TIMEOUT);
      return;
    }
    __nanosleep(200);
  }
}
// A thread's part of a state that is handed on.
template <int N>
__device__ __forceinline__ void give_state(float* between, const float (&S)[N][4], int threads) {
  float4* to = reinterpret_cast<float4*>(between) + threadIdx.x;
#pragma unroll
  for (int t = 0; t < N; ++t) to[t * threads] = make_float4(S[t][0], S[t][1], S[t][2], S[t][3]);
  __threadfence();
}
template <int N>
__device__ __forceinline__ void take_state(const float* between, float (&S)[N][4], int threads) {
  const float4* from = reinterpret_cast<const float4*>(between) + threadIdx.x;
#pragma unroll
  for (int t = 0; t < N; ++t) {
    const float4 x = __ldcg(from + t * threads);
    S[t][0] = x.x; S[t][1] = x.y; S[t][2] = x.z; S[t][3] = x.w;
  }
}

template <class E>
__device__ __forceinline__ size_t unit_of(const Args<E>& a, int chunk, int head) {
  return static_cast<size_t>(chunk) * a.heads + head;
}

// Behind the states, `carry` has the writes U, [n_tokens][heads*dv]: fp32, or for inputs of
// type bf16 two terms, one array behind the other.
template <class E>
__device__ __forceinline__ typename E::T* kept_writes(const Args<E>& a) {
  return reinterpret_cast<typename E::T*>(a.carry + static_cast<size_t>(a.max_chunks) * a.heads * saved_floats<E>(a.dk, a.dv));
}

// Behind those the chunks' triangles and gates, where either type's have their place.
inline size_t kept_triangles_at(int64_t n_tokens, int64_t chunks, int32_t heads, int32_t dk, int32_t dv) {  // bytes
  const size_t floats =
      static_cast<size_t>(chunks) * heads * saved_floats<train::Bf16>(dk, dv) + static_cast<size_t>(n_tokens) * heads * dv;
  return (floats * sizeof(float) + 15) & ~size_t(15);
}
template <class E>
void use_kept_triangles(Args<E>& a) {
  a.tri = reinterpret_cast<unsigned char*>(a.carry) + kept_triangles_at(a.n_tokens, a.max_chunks, a.heads, a.dk, a.dv);
  a.gates = reinterpret_cast<Gates*>(a.tri + static_cast<size_t>(a.max_chunks) * a.heads * kTriBytes);
}

// The outputs (y, or the values' gradient) of a sequence without a slot, and the states
// that it would have left for the backward pass.
template <class E>
__device__ __forceinline__ void padding_zeros(const Args<E>& a, int lo, int hi, int c0, int n, int h, int v0, int cols, int threads) {
  auto* out = a.y != nullptr ? a.y : a.dv_out;
  const int64_t stride = a.y != nullptr ? a.y_stride : a.dv_stride;
  for (int64_t i = threadIdx.x; i < static_cast<int64_t>(hi - lo) * cols; i += threads)
    E::store(out + (lo + i / cols) * stride + h * a.dv + v0 + i % cols, 0.f);
  if (a.y == nullptr || a.carry == nullptr) return;
  const int64_t wide = static_cast<int64_t>(a.heads) * a.dv;
  for (int64_t i = threadIdx.x; i < static_cast<int64_t>(hi - lo) * cols; i += threads) {
    auto* to = kept_writes<E>(a) + (lo + i / cols) * wide + static_cast<int64_t>(h) * a.dv + v0 + i % cols;
    E::store(to, 0.f);
    if (E::kBytes == 2) E::store(to + a.n_tokens * wide, 0.f);
  }
  const size_t saved = saved_floats<E>(a.dk, a.dv), at = v0 == 0 ? 0 : saved_floats<E>(a.dk, v0);
  const size_t mine = saved_floats<E>(a.dk, cols);
  for (int c = 0; c < n; ++c)
    for (size_t i = threadIdx.x; i < mine; i += threads) a.carry[unit_of(a, c0 + c, h) * saved + at + i] = 0.f;
}

// 16 of a chunk's rows, r0 on, of a quad's 16 columns, held transposed; masked rows (beta
// 0) get zeros.  `to` is the chunk's first row's column 0 of the head.
template <class E>
__device__ __forceinline__ void store_rows(typename E::T* to, int64_t stride, int r0, int len, int vw, int dv, bool pairs,
                                           const float* beta, const float (&y)[2][4]) {
  const int lane = lane_id(), g = lane >> 2, t2 = (lane & 3) * 2;
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if constexpr (E::kBytes == 2) {
        const uint32_t w = transposed(pack(y[t][2 * j], y[t][2 * j + 1]));  // row t * 8 + g, columns t2, t2 + 1
        const int r = r0 + t * 8 + g, v = vw + j * 8 + t2;
        if (r >= len) continue;
        const uint32_t x = beta[r] != 0.f ? w : 0u;
        typename E::T* at = to + r * stride + v;
        if (pairs) {
          if (v < dv) *reinterpret_cast<uint32_t*>(at) = x;
        } else {
          if (v < dv) at[0] = static_cast<uint16_t>(x);
          if (v + 1 < dv) at[1] = static_cast<uint16_t>(x >> 16);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = r0 + t * 8 + t2 + e, v = vw + j * 8 + g;
          if (r < len && v < dv) E::store(to + r * stride + v, beta[r] != 0.f ? y[t][2 * j + e] : 0.f);
        }
      }
    }
}

// ------------------------------------------------------------------- quads

// Four warps, a quad, follow a sequence in a head for 16 of the value columns.  The
// state is held transposed, S^T [16][dk], a quarter of its rows a warp, as an accumulator;
// an accumulator is the next product's operand A as it lies in the registers (see
// as_operand), so what the warps hand to one another are operands: 512 bytes a term,
// 16 a lane, written and read without conflicts.  Each warp makes a quarter of the
// chunk's positions of K S, U and Y, and its own rows of the state.  A block's quads share
// the chunk's inputs; their warps' roles are turned by one from quad to quad, so that the
// triangles' short and long rows are spread over the SM's four parts.
__device__ __forceinline__ void quad_sync(int quad) { asm volatile("bar.sync %0, 128;" ::"r"(quad + 1) : "memory"); }
// A block of one quad has more warps: four for the copies and, forwards, four for Y.  The
// quad's own, one on each of the SM's four parts, are bound by the instructions that they
// issue one after another (one sequence of 16,381 positions in 10 heads, us: 745 without
// either, 546 with those for the copies, 520 with both).
template <int NQ>
constexpr bool kAlone = NQ == 1;
constexpr int kCopiers = 128;
// The quads of a block of four go on by themselves, as far as the two stages of the chunks'
// inputs let them: `here` counts the threads whose copies have come, `done` the warps that
// no longer need a stage.  (201 chunks one after another, forwards: 1161 us with a barrier of
// the block at each, 1121 so.)
struct Stages {
  uint64_t here[2], done[2];
  int late;   // whether a wait has run out
  int begun;  // how often a stage's copies have been begun (its first thread's)
};
__device__ __forceinline__ void stages_begin(Stages& s, int threads, int warps) {
  if (threadIdx.x == 0) {
    for (int k = 0; k < 2; ++k) {
      mbar_init(smem_u32(&s.here[k]), threads + 1);
      mbar_init(smem_u32(&s.done[k]), warps);
    }
    s.late = s.begun = 0;
    fence_mbar_init();
  }
  __syncthreads();
}
// Where a wait runs out, that is reported, and the block goes to its end: no other wait lasts,
// and no thread arrives at a stage's barrier any more, whose phase may not have ended.
__device__ __forceinline__ bool stages_late(const Stages& s) { return *reinterpret_cast<const volatile int*>(&s.late) != 0; }
__device__ __forceinline__ void stage_wait(Stages& s, uint64_t& bar, int use, int32_t* status) {
  if (mbar_try_wait(smem_u32(&bar), use & 1)) return;
  if (stages_late(s) || mbar_wait_bounded(smem_u32(&bar), use & 1, &s.late)) return;
  *reinterpret_cast<volatile int*>(&s.late) = 1;
  if (status != nullptr) atomicOr(status, ENGRAM_ST_TIMEOUT);
}
// The rest of a stage behind its rows: the triangles (`tri` bytes) and gates by one thread's
// bulk copies.  A thread's own copies of rows count when they have come.
__device__ __forceinline__ void stage_copies(Stages& s, int stage, uint32_t to_tri, const unsigned char* from_tri, int tri,
                                             uint32_t to_gates, const Gates* from_gates, bool vec, uint32_t absent) {
  const uint32_t bar = smem_u32(&s.here[stage]);
  const bool on = !stages_late(s);
  if (threadIdx.x == 0 && on) {
    ++s.begun;
    mbar_arrive_expect_tx(bar, tri + static_cast<int>(sizeof(Gates)) + absent);
    bulk_g2s(to_tri, from_tri, tri, bar);
    bulk_g2s(to_gates, from_gates, sizeof(Gates), bar);
  }
  if (vec && on) asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(bar) : "memory");
  else if (on) mbar_arrive(bar);
}
// Copies that were begun and not waited for land before the shared memory is released: a
// thread's own, and the first thread's bulk copies of the last two stages, for which it waits
// as long as any wait lasts.
__device__ __forceinline__ void stages_end(Stages& s) {
  if (!stages_late(s)) return;
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (threadIdx.x != 0) return;
  for (int use = max(s.begun - 2, 0); use < s.begun; ++use) mbar_wait_bounded(smem_u32(&s.here[use & 1]), use >> 1 & 1, nullptr);
}
template <int N>
__device__ __forceinline__ void hand(uint32_t at, const uint32_t (&f)[N][4]) {
#pragma unroll
  for (int n = 0; n < N; ++n)
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at + n * 512 + lane_id() * 16), "r"(f[n][0]), "r"(f[n][1]),
                 "r"(f[n][2]), "r"(f[n][3])
                 : "memory");
}
template <int N>
__device__ __forceinline__ void take(uint32_t at, uint32_t (&f)[N][4]) {
#pragma unroll
  for (int n = 0; n < N; ++n)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(f[n][0]), "=r"(f[n][1]), "=r"(f[n][2]), "=r"(f[n][3])
                 : "r"(at + n * 512 + lane_id() * 16)
                 : "memory");
}
// Tiles of 8 columns that accumulate a product.  Where 24 bits are to be kept the small
// terms' products have accumulators of their own (see `product`).
template <int N, bool kApart>
struct Sums {
  float main[N][4], small[kApart ? N : 1][4];
  __device__ __forceinline__ void clear_all() {
    clear(main);
    if constexpr (kApart) clear(small);
  }
  // terms i of A and j of B
  __device__ __forceinline__ void add(int i, int j, const uint32_t (&a)[4], const uint32_t (*b)[2]) {
#pragma unroll
    for (int t = 0; t < N; ++t) {
      if constexpr (kApart) mma(i + j == 0 ? main[t] : small[t], a, b[t][0], b[t][1]);
      else mma(main[t], a, b[t][0], b[t][1]);
    }
  }
  __device__ __forceinline__ float sum(int t, int j) const {
    if constexpr (kApart) return main[t][j] + small[t][j];
    else return main[t][j];
  }
};
template <int TA, int kLimit, int N, bool kApart>
__device__ __forceinline__ void terms(Sums<N, kApart>& c, const uint32_t (&a)[TA][4], const uint32_t (&b)[N][2], int j) {
#pragma unroll
  for (int i = 0; i < TA; ++i)
    if (i + j < kLimit) c.add(i, j, a[i], b);
}

// ------------------------------------------------------------ host: launches

// The space behind a call's chunks.
struct Space {
  int32_t* first;
  int64_t* line;
  uint32_t* given;
  float* between;
  unsigned char* tri;
  Gates* gates;
  float* after;
  uint16_t* writes;
  float* shared;
  size_t bytes;
};
inline int64_t max_chunks(int64_t n_tokens, int64_t n_seqs) {
  return std::min(n_tokens, (n_tokens + (kC - 1) * n_seqs) / kC);
}
Space space(void* base, int64_t n_tokens, int64_t n_seqs, int32_t keys, int32_t heads, int32_t dk, int32_t dv, bool backward);

// The chunks' numbers and the blocks' shares of them.
template <class E>
int launch_first(const Args<E>& a, cudaStream_t st);

inline int opt_in(const void* kernel, int smem, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaGetDevice(&dev);
  const uint64_t bit = dev < 64 ? (uint64_t(1) << dev) : 0;
  if (bit != 0 && (done.load(std::memory_order_relaxed) & bit)) return ENGRAM_OK;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return fail(ENGRAM_E_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
  done.fetch_or(bit, std::memory_order_relaxed);
  return ENGRAM_OK;
}

// What the call of this thread leaves out for engram_selftest_delta_wait: 1 bytes of a stage,
// 2 the word that a state has been handed on.
extern thread_local int selftest_absent;
template <class E>
void set_absent(Args<E>& a) {
  a.absent = selftest_absent == 1 ? 16 : 0;
  a.withheld = selftest_absent == 2;
}

inline int slices_of(int dv, int quads) { return (dv + 16 * quads - 1) / (16 * quads); }

// Quads of a block: four, which share the copies of a chunk's inputs, where such blocks
// come to three quarters of the SMs or more; else one, so that few sequences and heads
// spread over more SMs.  (dk = dv = 128, bf16: a chunk takes a block of four quads 5.6 us
// and one of one 2.0, measured forwards: four blocks of one on an SM one after another
// take 8.0, three 6.0.)  Sequences are counted and not measured, as their lengths are not
// known here: where one is much longer than all others together, one quad would be
// better also for many (16,381 positions in 10 heads 580 us, with five sequences of 10
// beside them, which make it four quads, 1434; backwards 1099 and 2221).
template <class E>
bool many_quads(const Args<E>& a, int sms) {
  return E::kBytes == 2 && static_cast<int64_t>(a.n_seqs) * a.heads * slices_of(a.dv, 4) * 4 >= 3 * static_cast<int64_t>(sms);
}
// The blocks that follow the sequences: one on each SM at most (their shared memory and
// registers leave no room for two).
template <class E>
void set_blocks(Args<E>& a, int sms) {
  a.slices = slices_of(a.dv, many_quads(a, sms) ? 4 : 1);
  a.blocks = static_cast<int32_t>(
      std::min<int64_t>(std::min(sms, kMaxBlocks), static_cast<int64_t>(a.n_seqs) * a.heads * a.slices));
}

inline bool pieces(const void* p, int64_t stride, int bytes) { return aligned(p, 16) && stride * bytes % 16 == 0; }

inline int check_sizes(int32_t type, int64_t n_tokens, int32_t keys, int32_t heads, int32_t dk, int32_t dv, int64_t n_seqs,
                int64_t n_slots, bool has_state, float scale) {
  if (!train::known_type(type)) return fail(ENGRAM_E_INVALID, "type %d is not ENGRAM_T_BF16 or ENGRAM_T_F32", type);
  if (n_tokens < 0 || n_seqs < 0) return fail(ENGRAM_E_INVALID, "negative number of positions or sequences");
  if (n_tokens > 0x7ffffc00 || n_seqs > 0x7ffffc00) return fail(ENGRAM_E_RANGE, "too many positions or sequences");
  if (keys < 1 || heads < keys || heads % keys != 0 || heads > 65535)
    return fail(ENGRAM_E_SHAPE, "value heads must be a multiple of the key heads, and at most 65535");
  if (dk < 1 || dk > kMaxDim || dv < 1 || dv > kMaxDim) return fail(ENGRAM_E_SHAPE, "head widths must be in [1, %d]", kMaxDim);
  if (has_state && n_slots < 1) return fail(ENGRAM_E_INVALID, "a state needs n_slots >= 1");
  if (!(scale >= -3.0e38f && scale <= 3.0e38f)) return fail(ENGRAM_E_INVALID, "scale must be finite");
  return ENGRAM_OK;
}

inline int check_rows(const void* p, int32_t type, int64_t stride, int64_t width, const char* name) {
  if (stride < width) return fail(ENGRAM_E_SHAPE, "%s: row stride below its width", name);
  if (p == nullptr) return fail(ENGRAM_E_INVALID, "null device pointer: %s", name);
  if (!aligned(p, train::type_bytes(type))) return fail(ENGRAM_E_ALIGN, "%s must be aligned to its elements", name);
  return ENGRAM_OK;
}

}  // namespace delta
}  // namespace engram
