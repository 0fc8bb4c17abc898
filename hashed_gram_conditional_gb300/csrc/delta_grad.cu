// The gradients of the gated delta rule.
//
// With the names of delta_device.cuh, dS the gradient of the state behind a chunk
// and dV = M^T (P^T dY + e^(c_last - c) K dS):
//   dS <- e^c_last dS + Q^T (scale e^c dY) - K^T (e^c dV)       chunk after chunk, from the last
// and then, for all chunks at once, with F = scale D (dY U^T) on and below the
// diagonal and E = -D (dV U^T) below it:
//   dQ = scale e^c dY S^T + F K
//   dK = -e^c dV S^T + e^(c_last - c) U dS^T + E K + E^T K + F^T Q
//   db_t = (dV_t . U_t) (1 - beta_t) / beta_t
//   dg_t = (1 - f_t) (what crosses t: reads of S at t and later, writes before t that
//          reach dS, pairs of the two of them, and e^c_last S . dS)
// The states in front of the chunks, U, M and P come from the forward pass.  (M and P made
// again took 55 of 1020 us for 4096 positions of 40 heads, both passes together; they are a
// quarter of what is kept, and would take the same room here while they are used.)
#include "delta_device.cuh"

namespace engram {
namespace delta {
namespace {

// ------------------------------------------------ the state's gradient, backwards

// A quad goes backwards as scan_kernel's go forwards, with dS^T in its registers.  (4096
// positions in 7 sequences, 40 heads of 128, bf16: 287 us; the tensor cores are busy for
// 40 % of the time and shared memory for 66.)
template <class E, int KD, int NQ>
struct Back {
  static constexpr int kT = kAlone<NQ> ? kCopiers : NQ * 128, kThreads = kAlone<NQ> ? 128 + kCopiers : kT;
  static constexpr int kStages = E::kBytes == 2 ? 2 : 1, kB = kC / 16;
  static constexpr int kK = 0, kQ = kK + kIn<E> * mat_bytes(kC, KD), kY = kQ + kIn<E> * mat_bytes(kC, KD);
  static constexpr int kM = kY + kIn<E> * mat_bytes(kC, 16 * NQ), kP = kM + kStateTerms * kTerm, kG = kP + kStateTerms * kTerm;
  static constexpr int kStage = kG + static_cast<int>(sizeof(Gates)), kQuads = kStages * kStage;
  // a quad's operands: dS^T, then in its place (scale e^c dY)^T; dU^T, then (-e^c dV)^T
  static constexpr int kR = 0, kState = (KD / 16 > kB ? KD / 16 : kB) * kStateTerms * 512, kU = kState;
  static constexpr int kQuad = kU + kB * kStateTerms * 512;
  static constexpr int kSmem = kQuads + NQ * kQuad;
};

template <class E, int KD, int NQ>
__global__ void __launch_bounds__(Back<E, KD, NQ>::kThreads, 1) back_kernel(Args<E> a) {
  using L = Back<E, KD, NQ>;
  constexpr int kT = L::kT, kI = kIn<E>, kS = kStateTerms, kB = L::kB, kR = KD / 64;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ Stages stages;
  __shared__ Item item;
  const uint32_t base = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, g = lane >> 2, t2 = (lane & 3) * 2;
  const int quad = kAlone<NQ> ? 0 : tid >> 7, w = ((tid >> 5) + quad) & 3;
  const size_t matrix = static_cast<size_t>(a.dk) * a.dv, saved = saved_floats<E>(a.dk, a.dv);
  if (tid == 0) {
    item.seq = -1;
    item.give = false;
  }
  if (!kAlone<NQ>) stages_begin(stages, kT, kT / 32);
  for (int used = 0;;) {  // (used: how often the stages have been)
    __syncthreads();
    if (tid == 0) next_item(a, item, 16 * NQ);
    __syncthreads();
    if (!item.any) break;
    // its chunks, from the last of the sequence's backwards: first, first - 1, .. last
    const int h = uniform(item.h), v0 = uniform(item.v0), lo = uniform(item.lo), hi = uniform(item.hi), c0 = uniform(item.c0);
    const int first = uniform(item.n - 1 - item.from), last_one = uniform(item.n - item.to);
    const int cols = min(a.dv - v0, 16 * NQ);
    const int hk = h / (a.heads / a.keys), vw = v0 + quad * 16;
    int64_t slot;
    if (!live_slot(a, item.seq, c0, item.n, slot)) {
      if (tid == 0 && h == 0 && v0 == 0 && a.status != nullptr && slot >= 0) atomicOr(a.status, ENGRAM_ST_BAD_SLOT);
      padding_zeros(a, lo, hi, c0, item.n, h, v0, cols, blockDim.x);
      continue;
    }
    const uint32_t own = base + L::kQuads + quad * L::kQuad;
    float S[2 * kR][4];
    auto each = [&](auto f) {  // f(tile, place, the element's place in a state)
#pragma unroll
      for (int t = 0; t < 2 * kR; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int v = vw + g + (j >> 1) * 8, k = w * kR * 16 + t * 8 + t2 + (j & 1);
          if (v < a.dv && k < a.dk) f(t, j, static_cast<size_t>(k) * a.dv + v);
        }
    };
    const int share = gridDim.x - 1 - blockIdx.x;
    auto stage_of = [&](int i) { return kAlone<NQ> ? i % L::kStages : (used + first - i) & 1; };
    auto hand_state = [&](int i) {  // the gradient of the state behind chunk i
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        const int kb = w * kR + r;
        uint32_t f[kS][4];
        as_operand<kS>(f, S[2 * r], S[2 * r + 1]);
        hand<kS>(own + kb * (kS * 512), f);
        if (vw >= a.dv || kb * 16 >= a.dk) continue;
        float* to = a.after + unit_of(a, c0 + i, h) * saved;
        if constexpr (E::kBytes == 2) save_block(block_of(to, a.dk, vw >> 4, kb), f);
        else save_rows(to, a.dk, a.dv, vw, kb * 16, S[2 * r], S[2 * r + 1]);
      }
    };
    const int copier = tid - (kAlone<NQ> ? NQ * 128 : 0);  // a copying thread's number
    auto load = [&](int i) {
      const uint32_t stage = base + stage_of(i) * L::kStage;
      const int64_t p = lo + static_cast<int64_t>(i) * kC;
      const int len = hi - p < kC ? static_cast<int>(hi - p) : kC;
      const uint8_t* mask = a.mask != nullptr ? a.mask + p : nullptr;
      const size_t unit = unit_of(a, c0 + i, h);
      load_rows<E, KD, kT>(mat<kC, KD>(stage + L::kK), a.k + p * a.k_stride + hk * a.dk, a.k_stride, len, a.dk, mask, a.vec, copier);
      load_rows<E, KD, kT>(mat<kC, KD>(stage + L::kQ), a.q + p * a.q_stride + hk * a.dk, a.q_stride, len, a.dk, mask, a.vec, copier);
      load_rows<E, 16 * NQ, kT>(mat<kC, 16 * NQ>(stage + L::kY), a.dy + p * a.dy_stride + static_cast<int64_t>(h) * a.dv + v0,
                                a.dy_stride, len, cols, mask, a.vec, copier);
      if constexpr (kAlone<NQ>) {
        load_tri<kS, kT>(stage + L::kM, stage + L::kP, a.tri + unit * kTriBytes, copier);
        load_gates<kT>(stage + L::kG, a.gates + unit, copier);
        copies_begun();
      } else {
        stage_copies(stages, stage_of(i), stage + L::kM, a.tri + unit * kTriBytes, 2 * kS * kTerm, stage + L::kG, a.gates + unit,
                     a.vec, a.absent);
      }
    };
    if (kAlone<NQ> && copier >= 0) {
      if (first >= last_one) load(first);
      for (int i = first; i >= last_one; --i) {
        copies_done();
        __syncthreads();
        if (L::kStages == 1 && i > last_one) __syncthreads();
        if (i > last_one) load(i - 1);
      }
      continue;
    }
    if (!kAlone<NQ> && first >= last_one) load(first);
    clear(S);
    if (item.take) {
      take_state(a.between + static_cast<size_t>(share + 1) * kHandedOn, S, NQ * 128);
    } else if (a.state_out != nullptr) {
      const float* given = a.state_out + (slot * a.heads + h) * matrix;
      each([&](int t, int j, size_t at) { S[t][j] = given[at]; });
    }
    if (first >= last_one) hand_state(first);
    for (int i = first; i >= last_one; --i) {
      const uint32_t stage = base + stage_of(i) * L::kStage;
      const Mat K = mat<kC, KD>(stage + L::kK), Q = mat<kC, KD>(stage + L::kQ), Y = mat<kC, 16 * NQ>(stage + L::kY);
      const Gates& gt = *reinterpret_cast<const Gates*>(smem + stage_of(i) * L::kStage + L::kG);
      if constexpr (kAlone<NQ>) {
        __syncthreads();  // the chunk and the states' gradients are here, and the other stage is free
      } else {
        quad_sync(quad);  // the states' gradients are here
        stage_wait(stages, stages.here[stage_of(i)], (used + first - i) >> 1, a.status);
      }
      float2 into[2], last[2];  // of the warp's positions
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        into[t] = *reinterpret_cast<const float2*>(&gt.into[w * 16 + t * 8 + t2]);
        last[t] = *reinterpret_cast<const float2*>(&gt.last[w * 16 + t * 8 + t2]);
      }
      // ---- dU^T = e^(c_last - c) (K dS)^T + dY^T P
      Sums<2, true> x;
      x.clear_all();
#pragma unroll 4
      for (int kb = 0; kb < KD / 16; ++kb) {
        uint32_t fa[kS][4];
        take<kS>(own + kb * (kS * 512), fa);
#pragma unroll
        for (int j = 0; j < kI; ++j) {
          uint32_t fb[2][2];
          Across{K}.get<2>(fb, kb * 16, w * 16, j);
          terms<kS, kS>(x, fa, fb, j);
        }
      }
      float u[2][4];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) u[t][j] = x.sum(t, j) * (j & 1 ? last[t].y : last[t].x);
      x.clear_all();
      for (int tb = w; tb < kB; ++tb) {
        uint32_t fa[kI][4];
#pragma unroll
        for (int j = 0; j < kI; ++j) Cols{Y}(fa[j], quad * 16, tb * 16, j);
#pragma unroll
        for (int j = 0; j < kS; ++j) {
          uint32_t fb[2][2];
          TriDown{stage + L::kP}.get(fb, tb, w, j);
          terms<kI, kS>(x, fa, fb, j);
        }
      }
      {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j) u[t][j] += x.sum(t, j);
        uint32_t f[kS][4];
        as_operand<kS>(f, u[0], u[1]);
        hand<kS>(own + L::kU + w * (kS * 512), f);
      }
      quad_sync(quad);  // and dS^T is no longer needed
      {
        float r[2][4];
        clear(r);
#pragma unroll
        for (int j = kI - 1; j >= 0; --j) {
          uint32_t f[4];
          Cols{Y}(f, quad * 16, w * 16, j);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            r[q >> 1][(q & 1) * 2] += lo_of(f[q]);
            r[q >> 1][(q & 1) * 2 + 1] += hi_of(f[q]);
          }
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j) r[t][j] *= a.scale * (j & 1 ? into[t].y : into[t].x);
        uint32_t f[kS][4];
        as_operand<kS>(f, r[0], r[1]);
        hand<kS>(own + L::kR + w * (kS * 512), f);
      }
      // ---- dV^T = dU^T M
      x.clear_all();
      for (int tb = w; tb < kB; ++tb) {
        uint32_t fa[kS][4];
        take<kS>(own + L::kU + tb * (kS * 512), fa);
#pragma unroll
        for (int j = 0; j < kS; ++j) {
          uint32_t fb[2][2];
          TriDown{stage + L::kM}.get(fb, tb, w, j);
          terms<kS, kS>(x, fa, fb, j);
        }
      }
      float rest[2][4];  // what the output's rounding leaves
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          u[t][j] = x.sum(t, j);
          rest[t][j] = u[t][j] - lo_of(pack(u[t][j], 0.f));
        }
      {
        float c[2][4];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j) c[t][j] = -u[t][j] * (j & 1 ? into[t].y : into[t].x);
        uint32_t f[kS][4];
        as_operand<kS>(f, c[0], c[1]);
        quad_sync(quad);  // dU^T is no longer needed
        hand<kS>(own + L::kU + w * (kS * 512), f);
      }
      if (!kAlone<NQ> && i > last_one) {
        if (i < first) stage_wait(stages, stages.done[stage_of(i - 1)], (used + first - i - 1) >> 1, a.status);
        load(i - 1);
      }
      quad_sync(quad);
      // ---- dS^T
      {
        const float total = gt.into[kC - 1];
        Sums<2 * kR, true> d;
        d.clear_all();
#pragma unroll
        for (int cb = 0; cb < kB; ++cb) {
          uint32_t fr[kS][4], fw[kS][4];
          take<kS>(own + L::kR + cb * (kS * 512), fr);
          take<kS>(own + L::kU + cb * (kS * 512), fw);
#pragma unroll
          for (int j = 0; j < kI; ++j) {
            uint32_t fb[2 * kR][2];
            Down{Q}.get<2 * kR>(fb, cb * 16, w * kR * 16, j);
            terms<kS, kS>(d, fr, fb, j);
            Down{K}.get<2 * kR>(fb, cb * 16, w * kR * 16, j);
            terms<kS, kS>(d, fw, fb, j);
          }
        }
#pragma unroll
        for (int t = 0; t < 2 * kR; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j) S[t][j] = fmaf(S[t][j], total, d.sum(t, j));
      }
      if (i > last_one) {
        quad_sync(quad);  // the operands have been taken
        hand_state(i - 1);
      }
      const int64_t p = lo + static_cast<int64_t>(i) * kC;
      const int len = hi - p < kC ? static_cast<int>(hi - p) : kC;
      store_rows<E>(a.dv_out + p * a.dv_stride + static_cast<int64_t>(h) * a.dv, a.dv_stride, w * 16, len, vw, a.dv, a.pairs,
                    gt.beta, u);
      if constexpr (E::kBytes == 2) {
        const int64_t wide = static_cast<int64_t>(a.heads) * a.dv;
        auto* to = a.writes + p * wide + static_cast<int64_t>(h) * a.dv;
        store_rows<E>(to, wide, w * 16, len, vw, a.dv, a.dv % 2 == 0, gt.beta, rest);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j) rest[t][j] -= lo_of(pack(rest[t][j], 0.f));
        store_rows<E>(to + a.n_tokens * wide, wide, w * 16, len, vw, a.dv, a.dv % 2 == 0, gt.beta, rest);
      }
      if constexpr (kAlone<NQ>) {
        if (L::kStages == 1 && i > last_one) __syncthreads();  // the stage is free
      } else {
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&stages.done[stage_of(i)]));
      }
    }
    used += first + 1 - last_one;
    if (item.give) {
      give_state(a.between + static_cast<size_t>(share) * kHandedOn, S, NQ * 128);
    } else if (a.state_out != nullptr) {
      float* to = a.state_out + (slot * a.heads + h) * matrix;
      each([&](int t, int j, size_t at) { to[at] = S[t][j]; });
    }
  }
  if (!kAlone<NQ>) stages_end(stages);
}

// ------------------------------------------------------- all chunks' gradients

// A block has one chunk and the heads of one key head, one after another, and a head's
// value columns in slices of VS.  The next slice's inputs are copied while this one is
// used (bf16: all of them are operands as they lie in memory; fp32 are made terms on
// the way).  A warp has 16 rows and a part of the columns of each product: a quarter, or
// of type fp32, whose operands take more registers, half.  (The same 4096 x 40: 393 us, of
// which the tensor cores are busy for 35 %; the rest is the instructions of a head's end,
// where F and E are made, and the barriers around them.  Making U again in place of reading
// it took 561 us: two more barriers a slice.)
//
// dV is three terms for either type.  Where a write overwrites what its key held (beta near
// 1, keys that come back), dg is what is left of reads by queries and by corrections that
// cancel, and what does not cancel is dV's rounding: S, dS and U are the same in both.  With
// 16 bits of dV, and the products of second terms left out, dg was off by 2.3 % for one key
// again and again at beta = 0.9997, where it is off by 0.24 % (bf16's own rounding: 0.17 %);
// this kernel took 353 us and the backward scan 274.
template <class E, int KD, int VS>
struct Grads {
  static constexpr int kO = kOut<E>, kWT = kStateTerms, kStages = E::kBytes == 2 ? 2 : 1, kParts = E::kBytes == 2 ? 4 : 2;
  static constexpr int kT = 4 * kParts * 32;  // threads
  static constexpr int kK = 0, kQ = kK + kIn<E> * mat_bytes(kC, KD);
  static constexpr int kHead = kQ + kIn<E> * mat_bytes(kC, KD);  // the gates, of this head and the next
  static constexpr int kHeadBytes = static_cast<int>(sizeof(Gates));
  static constexpr int kNum = kHead + kStages * kHeadBytes;                   // sums
  static constexpr int kSums = kParts * kC * 4 + 4 * kC + 4 * kParts;         // floats
  static constexpr int kF = (kNum + kSums * 4 + 127) / 128 * 128, kE = kF + kO * mat_bytes(kC, kC);
  static constexpr int kEndF = kE + kO * mat_bytes(kC, kC);
  static constexpr int kSlice = kStages == 2 ? kEndF : kF;  // (fp32: F and E lie over the slice)
  // a slice of the value columns: S^T, dS^T, dY, dV, U
  static constexpr int kState = E::kBytes == 2 ? VS / 16 * (KD / 16) * kBlockBytes : kO * mat_bytes(VS, KD);
  static constexpr int kS = 0, kD = kS + kState, kY = kD + kState, kW = kY + kIn<E> * mat_bytes(kC, VS);
  static constexpr int kU = kW + kWT * mat_bytes(kC, VS), kSliceBytes = kU + kO * mat_bytes(kC, VS);
  static constexpr int kEnd = kSlice + kStages * kSliceBytes, kSmem = kEnd > kEndF ? kEnd : kEndF;
  static constexpr int kCN = kC / 8 / kParts, kKN = KD / 8 / kParts;  // a warp's tiles of 8 columns
};

// `cols` columns of a saved state, from column v0 on, zeros around them.
template <class E, int KD, int VS, int kT>
__device__ __forceinline__ void load_state(uint32_t to, const float* from, int v0, int cols, int dk) {
  if constexpr (E::kBytes == 2) {
    // blocks as they lie, and zeros where the head has none
    const int across = (dk + 15) / 16;
    const uint32_t* blocks = reinterpret_cast<const uint32_t*>(from) + static_cast<size_t>(v0 / 16) * across * (kBlockBytes / 4);
#pragma unroll
    for (int i0 = 0; i0 < VS / 16 * (KD / 16) * (kBlockBytes / 16); i0 += kT) {
      const int i = i0 + threadIdx.x, b = i / (kBlockBytes / 16), vb = b / (KD / 16), kb = b % (KD / 16);
      const bool on = vb * 16 < cols && kb < across;
      copy16(to + i * 16, on ? blocks + (vb * across + kb) * (kBlockBytes / 4) + i % (kBlockBytes / 16) * 4 : blocks, on);
    }
  } else {
    const Mat m = mat<VS, KD>(to);
    from += static_cast<size_t>(v0) * dk;
    constexpr int kAhead = 4;
    for (int i0 = threadIdx.x; i0 < VS * (KD / 2); i0 += kAhead * kT) {
      float x[kAhead][2];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = i0 + u * kT, r = i / (KD / 2), c = i % (KD / 2) * 2;
        const float* p = from + static_cast<size_t>(r) * dk + c;
        x[u][0] = r < cols && c < dk ? p[0] : 0.f;
        x[u][1] = r < cols && c + 1 < dk ? p[1] : 0.f;
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = i0 + u * kT, r = i / (KD / 2), c = i % (KD / 2) * 2;
        if (r < VS) put<kOut<E>>(m.base + r * m.pitch + c * 2, m.term, x[u][0], x[u][1]);
      }
    }
  }
}

// S^T in shared memory as an operand B, its columns as k.
template <class E, int KD, int VS>
__device__ __forceinline__ auto state_down(uint32_t at) {
  if constexpr (E::kBytes == 2) return BlocksDown{at, KD / 16};
  else return Down{mat<VS, KD>(at)};
}

// c += A B and d += A2 B, of TA, TB and (A2) TD terms, over k from 0 to k1: the products
// below 2^-8 TB of the first one are left out for A, those below 2^-8 TD for A2
template <int TA, int TB, int TD, int N, class A, class A2, class B>
__device__ __forceinline__ void both_products(float (&c)[N][4], float (&d)[N][4], const A& a, const A2& a2, const B& b, int m,
                                              int n, int k1) {
  if constexpr (TA == TB) {
    product<TA, TB, TB>(c, a, b, m, n, 0, k1);
    product<TD, TB, TD>(d, a2, b, m, n, 0, k1);
  } else {
#pragma unroll
    for (int k = 0; k < k1; k += 16) {
      uint32_t fa[TA][4], fd[TD][4];
#pragma unroll
      for (int i = 0; i < TA; ++i) a(fa[i], m, k, i);
#pragma unroll
      for (int i = 0; i < TD; ++i) a2(fd[i], m, k, i);
#pragma unroll
      for (int j = 0; j < TB; ++j) {
        uint32_t fb[N][2];
        b.template get<N>(fb, k, n, j);
#pragma unroll
        for (int i = 0; i < TD; ++i) {
#pragma unroll
          for (int t = 0; t < N; ++t) {
            if (i < TA && i + j < TB) mma(c[t], fa[i < TA ? i : 0], fb[t][0], fb[t][1]);
            if (i + j < TD) mma(d[t], fd[i], fb[t][0], fb[t][1]);
          }
        }
      }
    }
  }
}

__device__ __forceinline__ void ld128(uint32_t (&x)[4], uint32_t at) {
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(at) : "memory");
}
// four neighbouring values of N terms
template <int N>
__device__ __forceinline__ void get4(uint32_t at, int term, float (&x)[4]) {
  x[0] = x[1] = x[2] = x[3] = 0.f;
#pragma unroll
  for (int n = N - 1; n >= 0; --n) {
    uint32_t w0, w1;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w0), "=r"(w1) : "r"(at + n * term) : "memory");
    x[0] += lo_of(w0);
    x[1] += hi_of(w0);
    x[2] += lo_of(w1);
    x[3] += hi_of(w1);
  }
}
// an element of an operand's terms: of pair p its first or second
template <int N>
__device__ __forceinline__ float of_rows(const uint32_t (&f)[N][4], int p, int e) {
  float x = 0.f;
#pragma unroll
  for (int n = N - 1; n >= 0; --n) x += e ? hi_of(f[n][p]) : lo_of(f[n][p]);
  return x;
}

__device__ __forceinline__ float quad_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

template <class E, int KD, int VS>
__global__ void __launch_bounds__(Grads<E, KD, VS>::kT, 1) grads_kernel(Args<E> a) {
  using L = Grads<E, KD, VS>;
  constexpr int kO = L::kO, kT = L::kT, kParts = L::kParts;
  extern __shared__ __align__(128) unsigned char smem[];
  const uint32_t base = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t2 = (lane & 3) * 2;
  const int hk = blockIdx.y, group = a.heads / a.keys;
  Chunk ch;
  if (!chunk_at(a, blockIdx.x, ch)) return;
  const int64_t p = ch.start;
  if (!ch.live) {  // padding: zeros
    for (int i = tid; i < ch.len * a.dk; i += kT) {
      const int64_t r = p + i / a.dk;
      const int c = hk * a.dk + i % a.dk;
      E::store(a.dq + r * a.dq_stride + c, 0.f);
      E::store(a.dk_out + r * a.dk_stride + c, 0.f);
    }
    for (int i = tid; i < ch.len * group; i += kT) {
      const int64_t r = p + i / group;
      const int h = hk * group + i % group;
      E::store(a.dg + r * a.dg_stride + h, 0.f);
      E::store(a.db + r * a.db_stride + h, 0.f);
    }
    return;
  }
  const uint8_t* mask = a.mask != nullptr ? a.mask + p : nullptr;
  const size_t saved = saved_floats<E>(a.dk, a.dv);
  const Mat K = mat<kC, KD>(base + L::kK), Q = mat<kC, KD>(base + L::kQ);
  const Mat Fm = mat<kC, kC>(base + L::kF), Em = mat<kC, kC>(base + L::kE);
  float* sums = reinterpret_cast<float*>(smem + L::kNum);
  float *reads = sums, *writes = reads + kParts * kC, *rows = writes + kParts * kC, *own = rows + kParts * kC, *columns = own + kParts * kC,
        *wholes = columns + 4 * kC;
  const int slices = (a.dv + VS - 1) / VS, steps = group * slices;
  auto load = [&](int step) {  // of a head's slice, and with the first one the gates
    const int h = hk * group + step / slices, v0 = step % slices * VS, cols = a.dv - v0 < VS ? a.dv - v0 : VS;
    const size_t unit = unit_of(a, blockIdx.x, h);
    const uint32_t at = base + L::kSlice + (step % L::kStages) * L::kSliceBytes;
    const int64_t column = static_cast<int64_t>(h) * a.dv + v0;
    if (v0 == 0) load_gates<kT>(base + L::kHead + (h % L::kStages) * L::kHeadBytes, a.gates + unit);
    load_rows<E, VS, kT>(mat<kC, VS>(at + L::kY), a.dy + p * a.dy_stride + column, a.dy_stride, ch.len, cols, mask, a.vec);
    // of type bf16 dV's first term is the output, and its others and U's terms are kept apart
    const int64_t wide = static_cast<int64_t>(a.heads) * a.dv;
    const Mat W = mat<kC, VS>(at + L::kW), U = mat<kC, VS>(at + L::kU);
    const auto* kept = kept_writes<E>(a) + p * wide + column;
    load_rows<E, VS, kT>(W, a.dv_out + p * a.dv_stride + column, a.dv_stride, ch.len, cols, nullptr, a.vec);
    load_rows<E, VS, kT>(U, kept, wide, ch.len, cols, nullptr, a.vec);
    if constexpr (E::kBytes == 2) {
      auto term = [](const Mat& m, int n) { return Mat{m.base + static_cast<uint32_t>(n * m.term), m.pitch, m.term}; };
      const auto* rest = a.writes + p * wide + column;
      load_rows<E, VS, kT>(term(W, 1), rest, wide, ch.len, cols, nullptr, a.vec);
      load_rows<E, VS, kT>(term(W, 2), rest + a.n_tokens * wide, wide, ch.len, cols, nullptr, a.vec);
      load_rows<E, VS, kT>(term(U, 1), kept + a.n_tokens * wide, wide, ch.len, cols, nullptr, a.vec);
    }
    load_state<E, KD, VS, kT>(at + L::kS, a.carry + unit * saved, v0, cols, a.dk);
    load_state<E, KD, VS, kT>(at + L::kD, a.after + unit * saved, v0, cols, a.dk);
    copies_begun();
  };
  load_rows<E, KD, kT>(K, a.k + p * a.k_stride + hk * a.dk, a.k_stride, ch.len, a.dk, mask, a.vec);
  load_rows<E, KD, kT>(Q, a.q + p * a.q_stride + hk * a.dk, a.q_stride, ch.len, a.dk, mask, a.vec);
  load(0);
  copies_done();
  __syncthreads();
  // a warp's tiles: 16 rows, and a part of the columns
  const int m = (warp & 3) * 16, part = warp >> 2, nc = part * (kC / kParts), nk = part * (KD / kParts);
  const bool low = nc <= m;  // whether its tile of a triangle has anything
  float qk[L::kCN][4], kk[L::kCN][4];
  clear(qk);
  clear(kk);
  if (low) {
    product<kIn<E>, kIn<E>, kIn<E>>(qk, Rows{Q}, Across{K}, m, nc, 0, KD);
    product<kIn<E>, kIn<E>, kIn<E>>(kk, Rows{K}, Across{K}, m, nc, 0, KD);
  }
  for (int h = hk * group; h < (hk + 1) * group; ++h) {
    const Gates& gt = *reinterpret_cast<const Gates*>(smem + L::kHead + (h % L::kStages) * L::kHeadBytes);
    float cf[L::kCN][4], ce[L::kCN][4], cq[L::kKN][4], ck[L::kKN][4], cw[L::kKN][4];
    float whole = 0.f, dot = 0.f;
    clear(cf);
    clear(ce);
    clear(cq);
    clear(ck);
    clear(cw);
    for (int sl = 0; sl < slices; ++sl) {
      const int step = (h - hk * group) * slices + sl;
      const uint32_t at = base + L::kSlice + (step % L::kStages) * L::kSliceBytes;
      const auto S = state_down<E, KD, VS>(at + L::kS), D = state_down<E, KD, VS>(at + L::kD);
      const Mat Y = mat<kC, VS>(at + L::kY), W = mat<kC, VS>(at + L::kW), U = mat<kC, VS>(at + L::kU);
      if (L::kStages == 1 && step > 0) {
        __syncthreads();  // the slice before has been used
        load(step);
      }
      copies_done();
      __syncthreads();  // the slice is here, and the other stage is free
      if (L::kStages == 2 && step + 1 < steps) load(step + 1);
      // S . dS, wherever their values lie
      if constexpr (E::kBytes == 2) {
        if (VS / 16 * (KD / 16) * 32 == kT || tid < VS / 16 * (KD / 16) * 32) {
          const uint32_t to = at + (tid >> 5) * kBlockBytes + lane * 16;
          uint32_t s[2][4], d[2][4];
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            ld128(s[n], to + L::kS + n * 512);
            ld128(d[n], to + L::kD + n * 512);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            whole = fmaf(lo_of(s[0][j]) + lo_of(s[1][j]), lo_of(d[0][j]) + lo_of(d[1][j]), whole);
            whole = fmaf(hi_of(s[0][j]) + hi_of(s[1][j]), hi_of(d[0][j]) + hi_of(d[1][j]), whole);
          }
        }
      } else {
        const Mat sm = mat<VS, KD>(at + L::kS), dm = mat<VS, KD>(at + L::kD);
        for (int i = tid; i < VS * (KD / 2); i += kT) {
          const int r = i / (KD / 2), c = i % (KD / 2) * 2;
          float s[2], d[2];
          get<kO>(sm.base + r * sm.pitch + c * 2, sm.term, s[0], s[1]);
          get<kO>(dm.base + r * dm.pitch + c * 2, dm.term, d[0], d[1]);
          whole = fmaf(s[0], d[0], fmaf(s[1], d[1], whole));
        }
      }
      // dV . U of the block's positions: kT / 64 neighbouring threads a position
      {
        constexpr int kBy = kT / kC;
        static_assert(VS / kBy == 4, "four columns a thread");
        const uint32_t off = (tid / kBy) * W.pitch + tid % kBy * 8;
        float u[4], w[4];
        get4<kO>(U.base + off, U.term, u);
        get4<L::kWT>(W.base + off, W.term, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) dot = fmaf(u[i], w[i], dot);
      }
      both_products<kIn<E>, kO, L::kWT>(cq, ck, Rows{Y}, Rows{W}, S, m, nk, VS);
      product<kO, kO, kO>(cw, Rows{U}, D, m, nk, 0, VS);
      if (low) both_products<kIn<E>, kO, L::kWT>(cf, ce, Rows{Y}, Rows{W}, Across{U}, m, nc, VS);
    }
    // ---- F and E, the pairs of reads and writes, and what reads S and reaches dS
    float row[2] = {0.f, 0.f};
#pragma unroll
    for (int t = 0; t < L::kCN; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = nc + t * 8 + t2 + e;
        float column = 0.f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int r = m + g + j * 8;
          const float d = i <= r && low ? expf((gt.hi[r] - gt.hi[i]) + (gt.lo[r] - gt.lo[i])) : 0.f;
          float& f = cf[t][2 * j + e];
          float& w = ce[t][2 * j + e];
          f = i <= r && low ? a.scale * d * f : 0.f;
          w = i < r && low ? -d * w : 0.f;
          const float pair = i < r && low ? fmaf(f, qk[t][2 * j + e], w * kk[t][2 * j + e]) : 0.f;
          row[j] += pair;
          column += pair;
        }
        column += __shfl_xor_sync(0xffffffffu, column, 4);
        column += __shfl_xor_sync(0xffffffffu, column, 8);
        column += __shfl_xor_sync(0xffffffffu, column, 16);
        if (g == 0) columns[(m >> 4) * kC + i] = column;
      }
    // (an operand A's places are those of two neighbouring accumulators)
    uint32_t fq[L::kKN / 2][kIn<E>][4], fk[L::kKN / 2][kIn<E>][4];
#pragma unroll
    for (int t = 0; t < L::kKN / 2; ++t)
#pragma unroll
      for (int n = 0; n < kIn<E>; ++n) {
        Rows{Q}(fq[t][n], m, nk + t * 16, n);
        Rows{K}(fk[t][n], m, nk + t * 16, n);
      }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int r = m + g + j * 8;
      const float into = gt.into[r], last = gt.last[r];
      float read = 0.f, write = 0.f;
#pragma unroll
      for (int t = 0; t < L::kKN; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float q = of_rows<kIn<E>>(fq[t / 2], (t & 1) * 2 + j, e), k = of_rows<kIn<E>>(fk[t / 2], (t & 1) * 2 + j, e);
          cq[t][2 * j + e] *= a.scale * into;
          const float seen = -into * ck[t][2 * j + e], left = last * cw[t][2 * j + e];
          read = fmaf(q, cq[t][2 * j + e], fmaf(k, seen, read));
          write = fmaf(k, left, write);
          ck[t][2 * j + e] = seen + left;
        }
      const float sum_row = quad_sum(row[j]), sum_read = quad_sum(read), sum_write = quad_sum(write);
      if (t2 == 0) {
        rows[part * kC + r] = sum_row;
        reads[part * kC + r] = sum_read;
        writes[part * kC + r] = sum_write;
      }
    }
#pragma unroll
    for (int o = kT / kC / 2; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if (tid % (kT / kC) == 0) own[tid / (kT / kC)] = dot;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) whole += __shfl_xor_sync(0xffffffffu, whole, o);
    if (lane == 0) wholes[warp] = whole;
    __syncthreads();  // the slice is no longer needed
    if (low) {
#pragma unroll
      for (int t = 0; t < L::kCN; ++t)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t at = (m + g + j * 8) * Fm.pitch + (nc + t * 8 + t2) * 2;
          put<kO>(Fm.base + at, Fm.term, cf[t][2 * j], cf[t][2 * j + 1]);
          put<kO>(Em.base + at, Em.term, ce[t][2 * j], ce[t][2 * j + 1]);
        }
    }
    __syncthreads();
    product<kO, kIn<E>, kO>(cq, Rows{Fm}, Down{K}, m, nk, 0, m + 16);
    product<kO, kIn<E>, kO>(ck, Rows{Em}, Down{K}, m, nk, 0, m + 16);
    product<kO, kIn<E>, kO>(ck, Cols{Em}, Down{K}, m, nk, m, kC);
    product<kO, kIn<E>, kO>(ck, Cols{Fm}, Down{Q}, m, nk, m, kC);
    // ---- heads that share a key are added up in order, each thread its own elements
    const bool begins = h == hk * group, ends = h + 1 == (hk + 1) * group;
    if (!(begins && ends)) {
      float4* all = reinterpret_cast<float4*>(a.shared) +
                    (static_cast<size_t>(blockIdx.x) * a.keys + hk) * (2 * L::kKN * kT) + tid;
      if (!begins) {
        float4 x[2 * L::kKN];
#pragma unroll
        for (int t = 0; t < 2 * L::kKN; ++t) x[t] = all[t * kT];
#pragma unroll
        for (int t = 0; t < L::kKN; ++t) {
          cq[t][0] += x[t].x; cq[t][1] += x[t].y; cq[t][2] += x[t].z; cq[t][3] += x[t].w;
          const float4& y = x[t + L::kKN];
          ck[t][0] += y.x; ck[t][1] += y.y; ck[t][2] += y.z; ck[t][3] += y.w;
        }
      }
      if (!ends) {
#pragma unroll
        for (int t = 0; t < L::kKN; ++t) {
          all[t * kT] = make_float4(cq[t][0], cq[t][1], cq[t][2], cq[t][3]);
          all[(t + L::kKN) * kT] = make_float4(ck[t][0], ck[t][1], ck[t][2], ck[t][3]);
        }
      }
    }
    if (ends) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = m + g + j * 8;
        if (r >= ch.len) continue;
        const bool on = !(mask != nullptr && mask[r]);
        auto* to_q = a.dq + (p + r) * a.dq_stride + hk * a.dk;
        auto* to_k = a.dk_out + (p + r) * a.dk_stride + hk * a.dk;
#pragma unroll
        for (int t = 0; t < L::kKN; ++t) {
          const int c = nk + t * 8 + t2;
          if (c >= a.dk) continue;
          const float q0 = on ? cq[t][2 * j] : 0.f, q1 = on ? cq[t][2 * j + 1] : 0.f;
          const float k0 = on ? ck[t][2 * j] : 0.f, k1 = on ? ck[t][2 * j + 1] : 0.f;
          if (E::kBytes == 2 && a.key_pairs) {
            *reinterpret_cast<uint32_t*>(to_q + c) = pack(q0, q1);
            *reinterpret_cast<uint32_t*>(to_k + c) = pack(k0, k1);
          } else {
            E::store(to_q + c, q0);
            E::store(to_k + c, k0);
            if (c + 1 < a.dk) E::store(to_q + c + 1, q1);
            if (c + 1 < a.dk) E::store(to_k + c + 1, k1);
          }
        }
      }
    }
    if (warp == 0) {  // what crosses a position: two positions a lane
      float later[2], before[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = lane * 2 + j;
        float read = 0.f, row = 0.f, write = 0.f;
#pragma unroll
        for (int n = 0; n < kParts; ++n) {
          read += reads[n * kC + r];
          row += rows[n * kC + r];
          write += writes[n * kC + r];
        }
        later[j] = read + row - (((columns[r] + columns[kC + r]) + columns[2 * kC + r]) + columns[3 * kC + r]);
        before[j] = write;
      }
      float sum = later[0] + later[1], head = before[0] + before[1], all = 0.f;
      const float mine = head;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float x = __shfl_down_sync(0xffffffffu, sum, o), y = __shfl_up_sync(0xffffffffu, head, o);
        if (lane + o < 32) sum += x;
        if (lane >= o) head += y;
      }
#pragma unroll
      for (int w = 0; w < 4 * kParts; ++w) all += wholes[w];
      all *= gt.into[kC - 1];
      const float cross[2] = {sum + (head - mine) + all, (sum - later[0]) + (head - mine + before[0]) + all};
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = lane * 2 + j;
        if (r >= ch.len) continue;
        const bool on = gt.beta[r] != 0.f;
        const int64_t t = p + r;
        const float gr = E::load(a.g + t * a.g_stride + h), br = E::load(a.b + t * a.b_stride + h);
        E::store(a.dg + t * a.dg_stride + h, on ? cross[j] / (1.f + expf(gr)) : 0.f);
        E::store(a.db + t * a.db_stride + h, on ? own[r] / (gt.beta[r] * (1.f + expf(br))) : 0.f);
      }
    }
  }
}

template <class E>
int launch_grad(const Args<E>& a, int sms, cudaStream_t st) {
  int rc = launch_first<E>(a, st);
  if (rc) return rc;
  static std::atomic<uint64_t> done[4] = {{0}, {0}, {0}, {0}};
  auto go = [&](auto kernel, int smem, dim3 grid, std::atomic<uint64_t>& flag, const char* name, int threads = kThreads) {
    int r = opt_in(reinterpret_cast<const void*>(kernel), smem, flag);
    if (r) return r;
    kernel<<<grid, threads, smem, st>>>(a);
    return check_launch(name);
  };
  constexpr int VG = E::kBytes == 2 ? 32 : 16;
  const dim3 grads(a.max_chunks, a.keys);
  auto back = [&](auto kernel, int smem, int nq, std::atomic<uint64_t>& flag) {
    return go(kernel, smem, dim3(a.blocks), flag, "back_kernel",
              nq == 1 ? 128 + kCopiers : nq * 128);
  };
  bool many = false;
  if constexpr (E::kBytes == 2) {
    many = many_quads(a, sms);
    static std::atomic<uint64_t> flags[2] = {{0}, {0}};
    if (many)
      rc = a.dk <= 64 ? back(back_kernel<E, 64, 4>, Back<E, 64, 4>::kSmem, 4, flags[0])
                      : back(back_kernel<E, 128, 4>, Back<E, 128, 4>::kSmem, 4, flags[1]);
  }
  if (!many)
    rc = a.dk <= 64 ? back(back_kernel<E, 64, 1>, Back<E, 64, 1>::kSmem, 1, done[0])
                    : back(back_kernel<E, 128, 1>, Back<E, 128, 1>::kSmem, 1, done[1]);
  if (rc) return rc;
  return a.dk <= 64 ? go(grads_kernel<E, 64, VG>, Grads<E, 64, VG>::kSmem, grads, done[2], "grads_kernel", Grads<E, 64, VG>::kT)
                    : go(grads_kernel<E, 128, VG>, Grads<E, 128, VG>::kSmem, grads, done[3], "grads_kernel", Grads<E, 128, VG>::kT);
}

static_assert(Back<train::Bf16, 128, 4>::kSmem + sizeof(Stages) + sizeof(Item) <= 232448 && Back<train::F32, 128, 1>::kSmem <= 232448 &&
                  Grads<train::Bf16, 128, 32>::kSmem <= 232448 && Grads<train::F32, 128, 16>::kSmem <= 232448,
              "a block's shared memory");

}  // namespace
}  // namespace delta
}  // namespace engram

using namespace engram;
using namespace engram::delta;

extern "C" int engram_delta_grad(const void* dy_d, int64_t dy_stride, const void* q_d, int64_t q_stride, const void* k_d,
                                 int64_t k_stride, const void* v_d, int64_t v_stride, const void* g_d, int64_t g_stride,
                                 const void* b_d, int64_t b_stride, int32_t type, int64_t n_tokens, int32_t key_heads,
                                 int32_t heads, int32_t dk, int32_t dv, float scale, const int64_t* cu_seqlens_d,
                                 int64_t n_seqs, const int32_t* slots_d, const uint8_t* mask_d, const float* carry_d,
                                 float* dstate_d, int64_t n_slots, void* dq_d, int64_t dq_stride, void* dk_d,
                                 int64_t dk_stride, void* dv_d, int64_t dv_stride, void* dg_d, int64_t dg_stride,
                                 void* db_d, int64_t db_stride, void* workspace_d, size_t workspace_bytes,
                                 int32_t* status_d, void* stream) {
  int rc = check_sizes(type, n_tokens, key_heads, heads, dk, dv, n_seqs, n_slots, dstate_d != nullptr, scale);
  if (rc) return rc;
  if (n_seqs == 0) return n_tokens == 0 ? ENGRAM_OK : fail(ENGRAM_E_SHAPE, "positions without a sequence");
  if (n_tokens == 0) return ENGRAM_OK;  // the state's gradient passes through empty sequences
  if (!cu_seqlens_d || !carry_d) return fail(ENGRAM_E_INVALID, "null device pointer: cu_seqlens or carry");
  const int64_t wide_k = static_cast<int64_t>(key_heads) * dk, wide_v = static_cast<int64_t>(heads) * dv;
  if ((rc = check_rows(dy_d, type, dy_stride, wide_v, "dy"))) return rc;
  if ((rc = check_rows(q_d, type, q_stride, wide_k, "q"))) return rc;
  if ((rc = check_rows(k_d, type, k_stride, wide_k, "k"))) return rc;
  if (v_d != nullptr && (rc = check_rows(v_d, type, v_stride, wide_v, "v"))) return rc;  // (it is not read)
  if ((rc = check_rows(g_d, type, g_stride, heads, "g"))) return rc;
  if ((rc = check_rows(b_d, type, b_stride, heads, "b"))) return rc;
  if ((rc = check_rows(dq_d, type, dq_stride, wide_k, "dq"))) return rc;
  if ((rc = check_rows(dk_d, type, dk_stride, wide_k, "dk"))) return rc;
  if ((rc = check_rows(dv_d, type, dv_stride, wide_v, "dv"))) return rc;
  if ((rc = check_rows(dg_d, type, dg_stride, heads, "dg"))) return rc;
  if ((rc = check_rows(db_d, type, db_stride, heads, "db"))) return rc;
  if (!aligned(dstate_d, 4)) return fail(ENGRAM_E_ALIGN, "states must be aligned to their elements");
  if (!aligned(carry_d, 16)) return fail(ENGRAM_E_ALIGN, "carry must be 16-byte aligned");
  if (!workspace_d) return fail(ENGRAM_E_INVALID, "null device pointer: workspace");
  if (!aligned(workspace_d, 256)) return fail(ENGRAM_E_ALIGN, "workspace must be 256-byte aligned");
  if (workspace_bytes < engram_delta_workspace_bytes(n_tokens, n_seqs, key_heads, heads, dk, dv, 1))
    return fail(ENGRAM_E_RANGE, "workspace too small");
  int sms = 0;
  if ((rc = check_device(&sms))) return rc;
  auto go = [&](auto e) {
    using E = decltype(e);
    using T = typename E::T;
    Args<E> a{};
    a.dy = static_cast<const T*>(dy_d);
    a.q = static_cast<const T*>(q_d);
    a.k = static_cast<const T*>(k_d);
    a.g = static_cast<const T*>(g_d);
    a.b = static_cast<const T*>(b_d);
    a.dq = static_cast<T*>(dq_d);
    a.dk_out = static_cast<T*>(dk_d);
    a.dv_out = static_cast<T*>(dv_d);
    a.dg = static_cast<T*>(dg_d);
    a.db = static_cast<T*>(db_d);
    a.dy_stride = dy_stride;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.g_stride = g_stride;
    a.b_stride = b_stride;
    a.dq_stride = dq_stride;
    a.dk_stride = dk_stride;
    a.dv_stride = dv_stride;
    a.dg_stride = dg_stride;
    a.db_stride = db_stride;
    a.cu = cu_seqlens_d;
    a.slots = slots_d;
    a.mask = mask_d;
    a.state_out = dstate_d;
    a.carry = const_cast<float*>(carry_d);
    a.n_slots = n_slots;
    a.has_state = dstate_d != nullptr;
    a.n_tokens = static_cast<int32_t>(n_tokens);
    a.n_seqs = static_cast<int32_t>(n_seqs);
    a.max_chunks = static_cast<int32_t>(max_chunks(n_tokens, n_seqs));
    a.keys = key_heads;
    a.heads = heads;
    a.dk = dk;
    a.dv = dv;
    a.scale = scale;
    a.vec = pieces(q_d, q_stride, E::kBytes) && pieces(k_d, k_stride, E::kBytes) &&
            pieces(dy_d, dy_stride, E::kBytes) && pieces(dv_d, dv_stride, E::kBytes) && dk % 8 == 0 && dv % 8 == 0;
    a.pairs = dv % 2 == 0 && dv_stride % 2 == 0 && aligned(dv_d, 2 * E::kBytes);
    a.key_pairs = dk % 2 == 0 && dq_stride % 2 == 0 && dk_stride % 2 == 0 && aligned(dq_d, 2 * E::kBytes) &&
                  aligned(dk_d, 2 * E::kBytes);
    a.status = status_d;
    const Space s = space(workspace_d, n_tokens, n_seqs, key_heads, heads, dk, dv, true);
    a.first = s.first;
    a.line = s.line;
    a.given = s.given;
    a.between = s.between;
    set_blocks(a, sms);
    use_kept_triangles(a);
    a.after = s.after;
    a.writes = s.writes;
    a.shared = s.shared;
    set_absent(a);
    return launch_grad<E>(a, sms, as_stream(stream));
  };
  return type == ENGRAM_T_BF16 ? go(train::Bf16{}) : go(train::F32{});
}
