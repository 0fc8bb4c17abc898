// The gated delta rule: a memory of each head that is a matrix, read by queries and
// corrected towards a value at its key.
//
//   S <- f S,  u = beta (v - S^T k),  S <- S + k u^T,  y = scale S^T q
// with f = sigmoid(g) and beta = sigmoid(b).  A whole sequence goes in chunks of 64
// positions (delta_device.cuh), a decode step token by token.
#include "delta_device.cuh"

namespace engram {
namespace delta {

// ------------------------------------------------------------------- chunks

// first[s]: how many chunks the sequences before s have.
template <class E>
__global__ void __launch_bounds__(1024) first_kernel(Args<E> a) {
  __shared__ int warp_sum[32];
  __shared__ int64_t before;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) before = 0;
  for (int s0 = 0; s0 < a.n_seqs; s0 += 1024) {
    const int s = s0 + threadIdx.x;
    int n = 0;
    if (s < a.n_seqs) {
      int lo, hi;
      bounds(a, s, lo, hi);
      n = (hi - lo + kC - 1) / kC;
    }
    int sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += x;
    }
    __syncthreads();
    if (lane == 31) warp_sum[warp] = sum;
    __syncthreads();
    int64_t at = before + sum - n;
    for (int w = 0; w < warp; ++w) at += warp_sum[w];
    // (sequences that lie over one another could give more chunks than there is room for)
    if (s < a.n_seqs) a.first[s] = static_cast<int>(at < a.max_chunks ? at : a.max_chunks);
    __syncthreads();
    if (threadIdx.x == 1023) before = at + n;
  }
  __syncthreads();
  if (threadIdx.x == 0) a.first[a.n_seqs] = static_cast<int>(before < a.max_chunks ? before : a.max_chunks);
}

// ---------------------------------------------------------------- M, P, gates

constexpr int kPitch = kC + 4;  // of fp32 64 x 64 matrices

// dst = sign A B, 16 x 16, by a warp, in fp32's precision: each operand as two tf32
// terms (22 bits), three products.
__device__ __forceinline__ void small_product(float* dst, const float* a, const float* b, int depth, float sign) {
  const int l = lane_id(), g = l >> 2, t = l & 3;
  float c[2][4] = {};
  auto tf32 = [](float x) {
    uint32_t r;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
    return r;
  };
  for (int k = 0; k < depth; k += 8) {
    uint32_t ah[4], al[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float x = a[(g + (j & 1) * 8) * kPitch + k + t + (j >> 1) * 4];
      ah[j] = tf32(x);
      al[j] = tf32(x - __uint_as_float(ah[j]));
    }
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      uint32_t bh[2], bl[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float x = b[(k + t + j * 4) * kPitch + n * 8 + g];
        bh[j] = tf32(x);
        bl[j] = tf32(x - __uint_as_float(bh[j]));
      }
      auto step = [&](const uint32_t (&x)[4], const uint32_t (&y)[2]) {
        asm volatile(
            "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
            "%3};"
            : "+f"(c[n][0]), "+f"(c[n][1]), "+f"(c[n][2]), "+f"(c[n][3])
            : "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(y[0]), "r"(y[1]));
      };
      step(al, bh);
      step(ah, bl);
      step(ah, bh);
    }
  }
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j) dst[(g + (j >> 1) * 8) * kPitch + n * 8 + 2 * t + (j & 1)] = sign * c[n][j];
}

// A pair of neighbouring columns of a triangle as N terms in the workspace.
template <int N>
__device__ __forceinline__ void put_tri(unsigned char* base, int t, int i, float x0, float x1) {
  const int bi = t >> 4, bj = i >> 4, r = t & 15;
  unsigned char* at = base + (bi * (bi + 1) / 2 + bj) * 512 + tri_at(r, (i >> 3) & 1) + (i & 7) * 2;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const uint32_t w = pack(x0, x1);
    *reinterpret_cast<uint32_t*>(at + n * kTerm) = w;
    x0 -= lo_of(w);
    x1 -= hi_of(w);
  }
}

template <class E, int KD>
constexpr int kPrepareSmem = 2 * kIn<E>* mat_bytes(kC, KD) + 4 * kC * kPitch * 4 + static_cast<int>(sizeof(Gates));

// A block makes M and P for the heads that share a key head, in one chunk.
template <class E, int KD>
__global__ void __launch_bounds__(kThreads) prepare_kernel(Args<E> a) {
  extern __shared__ __align__(128) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Chunk ch;
  if (!chunk_at(a, blockIdx.x, ch) || !ch.live) return;
  const Mat K = mat<kC, KD>(smem_u32(smem)), Q = mat<kC, KD>(K.base + kIn<E> * K.term);
  float* kk = reinterpret_cast<float*>(smem + 2 * kIn<E> * mat_bytes(kC, KD));
  float *qk = kk + kC * kPitch, *A = qk + kC * kPitch, *M = A + kC * kPitch;
  Gates& gt = *reinterpret_cast<Gates*>(M + kC * kPitch);
  const uint8_t* mask = a.mask != nullptr ? a.mask + ch.start : nullptr;
  const int hk = blockIdx.y, group = a.heads / a.keys;
  load_rows<E, KD>(K, a.k + ch.start * a.k_stride + hk * a.dk, a.k_stride, ch.len, a.dk, mask, a.vec);
  load_rows<E, KD>(Q, a.q + ch.start * a.q_stride + hk * a.dk, a.q_stride, ch.len, a.dk, mask, a.vec);
  copies_begun();
  copies_done();
  __syncthreads();
  {  // K K^T and Q K^T: a warp has 16 rows and 32 columns of each
    const int m = (warp & 3) * 16, n = (warp >> 2) * 32;
    if (n <= m) {
      float ck[4][4], cq[4][4];
      clear(ck);
      clear(cq);
      product<kIn<E>, kIn<E>, kIn<E>>(ck, Rows{K}, Across{K}, m, n, 0, KD);
      product<kIn<E>, kIn<E>, kIn<E>>(cq, Rows{Q}, Across{K}, m, n, 0, KD);
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int at = (m + (lane >> 2) + (j >> 1) * 8) * kPitch + n + t * 8 + (lane & 3) * 2 + (j & 1);
          kk[at] = ck[t][j];
          qk[at] = cq[t][j];
        }
    }
  }
  for (int h = hk * group; h < (hk + 1) * group; ++h) {
    unsigned char* tri = a.tri + unit_of(a, blockIdx.x, h) * kTriBytes;
    if (warp == 0) {  // c, two positions a lane
      double c[2], sum;
      float beta[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = lane * 2 + j;
        const bool on = r < ch.len && !(mask != nullptr && mask[r]);
        const int64_t t = ch.start + (on ? r : 0);
        // gates below -80 count as -80, b below -40 as -40 (a NaN stays)
        float g = E::load(a.g + t * a.g_stride + h), b = E::load(a.b + t * a.b_stride + h);
        g = g < -80.f ? -80.f : g;
        b = b < -40.f ? -40.f : b;
        c[j] = on ? static_cast<double>(g < 0.f ? g - log1pf(expf(g)) : -log1pf(expf(-g))) : 0.0;
        beta[j] = on ? 1.f / (1.f + expf(-b)) : 0.f;
      }
      c[1] += c[0];
      sum = c[1];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double x = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += x;
      }
      const double before = sum - c[1], all = __shfl_sync(0xffffffffu, sum, 31);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = lane * 2 + j;
        const double x = before + c[j];
        // c = hi + lo, hi a multiple of 1/16: differences of hi are exact
        const float hi = rintf(static_cast<float>(x) * 16.f) * 0.0625f;
        gt.hi[r] = hi;
        gt.lo[r] = static_cast<float>(x - hi);
        gt.into[r] = expf(static_cast<float>(x));
        gt.last[r] = expf(static_cast<float>(all - x));
        gt.beta[r] = beta[j];
      }
    }
    __syncthreads();
    for (int i = tid; i < static_cast<int>(sizeof(Gates)) / 4; i += kThreads)
      reinterpret_cast<float*>(a.gates + unit_of(a, blockIdx.x, h))[i] = reinterpret_cast<const float*>(&gt)[i];
    for (int p = tid; p < kC * kC / 2; p += kThreads) {
      const int t = p >> 5, i = (p & 31) * 2;
      if ((i >> 4) > (t >> 4)) continue;
      float x[2], y[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const bool in = i + j <= t;
        const float d = in ? expf((gt.hi[t] - gt.hi[i + j]) + (gt.lo[t] - gt.lo[i + j])) : 0.f;
        x[j] = i + j < t ? gt.beta[t] * d * kk[t * kPitch + i + j] : 0.f;
        y[j] = in ? a.scale * d * qk[t * kPitch + i + j] : 0.f;
      }
      A[t * kPitch + i] = x[0];
      A[t * kPitch + i + 1] = x[1];
      put_tri<kStateTerms>(tri + kStateTerms * kTerm, t, i, y[0], y[1]);
    }
    __syncthreads();
    // (I + A)^-1: blocks of 16 by substitution, a column a lane; then [M11 0; -M22 A21 M11 M22]
    if (warp < 4 && lane < 16) {
      const float* D = A + warp * 16 * (kPitch + 1);
      float x[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float s = i == lane ? 1.f : 0.f;
#pragma unroll
        for (int j = 0; j < i; ++j) s = fmaf(-D[i * kPitch + j], x[j], s);
        x[i] = s;
        M[(warp * 16 + i) * kPitch + warp * 16 + lane] = s;
      }
    }
    __syncthreads();
    if (warp < 2) {  // (A's blocks above the diagonal are free for the products in between)
      const int o = warp * 32 * (kPitch + 1), down = 16 * kPitch;
      small_product(A + o + 16, A + o + down, M + o, 16, 1.f);
      __syncwarp();
      small_product(M + o + down, M + o + down + 16, A + o + 16, 16, -1.f);
    }
    __syncthreads();
    const int bm = (warp & 1) * 16, bn = (warp >> 1) * 16;
    // (M's upper block of the first half is not written above: the product of the second
    // half of the columns starts below it)
    if (warp < 4) small_product(A + bm * kPitch + 32 + bn, A + (32 + bm) * kPitch + bn, M + bn * kPitch + bn, 32 - bn, 1.f);
    __syncthreads();
    if (warp < 4) small_product(M + (32 + bm) * kPitch + bn, M + (32 + bm) * kPitch + 32, A + 32 + bn, 16 + bm, -1.f);
    __syncthreads();
    for (int p = tid; p < kC * kC / 2; p += kThreads) {
      const int t = p >> 5, i = (p & 31) * 2;
      if ((i >> 4) > (t >> 4)) continue;
      put_tri<kStateTerms>(tri, t, i, i <= t ? M[t * kPitch + i] * gt.beta[i] : 0.f,
                           i + 1 <= t ? M[t * kPitch + i + 1] * gt.beta[i + 1] : 0.f);
    }
    __syncthreads();
  }
}

template <class E>
int launch_prepare(const Args<E>& a, cudaStream_t st) {
  first_kernel<E><<<1, 1024, 0, st>>>(a);
  int rc = check_launch("first_kernel");
  if (rc || a.max_chunks == 0) return rc;
  auto go = [&](auto kernel, int smem, std::atomic<uint64_t>& done) {
    int r = opt_in(reinterpret_cast<const void*>(kernel), smem, done);
    if (r) return r;
    kernel<<<dim3(a.max_chunks, a.keys), kThreads, smem, st>>>(a);
    return check_launch("prepare_kernel");
  };
  static std::atomic<uint64_t> done[2] = {{0}, {0}};
  return a.dk <= 64 ? go(prepare_kernel<E, 64>, kPrepareSmem<E, 64>, done[0])
                    : go(prepare_kernel<E, 128>, kPrepareSmem<E, 128>, done[1]);
}
template int launch_prepare<train::Bf16>(const Args<train::Bf16>&, cudaStream_t);
template int launch_prepare<train::F32>(const Args<train::F32>&, cudaStream_t);

// --------------------------------------------------------------------- scan

// A block follows one sequence's chunks in one head, for kVS of the value columns.
// The state stays in registers as the products' accumulator; its terms go to shared
// memory, where they are an operand.  The next chunk's inputs are copied meanwhile
// (bf16; fp32's terms are made on the way to shared memory and take the room).
template <class E, int KD, int VS>
struct Scan {
  static constexpr int kStages = E::kBytes == 2 ? 2 : 1;
  static constexpr int kQ = 0, kK = kQ + kIn<E> * mat_bytes(kC, KD), kV = kK + kIn<E> * mat_bytes(kC, KD);
  static constexpr int kM = kV + kIn<E> * mat_bytes(kC, VS), kP = kM + kStateTerms * kTerm, kG = kP + kOut<E> * kTerm;
  static constexpr int kStage = kG + static_cast<int>(sizeof(Gates));
  static constexpr int kS = kStages * kStage;                         // the state
  static constexpr int kX = kS + kStateTerms * mat_bytes(KD, VS);     // V - e^c K S, then e^(c_last - c) U
  static constexpr int kU = kX + kStateTerms * mat_bytes(kC, VS);
  static constexpr int kSmem = kU + kOut<E> * mat_bytes(kC, VS);
  static constexpr int kAcross = kWarps / (KD / 16);  // warps that share 16 rows of the state
  static constexpr int kN = VS / 16;                  // a warp's tiles of 8 columns of a chunk's rows
  static constexpr int kSN = VS / 8 / kAcross;        // and of the state's
};

template <class E, int KD, int VS>
__global__ void __launch_bounds__(kThreads, 1) scan_kernel(Args<E> a) {
  using L = Scan<E, KD, VS>;
  extern __shared__ __align__(128) unsigned char smem[];
  const uint32_t base = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t2 = (lane & 3) * 2;
  const int seq = blockIdx.x, h = blockIdx.y, v0 = blockIdx.z * VS, cols = a.dv - v0 < VS ? a.dv - v0 : VS;
  const int hk = h / (a.heads / a.keys);
  int lo, hi;
  bounds(a, seq, lo, hi);
  const int c0 = a.first[seq], n = min((hi - lo + kC - 1) / kC, a.max_chunks - c0);
  int64_t slot;
  const bool live = live_slot(a, seq, slot);
  if (!live && tid == 0 && h == 0 && v0 == 0 && a.status != nullptr && slot >= 0) atomicOr(a.status, ENGRAM_ST_BAD_SLOT);
  const size_t matrix = static_cast<size_t>(a.dk) * a.dv;
  if (!live) {  // padding: zeros
    for (int64_t i = tid; i < static_cast<int64_t>(hi - lo) * cols; i += kThreads)
      E::store(a.y + (lo + i / cols) * a.y_stride + h * a.dv + v0 + i % cols, 0.f);
    for (int c = 0; a.carry != nullptr && c < n; ++c)
      for (int i = tid; i < a.dk * cols; i += kThreads)
        a.carry[unit_of(a, c0 + c, h) * matrix + static_cast<size_t>(i / cols) * a.dv + v0 + i % cols] = 0.f;
    return;
  }
  // the rows and columns of the state that this thread holds
  const int sm = warp % (KD / 16) * 16, sn = warp / (KD / 16) * (L::kSN * 8);
  auto each = [&](auto f) {  // f(accumulator's tile and place, row, column)
#pragma unroll
    for (int t = 0; t < L::kSN; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = sm + g + (j >> 1) * 8, c = sn + t * 8 + t2 + (j & 1);
        if (r < a.dk && c < cols) f(t, j, static_cast<size_t>(r) * a.dv + v0 + c);
      }
  };
  float S[L::kSN][4];
  clear(S);
  if (a.state != nullptr) {
    const float* from = a.state + (slot * a.heads + h) * matrix;
    each([&](int t, int j, size_t at) { S[t][j] = from[at]; });
  }
  const Mat St = mat<KD, VS>(base + L::kS), X = mat<kC, VS>(base + L::kX), U = mat<kC, VS>(base + L::kU);
  auto keep = [&]() {
#pragma unroll
    for (int t = 0; t < L::kSN; ++t)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        put<kStateTerms>(St.base + (sm + g + j * 8) * St.pitch + (sn + t * 8 + t2) * 2, St.term, S[t][2 * j], S[t][2 * j + 1]);
  };
  auto load = [&](int i) {
    const uint32_t stage = base + (i % L::kStages) * L::kStage;
    const int64_t p = lo + static_cast<int64_t>(i) * kC;
    const int len = hi - p < kC ? static_cast<int>(hi - p) : kC;
    const uint8_t* mask = a.mask != nullptr ? a.mask + p : nullptr;
    const size_t unit = unit_of(a, c0 + i, h);
    load_rows<E, KD>(mat<kC, KD>(stage + L::kK), a.k + p * a.k_stride + hk * a.dk, a.k_stride, len, a.dk, mask, a.vec);
    load_rows<E, KD>(mat<kC, KD>(stage + L::kQ), a.q + p * a.q_stride + hk * a.dk, a.q_stride, len, a.dk, mask, a.vec);
    load_rows<E, VS>(mat<kC, VS>(stage + L::kV), a.v + p * a.v_stride + h * a.dv + v0, a.v_stride, len, cols, mask, a.vec);
    load_tri<kOut<E>>(stage + L::kM, stage + L::kP, a.tri + unit * kTriBytes);
    load_gates(stage + L::kG, a.gates + unit);
    copies_begun();
  };
  keep();
  if (n > 0) load(0);
  const int m = (warp & 3) * 16, nn = (warp >> 2) * (VS / 2);  // the warp's tile of a chunk's rows
  for (int i = 0; i < n; ++i) {
    const uint32_t stage = base + (i % L::kStages) * L::kStage;
    const Mat K = mat<kC, KD>(stage + L::kK), Q = mat<kC, KD>(stage + L::kQ), V = mat<kC, VS>(stage + L::kV);
    const Gates& gt = *reinterpret_cast<const Gates*>(smem + (i % L::kStages) * L::kStage + L::kG);
    copies_done();
    __syncthreads();  // the chunk and the state are here, and the other stage is free
    if (L::kStages == 2 && i + 1 < n) load(i + 1);
    if (a.carry != nullptr) {
      float* to = a.carry + unit_of(a, c0 + i, h) * matrix;
      each([&](int t, int j, size_t at) { to[at] = S[t][j]; });
    }
    float x[L::kN][4], y[L::kN][4];
    clear(x);
    clear(y);
    product<kIn<E>, kStateTerms, kStateTerms>(x, Rows{K}, Down{St}, m, nn, 0, KD);
    product<kIn<E>, kOut<E>, kOut<E>>(y, Rows{Q}, Down{St}, m, nn, 0, KD);
#pragma unroll
    for (int t = 0; t < L::kN; ++t)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = m + g + j * 8, c = nn + t * 8 + t2;
        float v[2];
        get<kIn<E>>(V.base + r * V.pitch + c * 2, V.term, v[0], v[1]);
        const float into = gt.into[r];
        put<kStateTerms>(X.base + r * X.pitch + c * 2, X.term, fmaf(-into, x[t][2 * j], v[0]), fmaf(-into, x[t][2 * j + 1], v[1]));
        y[t][2 * j] *= a.scale * into;
        y[t][2 * j + 1] *= a.scale * into;
      }
    __syncthreads();
    float u[L::kN][4];
    clear(u);
    product<kStateTerms, kStateTerms, kStateTerms>(u, TriRows{stage + L::kM}, Down{X}, m, nn, 0, m + 16);
    __syncthreads();  // X is free
#pragma unroll
    for (int t = 0; t < L::kN; ++t)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = m + g + j * 8, c = nn + t * 8 + t2;
        const float last = gt.last[r];
        put<kOut<E>>(U.base + r * U.pitch + c * 2, U.term, u[t][2 * j], u[t][2 * j + 1]);
        put<kStateTerms>(X.base + r * X.pitch + c * 2, X.term, last * u[t][2 * j], last * u[t][2 * j + 1]);
      }
    __syncthreads();
    const float total = gt.into[kC - 1];
#pragma unroll
    for (int t = 0; t < L::kSN; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) S[t][j] *= total;
    product<kIn<E>, kStateTerms, kStateTerms>(S, Cols{K}, Down{X}, sm, sn, 0, kC);
    keep();
    product<kOut<E>, kOut<E>, kOut<E>>(y, TriRows{stage + L::kP}, Down{U}, m, nn, 0, m + 16);
    const int64_t p = lo + static_cast<int64_t>(i) * kC;
#pragma unroll
    for (int t = 0; t < L::kN; ++t)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = m + g + j * 8, c = nn + t * 8 + t2;
        if (p + r >= hi) continue;
        const bool on = gt.beta[r] != 0.f;  // a masked position gives 0
        auto* to = a.y + (p + r) * a.y_stride + h * a.dv + v0 + c;
        if (c < cols) E::store(to, on ? y[t][2 * j] : 0.f);
        if (c + 1 < cols) E::store(to + 1, on ? y[t][2 * j + 1] : 0.f);
      }
    if (L::kStages == 1 && i + 1 < n) {
      __syncthreads();  // the stage is free
      load(i + 1);
    }
  }
  if (a.state_out != nullptr) {
    float* to = a.state_out + (slot * a.heads + h) * matrix;
    each([&](int t, int j, size_t at) { to[at] = S[t][j]; });
  }
}

template <class E>
int launch_scan(const Args<E>& a, cudaStream_t st) {
  static std::atomic<uint64_t> done[2] = {{0}, {0}};
  auto go = [&](auto kernel, int smem, int vs, std::atomic<uint64_t>& flag) {
    int r = opt_in(reinterpret_cast<const void*>(kernel), smem, flag);
    if (r) return r;
    kernel<<<dim3(a.n_seqs, a.heads, (a.dv + vs - 1) / vs), kThreads, smem, st>>>(a);
    return check_launch("scan_kernel");
  };
  return a.dk <= 64 ? go(scan_kernel<E, 64, 32>, Scan<E, 64, 32>::kSmem, 32, done[0])
                    : go(scan_kernel<E, 128, 32>, Scan<E, 128, 32>::kSmem, 32, done[1]);
}

// --------------------------------------------------------------------- step

// One token: a block has one sequence's state in one head, kV x 32 of the value
// columns, in registers from the load to the store.  Bound by memory: the state is
// read once and written once.
constexpr int kStepRows = kMaxDim / kWarps;  // a thread's rows: one in eight

template <class E, int kV>
__global__ void __launch_bounds__(kThreads) step_kernel(Args<E> a) {
  __shared__ float part[kWarps][32 * kV];
  __shared__ float qs[kMaxDim], ks[kMaxDim];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.x, h = blockIdx.y, hk = h / (a.heads / a.keys);
  const int c = (blockIdx.z * 32 + lane) * kV;
  const int64_t slot = a.slots[row];
  if (slot < 0 || slot >= a.n_slots) {  // padding
    if (slot >= 0 && a.status != nullptr && threadIdx.x == 0 && h == 0 && blockIdx.z == 0)
      atomicOr(a.status, ENGRAM_ST_BAD_SLOT);
    if (warp == 0)
      for (int j = 0; j < kV; ++j)
        if (c + j < a.dv) E::store(a.y + row * a.y_stride + h * a.dv + c + j, 0.f);
    return;
  }
  const size_t at = (slot * a.heads + h) * (static_cast<size_t>(a.dk) * a.dv) + c;
  const bool in = c < a.dv;
  float S[kStepRows][kV];
#pragma unroll
  for (int i = 0; i < kStepRows; ++i) {
    const int r = warp + i * kWarps;
#pragma unroll
    for (int j = 0; j < kV; ++j) S[i][j] = 0.f;
    if (in && r < a.dk) {
      const float* from = a.state + at + static_cast<size_t>(r) * a.dv;
      if constexpr (kV == 4) {
        const float4 x = *reinterpret_cast<const float4*>(from);
        S[i][0] = x.x; S[i][1] = x.y; S[i][2] = x.z; S[i][3] = x.w;
      } else {
        S[i][0] = *from;
      }
    }
  }
  for (int i = threadIdx.x; i < kMaxDim; i += kThreads) {
    qs[i] = i < a.dk ? E::load(a.q + row * a.q_stride + hk * a.dk + i) : 0.f;
    ks[i] = i < a.dk ? E::load(a.k + row * a.k_stride + hk * a.dk + i) : 0.f;
  }
  const float f = 1.f / (1.f + expf(-E::load(a.g + row * a.g_stride + h)));
  const float beta = 1.f / (1.f + expf(-E::load(a.b + row * a.b_stride + h)));
  float v[kV], sum[kV];
#pragma unroll
  for (int j = 0; j < kV; ++j) {
    v[j] = c + j < a.dv ? E::load(a.v + row * a.v_stride + h * a.dv + c + j) : 0.f;
    sum[j] = 0.f;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kStepRows; ++i)
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      S[i][j] *= f;
      sum[j] = fmaf(S[i][j], ks[warp + i * kWarps], sum[j]);
    }
#pragma unroll
  for (int j = 0; j < kV; ++j) part[warp][lane * kV + j] = sum[j];
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kV; ++j) {
    float seen = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) seen += part[w][lane * kV + j];
    const float u = beta * (v[j] - seen);
    sum[j] = 0.f;
#pragma unroll
    for (int i = 0; i < kStepRows; ++i) {
      S[i][j] = fmaf(ks[warp + i * kWarps], u, S[i][j]);
      sum[j] = fmaf(S[i][j], qs[warp + i * kWarps], sum[j]);
    }
  }
#pragma unroll
  for (int i = 0; i < kStepRows; ++i) {
    const int r = warp + i * kWarps;
    if (!in || r >= a.dk) continue;
    float* to = a.state_out + at + static_cast<size_t>(r) * a.dv;
    if constexpr (kV == 4) *reinterpret_cast<float4*>(to) = make_float4(S[i][0], S[i][1], S[i][2], S[i][3]);
    else *to = S[i][0];
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kV; ++j) part[warp][lane * kV + j] = sum[j];
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int j = 0; j < kV; ++j) {
      float y = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) y += part[w][lane * kV + j];
      if (c + j < a.dv) E::store(a.y + row * a.y_stride + h * a.dv + c + j, a.scale * y);
    }
  }
}

template <class E>
int launch_step(const Args<E>& a, int64_t batch, cudaStream_t st) {
  const bool vec = a.dv % 4 == 0 && aligned(a.state, 16) && aligned(a.state_out, 16);
  const int wide = vec ? 128 : 32;
  const dim3 grid(static_cast<unsigned>(batch), a.heads, (a.dv + wide - 1) / wide);
  if (vec) step_kernel<E, 4><<<grid, kThreads, 0, st>>>(a);
  else step_kernel<E, 1><<<grid, kThreads, 0, st>>>(a);
  return check_launch("step_kernel");
}

Space space(void* base, int64_t n_tokens, int64_t n_seqs, int32_t keys, int32_t heads, int32_t dk, int32_t dv, bool backward) {
  Space s{};
  const size_t units = static_cast<size_t>(max_chunks(n_tokens, n_seqs)) * heads;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    unsigned char* p = base == nullptr ? nullptr : static_cast<unsigned char*>(base) + at;
    at += train::round256(bytes);
    return p;
  };
  s.first = reinterpret_cast<int32_t*>(take(sizeof(int32_t) * (n_seqs + 1)));
  s.tri = take(units * kTriBytes);
  s.gates = reinterpret_cast<Gates*>(take(units * sizeof(Gates)));
  if (backward) {
    s.after = reinterpret_cast<float*>(take(units * dk * dv * sizeof(float)));
    s.writes = reinterpret_cast<float*>(take(static_cast<size_t>(n_tokens) * heads * dv * sizeof(float)));
    if (heads > keys) s.shared = reinterpret_cast<float*>(take(2 * static_cast<size_t>(n_tokens) * keys * dk * sizeof(float)));
  }
  s.bytes = at;
  return s;
}

}  // namespace delta
}  // namespace engram

using namespace engram;
using namespace engram::delta;

extern "C" size_t engram_delta_carry_bytes(int64_t n_tokens, int64_t n_seqs, int32_t heads, int32_t dk, int32_t dv) {
  if (n_tokens < 0 || n_seqs < 0 || heads < 1 || dk < 1 || dv < 1) return 0;
  return static_cast<size_t>(max_chunks(n_tokens, n_seqs)) * heads * dk * dv * sizeof(float);
}

extern "C" size_t engram_delta_workspace_bytes(int64_t n_tokens, int64_t n_seqs, int32_t key_heads, int32_t heads, int32_t dk,
                                               int32_t dv, int32_t backward) {
  if (n_tokens < 0 || n_seqs < 0 || key_heads < 1 || heads < 1 || dk < 1 || dv < 1) return 0;
  return space(nullptr, n_tokens, n_seqs, key_heads, heads, dk, dv, backward != 0).bytes;
}

extern "C" int engram_delta(const void* q_d, int64_t q_stride, const void* k_d, int64_t k_stride, const void* v_d,
                            int64_t v_stride, const void* g_d, int64_t g_stride, const void* b_d, int64_t b_stride,
                            int32_t type, int64_t n_tokens, int32_t key_heads, int32_t heads, int32_t dk, int32_t dv,
                            float scale, const int64_t* cu_seqlens_d, int64_t n_seqs, const int32_t* slots_d,
                            const uint8_t* mask_d, const float* state_d, float* state_out_d, int64_t n_slots, void* y_d,
                            int64_t y_stride, float* carry_d, void* workspace_d, size_t workspace_bytes,
                            int32_t* status_d, void* stream) {
  const bool has_state = state_d != nullptr || state_out_d != nullptr;
  int rc = check_sizes(type, n_tokens, key_heads, heads, dk, dv, n_seqs, n_slots, has_state, scale);
  if (rc) return rc;
  if (n_seqs == 0) return n_tokens == 0 ? ENGRAM_OK : fail(ENGRAM_E_SHAPE, "positions without a sequence");
  if (!cu_seqlens_d) return fail(ENGRAM_E_INVALID, "null device pointer: cu_seqlens");
  if (n_tokens > 0) {
    if ((rc = check_rows(q_d, type, q_stride, static_cast<int64_t>(key_heads) * dk, "q"))) return rc;
    if ((rc = check_rows(k_d, type, k_stride, static_cast<int64_t>(key_heads) * dk, "k"))) return rc;
    if ((rc = check_rows(v_d, type, v_stride, static_cast<int64_t>(heads) * dv, "v"))) return rc;
    if ((rc = check_rows(g_d, type, g_stride, heads, "g"))) return rc;
    if ((rc = check_rows(b_d, type, b_stride, heads, "b"))) return rc;
    if ((rc = check_rows(y_d, type, y_stride, static_cast<int64_t>(heads) * dv, "y"))) return rc;
  } else if (state_out_d == nullptr || state_out_d == state_d) {
    return ENGRAM_OK;
  }
  if (!aligned(state_d, 4) || !aligned(state_out_d, 4) || !aligned(carry_d, 4))
    return fail(ENGRAM_E_ALIGN, "states and carry must be aligned to their elements");
  if (!workspace_d) return fail(ENGRAM_E_INVALID, "null device pointer: workspace");
  if (!aligned(workspace_d, 256)) return fail(ENGRAM_E_ALIGN, "workspace must be 256-byte aligned");
  if (workspace_bytes < engram_delta_workspace_bytes(n_tokens, n_seqs, key_heads, heads, dk, dv, 0))
    return fail(ENGRAM_E_RANGE, "workspace too small");
  if ((rc = check_device(nullptr))) return rc;
  auto go = [&](auto e) {
    using E = decltype(e);
    using T = typename E::T;
    Args<E> a{};
    a.q = static_cast<const T*>(q_d);
    a.k = static_cast<const T*>(k_d);
    a.v = static_cast<const T*>(v_d);
    a.g = static_cast<const T*>(g_d);
    a.b = static_cast<const T*>(b_d);
    a.y = static_cast<T*>(y_d);
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.g_stride = g_stride;
    a.b_stride = b_stride;
    a.y_stride = y_stride;
    a.cu = cu_seqlens_d;
    a.slots = slots_d;
    a.mask = mask_d;
    a.state = state_d;
    a.state_out = state_out_d;
    a.carry = carry_d;
    a.n_slots = n_slots;
    a.has_state = has_state;
    a.n_tokens = static_cast<int32_t>(n_tokens);
    a.n_seqs = static_cast<int32_t>(n_seqs);
    a.max_chunks = static_cast<int32_t>(max_chunks(n_tokens, n_seqs));
    a.keys = key_heads;
    a.heads = heads;
    a.dk = dk;
    a.dv = dv;
    a.scale = scale;
    a.vec = pieces(q_d, q_stride, E::kBytes) && pieces(k_d, k_stride, E::kBytes) && pieces(v_d, v_stride, E::kBytes) &&
            dk % 8 == 0 && dv % 8 == 0;
    a.status = status_d;
    const Space s = space(workspace_d, n_tokens, n_seqs, key_heads, heads, dk, dv, false);
    a.first = s.first;
    a.tri = s.tri;
    a.gates = s.gates;
    int r = launch_prepare<E>(a, as_stream(stream));
    return r ? r : launch_scan<E>(a, as_stream(stream));
  };
  return type == ENGRAM_T_BF16 ? go(train::Bf16{}) : go(train::F32{});
}

extern "C" int engram_delta_step(const void* q_d, int64_t q_stride, const void* k_d, int64_t k_stride, const void* v_d,
                                 int64_t v_stride, const void* g_d, int64_t g_stride, const void* b_d, int64_t b_stride,
                                 int32_t type, int64_t batch, int32_t key_heads, int32_t heads, int32_t dk, int32_t dv,
                                 float scale, const int32_t* slots_d, const float* state_d, float* state_out_d,
                                 int64_t n_slots, void* y_d, int64_t y_stride, int32_t* status_d, void* stream) {
  int rc = check_sizes(type, batch, key_heads, heads, dk, dv, 0, n_slots, true, scale);
  if (rc) return rc;
  if (batch == 0) return ENGRAM_OK;
  if (!slots_d || !state_d || !state_out_d) return fail(ENGRAM_E_INVALID, "null device pointer: slots or state");
  if ((rc = check_rows(q_d, type, q_stride, static_cast<int64_t>(key_heads) * dk, "q"))) return rc;
  if ((rc = check_rows(k_d, type, k_stride, static_cast<int64_t>(key_heads) * dk, "k"))) return rc;
  if ((rc = check_rows(v_d, type, v_stride, static_cast<int64_t>(heads) * dv, "v"))) return rc;
  if ((rc = check_rows(g_d, type, g_stride, heads, "g"))) return rc;
  if ((rc = check_rows(b_d, type, b_stride, heads, "b"))) return rc;
  if ((rc = check_rows(y_d, type, y_stride, static_cast<int64_t>(heads) * dv, "y"))) return rc;
  if (!aligned(state_d, 4) || !aligned(state_out_d, 4)) return fail(ENGRAM_E_ALIGN, "states must be aligned to their elements");
  if ((rc = check_device(nullptr))) return rc;
  auto go = [&](auto e) {
    using E = decltype(e);
    using T = typename E::T;
    Args<E> a{};
    a.q = static_cast<const T*>(q_d);
    a.k = static_cast<const T*>(k_d);
    a.v = static_cast<const T*>(v_d);
    a.g = static_cast<const T*>(g_d);
    a.b = static_cast<const T*>(b_d);
    a.y = static_cast<T*>(y_d);
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.g_stride = g_stride;
    a.b_stride = b_stride;
    a.y_stride = y_stride;
    a.slots = slots_d;
    a.state = state_d;
    a.state_out = state_out_d;
    a.n_slots = n_slots;
    a.keys = key_heads;
    a.heads = heads;
    a.dk = dk;
    a.dv = dv;
    a.scale = scale;
    a.status = status_d;
    return launch_step<E>(a, batch, as_stream(stream));
  };
  return type == ENGRAM_T_BF16 ? go(train::Bf16{}) : go(train::F32{});
}
