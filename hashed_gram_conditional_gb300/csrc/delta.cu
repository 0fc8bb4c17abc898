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

// first[s]: how many chunks the sequences before s have.  line[s]: how much of a head's line
// they take (see Item), and behind the last one the blocks' share of it.
template <class E>
__global__ void __launch_bounds__(1024) first_kernel(Args<E> a) {
  __shared__ int64_t sums[2][32], before[2];
  __shared__ int most[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x < 2) before[threadIdx.x] = 0;
  for (int k = threadIdx.x; k < a.blocks; k += 1024) a.given[k] = 0;
  // the sum over the block's threads before this one and over what came before, and on to the next 1024
  auto sum_before = [&](int64_t n, int which) {
    int64_t sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += x;
    }
    __syncthreads();
    if (lane == 31) sums[which][warp] = sum;
    __syncthreads();
    int64_t at = before[which] + sum - n;
    for (int w = 0; w < warp; ++w) at += sums[which][w];
    __syncthreads();
    if (threadIdx.x == 1023) before[which] = at + n;
    return at;
  };
  int longest = 1;
  for (int s0 = 0; s0 < a.n_seqs; s0 += 1024) {
    const int s = s0 + threadIdx.x;
    int n = 0, cost = 0;
    if (s < a.n_seqs) {
      int lo, hi;
      bounds(a, s, lo, hi);
      n = (hi - lo + kC - 1) / kC;
    }
    // (sequences that lie over one another could give more chunks than there is room for)
    const int64_t all = sum_before(n, 0);
    const int at = static_cast<int>(all < a.max_chunks ? all : a.max_chunks);
    if (s < a.n_seqs) {
      int64_t slot;
      n = min(n, a.max_chunks - at);
      cost = live_slot(a, s, at, n, slot) ? n + 1 : 1;
      longest = max(longest, cost);
      a.first[s] = at;
    }
    const int64_t line = sum_before(cost, 1);
    if (s < a.n_seqs) a.line[s] = line;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, o));
  if (lane == 0) most[warp] = longest;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int w = 1; w < 32; ++w) longest = max(longest, most[w]);
  a.first[a.n_seqs] = static_cast<int>(before[0] < a.max_chunks ? before[0] : a.max_chunks);
  const int64_t share = (before[1] * a.heads * a.slices + a.blocks - 1) / a.blocks;
  a.line[a.n_seqs] = before[1];
  a.line[a.n_seqs + 1] = share > longest ? share : longest;
}

// ---------------------------------------------------------------- M, P, gates

constexpr int kPitch = kC + 4;  // of fp32 64 x 64 matrices

// dst = sign A B, 16 x 16, by a warp, in fp32's precision: each operand as two tf32
// terms (22 bits), three products.
__device__ __forceinline__ void small_product(float* dst, const float* a, const float* b, int depth, float sign) {
  const int l = lane_id(), g = l >> 2, t = l & 3;
  float c[2][4] = {}, small[2][4] = {};
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
      auto step = [&](float (&c)[4], const uint32_t (&x)[4], const uint32_t (&y)[2]) {
        asm volatile(
            "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
            "%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(y[0]), "r"(y[1]));
      };
      step(small[n], al, bh);
      step(small[n], ah, bl);
      step(c[n], ah, bh);
    }
  }
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j) dst[(g + (j >> 1) * 8) * kPitch + n * 8 + 2 * t + (j & 1)] = sign * (c[n][j] + small[n][j]);
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

constexpr int kPrepareThreads = 128;
// Factors of D between two blocks of 16 positions: from a block's first position to its
// others, and from positions before it to its first.
struct Factors {
  float row[kC], column[3][kC];  // column[bt - 1][i], i < 16 bt
};
template <class E, int KD>
constexpr int kPrepareRoom = std::max(2 * kIn<E> * mat_bytes(kC, KD), 2 * kC * kPitch * 4);
template <class E, int KD>
constexpr int kPrepareSmem = kPrepareRoom<E, KD> + static_cast<int>(sizeof(Gates) + sizeof(Factors));

// A block of four warps makes M and P of one head in one chunk.  K K^T and Q K^T stay in
// the registers until they are A and P; A and M take the place of K and Q.  Heads that
// share a key head compute its products again, which is little beside the rest; blocks of
// eight warps for all of them took twice as long (110 us against 52, now 48, for 2560 chunks
// and heads, dk = 128).  Bound by instructions issued (2.0 a clock and SM) and the waits
// between the inverse's steps.
template <class E, int KD>
__global__ void __launch_bounds__(kPrepareThreads) prepare_kernel(Args<E> a) {
  constexpr int kRoom = kPrepareRoom<E, KD>;
  extern __shared__ __align__(128) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t2 = (lane & 3) * 2;
  Chunk ch;
  if (!chunk_at(a, blockIdx.x, ch)) return;
  if (!ch.live) {
    if (a.carry != nullptr && tid == 0) a.gates[unit_of(a, blockIdx.x, blockIdx.y)].into[0] = kPadding;
    return;
  }
  const Mat K = mat<kC, KD>(smem_u32(smem)), Q = mat<kC, KD>(K.base + kIn<E> * K.term);
  float *A = reinterpret_cast<float*>(smem), *M = A + kC * kPitch;
  Gates& gt = *reinterpret_cast<Gates*>(smem + kRoom);
  Factors& fc = *reinterpret_cast<Factors*>(smem + kRoom + sizeof(Gates));
  const uint8_t* mask = a.mask != nullptr ? a.mask + ch.start : nullptr;
  const int h = blockIdx.y, hk = h / (a.heads / a.keys);
  load_rows<E, KD, kPrepareThreads>(K, a.k + ch.start * a.k_stride + hk * a.dk, a.k_stride, ch.len, a.dk, mask, a.vec);
  load_rows<E, KD, kPrepareThreads>(Q, a.q + ch.start * a.q_stride + hk * a.dk, a.q_stride, ch.len, a.dk, mask, a.vec);
  copies_begun();
  if (warp == 0) {  // c, two positions a lane: multiples of 1/256 as integers, and the rest
    int hi[2];
    float lo[2], beta[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int r = lane * 2 + j;
      const bool on = r < ch.len && !(mask != nullptr && mask[r]);
      const int64_t t = ch.start + (on ? r : 0);
      // gates below -80 count as -80, b below -40 as -40 (a NaN stays)
      float x = E::load(a.g + t * a.g_stride + h), b = E::load(a.b + t * a.b_stride + h);
      x = x < -80.f ? -80.f : x;
      b = b < -40.f ? -40.f : b;
      x = on ? (x < 0.f ? x - log1pf(expf(x)) : -log1pf(expf(-x))) : 0.f;
      beta[j] = on ? 1.f / (1.f + expf(-b)) : 0.f;
      hi[j] = __float2int_rn(x * 256.f);  // (0 for a NaN, which the rest then is)
      lo[j] = x - static_cast<float>(hi[j]) * (1.f / 256.f);
    }
    int sum_hi = hi[0] + hi[1];
    float sum_lo = lo[0] + lo[1];
    const int own_hi = sum_hi;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, sum_hi, o);
      const float y = __shfl_up_sync(0xffffffffu, sum_lo, o);
      if (lane >= o) {
        sum_hi += x;
        sum_lo += y;
      }
    }
    float before = __shfl_up_sync(0xffffffffu, sum_lo, 1);
    before = lane == 0 ? 0.f : before;
    const int all_hi = __shfl_sync(0xffffffffu, sum_hi, 31);
    const float all_lo = __shfl_sync(0xffffffffu, sum_lo, 31);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int r = lane * 2 + j, to = sum_hi - own_hi + hi[0] + (j ? hi[1] : 0);
      const float rest = j ? sum_lo : before + lo[0];
      gt.hi[r] = static_cast<float>(to) * (1.f / 256.f);  // exact: below 2^24 / 256
      gt.lo[r] = rest;
      gt.into[r] = expf(static_cast<float>(to) * (1.f / 256.f) + rest);
      gt.last[r] = expf(static_cast<float>(all_hi - to) * (1.f / 256.f) + (all_lo - rest));
      gt.beta[r] = beta[j];
    }
  }
  copies_done();
  __syncthreads();
  // (each factor is at most 1: what underflows is nothing beside D's own 2^-126)
  for (int i = tid; i < 4 * kC; i += kPrepareThreads) {
    const int bt = i < kC ? (i >> 4) : (i >> 6), to = i < kC ? i : bt * 16, from = i < kC ? bt * 16 : i & 63;
    if (from <= to) (&fc.row[0])[i] = expf((gt.hi[to] - gt.hi[from]) + (gt.lo[to] - gt.lo[from]));
  }
  // K K^T and Q K^T: the triangle's ten blocks of 16 x 16 in turn, three a warp at most
  float ck[3][2][4], cq[3][2][4];
  auto block = [&](int n, int& bt, int& bi) {
    const int b = warp + n * 4;
    bt = b >= 6 ? 3 : b >= 3 ? 2 : b >= 1 ? 1 : 0;
    bi = b - bt * (bt + 1) / 2;
    return b < kBlocks;
  };
#pragma unroll
  for (int n = 0; n < 3; ++n) {
    clear(ck[n]);
    clear(cq[n]);
    int bt, bi;
    if (!block(n, bt, bi)) continue;
    if constexpr (kIn<E> == 1) {
#pragma unroll 4
      for (int k = 0; k < KD; k += 16) {
        uint32_t fk[4], fq[4], fb[2][2];
        Rows{K}(fk, bt * 16, k, 0);
        Rows{Q}(fq, bt * 16, k, 0);
        Across{K}.get<2>(fb, k, bi * 16, 0);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mma(ck[n][e], fk, fb[e][0], fb[e][1]);
          mma(cq[n][e], fq, fb[e][0], fb[e][1]);
        }
      }
    } else {
      product<kIn<E>, kIn<E>, kIn<E>>(ck[n], Rows{K}, Across{K}, bt * 16, bi * 16, 0, KD);
      product<kIn<E>, kIn<E>, kIn<E>>(cq[n], Rows{Q}, Across{K}, bt * 16, bi * 16, 0, KD);
    }
  }
  __syncthreads();  // K and Q are no longer needed
  const size_t unit = unit_of(a, blockIdx.x, h);
  unsigned char* tri = a.tri + unit * kTriBytes;
  for (int i = tid; i < static_cast<int>(sizeof(Gates)) / 4; i += kPrepareThreads)
    reinterpret_cast<float*>(a.gates + unit)[i] = reinterpret_cast<const float*>(&gt)[i];
#pragma unroll
  for (int n = 0; n < 3; ++n) {
    int bt, bi;
    if (!block(n, bt, bi)) continue;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = bi * 16 + e * 8 + t2;
      const float2 hi = *reinterpret_cast<const float2*>(&gt.hi[i]), lo = *reinterpret_cast<const float2*>(&gt.lo[i]);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int t = bt * 16 + g + j * 8;
        float d0, d1;
        if (bt > bi) {
          const float2 c = *reinterpret_cast<const float2*>(&fc.column[bt - 1][i]);
          d0 = fc.row[t] * c.x;
          d1 = fc.row[t] * c.y;
        } else {
          d0 = expf((gt.hi[t] - hi.x) + (gt.lo[t] - lo.x));
          d1 = expf((gt.hi[t] - hi.y) + (gt.lo[t] - lo.y));
        }
        const float beta = gt.beta[t];
        float k0 = beta * d0 * ck[n][e][2 * j], k1 = beta * d1 * ck[n][e][2 * j + 1];
        float q0 = a.scale * d0 * cq[n][e][2 * j], q1 = a.scale * d1 * cq[n][e][2 * j + 1];
        if (bt == bi) {  // (above the diagonal there may be anything)
          if (i >= t) k0 = 0.f;
          if (i + 1 >= t) k1 = 0.f;
          if (i > t) q0 = 0.f;
          if (i + 1 > t) q1 = 0.f;
        }
        *reinterpret_cast<float2*>(A + t * kPitch + i) = make_float2(k0, k1);
        if (E::kBytes == 4 || a.carry != nullptr) put_tri<kStateTerms>(tri + kStateTerms * kTerm, t, i, q0, q1);
        else put_tri<kOut<E>>(tri + kStateTerms * kTerm, t, i, q0, q1);
      }
    }
  }
  __syncthreads();
  const int m = warp * 16;
  // (I + A)^-1: a warp's block of 16 by substitution, a column a lane; then twice
  // [M11 0; -M22 A21 M11 M22].  A's blocks above the diagonal hold what comes in between.
  if (lane < 16) {
    const float* D = A + m * (kPitch + 1);
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s0 = i == lane ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
      for (int j = 0; j < i; ++j) {
        float& s = j & 1 ? s1 : s0;
        s = fmaf(-D[i * kPitch + j], x[j], s);
      }
      x[i] = s0 + s1;
      M[(m + i) * kPitch + m + lane] = x[i];
    }
  }
  __syncthreads();
  if (warp < 2) {
    const int o = warp * 32 * (kPitch + 1), down = 16 * kPitch;
    small_product(A + o + 16, A + o + down, M + o, 16, 1.f);
    __syncwarp();
    small_product(M + o + down, M + o + down + 16, A + o + 16, 16, -1.f);
  }
  __syncthreads();
  const int bm = (warp & 1) * 16, bn = (warp >> 1) * 16;
  // (a column block's upper half begins at its own rows)
  small_product(A + bm * kPitch + 32 + bn, A + (32 + bm) * kPitch + bn, M + bn * kPitch + bn, 32 - bn, 1.f);
  __syncthreads();
  small_product(M + (32 + bm) * kPitch + bn, M + (32 + bm) * kPitch + 32, A + 32 + bn, 16 + bm, -1.f);
  __syncthreads();
#pragma unroll 4
  for (int p = tid; p < kBlocks * 128; p += kPrepareThreads) {
    const int b = p >> 7, bt = b >= 6 ? 3 : b >= 3 ? 2 : b >= 1 ? 1 : 0, bi = b - bt * (bt + 1) / 2;
    const int t = bt * 16 + ((p >> 3) & 15), i = bi * 16 + (p & 7) * 2;
    const float2 x = *reinterpret_cast<const float2*>(M + t * kPitch + i);
    put_tri<kStateTerms>(tri, t, i, i <= t ? x.x * gt.beta[i] : 0.f, i + 1 <= t ? x.y * gt.beta[i + 1] : 0.f);
  }
}

template <class E>
int launch_first(const Args<E>& a, cudaStream_t st) {
  first_kernel<E><<<1, 1024, 0, st>>>(a);
  return check_launch("first_kernel");
}
template int launch_first<train::Bf16>(const Args<train::Bf16>&, cudaStream_t);
template int launch_first<train::F32>(const Args<train::F32>&, cudaStream_t);

// M, P and the gates of all chunks.
template <class E>
int launch_prepare(const Args<E>& a, cudaStream_t st) {
  if (a.max_chunks == 0) return ENGRAM_OK;
  auto go = [&](auto kernel, int smem, std::atomic<uint64_t>& done) {
    int r = opt_in(reinterpret_cast<const void*>(kernel), smem, done);
    if (r) return r;
    kernel<<<dim3(a.max_chunks, a.heads), kPrepareThreads, smem, st>>>(a);
    return check_launch("prepare_kernel");
  };
  static std::atomic<uint64_t> done[2] = {{0}, {0}};
  return a.dk <= 64 ? go(prepare_kernel<E, 64>, kPrepareSmem<E, 64>, done[0])
                    : go(prepare_kernel<E, 128>, kPrepareSmem<E, 128>, done[1]);
}

// --------------------------------------------------------------------- scan

// A chunk in a quad (16 value columns, dk = 128) is 48 + 32 + 48 + 24 + 48 tensor
// instructions a warp at most: K S and U and what is added to S in three terms, Q S and
// P U in two.  bf16: the next chunk's inputs are copied meanwhile; fp32's terms are made
// on the way to shared memory and take the room.
//
// Four quads a block (16,384 positions in 4 sequences, 40 heads of 128, bf16: 768 us where no
// sequence is longer than a block's share, 5.6 a chunk): the tensor cores are busy for 42 %
// of the time and shared memory for 72; what is left are waits of warps that have nothing
// else to do between a quad's barriers.  One quad (16,381
// positions, 10 heads: 520 us, 2.0 a chunk): instructions that follow one another.  A form
// with 16 columns and the whole of their state a warp, without anything handed on, read a
// third of the shared memory and took as long: two warps on each part of an SM are all
// that its registers allow.
template <class E, int KD, int NQ>
struct Scan {
  static constexpr int kT = kAlone<NQ> ? kCopiers : NQ * 128, kThreads = kAlone<NQ> ? 256 + kCopiers : kT;
  static constexpr int kStages = E::kBytes == 2 ? 2 : 1, kB = kC / 16;
  static constexpr int kK = 0, kQ = kK + kIn<E> * mat_bytes(kC, KD), kV = kQ + kIn<E> * mat_bytes(kC, KD);
  static constexpr int kM = kV + kIn<E> * mat_bytes(kC, 16 * NQ), kP = kM + kStateTerms * kTerm, kG = kP + kOut<E> * kTerm;
  static constexpr int kStage = kG + static_cast<int>(sizeof(Gates)), kQuads = kStages * kStage;
  // a quad's operands: S^T; X^T, and (where there are four quads in its place) (e^(c_last - c)
  // U)^T; U^T
  static constexpr int kX = KD / 16 * kStateTerms * 512, kL = kAlone<NQ> ? kX + kB * kStateTerms * 512 : kX;
  static constexpr int kU = kL + kB * kStateTerms * 512, kQuad = kU + kB * kOut<E> * 512;
  static constexpr int kSmem = kQuads + NQ * kQuad;
};

template <class E, int KD, int NQ>
__global__ void __launch_bounds__(Scan<E, KD, NQ>::kThreads, 1) scan_kernel(Args<E> a) {
  using L = Scan<E, KD, NQ>;
  constexpr int kT = L::kT, kI = kIn<E>, kO = kOut<E>, kS = kStateTerms, kB = L::kB, kR = KD / 64;  // kR: a warp's blocks of S^T
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ Stages stages;
  __shared__ Item item;
  const uint32_t base = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, g = lane >> 2, t2 = (lane & 3) * 2;
  const int quad = kAlone<NQ> ? 0 : tid >> 7, w = ((tid >> 5) + quad) & 3;  // w: the warp's quarter
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
    const int h = uniform(item.h), v0 = uniform(item.v0), lo = uniform(item.lo), hi = uniform(item.hi), c0 = uniform(item.c0),
              from = uniform(item.from), n = uniform(item.to);
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
    auto stage_of = [&](int i) { return kAlone<NQ> ? i % L::kStages : (used + i - from) & 1; };
    auto hand_state = [&](int i) {  // the state in front of chunk i
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        const int kb = w * kR + r;
        uint32_t f[kS][4];
        as_operand<kS>(f, S[2 * r], S[2 * r + 1]);
        hand<kS>(own + kb * (kS * 512), f);
        if (a.carry == nullptr || vw >= a.dv || kb * 16 >= a.dk) continue;
        float* to = a.carry + unit_of(a, c0 + i, h) * saved;
        if constexpr (E::kBytes == 2) save_block(block_of(to, a.dk, vw >> 4, kb), f);
        else save_rows(to, a.dk, a.dv, vw, kb * 16, S[2 * r], S[2 * r + 1]);
      }
    };
    const int copier = tid - (kAlone<NQ> ? 256 : 0);  // a copying thread's number
    auto load = [&](int i) {
      const uint32_t stage = base + stage_of(i) * L::kStage;
      const int64_t p = lo + static_cast<int64_t>(i) * kC;
      const int len = hi - p < kC ? static_cast<int>(hi - p) : kC;
      const uint8_t* mask = a.mask != nullptr ? a.mask + p : nullptr;
      const size_t unit = unit_of(a, c0 + i, h);
      load_rows<E, KD, kT>(mat<kC, KD>(stage + L::kK), a.k + p * a.k_stride + hk * a.dk, a.k_stride, len, a.dk, mask, a.vec, copier);
      load_rows<E, KD, kT>(mat<kC, KD>(stage + L::kQ), a.q + p * a.q_stride + hk * a.dk, a.q_stride, len, a.dk, mask, a.vec, copier);
      load_rows<E, 16 * NQ, kT>(mat<kC, 16 * NQ>(stage + L::kV), a.v + p * a.v_stride + static_cast<int64_t>(h) * a.dv + v0,
                                a.v_stride, len, cols, mask, a.vec, copier);
      if constexpr (kAlone<NQ>) {
        load_tri<kO, kT>(stage + L::kM, stage + L::kP, a.tri + unit * kTriBytes, copier);
        load_gates<kT>(stage + L::kG, a.gates + unit, copier);
        copies_begun();
      } else {
        stage_copies(stages, stage_of(i), stage + L::kM, a.tri + unit * kTriBytes, (kS + kO) * kTerm, stage + L::kG, a.gates + unit,
                     a.vec, a.absent);
      }
    };
    if (!kAlone<NQ> && n > from) load(from);
    // Y^T of the warp's positions: first what Q reads of the state, then of the chunk's writes
    using Out = Sums<2, kO == 3>;
    auto scaled = [&](Out& y, const Gates& gt) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const float2 into = *reinterpret_cast<const float2*>(&gt.into[w * 16 + t * 8 + t2]);
#pragma unroll
        for (int j = 0; j < 4; ++j) y.main[t][j] = y.sum(t, j) * (a.scale * (j & 1 ? into.y : into.x));
      }
      if constexpr (kO == 3) clear(y.small);
    };
    auto finish = [&](Out& y, const Gates& gt, uint32_t stage, int i) {
      for (int ib = 0; ib <= w; ++ib) {
        uint32_t fa[kO][4];
        take<kO>(own + L::kU + ib * (kO * 512), fa);
#pragma unroll
        for (int j = 0; j < kO; ++j) {
          uint32_t fb[2][2];
          TriAcross{stage + L::kP}.get(fb, ib, w, j);
          terms<kO, kO>(y, fa, fb, j);
        }
      }
      float out[2][4];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) out[t][j] = y.sum(t, j);
      const int64_t p = lo + static_cast<int64_t>(i) * kC;
      store_rows<E>(a.y + p * a.y_stride + static_cast<int64_t>(h) * a.dv, a.y_stride, w * 16,
                    hi - p < kC ? static_cast<int>(hi - p) : kC, vw, a.dv, a.pairs, gt.beta, out);
    };
    if (kAlone<NQ> && copier >= 0) {
      if (n > from) load(from);
      for (int i = from; i < n; ++i) {
        copies_done();
        __syncthreads();
        if (L::kStages == 1 && i + 1 < n) __syncthreads();
        if (i + 1 < n) load(i + 1);
      }
      continue;
    }
    if (kAlone<NQ> && tid >= 128) {  // the quad's Y
      for (int i = from; i < n; ++i) {
        const uint32_t stage = base + (i % L::kStages) * L::kStage;
        const Mat Q = mat<kC, KD>(stage + L::kQ);
        const Gates& gt = *reinterpret_cast<const Gates*>(smem + (i % L::kStages) * L::kStage + L::kG);
        __syncthreads();
        Out y;
        y.clear_all();
#pragma unroll 4
        for (int kb = 0; kb < KD / 16; ++kb) {
          uint32_t fa[kO][4];
          take<kO>(own + kb * (kS * 512), fa);
#pragma unroll
          for (int j = 0; j < kI; ++j) {
            uint32_t fb[2][2];
            Across{Q}.get<2>(fb, kb * 16, w * 16, j);
            terms<kO, kO>(y, fa, fb, j);
          }
        }
        asm volatile("bar.arrive 6, 256;" ::: "memory");  // S^T is no longer needed here
        scaled(y, gt);
        asm volatile("bar.sync 5, 256;" ::: "memory");  // U^T is here
        finish(y, gt, stage, i);
        if (L::kStages == 1 && i + 1 < n) __syncthreads();
      }
      continue;
    }
    clear(S);
    if (item.take) {
      take_state(a.between + static_cast<size_t>(share + 1) * kHandedOn, S, NQ * 128);
    } else if (a.state != nullptr) {
      const float* given = a.state + (slot * a.heads + h) * matrix;
      each([&](int t, int j, size_t at) { S[t][j] = given[at]; });
    }
    if (n > from) hand_state(from);
    for (int i = from; i < n; ++i) {
      const uint32_t stage = base + stage_of(i) * L::kStage;
      const Mat K = mat<kC, KD>(stage + L::kK), Q = mat<kC, KD>(stage + L::kQ), V = mat<kC, 16 * NQ>(stage + L::kV);
      const Gates& gt = *reinterpret_cast<const Gates*>(smem + stage_of(i) * L::kStage + L::kG);
      if constexpr (kAlone<NQ>) {
        __syncthreads();  // the chunk and the states are here, and the other stage is free
      } else {
        quad_sync(quad);  // the states are here
        stage_wait(stages, stages.here[stage_of(i)], (used + i - from) >> 1, a.status);
      }
      // ---- (K S)^T and (Q S)^T
      Sums<2, true> x;
      Out y;
      x.clear_all();
      if (!kAlone<NQ>) y.clear_all();
#pragma unroll 4
      for (int kb = 0; kb < KD / 16; ++kb) {
        uint32_t fa[kS][4];
        take<kS>(own + kb * (kS * 512), fa);
#pragma unroll
        for (int j = 0; j < kI; ++j) {
          uint32_t fk[2][2], fq[2][2];
          Across{K}.get<2>(fk, kb * 16, w * 16, j);
          if (!kAlone<NQ>) Across{Q}.get<2>(fq, kb * 16, w * 16, j);
#pragma unroll
          for (int e = 0; e < kS; ++e) {
            if (e + j < kS) x.add(e, j, fa[e], fk);
            if (!kAlone<NQ> && e + j < kO) y.add(e, j, fa[e], fq);
          }
        }
      }
      // ---- X^T, of the warp's positions: rows w * 16 + t2 (+ 1, + 8), columns vw + g (+ 8)
      {
        float c[2][4];
        clear(c);
#pragma unroll
        for (int j = kI - 1; j >= 0; --j) {
          uint32_t f[4];
          Cols{V}(f, quad * 16, w * 16, j);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            c[q >> 1][(q & 1) * 2] += lo_of(f[q]);
            c[q >> 1][(q & 1) * 2 + 1] += hi_of(f[q]);
          }
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const float2 into = *reinterpret_cast<const float2*>(&gt.into[w * 16 + t * 8 + t2]);
#pragma unroll
          for (int j = 0; j < 4; ++j) c[t][j] = fmaf(-(j & 1 ? into.y : into.x), x.sum(t, j), c[t][j]);
        }
        if (!kAlone<NQ>) scaled(y, gt);
        uint32_t f[kS][4];
        as_operand<kS>(f, c[0], c[1]);
        hand<kS>(own + L::kX + w * (kS * 512), f);
      }
      quad_sync(quad);
      // ---- U^T
      x.clear_all();
      for (int ib = 0; ib <= w; ++ib) {
        uint32_t fa[kS][4];
        take<kS>(own + L::kX + ib * (kS * 512), fa);
#pragma unroll
        for (int j = 0; j < kS; ++j) {
          uint32_t fb[2][2];
          TriAcross{stage + L::kM}.get(fb, ib, w, j);
          terms<kS, kS>(x, fa, fb, j);
        }
      }
      {
        float u[2][4];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j) u[t][j] = x.sum(t, j);
        uint32_t f[kO][4], fl[kS][4];
        as_operand<kO>(f, u[0], u[1]);
        hand<kO>(own + L::kU + w * (kO * 512), f);
        if (kAlone<NQ>) asm volatile("bar.arrive 5, 256;" ::: "memory");
        if (a.carry != nullptr) {  // for the backward pass
          const int64_t p = lo + static_cast<int64_t>(i) * kC, wide = static_cast<int64_t>(a.heads) * a.dv;
          auto* to = kept_writes<E>(a) + p * wide + static_cast<int64_t>(h) * a.dv;
          const int len = hi - p < kC ? static_cast<int>(hi - p) : kC;
          store_rows<E>(to, wide, w * 16, len, vw, a.dv, a.dv % 2 == 0, gt.beta, u);
          if constexpr (E::kBytes == 2) {
            float rest[2][4];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int j = 0; j < 4; ++j) rest[t][j] = u[t][j] - lo_of(pack(u[t][j], 0.f));
            store_rows<E>(to + a.n_tokens * wide, wide, w * 16, len, vw, a.dv, a.dv % 2 == 0, gt.beta, rest);
          }
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const float2 last = *reinterpret_cast<const float2*>(&gt.last[w * 16 + t * 8 + t2]);
#pragma unroll
          for (int j = 0; j < 4; ++j) u[t][j] *= j & 1 ? last.y : last.x;
        }
        as_operand<kS>(fl, u[0], u[1]);
        if (!kAlone<NQ>) quad_sync(quad);  // X^T is no longer needed
        hand<kS>(own + L::kL + w * (kS * 512), fl);
      }
      if (!kAlone<NQ> && i + 1 < n) {
        if (i > from) stage_wait(stages, stages.done[stage_of(i + 1)], (used + i - 1 - from) >> 1, a.status);
        load(i + 1);
      }
      quad_sync(quad);
      // ---- S^T
      {
        const float total = gt.into[kC - 1];
        Sums<2 * kR, true> d;
        d.clear_all();
#pragma unroll
        for (int cb = 0; cb < kB; ++cb) {
          uint32_t fa[kS][4];
          take<kS>(own + L::kL + cb * (kS * 512), fa);
#pragma unroll
          for (int j = 0; j < kI; ++j) {
            uint32_t fb[2 * kR][2];
            Down{K}.get<2 * kR>(fb, cb * 16, w * kR * 16, j);
            terms<kS, kS>(d, fa, fb, j);
          }
        }
#pragma unroll
        for (int t = 0; t < 2 * kR; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j) S[t][j] = fmaf(S[t][j], total, d.sum(t, j));
      }
      if (kAlone<NQ>) asm volatile("bar.sync 6, 256;" ::: "memory");  // Q has read S^T
      if (i + 1 < n) hand_state(i + 1);
      if constexpr (kAlone<NQ>) {
        if (L::kStages == 1 && i + 1 < n) __syncthreads();  // the stage is free
      } else {
        finish(y, gt, stage, i);
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&stages.done[stage_of(i)]));
      }
    }
    used += n - from;
    if (item.give) {
      give_state(a.between + static_cast<size_t>(share) * kHandedOn, S, NQ * 128);
    } else if (a.state_out != nullptr) {
      float* to = a.state_out + (slot * a.heads + h) * matrix;
      each([&](int t, int j, size_t at) { to[at] = S[t][j]; });
    }
  }
  if (!kAlone<NQ>) stages_end(stages);
}

template <class E>
int launch_scan(const Args<E>& a, int sms, cudaStream_t st) {
  auto go = [&](auto kernel, int smem, int nq, std::atomic<uint64_t>& flag) {
    int r = opt_in(reinterpret_cast<const void*>(kernel), smem, flag);
    if (r) return r;
    kernel<<<a.blocks, nq == 1 ? 256 + kCopiers : nq * 128, smem, st>>>(a);
    return check_launch("scan_kernel");
  };
  static std::atomic<uint64_t> done[4] = {{0}, {0}, {0}, {0}};
  if constexpr (E::kBytes == 2)
    if (many_quads(a, sms))
      return a.dk <= 64 ? go(scan_kernel<E, 64, 4>, Scan<E, 64, 4>::kSmem, 4, done[0])
                        : go(scan_kernel<E, 128, 4>, Scan<E, 128, 4>::kSmem, 4, done[1]);
  return a.dk <= 64 ? go(scan_kernel<E, 64, 1>, Scan<E, 64, 1>::kSmem, 1, done[2])
                    : go(scan_kernel<E, 128, 1>, Scan<E, 128, 1>::kSmem, 1, done[3]);
}
static_assert(Scan<train::Bf16, 128, 4>::kSmem + sizeof(Stages) + sizeof(Item) <= 232448 && Scan<train::F32, 128, 1>::kSmem <= 232448, "a block's shared memory");

// --------------------------------------------------------------------- step

// One token: a block has one sequence's state in one head, kV x 32 of the value
// columns, in registers from the load to the store.  Bound by memory: the state is
// read once and written once (256 sequences of 40 heads of 128 x 128, 1.35 GB: 212 us, 6.4
// TB/s, 95 % of a copy's rate).
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

thread_local int selftest_absent = 0;

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
  s.line = reinterpret_cast<int64_t*>(take(sizeof(int64_t) * (n_seqs + 2)));
  const int64_t blocks = std::min<int64_t>(kMaxBlocks, n_seqs * heads * slices_of(dv, 1));
  s.given = reinterpret_cast<uint32_t*>(take(sizeof(uint32_t) * blocks));
  s.between = reinterpret_cast<float*>(take(sizeof(float) * kHandedOn * blocks));
  if (!backward) {
    s.tri = take(units * kTriBytes);
    s.gates = reinterpret_cast<Gates*>(take(units * sizeof(Gates)));
  } else {
    s.after = reinterpret_cast<float*>(take(units * saved_floats<train::Bf16>(dk, dv) * sizeof(float)));
    s.writes = reinterpret_cast<uint16_t*>(take(static_cast<size_t>(n_tokens) * heads * dv * 2 * sizeof(uint16_t)));
    // (a block's threads leave a chunk's sums, 64 x 128 of queries and of keys, as they hold them)
    if (heads > keys)
      s.shared = reinterpret_cast<float*>(
          take(static_cast<size_t>(max_chunks(n_tokens, n_seqs)) * keys * 2 * kC * (dk <= 64 ? 64 : 128) * sizeof(float)));
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
  // (both types' room: bf16's blocks are padded, fp32's matrices are not)
  const int64_t chunks = max_chunks(n_tokens, n_seqs);
  return kept_triangles_at(n_tokens, chunks, heads, dk, dv) + static_cast<size_t>(chunks) * heads * (kTriBytes + sizeof(Gates));
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
  if (!aligned(state_d, 4) || !aligned(state_out_d, 4)) return fail(ENGRAM_E_ALIGN, "states must be aligned to their elements");
  if (!aligned(carry_d, 16)) return fail(ENGRAM_E_ALIGN, "carry must be 16-byte aligned");
  if (!workspace_d) return fail(ENGRAM_E_INVALID, "null device pointer: workspace");
  if (!aligned(workspace_d, 256)) return fail(ENGRAM_E_ALIGN, "workspace must be 256-byte aligned");
  if (workspace_bytes < engram_delta_workspace_bytes(n_tokens, n_seqs, key_heads, heads, dk, dv, 0))
    return fail(ENGRAM_E_RANGE, "workspace too small");
  int sms = 0;
  if ((rc = check_device(&sms))) return rc;
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
    a.pairs = dv % 2 == 0 && y_stride % 2 == 0 && aligned(y_d, 2 * E::kBytes);
    a.status = status_d;
    const Space s = space(workspace_d, n_tokens, n_seqs, key_heads, heads, dk, dv, false);
    a.first = s.first;
    a.line = s.line;
    a.given = s.given;
    a.between = s.between;
    set_blocks(a, sms);
    a.tri = s.tri;
    a.gates = s.gates;
    if (a.carry != nullptr) use_kept_triangles(a);
    set_absent(a);
    int r = launch_first<E>(a, as_stream(stream));
    if (!r) r = launch_prepare<E>(a, as_stream(stream));
    return r ? r : launch_scan<E>(a, sms, as_stream(stream));
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

extern "C" int engram_selftest_delta_wait(int32_t which, const void* dy_d, const void* q_d, const void* k_d, const void* v_d,
                                          const void* g_d, const void* b_d, int32_t type, int64_t n_tokens, int32_t key_heads,
                                          int32_t heads, int32_t dk, int32_t dv, const int64_t* cu_seqlens_d, int64_t n_seqs,
                                          void* y_d, float* carry_d, void* dq_d, void* dk_d, void* dv_d, void* dg_d, void* db_d,
                                          void* workspace_d, size_t workspace_bytes, int32_t* status_d, void* stream) {
  if (which != 0 && which != 1) return fail(ENGRAM_E_INVALID, "which %d is not 0 or 1", which);
  const int64_t wk = static_cast<int64_t>(key_heads) * dk, wv = static_cast<int64_t>(heads) * dv;
  selftest_absent = which + 1;
  const int rc =
      dy_d == nullptr
          ? engram_delta(q_d, wk, k_d, wk, v_d, wv, g_d, heads, b_d, heads, type, n_tokens, key_heads, heads, dk, dv, 1.f,
                         cu_seqlens_d, n_seqs, nullptr, nullptr, nullptr, nullptr, 0, y_d, wv, carry_d, workspace_d,
                         workspace_bytes, status_d, stream)
          : engram_delta_grad(dy_d, wv, q_d, wk, k_d, wk, v_d, wv, g_d, heads, b_d, heads, type, n_tokens, key_heads, heads, dk,
                              dv, 1.f, cu_seqlens_d, n_seqs, nullptr, nullptr, carry_d, nullptr, 0, dq_d, wk, dk_d, wk, dv_d, wv,
                              dg_d, heads, db_d, heads, workspace_d, workspace_bytes, status_d, stream);
  selftest_absent = 0;
  return rc;
}
