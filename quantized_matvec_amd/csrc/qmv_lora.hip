// Low-rank adapters beside a 4-bit projection (include/qmv/tuning.h):
//   y[t] = W^ x[t] + bias + up[a] u[t],   u[t] = scale[a] down[a] x[t],   a = index[t]
// and, with g = dy and v[t] = scale[a] up[a]^T g[t],
//   dx[t] = W^^T g[t] + down[a]^T v[t],   d_down[a] = sum v[t] x[t]^T,   d_up[a] = sum g[t] u[t]^T.
//
// A few tokens: the projection in fp32 by gemv_4bit's kernels, gemm_4bit's or those of
// qmv_skinny.hip, then
// a workgroup for each token and part of the columns.  More: tokens are put in
// order of their adapters, so that tiles of the matrix cores meet one adapter,
// or few; u and v, a handful of values a token, are summed in fp32 and carried
// into the second products as two 16-bit terms (fp16: times a power of two).  Many: the weight is decoded
// once, and the adapters' part is added to the tile product's sums before they
// are rounded.
#include "qmv_tile.hpp"

namespace qmv {

typedef __attribute__((__vector_size__(4 * sizeof(float)))) float acc4_t;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4_t;

// The smaller kernels ask for two waves a SIMD: with one the compiler may use 512
// registers, puts sums into the accumulation half, and moves loads in flight there
// as well, each with a wait of its own (a gradient's step then takes six round trips
// to memory, 123 us for 4096 tokens x 14336).
template <int DT>
__device__ __forceinline__ acc4_t mma16(const frag_t &a, const frag_t &b, const acc4_t &c) {
  if constexpr (DT == kBF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(frag_h_t, a), __builtin_bit_cast(frag_h_t, b), c, 0, 0, 0);
}

__device__ __forceinline__ frag_t no_frag() { return __builtin_bit_cast(frag_t, make_uint4(0, 0, 0, 0)); }

// Eight values of one column out of rows in LDS (16-bit, `pitch` apart): within 16
// lanes, lane 4 e + q names 4 columns of row e, and lane i gets column i of rows 0 .. 3.
// p: this lane's first address; the second four rows lie 4 pitches on.
__device__ __forceinline__ frag_t read_column(const uint16_t *p, int pitch) {
  typedef short s4_t __attribute__((ext_vector_type(4)));
  typedef __attribute__((address_space(3))) s4_t lds_s4_t;
  const s4_t x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4_t *)p);
  const s4_t y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4_t *)(p + 4 * pitch));
  const uint2 a = __builtin_bit_cast(uint2, x), b = __builtin_bit_cast(uint2, y);
  return __builtin_bit_cast(frag_t, make_uint4(a.x, a.y, b.x, b.y));
}

// ---------------------------------------------------------------------------
// A few tokens
//
// u[s][t][r] = scale[a] * sum over piece s of x[t][k] down[a][r][k]: a workgroup of
// 4 waves takes one token and one piece of 512 terms; a wave goes through every
// fourth r, its lanes along k (16-byte loads, four rows of down in flight).  Bound by latency:
// 32 tokens x 4096 of rank 16 4.7 us, the up side for 14336 columns 5.9 us.
// ---------------------------------------------------------------------------
constexpr int kPiece = 512;

template <int DT>
__global__ __launch_bounds__(256) void lora_down_kernel(const uint16_t *__restrict__ x, int64_t K,
                                                        const uint16_t *__restrict__ down,
                                                        const float *__restrict__ scale, int count, int R,
                                                        const int32_t *__restrict__ index, float *__restrict__ u,
                                                        int64_t T) {
  const int64_t t = blockIdx.x;
  const int a = index[t];
  if (a < 0 || a >= count) return;  // nothing reads this token's u
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t k = (int64_t)blockIdx.y * kPiece + 8 * lane;
  const bool in = k < K;  // K is a multiple of 32
  float xf[8] = {};
  if (in) unpack8<DT>(*reinterpret_cast<const uint4 *>(x + t * K + k), xf);
  const float s = scale[a];
  const uint16_t *rows = down + (int64_t)a * R * K + (in ? k : 0);
  for (int r0 = wave; r0 < R; r0 += 16) {
    uint4 w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) w[q] = *reinterpret_cast<const uint4 *>(rows + (int64_t)min(r0 + 4 * q, R - 1) * K);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float af[8], acc = 0.f;
      unpack8<DT>(w[q], af);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc = fmaf(xf[i], in ? af[i] : 0.f, acc);
      acc = wave_sum(acc);
      if (lane == 0 && r0 + 4 * q < R) u[((int64_t)blockIdx.y * T + t) * R + r0 + 4 * q] = s * acc;
    }
  }
}

// out[t][n] = round(base[t][n] + bias[n] + sum_r up[a][n][r] u[t][r]), base in parts
// that are added up in order, and u's pieces: 256 / R of them side by side, then those sums
template <int DT, int ODT>
__global__ __launch_bounds__(256) void lora_up_kernel(const float *__restrict__ base, int base_parts, int64_t N,
                                                      const uint16_t *__restrict__ up, int count, int R,
                                                      const int32_t *__restrict__ index, const float *__restrict__ u,
                                                      int pieces, int64_t T, const uint16_t *__restrict__ bias,
                                                      typename Storage<ODT>::type *__restrict__ out) {
  __shared__ float part[256], us[128];
  const int64_t t = blockIdx.y;
  const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int a = index[t];
  float acc = 0.f, more = 0.f;
  if (n < N) {
    acc = base[t * N + n];
#pragma unroll 8
    for (int s = 1; s < base_parts; ++s) acc += base[(s * T + t) * N + n];
    if (bias) more = bits16_to_f32<DT>(bias[n]);
  }
  if (a >= 0 && a < count) {
    const uint16_t *row = up + ((int64_t)a * N + (n < N ? n : N - 1)) * R;
    uint4 first[2];  // in flight while u is added up
    first[0] = *reinterpret_cast<const uint4 *>(row);
    first[1] = *reinterpret_cast<const uint4 *>(row + (R > 8 ? 8 : 0));
    const int side = 256 / R, r = threadIdx.x % R, g = threadIdx.x / R;
    float sum = 0.f;
    if (g < side)
      for (int s = g; s < pieces; s += side) sum += u[((int64_t)s * T + t) * R + r];
    part[threadIdx.x] = sum;
    __syncthreads();
    if ((int)threadIdx.x < R) {
      sum = part[r];
      for (int j = 1; j < side && j < pieces; ++j) sum += part[j * R + r];
      us[r] = sum;
    }
    __syncthreads();
    float adapter = 0.f;
#pragma unroll 2
    for (int c = 0; c < R; c += 8) {
      float b[8];
      unpack8<DT>(c == 0 ? first[0] : c == 8 ? first[1] : *reinterpret_cast<const uint4 *>(row + c), b);
#pragma unroll
      for (int i = 0; i < 8; ++i) adapter = fmaf(us[c + i], b[i], adapter);
    }
    acc += adapter;
  }
  if (n < N) store_elem<ODT>(out, t * N + n, acc + more);
}

// ---------------------------------------------------------------------------
// Tokens in order of their adapters
// ---------------------------------------------------------------------------
constexpr int kMostAdapters = 4096;
constexpr int kUnit = 64;  // most places of a unit

struct Places {
  int32_t *order;    // [T] token at a place; those without an adapter come last
  int32_t *adapter;  // [T] its adapter (count: none)
  int32_t *start;    // [count + 2] first place of each adapter, of those without, and T
  int4 *units;       // (adapter, first place, last place + 1): at most 64 places of one adapter
  int32_t *n_units;
};

// Every workgroup counts all tokens (and those before its own 256), so that one
// launch without atomics on global memory gives a stable order; the first one
// writes the adapters' places and the units as well.  4096 tokens 9.4 us: two trips to
// memory, LDS counts and the scan, one after the other.
__global__ __launch_bounds__(256) void lora_order_kernel(const int32_t *__restrict__ index, int T, int count, Places pl) {
  __shared__ int total[kMostAdapters + 1], before[kMostAdapters + 1], sums[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, t0 = blockIdx.x * 256;
  const int buckets = count + 1;
  auto bucket = [&](int t) {
    const int a = index[t];
    return a >= 0 && a < count ? a : count;
  };
  for (int b = tid; b < buckets; b += 256) total[b] = before[b] = 0;
  const int my = t0 + tid < T ? bucket(t0 + tid) : -1;
  __syncthreads();
  for (int base = 0; base < T; base += 4096) {
    int held[16];  // loads in flight
#pragma unroll
    for (int q = 0; q < 16; ++q) held[q] = index[min(base + 256 * q + tid, T - 1)];
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      const int chunk = base + 256 * q;
      if (chunk + tid >= T) break;
      const int b = held[q] >= 0 && held[q] < count ? held[q] : count;
      const int one = __builtin_amdgcn_readfirstlane(b);
      const uint64_t here = __ballot(1);
      if (__ballot(b == one) == here) {  // prompts: neighbours have one adapter
        if (lane == __builtin_ctzll(here)) {
          atomicAdd(&total[one], __builtin_popcountll(here));
          if (chunk < t0) atomicAdd(&before[one], __builtin_popcountll(here));
        }
      } else {
        atomicAdd(&total[b], 1);
        if (chunk < t0) atomicAdd(&before[b], 1);
      }
    }
  }
  __syncthreads();
  // totals (and, in the first workgroup, units) to the sums before them
  const int each = (buckets + 255) / 256, b0 = min(tid * each, buckets), b1 = min(b0 + each, buckets);
  auto scan = [&](int v) {  // exclusive over the threads; the same barriers in every thread
    int upto = v;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int w = __shfl_up(upto, o);
      if (lane >= o) upto += w;
    }
    __syncthreads();
    if (lane == 63) sums[wave] = upto;
    __syncthreads();
    for (int w = 0; w < wave; ++w) upto += sums[w];
    return upto - v;
  };
  int tokens = 0, units = 0;
  for (int b = b0; b < b1; ++b) {
    tokens += total[b];
    units += (total[b] + kUnit - 1) / kUnit;
  }
  int at = scan(tokens), unit = scan(units);
  if (blockIdx.x == 0) {
    int place = at;
    for (int b = b0; b < b1; ++b) {
      pl.start[b] = place;
      const int end = place + total[b];
      const int n = (end - place + kUnit - 1) / kUnit;
#pragma unroll 4
      for (int i = 0; i < n; ++i) pl.units[unit + i] = make_int4(b, place + kUnit * i, min(place + kUnit * (i + 1), end), 0);
      unit += n;
      place = end;
    }
    if (tid == 255) {
      pl.start[buckets] = T;
      *pl.n_units = unit;
    }
  }
  for (int b = b0; b < b1; ++b) {
    const int n = total[b];
    total[b] = at;
    at += n;
  }
  __syncthreads();
  // this workgroup's tokens take the next places of their adapters, wave by wave
  int place = 0;
  for (int w = 0; w < 4; ++w) {
    if (w == wave) {
      for (uint64_t left = __ballot(my >= 0); left;) {
        const int one = __builtin_amdgcn_readlane(my, __builtin_ctzll(left));
        const uint64_t same = __ballot(my == one);
        const int next = before[one];
        if (my == one) place = total[one] + next + __builtin_popcountll(same & ((1ull << lane) - 1));
        if (lane == 0) before[one] = next + __builtin_popcountll(same);
        left &= ~same;
      }
    }
    __syncthreads();
  }
  if (my < 0) return;
  pl.order[place] = t0 + tid;
  pl.adapter[place] = my;
}

// ---------------------------------------------------------------------------
// parts[s][p][r] = scale[a] * sum over piece s of x[order[p]][l] down[a][r][l], or with
// TRANS of dy[..][l] up[a][l][r]: the inner values of the tokens, by place.
//
// A workgroup takes a unit and a piece of the sum, a wave every fourth 64 terms of
// it: 4 x NT tiles of v_mfma_f32_16x16x32, whose operands come straight from
// memory (rows are read once, an adapter's factor from L2).  With TRANS the
// factor's rows run the other way: 32 of them go through a part of LDS that is
// the wave's own, and come back by columns.  Waves are added up through LDS in
// order.  Bound by the read of the rows: 4099 tokens x 4096, rank 32 19 us (1.8 TB/s, with the factor's
// reads and the parts' writes), with TRANS 4096 x 14336, rank 16 35 us (3.4 TB/s).
// ---------------------------------------------------------------------------
template <int DT, int NT, bool TRANS>
__global__ __launch_bounds__(256, 2) void lora_shrink_kernel(const uint16_t *__restrict__ x, int64_t L, int piece,
                                                          const uint16_t *__restrict__ factor,
                                                          const float *__restrict__ scale, int count, int R, Places pl,
                                                          float *__restrict__ parts, int64_t T) {
  constexpr int kPitch = 16 * NT + (NT == 1 ? 0 : 16);  // rows 8 (mod 64) banks apart
  __shared__ __attribute__((aligned(16))) union {
    float red[4][4 * NT][64];
    uint16_t turn[TRANS ? 4 : 1][TRANS ? 32 * kPitch : 1];
  } sh;
  if ((int)blockIdx.x >= *pl.n_units) return;
  const int4 unit = pl.units[blockIdx.x];
  const int a = unit.x, places = unit.z - unit.y;
  if (a >= count) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, g = lane >> 4;
  const uint16_t *row[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) row[i] = x + (int64_t)pl.order[unit.y + min(16 * i + l16, places - 1)] * L + 8 * g;
  const uint16_t *frow[NT];  // columns past R: the last one again, not stored
#pragma unroll
  for (int j = 0; j < NT; ++j) frow[j] = factor + ((int64_t)a * R + min(16 * j + l16, R - 1)) * L + 8 * g;
  int turn_from[NT], turn_to[NT];  // TRANS: 16-byte chunks of 32 rows of R
  uint16_t *turn = sh.turn[TRANS ? wave : 0];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int c = 64 * j + lane, per = R / 8;
    turn_from[j] = c < 32 * per ? c * 8 : -1;
    turn_to[j] = (c / per) * kPitch + 8 * (c % per);
  }
  acc4_t acc[4][NT];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = acc4_t{0.f, 0.f, 0.f, 0.f};
  const int64_t l0 = (int64_t)blockIdx.y * piece, l1 = l0 + piece < L ? l0 + piece : L;
  for (int64_t l = l0 + 64 * wave; l < l1; l += 256) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int64_t k = l + 32 * s;
      if (k >= l1) break;  // L is a multiple of 32
      frag_t xa[4], fb[NT];
#pragma unroll
      for (int i = 0; i < 4; ++i) xa[i] = __builtin_bit_cast(frag_t, *reinterpret_cast<const uint4 *>(row[i] + k));
      if constexpr (TRANS) {
        const uint16_t *from = factor + ((int64_t)a * L + k) * R;
        uint4 v[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j)
          if (turn_from[j] >= 0) v[j] = *reinterpret_cast<const uint4 *>(from + turn_from[j]);
#pragma unroll
        for (int j = 0; j < NT; ++j)
          if (turn_from[j] >= 0) *reinterpret_cast<uint4 *>(turn + turn_to[j]) = v[j];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // the wave's own LDS, in order
#pragma unroll
        for (int j = 0; j < NT; ++j) fb[j] = read_column(turn + (8 * g + (l16 >> 2)) * kPitch + 16 * j + 4 * (l16 & 3), kPitch);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      } else {
#pragma unroll
        for (int j = 0; j < NT; ++j) fb[j] = __builtin_bit_cast(frag_t, *reinterpret_cast<const uint4 *>(frow[j] + k));
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = mma16<DT>(xa[i], fb[j], acc[i][j]);
    }
  }
  const float sc = scale[a];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (16 * i >= places) break;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) sh.red[wave][4 * j + q][lane] = acc[i][j][q];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const float sum = ((sh.red[0][4 * j + wave][lane] + sh.red[1][4 * j + wave][lane]) + sh.red[2][4 * j + wave][lane]) +
                        sh.red[3][4 * j + wave][lane];
      const int p = 16 * i + 4 * g + wave, r = 16 * j + l16;
      if (p < places && r < R) parts[((int64_t)blockIdx.y * T + unit.y + p) * R + r] = sc * sum;
    }
  }
}

// The parts added up in order, as two 16-bit terms [T][Rp] (Rp: R up to a multiple
// of 16, zeros past R): the first is off by half a step, the second by half a step of that.
// fp16 reaches from 2^-24 to 65504 only, and v, a product of two small numbers where a
// training starts, lies below that: there a place's values are held times a power of two,
// its gain, that brings the largest of them to 2^14 or more.  Then what is 2^-17 of the
// largest or more keeps its 22 bits, and nothing is off by more than 2^-39 of the largest; the
// products are divided by the gain in fp32, exactly.  Each place has a gain of its own, so that
// no token's part depends on another's.  Gains end at 2^+-78: projections, which are whole
// multiples of 2^-48 up to 2^48, can be multiplied by one and divided again.
// A place's values are 16 lanes', 16 places a workgroup: u and v of 4096 tokens, rank 16 4.9 us.
struct Split {
  const float *parts;
  int pieces;
  uint16_t *hi, *lo;
  float *gain;  // [T], fp16 only
};
constexpr int kMostGain = 78;

__device__ __forceinline__ float one_over(float power_of_two) { return __uint_as_float(0x7f000000u - __float_as_uint(power_of_two)); }

template <int DT, int NT>
__global__ __launch_bounds__(256) void lora_split_kernel(Split one, Split two, int64_t T, int R, int Rp, int count,
                                                         const int32_t *__restrict__ start) {
  const Split s = blockIdx.y ? two : one;
  const int64_t p = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  const int l16 = threadIdx.x & 15;
  if (p >= T) return;
  const bool there = p < start[count];
  float v[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) v[j] = 0.f;
  if (there)
#pragma unroll 4
    for (int k = 0; k < s.pieces; ++k)
#pragma unroll
      for (int j = 0; j < NT; ++j) v[j] += s.parts[(k * T + p) * R + min(16 * j + l16, R - 1)];
  float gain = 1.f;
  if constexpr (DT == kF16) {
    float most = 0.f;  // of the finite ones: the others spoil their token whatever the gain
#pragma unroll
    for (int j = 0; j < NT; ++j) most = fmaxf(most, fabsf(v[j]) < INFINITY ? fabsf(v[j]) : 0.f);
    most = group_max(most, 16);
    const int e = 14 - ((int)(__float_as_uint(most) >> 23) - 127);
    if (there) gain = __uint_as_float((uint32_t)(127 + max(-kMostGain, min(e, kMostGain))) << 23);
    if (l16 == 0) s.gain[p] = gain;
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int r = 16 * j + l16;
    if (r >= Rp) break;
    const float value = r < R ? v[j] * gain : 0.f;
    const uint32_t hi = f32_to_bits16<DT>(value);
    s.hi[p * Rp + r] = (uint16_t)hi;
    s.lo[p * Rp + r] = (uint16_t)f32_to_bits16<DT>(value - bits16_to_f32<DT>(hi));
  }
}

// ---------------------------------------------------------------------------
// The adapters' part of sums over places [p0, p0 + 32 MI) and columns: for each
// run of one adapter, its inner values (rows of other runs as zeros) times its
// factor, 16 ranks an instruction, the two terms one after the other.  SHARED: there
// may be rows of other runs, whose zeros a factor that is not finite would turn into NaN; its
// values that are not are left out of the products, and the result says that there are
// some: mark_low_rank then writes the run's own rows.  (With selects on the sums instead the
// compiler spills a hundred registers: 548 instead of 520 us for 4099 tokens x 14336 x 4096.)
// ---------------------------------------------------------------------------
struct LowRank {
  const uint16_t *hi, *lo;  // [T][Rp]
  const float *gain;        // [T], fp16: what hi and lo have been multiplied by
  const uint16_t *factor;   // up [count][width][R], or down [count][R][width]
  int64_t width;
  int R, Rp, count;
  const int32_t *adapter, *start;
};

// Values that are not finite to zeros; whether there were any
template <int DT>
__device__ __forceinline__ bool drop_not_finite(uint32_t (&v)[4]) {
  constexpr uint32_t kExp = DT == kBF16 ? 0x7f80u : 0x7c00u;
  bool any = false;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const bool lo = (v[e] & kExp) == kExp, hi = (v[e] >> 16 & kExp) == kExp;
    v[e] &= (lo ? 0u : 0xffffu) | (hi ? 0u : 0xffff0000u);
    any |= lo | hi;
  }
  return any;
}

// ranks k .. k + 7 of column c of adapter a's factor
template <bool TRANS>
__device__ __forceinline__ void low_rank_factor(const LowRank &lr, int a, int k, int64_t c, uint32_t (&v)[4]) {
  if constexpr (TRANS) {
    const uint16_t *f = lr.factor + ((int64_t)a * lr.R + k) * lr.width + c;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = f[2 * e * lr.width] | (uint32_t)f[(2 * e + 1) * lr.width] << 16;
  } else {
    const uint4 w = *reinterpret_cast<const uint4 *>(lr.factor + ((int64_t)a * lr.width + c) * lr.R + k);
    v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
  }
}

template <int DT, bool TRANS, bool SHARED, int MI, int NJ>
__device__ __forceinline__ bool add_low_rank(tile_acc_t (&acc)[MI][NJ], const LowRank &lr, int p0, int end, int64_t c0,
                                             int64_t cols, int lane) {
  const int h = lane >> 5, l32 = lane & 31;
  bool dropped = false;
  for (int p = p0; p < end;) {
    const int a = __builtin_amdgcn_readfirstlane(lr.adapter[p]);
    if (a >= lr.count) break;  // those without an adapter come last
    const int past = __builtin_amdgcn_readfirstlane(min(lr.start[a + 1], end));
    for (int k0 = 0; k0 < lr.Rp; k0 += 16) {
      const int k = k0 + 8 * h;
      frag_t b[NJ];
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const int64_t c = c0 + 32 * j + l32;
        b[j] = no_frag();
        if (k < lr.R && c < cols) {
          uint32_t v[4];
          low_rank_factor<TRANS>(lr, a, k, c, v);
          if constexpr (SHARED) dropped |= drop_not_finite<DT>(v);
          b[j] = __builtin_bit_cast(frag_t, make_uint4(v[0], v[1], v[2], v[3]));
        }
      }
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const int q = p0 + 32 * i + l32;
        const bool in = q >= p && q < past;
        const int64_t at = (int64_t)(in ? q : p) * lr.Rp + k;
        const uint4 vh = *reinterpret_cast<const uint4 *>(lr.hi + at), vl = *reinterpret_cast<const uint4 *>(lr.lo + at);
        const frag_t hi = in ? __builtin_bit_cast(frag_t, vh) : no_frag();
        const frag_t lo = in ? __builtin_bit_cast(frag_t, vl) : no_frag();
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = tile_mma<DT>(lo, b[j], tile_mma<DT>(hi, b[j], acc[i][j]));
      }
    }
    p = past;
  }
  return __ballot(dropped) != 0;
}

// NaN to the rows out[order[p]] of places [p0, end) in the columns (32 NJ from c0 on) where their adapter's factor
// holds a value that is not finite
template <int DT, int ODT, bool TRANS, int NJ>
__device__ __forceinline__ void mark_low_rank(const LowRank &lr, int p0, int end, int64_t c0, int64_t cols, int lane,
                                           const int32_t *order, typename Storage<ODT>::type *out, int64_t ld) {
  const int h = lane >> 5, l32 = lane & 31;
  __threadfence();  // after the rows' own stores
  for (int p = p0; p < end;) {
    const int a = __builtin_amdgcn_readfirstlane(lr.adapter[p]);
    if (a >= lr.count) break;
    const int past = __builtin_amdgcn_readfirstlane(min(lr.start[a + 1], end));
#pragma unroll 1
    for (int64_t c = c0 + l32; c < cols && c < c0 + 32 * NJ; c += 32) {
      bool any = false;
#pragma unroll 1
      for (int k = 0; k < lr.R; k += 8) {
        uint32_t v[4];
        low_rank_factor<TRANS>(lr, a, k, c, v);
        any |= drop_not_finite<DT>(v);
      }
      if (any)
        for (int q = p + h; q < past; q += 2) store_elem<ODT>(out, order[q] * ld + c, NAN);
    }
    p = past;
  }
}

// out[t][c] = round(base[t][c] + bias[c] + the adapter's part): a unit and 128 columns
// a workgroup, 32 columns a wave; base's loads go out first.  Bound by base and out, and few
// workgroups: 301 tokens x 8192, rank 64, fp16 14.6 us.
template <int DT, int ODT, bool TRANS>
__global__ __launch_bounds__(256, 2) void lora_expand_kernel(const float *__restrict__ base, LowRank lr, Places pl,
                                                          const uint16_t *__restrict__ bias,
                                                          typename Storage<ODT>::type *__restrict__ out) {
  if ((int)blockIdx.x >= *pl.n_units) return;
  const int4 unit = pl.units[blockIdx.x];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, h = lane >> 5, l32 = lane & 31;
  const int64_t c0 = (int64_t)blockIdx.y * 128 + 32 * wave, c = c0 + l32, cin = min(c, lr.width - 1);
  if (c0 >= lr.width) return;
  float old[2][16], gain[2][16];
  int64_t token[2][16];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int p = min(unit.y + 32 * i + 8 * (r >> 2) + 4 * h + (r & 3), unit.z - 1);
      token[i][r] = pl.order[p];
      gain[i][r] = DT == kF16 ? lr.gain[p] : 1.f;
      old[i][r] = base[token[i][r] * lr.width + cin];
    }
  const float more = bias ? bits16_to_f32<DT>(bias[cin]) : 0.f;
  tile_acc_t acc[2][1];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[i][0][r] = 0.f;
  if (unit.x < lr.count) add_low_rank<DT, TRANS, false>(acc, lr, unit.y, unit.z, c0, lr.width, lane);
  if (c >= lr.width) return;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r)
      if (unit.y + 32 * i + 8 * (r >> 2) + 4 * h + (r & 3) < unit.z)
        store_elem<ODT>(out, token[i][r] * lr.width + c, acc[i][0][r] * one_over(gain[i][r]) + old[i][r] + more);
}

// The tile product's sums, rows by place, with the adapters' part and the bias; row's token
template <int DT, int ODT, bool TRANS>
struct EpilogueLora : EpilogueBase {
  using OT = typename Storage<ODT>::type;
  LowRank lr;           // factor from this piece's first column on
  const int32_t *order;
  const uint16_t *bias;
  OT *out;
  int64_t ld;
  struct Row {
    OT *out;
    float scale;  // 1 / gain
  };
  __device__ __forceinline__ bool begin(tile_acc_t (&acc)[4][4], int N, int m, int end, int n, int lane) const {
    if constexpr (DT == kF16) {  // the sums so far times their rows' gains (there is room for whole tiles of these)
      if (m < end)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float4 g = *reinterpret_cast<const float4 *>(lr.gain + m + 32 * i + 8 * q + 4 * (lane >> 5));
#pragma unroll
            for (int j = 0; j < 4; ++j)
              acc[i][j][4 * q] *= g.x, acc[i][j][4 * q + 1] *= g.y, acc[i][j][4 * q + 2] *= g.z, acc[i][j][4 * q + 3] *= g.w;
          }
    }
    return add_low_rank<DT, TRANS, true>(acc, lr, m, end, n, N, lane);
  }
  __device__ __forceinline__ void end(int N, int m, int past, int n, int lane) const {
    mark_low_rank<DT, ODT, TRANS, 4>(lr, m, past, n, N, lane, order, out, ld);
  }
  __device__ __forceinline__ Row row(int m) const {
    return Row{out + order[m] * ld, DT == kF16 ? one_over(lr.gain[m]) : 1.f};
  }
  __device__ __forceinline__ void store(const Row &row, int n, float v) const {
    v *= row.scale;
    store_elem<ODT>(row.out, n, bias ? v + bits16_to_f32<DT>(bias[n]) : v);
  }
};

// ---------------------------------------------------------------------------
// The adapters' gradients: sum over the places p of adapter a of g[order[p]][w] h[p][r],
// at [a][w][r] (UP: g = dy, h = u) or [a][r][w] (g = x, h = v).
//
// A workgroup takes a window of places and 128 columns w; for each run of one
// adapter in the window it multiplies 64 places at a time, rows outside of the
// run as zeros: both operands are wanted by columns, and come out of LDS so.
// A wave has 32 columns and all ranks.  An adapter whose places lie in one
// window is done then; a part of a run that goes on is left in fp32 (a window
// has two at most: one that began before it, and one that goes on after), and
// lora_join_kernel adds an adapter's parts in order.  In fp16 the places' gains differ, and a
// sum over places needs one: the smallest of the run, to which the others' terms are brought on
// their way into LDS (off by at most 2^-37 of the run's largest value; 1537 tokens x 14336, rank 64
// 26 instead of 21 us).  Bound by the read of g and the
// parts' writes: 4096 tokens x 14336, rank 16 27.5 us (4.3 TB/s of g).
// ---------------------------------------------------------------------------
// Eight fp16 values held times `own`, brought to the gain `all`, which is no larger.  Both are powers of two; the factor is
// below fp16's smallest normal number for a place far below the run's largest: then in two steps, and
// from 2^-39 on, where nothing of a value up to 2^15 is left, zero (which keeps a NaN, and makes one of an infinity)
__device__ __forceinline__ u32x4_t to_gain(const u32x4_t &v, float own, float all) {
  typedef __attribute__((ext_vector_type(8))) _Float16 half8_t;
  const int down = (int)((__float_as_uint(own) - __float_as_uint(all)) >> 23);
  const int one = min(down, 14), two = min(down - one, 24);
  const _Float16 a = (_Float16)__uint_as_float((uint32_t)(127 - one) << 23);
  const _Float16 b = down < 39 ? (_Float16)__uint_as_float((uint32_t)(127 - two) << 23) : (_Float16)0.f;
  return __builtin_bit_cast(u32x4_t, __builtin_bit_cast(half8_t, v) * a * b);
}

template <int DT, int ODT, int NT, bool UP>
__global__ __launch_bounds__(256, 2) void lora_grad_kernel(const uint16_t *__restrict__ gp, int64_t W,
                                                        const uint16_t *__restrict__ hi, const uint16_t *__restrict__ lo,
                                                        const float *__restrict__ gain, int R, int Rp, int count,
                                                        int window, Places pl,
                                                        float *__restrict__ parts,
                                                        typename Storage<ODT>::type *__restrict__ out) {
  constexpr int kG = 128 + 16, kH = 32 * NT + 16;  // pitches: rows 8 (mod 64) banks apart
  __shared__ __attribute__((aligned(16))) uint16_t gs[64 * kG], hs[2][64 * kH];
  __shared__ float least[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l32 = lane & 31, h = lane >> 5;
  const int64_t w0 = (int64_t)blockIdx.x * 128;
  const int first = blockIdx.y * window, there = pl.start[count];
  const int last = min(first + window, there);
  const int grow = tid >> 4, gcol = 8 * (tid & 15);
  const bool gin = w0 + gcol < W;
  // this lane's address for a column of 8 places: read_column
  const int i16 = lane & 15, part = (lane >> 4) & 1;
  const int place = 8 * h + (i16 >> 2), col = 16 * part + 4 * (i16 & 3);
  for (int p = first; p < last;) {
    const int a = __builtin_amdgcn_readfirstlane(pl.adapter[p]);
    const int begin = __builtin_amdgcn_readfirstlane(pl.start[a]), past = __builtin_amdgcn_readfirstlane(pl.start[a + 1]);
    const int end = min(past, last);
    tile_acc_t acc[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[j][r] = 0.f;
    // 64 places of 128 columns and of 32 NT ranks (two terms); their tokens a step before that.
    // Loads without conditions, so that they are in flight together: what is not there is
    // read at the run's last place, and zeroed on its way into LDS.  (As vectors: taken apart into
    // words they would be copied, each with a wait, before the loop's end.)
    u32x4_t gv[4], hv[2][NT];
    float own[NT];
    int token[4];
    auto find = [&](int q) __attribute__((always_inline)) {
#pragma unroll
      for (int s = 0; s < 4; ++s) token[s] = pl.order[min(q + grow + 16 * s, end - 1)];
    };
    auto load = [&](int q) __attribute__((always_inline)) {
#pragma unroll
      for (int s = 0; s < 4; ++s) gv[s] = *reinterpret_cast<const u32x4_t *>(gp + (int64_t)token[s] * W + (gin ? w0 + gcol : 0));
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int c = 256 * j + tid;
        const int at = min(q + c / (4 * NT), end - 1);
        const int64_t from = (int64_t)at * Rp + min(8 * (c % (4 * NT)), Rp - 8);
        if constexpr (DT == kF16) own[j] = gain[at];
        hv[0][j] = *reinterpret_cast<const u32x4_t *>(hi + from);
        hv[1][j] = *reinterpret_cast<const u32x4_t *>(lo + from);
      }
    };
    find(p);
    load(p);
    find(p + 64);
    float all = 1.f;  // the run's gain
    if constexpr (DT == kF16) {
      all = INFINITY;
      for (int q = p + tid; q < end; q += 256) all = fminf(all, gain[q]);
      all = -wave_max(-all);
      if (lane == 0) least[wave] = all;
      __syncthreads();  // read by all before the next run's: the steps' barriers are between
      all = fminf(fminf(least[0], least[1]), fminf(least[2], least[3]));
    }
    for (int q = p; q < end; q += 64) {
      __syncthreads();
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const int row = grow + 16 * s;
        *reinterpret_cast<u32x4_t *>(gs + row * kG + gcol) = gv[s] & (q + row < end ? ~0u : 0u);
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int c = 256 * j + tid, row = c / (4 * NT), at = row * kH + 8 * (c % (4 * NT));
        const uint32_t in = q + row < end ? ~0u : 0u;
        if constexpr (DT == kF16) {
          hv[0][j] = to_gain(hv[0][j], own[j], all);
          hv[1][j] = to_gain(hv[1][j], own[j], all);
        }
        *reinterpret_cast<u32x4_t *>(hs[0] + at) = hv[0][j] & in;
        *reinterpret_cast<u32x4_t *>(hs[1] + at) = hv[1][j] & in;
      }
      __syncthreads();
      load(q + 64);
      find(q + 128);
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const frag_t gf = read_column(gs + (16 * s + place) * kG + 32 * wave + col, kG);
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int term = 0; term < 2; ++term) {
            const frag_t hf = read_column(hs[term] + (16 * s + place) * kH + 32 * j + col, kH);
            acc[j] = UP ? tile_mma<DT>(gf, hf, acc[j]) : tile_mma<DT>(hf, gf, acc[j]);
          }
      }
    }
    const bool whole = begin >= first && past <= last;
    float *keep = parts + (int64_t)(2 * blockIdx.y + (begin >= first)) * W * R;
    const float scale = one_over(all);
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int in = 8 * (r >> 2) + 4 * h + (r & 3);  // row of the 32 x 32 sums, l32 its column
        const int64_t w = w0 + 32 * wave + (UP ? in : l32);
        const int rank = 32 * j + (UP ? l32 : in);
        if (w >= W || rank >= R) continue;
        const int64_t at = UP ? w * R + rank : rank * W + w;
        const float sum = DT == kF16 ? acc[j][r] * scale : acc[j][r];
        if (whole) store_elem<ODT>(out, (int64_t)a * W * R + at, sum);
        else keep[at] = sum;
      }
    p = end;
  }
}

// What lora_grad_kernel left: sums of an adapter's parts, and zeros for one without tokens.
template <int ODT>
__global__ __launch_bounds__(256) void lora_join_kernel(const float *__restrict__ parts, int64_t n, int window,
                                                        const int32_t *__restrict__ start,
                                                        typename Storage<ODT>::type *__restrict__ out) {
  const int a = blockIdx.y, begin = start[a], past = start[a + 1];
  const int from = begin / window, to = (past - 1) / window;
  if (begin < past && from == to) return;
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;  // n is a multiple of 8
  if (i >= n) return;
  float sum[4] = {};
  if (begin < past) {
    const float4 v = *reinterpret_cast<const float4 *>(parts + (int64_t)(2 * from + 1) * n + i);
    sum[0] = v.x, sum[1] = v.y, sum[2] = v.z, sum[3] = v.w;
#pragma unroll 4
    for (int w = from + 1; w <= to; ++w) {
      const float4 u = *reinterpret_cast<const float4 *>(parts + (int64_t)(2 * w) * n + i);
      sum[0] += u.x, sum[1] += u.y, sum[2] += u.z, sum[3] += u.w;
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) store_elem<ODT>(out, a * n + i + e, sum[e]);
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
constexpr int64_t kFew = 64;        // tokens up to which a token is a workgroup's
constexpr int64_t kTiledFrom = 640, kTiledTiles = 144;  // tokens and tiles from which the tile product is used
constexpr int64_t kRows = 4096;     // tokens of a fp32 projection in the workspace
constexpr int64_t kTiledRows = 8192;  // by order: offsets of 8192 rows of 65536 fit 31 bits
constexpr int64_t kDecoded = (int64_t)1 << 27;  // elements of a decoded piece, about

static int few_pieces(int64_t width) { return (int)((width + kPiece - 1) / kPiece); }
static int64_t most_units(int64_t T, int count) { return (T + kUnit - 1) / kUnit + (T < count + 1 ? T : count + 1); }

// Pieces of the inner values' sums: a workgroup for each of about 1024 units and pieces, 256 terms
// at least, and no more parts than about 32 MB of them
static int inner_pieces(int64_t T, int64_t L, int count, int R) {
  int64_t s = 1024 / most_units(T, count);
  if (s > L / 256) s = L / 256;
  if (s > (32 << 20) / (T * R * 4)) s = (32 << 20) / (T * R * 4);
  return s < 1 ? 1 : (int)s;
}
static int inner_piece(int64_t L, int pieces) { return (int)(((L + pieces - 1) / pieces + 63) & ~(int64_t)63); }

struct InnerPlan {
  int pieces, piece;
  size_t parts, hi, lo, gain;
};
static InnerPlan inner_plan(Carver &c, int64_t T, int64_t L, int R, int count) {
  InnerPlan p{};
  p.piece = inner_piece(L, inner_pieces(T, L, count, R));
  p.pieces = (int)((L + p.piece - 1) / p.piece);
  const int64_t Rp = (R + 15) & ~15;
  p.parts = c.take((size_t)p.pieces * T * R * 4);
  p.hi = c.take((size_t)T * Rp * 2), p.lo = c.take((size_t)T * Rp * 2);
  p.gain = c.take((size_t)((T + kTileM - 1) / kTileM) * kTileM * 4);  // read by whole tiles
  return p;
}

struct PlacesPlan {
  size_t order, adapter, start, units, n_units;
};
static PlacesPlan places_plan(Carver &c, int64_t T, int count) {
  PlacesPlan p{};
  p.order = c.take((size_t)T * 4), p.adapter = c.take((size_t)T * 4), p.start = c.take((size_t)(count + 2) * 4);
  p.units = c.take((size_t)most_units(T, count) * 16), p.n_units = c.take(4);
  return p;
}
static Places places_at(const PlacesPlan &p, char *ws) {
  return Places{reinterpret_cast<int32_t *>(ws + p.order), reinterpret_cast<int32_t *>(ws + p.adapter),
                reinterpret_cast<int32_t *>(ws + p.start), reinterpret_cast<int4 *>(ws + p.units),
                reinterpret_cast<int32_t *>(ws + p.n_units)};
}

// The product of tokens with a 4-bit weight: width [N] outputs of sums over [K] (forward) or the other way round
struct ProductPlan {
  // tiled: the tile product, with the adapters' part added to its sums; parts > 0: the tile product in
  // fp32, in parts of the sum; else gemm_4bit's kernels in fp32
  bool tiled;
  int parts;
  int64_t split, tokens, piece, Lp;  // terms of a part, tokens at a time, columns whose weights are decoded at a time
  size_t base, back, decoded, x;     // fp32 projection, gemm_4bit_backward's own, decoded weights, rows padded to Lp
};
static ProductPlan product_plan(Carver &c, int64_t T, int64_t N, int64_t K, int log2bs, bool backward, bool few) {
  ProductPlan p{};
  const int64_t L = backward ? N : K, width = backward ? K : N;
  // The tile product wants the decoding spread over many tokens, and tiles for half the compute units
  // or more.  Both sides, us of a call with it / with gemm_4bit's kernels (rank 16): 14336 x 4096 outputs x
  // sums, 448 tokens 155 / 108, 768 tokens (168 tiles) 151 / 187, 4096 tokens 495 / 727; 4096 x 4096, 2048 tokens
  // (128 tiles) 126 / 122, 4096 tokens 154 / 226; 4096 x 14336, 2048 tokens 357 / 303, 4096 tokens 429 / 588
  const int64_t tiles = ((T + kTileM - 1) / kTileM) * ((width + kTileN - 1) / kTileN);
  const bool can = L <= 65536 && width <= ((int64_t)1 << 30);
  p.tiled = can && T >= kTiledFrom && tiles >= kTiledTiles;
  // the plain epilogue's offsets: 256 rows of fp32 sums in less than 2^31 bytes
  const bool parts = can && width <= ((int64_t)1 << 20) && !p.tiled && backward && !fast_backward(T, N, K, log2bs);
  const int64_t most = p.tiled ? kTiledRows : kRows, turns = (T + most - 1) / most;
  p.tokens = (T + turns - 1) / turns;
  p.Lp = to64(L);
  if (p.tiled || parts) {
    p.piece = kDecoded / p.Lp & ~(int64_t)4095;  // L is at most 2^16: 2048 .. ; rows_of wants 4096 rows
    if (p.piece < 4096) p.piece = 4096;
    if (p.piece > width) p.piece = width;
    p.decoded = c.take((size_t)p.piece * p.Lp * 2);
    if (p.Lp != L) p.x = c.take((size_t)p.tokens * p.Lp * 2);
  }
  if (parts) {
    const int64_t there = ((p.tokens + kTileM - 1) / kTileM) * ((width + kTileN - 1) / kTileN);
    int64_t n = there >= 256 ? 1 : 256 / there;
    if (n > p.Lp / 256) n = p.Lp / 256 > 0 ? p.Lp / 256 : 1;
    p.split = to64((p.Lp + n - 1) / n);
    p.parts = (int)((p.Lp + p.split - 1) / p.split);
  }
  if (!p.tiled) {
    const int in = parts ? p.parts : few && skinny_fits(T, K, log2bs) ? skinny_parts(K) : 1;
    p.base = c.take((size_t)p.tokens * width * 4 * in);
    if (backward && !parts) {
      size_t need = 0;
      for (int64_t m : {p.tokens, T % p.tokens})
        if (m > 0) {
          const size_t b = gemm_backward_workspace_bytes(m, N, K, log2bs);
          need = b > need ? b : need;
        }
      p.back = c.take(need);
    }
  }
  return p;
}

// Windows of the gradients: about 2048 workgroups, no more parts than about 32 MB of them, and 128
// places at least; fewer where there are few tokens, whose adapters a workgroup takes one after
// the other (43 tokens of 43 adapters, 6976 wide: 47 us in one window)
static int grad_window(int64_t T, int64_t W, int R, int count) {
  const int64_t tiles = (W + 127) / 128, part = W * R * 4, least = T >= 512 ? 128 : count >= 8 ? 16 : 64;
  int64_t windows = 2048 / tiles;
  if (windows > (32 << 20) / part) windows = (32 << 20) / part;
  if (windows < 4) windows = 4;
  int64_t w = ((T + windows - 1) / windows + least - 1) / least * least;
  if (T >= 512) w = to64(w);
  return (int)(w < T ? w : T);
}

struct LoraPlan {
  bool few;
  ProductPlan product;
  int64_t tokens;
  size_t u_few;
  PlacesPlan places;
  InnerPlan inner;  // of the product: u forward, v backward
  // backward: for all tokens
  PlacesPlan all;
  InnerPlan u, v;
  int window_down, window_up;
  size_t parts, total;
};

static LoraPlan lora_plan(int64_t T, int64_t N, int64_t K, int log2bs, int count, int R, bool backward) {
  LoraPlan p{};
  Carver c;
  p.few = !backward && T <= kFew;
  p.product = product_plan(c, T, N, K, log2bs, backward, p.few);
  p.tokens = p.product.tokens;
  if (p.few) {
    p.u_few = c.take((size_t)few_pieces(K) * T * R * 4);
  } else {
    p.places = places_plan(c, p.tokens, count);
    p.inner = inner_plan(c, p.tokens, backward ? N : K, R, count);
  }
  if (backward) {
    if (p.tokens < T) {
      p.all = places_plan(c, T, count);
      p.v = inner_plan(c, T, N, R, count);
    } else {
      p.all = p.places;
      p.v = p.inner;
    }
    p.u = inner_plan(c, T, K, R, count);
    p.window_down = grad_window(T, K, R, count), p.window_up = grad_window(T, N, R, count);
    const size_t a = 2 * (size_t)((T + p.window_down - 1) / p.window_down) * K * R * 4;
    const size_t b = 2 * (size_t)((T + p.window_up - 1) / p.window_up) * N * R * 4;
    p.parts = c.take(a > b ? a : b);
  }
  p.total = c.at;
  return p;
}

size_t lora_workspace(int64_t T, int64_t N, int64_t K, int log2bs, int count, int rank, bool backward) {
  return lora_plan(T, N, K, log2bs, count, rank, backward).total;
}

#define QMV_RANKS(NT_OF, CALL)        \
  switch (NT_OF) {                    \
    case 1: { constexpr int NT = 1; CALL; break; } \
    case 2: { constexpr int NT = 2; CALL; break; } \
    case 3: case 4: { constexpr int NT = 4; CALL; break; } \
    default: { constexpr int NT = 8; CALL; break; } \
  }

template <int DT, bool TRANS>
static void shrink(const uint16_t *x, int64_t T, int64_t L, const uint16_t *factor, const Lora &l, const InnerPlan &p,
                   const Places &pl, char *ws, hipStream_t st) {
  const dim3 grid((unsigned)most_units(T, l.count), (unsigned)p.pieces);
  QMV_RANKS((l.rank + 15) / 16,
            hipLaunchKernelGGL((lora_shrink_kernel<DT, NT, TRANS>), grid, dim3(256), 0, st, x, L, p.piece, factor, l.scale,
                               l.count, l.rank, pl, reinterpret_cast<float *>(ws + p.parts), T))
}

static Split split_of(const InnerPlan &p, char *ws) {
  return Split{reinterpret_cast<float *>(ws + p.parts), p.pieces, reinterpret_cast<uint16_t *>(ws + p.hi),
               reinterpret_cast<uint16_t *>(ws + p.lo), reinterpret_cast<float *>(ws + p.gain)};
}

template <int DT>
static void split(const Split &one, const Split *two, int64_t T, const Lora &l, const Places &pl, hipStream_t st) {
  const int Rp = (l.rank + 15) & ~15;
  QMV_RANKS(Rp / 16, hipLaunchKernelGGL((lora_split_kernel<DT, NT>), dim3((unsigned)((T + 15) / 16), two ? 2 : 1), dim3(256), 0,
                                        st, one, two ? *two : one, T, l.rank, Rp, l.count, pl.start))
}

static void order(const int32_t *index, int64_t T, const Lora &l, const Places &pl, hipStream_t st) {
  hipLaunchKernelGGL(lora_order_kernel, dim3((unsigned)((T + 255) / 256)), dim3(256), 0, st, index, (int)T, l.count, pl);
}

// out = the product of m tokens with the weight, its transpose with TRANS, and the adapters' part
template <int DT, int ODT, bool TRANS>
static hipError_t product(const LoraPlan &p, const uint16_t *x, int64_t m, const Weight4 &w, const Lora &l,
                          const Places &pl, const uint16_t *bias, typename Storage<ODT>::type *out, char *ws,
                          hipStream_t st) {
  const int64_t L = TRANS ? w.N : w.K, width = TRANS ? w.K : w.N;
  const Split s = split_of(p.inner, ws);
  const int Rp = (l.rank + 15) & ~15;
  const LowRank lr{s.hi, s.lo, s.gain, TRANS ? l.down : l.up, width, l.rank, Rp, l.count, pl.adapter, pl.start};
  const ProductPlan &pp = p.product;
  float *base = reinterpret_cast<float *>(ws + pp.base);
  if (pp.tiled || pp.parts) {
    uint16_t *W = reinterpret_cast<uint16_t *>(ws + pp.decoded);
    if (pp.Lp != L) {
      uint16_t *padded = reinterpret_cast<uint16_t *>(ws + pp.x);
      const hipError_t e = launch_pad_rows(x, m, L, pp.Lp, padded, st);
      if (e != hipSuccess) return e;
      x = padded;
    }
    for (int64_t c = 0; c < width; c += pp.piece) {
      const int64_t n = width - c < pp.piece ? width - c : pp.piece;
      const hipError_t e = TRANS ? launch_decode_piece(w, DT, c, n, nullptr, 0, W, pp.Lp, st)
                                 : launch_decode_rows(rows_of(w, c, n), DT, W, pp.Lp, st);
      if (e != hipSuccess) return e;
      TileArgs a = tile_args(x, pp.Lp, W, pp.Lp, m, n, pp.Lp);
      if (pp.tiled) {
        a.rows = pl.order;
        EpilogueLora<DT, ODT, TRANS> epi;
        epi.lr = lr;
        epi.lr.factor += TRANS ? c : c * l.rank;
        epi.order = pl.order, epi.bias = bias ? bias + c : nullptr, epi.out = out + c, epi.ld = width;
        hipLaunchKernelGGL((tile_kernel<DT, EpilogueLora<DT, ODT, TRANS>>), dim3(a.ncol * a.nrow), dim3(256), 0, st, a, epi);
      } else {
        a.split = (int)pp.split;
        EpilogueF32 epi;
        epi.C = base + c, epi.ld = width, epi.part = m * width;
        hipLaunchKernelGGL((tile_kernel<DT, EpilogueF32>), dim3(a.ncol * a.nrow, pp.parts), dim3(256), 0, st, a, epi);
      }
    }
    if (pp.tiled) return hipGetLastError();
    if (pp.parts > 1) {
      const hipError_t e = launch_sum_parts(base, pp.parts, m * width, st);
      if (e != hipSuccess) return e;
    }
  } else {
    const hipError_t e =
        TRANS ? launch_gemm_4bit_backward(x, DT, m, w.N, w.K, w.packed, w.sc, w.dq, w.log2bs, w.qt, base, kF32,
                                          ws + pp.back, st)
              : launch_gemm_4bit(x, DT, m, w.N, w.K, w.packed, w.sc, w.dq, w.log2bs, w.qt, base, kF32, nullptr, st);
    if (e != hipSuccess) return e;
  }
  const dim3 grid((unsigned)most_units(m, l.count), (unsigned)((width + 127) / 128));
  hipLaunchKernelGGL((lora_expand_kernel<DT, ODT, TRANS>), grid, dim3(256), 0, st, base, lr, pl, bias, out);
  return hipGetLastError();
}

template <int DT, int ODT>
static hipError_t lora_t(const uint16_t *x, int64_t T, const Weight4 &w, const Lora &l, const int32_t *index,
                         const uint16_t *bias, typename Storage<ODT>::type *y, char *ws, hipStream_t st) {
  const LoraPlan p = lora_plan(T, w.N, w.K, w.log2bs, l.count, l.rank, false);
  if (p.few) {
    float *base = reinterpret_cast<float *>(ws + p.product.base), *u = reinterpret_cast<float *>(ws + p.u_few);
    const int pieces = few_pieces(w.K);
    hipLaunchKernelGGL(lora_down_kernel<DT>, dim3((unsigned)T, (unsigned)pieces), dim3(256), 0, st, x, w.K, l.down, l.scale,
                       l.count, l.rank, index, u, T);
    const bool skinny = skinny_fits(T, w.K, w.log2bs);
    const hipError_t e =
        skinny   ? launch_skinny(x, DT, T, w, base, st)
        : T <= 8 ? launch_gemv_4bit(x, DT, (int)T, w.N, w.K, w.packed, w.sc, w.dq, w.log2bs, w.qt, base, kF32, nullptr, st)
                 : launch_gemm_4bit(x, DT, T, w.N, w.K, w.packed, w.sc, w.dq, w.log2bs, w.qt, base, kF32, nullptr, st);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((lora_up_kernel<DT, ODT>), dim3((unsigned)((w.N + 255) / 256), (unsigned)T), dim3(256), 0, st, base,
                       skinny ? skinny_parts(w.K) : 1, w.N, l.up, l.count, l.rank, index, u, pieces, T, bias, y);
    return hipGetLastError();
  }
  const Places pl = places_at(p.places, ws);
  for (int64_t t = 0; t < T; t += p.tokens) {
    const int64_t m = T - t < p.tokens ? T - t : p.tokens;
    order(index + t, m, l, pl, st);
    shrink<DT, false>(x + t * w.K, m, w.K, l.down, l, p.inner, pl, ws, st);
    split<DT>(split_of(p.inner, ws), nullptr, m, l, pl, st);
    const hipError_t e = product<DT, ODT, false>(p, x + t * w.K, m, w, l, pl, bias, y + t * w.N, ws, st);
    if (e != hipSuccess) return e;
  }
  return hipGetLastError();
}

template <int DT, int ODT>
static hipError_t lora_backward_t(const uint16_t *dy, const uint16_t *x, int64_t T, const Weight4 &w, const Lora &l,
                                  const int32_t *index, uint16_t *dx, void *d_down, void *d_up, char *ws, hipStream_t st) {
  using OT = typename Storage<ODT>::type;
  const LoraPlan p = lora_plan(T, w.N, w.K, w.log2bs, l.count, l.rank, true);
  const int R = l.rank, Rp = (R + 15) & ~15;
  const bool once = p.tokens >= T;
  if (!once) {  // the input's gradient in turns, with an order of its own each time
    const Places pl = places_at(p.places, ws);
    for (int64_t t = 0; t < T; t += p.tokens) {
      const int64_t m = T - t < p.tokens ? T - t : p.tokens;
      order(index + t, m, l, pl, st);
      shrink<DT, true>(dy + t * w.N, m, w.N, l.up, l, p.inner, pl, ws, st);
      split<DT>(split_of(p.inner, ws), nullptr, m, l, pl, st);
      const hipError_t e = product<DT, DT, true>(p, dy + t * w.N, m, w, l, pl, nullptr, dx + t * w.K, ws, st);
      if (e != hipSuccess) return e;
    }
  }
  const Places pl = places_at(p.all, ws);
  order(index, T, l, pl, st);
  shrink<DT, true>(dy, T, w.N, l.up, l, p.v, pl, ws, st);
  shrink<DT, false>(x, T, w.K, l.down, l, p.u, pl, ws, st);
  const Split v = split_of(p.v, ws), u = split_of(p.u, ws);
  split<DT>(v, &u, T, l, pl, st);
  if (once) {
    const hipError_t e = product<DT, DT, true>(p, dy, T, w, l, pl, nullptr, dx, ws, st);
    if (e != hipSuccess) return e;
  }
  float *parts = reinterpret_cast<float *>(ws + p.parts);
  auto grads = [&](const uint16_t *g, int64_t W, const Split &h, int window, auto up, void *out) {
    constexpr bool UP = decltype(up)::value;
    const dim3 grid((unsigned)((W + 127) / 128), (unsigned)((T + window - 1) / window));
    QMV_RANKS((R + 31) / 32, hipLaunchKernelGGL((lora_grad_kernel<DT, ODT, (NT > 4 ? 4 : NT), UP>), grid, dim3(256), 0, st,
                                                g, W, h.hi, h.lo, h.gain, R, Rp, l.count, window, pl, parts, static_cast<OT *>(out)))
    const int64_t n = W * R;
    hipLaunchKernelGGL((lora_join_kernel<ODT>), dim3((unsigned)((n + 1023) / 1024), (unsigned)l.count), dim3(256), 0, st,
                       parts, n, window, pl.start, static_cast<OT *>(out));
  };
  grads(x, w.K, v, p.window_down, std::false_type{}, d_down);
  grads(dy, w.N, u, p.window_up, std::true_type{}, d_up);
  return hipGetLastError();
}

hipError_t launch_lora(const void *x, int dt, int64_t T, const Weight4 &w, const Lora &l, const int32_t *index,
                       const void *bias, void *y, int y_dt, char *ws, hipStream_t st) {
  const uint16_t *xp = static_cast<const uint16_t *>(x), *b = static_cast<const uint16_t *>(bias);
  if (y_dt == kF32) {
    float *o = static_cast<float *>(y);
    return dt == kF16 ? lora_t<kF16, kF32>(xp, T, w, l, index, b, o, ws, st) : lora_t<kBF16, kF32>(xp, T, w, l, index, b, o, ws, st);
  }
  uint16_t *o = static_cast<uint16_t *>(y);
  return dt == kF16 ? lora_t<kF16, kF16>(xp, T, w, l, index, b, o, ws, st) : lora_t<kBF16, kBF16>(xp, T, w, l, index, b, o, ws, st);
}

hipError_t launch_lora_backward(const void *dy, const void *x, int dt, int64_t T, const Weight4 &w, const Lora &l,
                                const int32_t *index, void *dx, void *d_down, void *d_up, int grad_dt, char *ws,
                                hipStream_t st) {
  const uint16_t *g = static_cast<const uint16_t *>(dy), *xp = static_cast<const uint16_t *>(x);
  uint16_t *o = static_cast<uint16_t *>(dx);
  if (grad_dt == kF32)
    return dt == kF16 ? lora_backward_t<kF16, kF32>(g, xp, T, w, l, index, o, d_down, d_up, ws, st)
                      : lora_backward_t<kBF16, kF32>(g, xp, T, w, l, index, o, d_down, d_up, ws, st);
  return dt == kF16 ? lora_backward_t<kF16, kF16>(g, xp, T, w, l, index, o, d_down, d_up, ws, st)
                    : lora_backward_t<kBF16, kBF16>(g, xp, T, w, l, index, o, d_down, d_up, ws, st);
}

}  // namespace qmv
