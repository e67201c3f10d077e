// Rotary positions on q and k, and the backward's finalize step with their
// adjoint.
//
// Column pair i of a row at position p turns by the angle theta = p w_i:
//   a' = m (a cos theta - b sin theta),  b' = m (a sin theta + b cos theta),
// with the pair (a, b) in columns (i, i + rot / 2) ("half" layout) or
// (2 i, 2 i + 1) ("interleaved"); columns from rot on are copied. The map is
// m times a rotation, so its adjoint is the same with -theta.
//
// Angles are exact: the frequency is given as F_i, the turns per position as
// a 64-bit fraction (w_i = 2 pi F_i / 2^64), and p F_i modulo 2^64 is the
// angle's fraction of a turn in integers, however far the position. Its top
// bits give the quadrant, the rest an angle in [-pi/4, pi/4], whose sine and
// cosine are their Taylor sums. No table of cosines is stored or read.
#include <cmath>
#include <cstdint>

#include "element.cuh"
#include "grid_ptx.cuh"

namespace attn {
namespace rotary {

// One of the two tensors of a call: q (0) or k (1). Strides in elements of
// batch, head and row; the row's d elements are contiguous.
struct Side {
  const void* in;
  void* out;
  long long in_stride[3], out_stride[3];
  int heads;
  float scale;  // multiplies the input (tau of the finalize step, else 1)
};

struct Args {
  Side side[2];
  const unsigned long long* turns;  // [rot / 2]
  const long long* positions;       // [B, N] with batch stride pos_stride, or NULL: row index
  long long pos_stride;
  int B, N, d, half;  // half = rot / 2
  float magnitude;
  float sign;  // +1, or -1 for the adjoint
  int interleaved;
};

// cos and sin of 2 pi p F / 2^64. |theta| <= pi / 4 after the quadrant is
// taken off; the Taylor sums' first left-out terms are theta^11 / 11! < 2e-9
// and theta^12 / 12! < 2e-10, below half an fp32 step of the values.
__device__ __forceinline__ void angle(long long p, unsigned long long f, float& c, float& s) {
  const uint32_t t = static_cast<uint32_t>((static_cast<unsigned long long>(p) * f) >> 32);
  const uint32_t quadrant = (t + 0x20000000u) >> 30;
  const int32_t rest = static_cast<int32_t>(t - (quadrant << 30));
  const float x = static_cast<float>(rest) * 1.4629180792671596e-09f;  // 2 pi / 2^32
  const float x2 = x * x;
  float sn = fmaf(x2, 2.7557319e-6f, -1.9841270e-4f);
  sn = fmaf(sn, x2, 8.3333333e-3f);
  sn = fmaf(sn, x2, -1.6666667e-1f);
  sn = fmaf(sn * x2, x, x);
  float cs = fmaf(x2, -2.7557319e-7f, 2.4801587e-5f);
  cs = fmaf(cs, x2, -1.3888889e-3f);
  cs = fmaf(cs, x2, 4.1666667e-2f);
  cs = fmaf(cs, x2, -0.5f);
  cs = fmaf(cs, x2, 1.0f);
  const float a = (quadrant & 1u) ? sn : cs, b = (quadrant & 1u) ? cs : sn;
  c = (quadrant == 1u || quadrant == 2u) ? -a : a;
  s = (quadrant & 2u) ? -b : b;
}

// Fallback for rows that 16-byte groups do not divide (odd d, strides or
// rot): one thread per column pair (or copied column) of a row.
template <typename TQ, typename TK, typename TO>
__global__ void __launch_bounds__(256) rotary_any_kernel(Args p) {
  ptx::grid_dependency_wait();
  const int items = p.half + (p.d - 2 * p.half);
  const int heads = p.side[0].heads + p.side[1].heads;
  const long long total = static_cast<long long>(p.B) * p.N * heads * items;
  const long long stride = static_cast<long long>(gridDim.x) * blockDim.x;
  for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
       i += stride) {
    const int j = static_cast<int>(i % items);
    long long rest = i / items;
    int h = static_cast<int>(rest % heads);
    rest /= heads;
    const long long n = rest % p.N, b = rest / p.N;
    const bool is_k = h >= p.side[0].heads;
    if (is_k) h -= p.side[0].heads;
    const Side& s = p.side[is_k ? 1 : 0];
    const long long in = b * s.in_stride[0] + h * s.in_stride[1] + n * s.in_stride[2];
    const long long out = b * s.out_stride[0] + h * s.out_stride[1] + n * s.out_stride[2];
    auto load = [&](int c) {
      return s.scale * (is_k ? to_f32(static_cast<const TK*>(s.in)[in + c])
                             : to_f32(static_cast<const TQ*>(s.in)[in + c]));
    };
    auto store = [&](int c, float v) { static_cast<TO*>(s.out)[out + c] = from_f32<TO>(v); };
    if (j >= p.half) {
      const int c = j + p.half;
      store(c, load(c));
      continue;
    }
    const long long pos = p.positions != nullptr ? p.positions[b * p.pos_stride + n] : n;
    float cs, sn;
    angle(pos, p.turns[j], cs, sn);
    cs *= p.magnitude;
    sn *= p.magnitude * p.sign;
    const int ca = p.interleaved ? 2 * j : j, cb = p.interleaved ? 2 * j + 1 : j + p.half;
    const float a = load(ca), v = load(cb);
    store(ca, a * cs - v * sn);
    store(cb, a * sn + v * cs);
  }
}

constexpr int kThreads = 128;

// E consecutive elements in fp32 from T (E = the output type's 16 bytes).
template <typename T, int E>
struct Group {
  static constexpr int kVecs = E * static_cast<int>(sizeof(T)) / 16;
  Vec<T> v[kVecs];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) v[i] = load_vec(p + i * Vec<T>::kElems);
  }
  __device__ __forceinline__ void get(float (&f)[E]) const {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      float part[Vec<T>::kElems];
      unpack(v[i], part);
#pragma unroll
      for (int j = 0; j < Vec<T>::kElems; ++j) f[i * Vec<T>::kElems + j] = part[j];
    }
  }
};

// One thread keeps the cosines and sines of E column pairs of one token and
// takes them through `per` heads, U heads' loads in flight at a time: of two
// 16-byte groups a row, the pairs' two halves (half layout), or two groups
// apart of the turning columns (interleaved) or of the copied ones. Neighbour
// lanes have neighbour groups, so that requests are whole sectors (with two
// neighbouring groups a lane the interleaved d = 64 case took 14.8 us, not
// 14.0). The angles cost about as much as four heads' arithmetic; the loads
// and stores are what bounds it: B=2 H=32 H_kv=8 N=4096 d=128 bf16 takes 27.4
// us for 168 MB (6.1 TB/s), the finalize step of that shape 36.0 us for 235 MB
// (6.5 TB/s).
template <typename TI, typename TO, int U, bool INTERLEAVED>
__device__ __forceinline__ void rotate_heads(const Args& p, const Side& s, int h0, int h1,
                                             long long b, long long n, int item) {
  constexpr int E = Vec<TO>::kElems;
  int ca, cb;
  bool turn_a, turn_b;
  const int turning = INTERLEAVED ? 0 : p.half / E;  // items that turn (half layout)
  if (!INTERLEAVED && item < turning) {
    ca = item * E;
    cb = ca + p.half;
    turn_a = turn_b = true;
  } else {
    const int start = INTERLEAVED ? 0 : 2 * p.half;  // groups from here on, two an item
    const int items = ((p.d - start) / E + 1) / 2;
    ca = start + (item - turning) * E;
    cb = ca + items * E;
    turn_a = ca < 2 * p.half;
    turn_b = cb < 2 * p.half;
  }
  const bool has_b = cb < p.d;
  const TI* in = static_cast<const TI*>(s.in) + b * s.in_stride[0] + h0 * s.in_stride[1] +
                 n * s.in_stride[2];
  TO* out = static_cast<TO*>(s.out) + b * s.out_stride[0] + h0 * s.out_stride[1] +
            n * s.out_stride[2];
  float cs[E], sn[E];
  bool ready = false;
  for (int h = h0; h < h1; h += U) {
    Group<TI, E> ga[U], gb[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (h + u < h1) {
        ga[u].load(in + u * s.in_stride[1] + ca);
        if (has_b) gb[u].load(in + u * s.in_stride[1] + cb);
      }
    }
    if (!ready) {  // behind the first loads, so that their latency covers it
      ready = true;
      if (turn_a) {
        const long long pos = p.positions != nullptr ? p.positions[b * p.pos_stride + n] : n;
        const float m = p.magnitude * s.scale, ms = m * p.sign;
#pragma unroll
        for (int i = 0; i < E; i += 2) {  // pairs come in twos: so does rot / 2 here
          // interleaved: the first E / 2 pairs are those of group a
          const int pair = !INTERLEAVED ? ca + i : i < E / 2 ? ca / 2 + i : cb / 2 + i - E / 2;
          ulonglong2 f = make_ulonglong2(0, 0);
          if (pair < p.half) f = *reinterpret_cast<const ulonglong2*>(p.turns + pair);
          angle(pos, f.x, cs[i], sn[i]);
          angle(pos, f.y, cs[i + 1], sn[i + 1]);
          cs[i] *= m;
          cs[i + 1] *= m;
          sn[i] *= ms;
          sn[i + 1] *= ms;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (h + u >= h1) continue;
      float a[E], v[E];
      ga[u].get(a);
      gb[u].get(v);
      if (INTERLEAVED) {
#pragma unroll
        for (int i = 0; i < E; i += 2) {
          if (turn_a) {
            const float x = a[i], y = a[i + 1];
            a[i] = x * cs[i / 2] - y * sn[i / 2];
            a[i + 1] = x * sn[i / 2] + y * cs[i / 2];
          } else {
            a[i] *= s.scale;
            a[i + 1] *= s.scale;
          }
          if (turn_b) {
            const float x = v[i], y = v[i + 1];
            v[i] = x * cs[(E + i) / 2] - y * sn[(E + i) / 2];
            v[i + 1] = x * sn[(E + i) / 2] + y * cs[(E + i) / 2];
          } else {
            v[i] *= s.scale;
            v[i + 1] *= s.scale;
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const float x = a[i], y = v[i];
          a[i] = turn_a ? x * cs[i] - y * sn[i] : x * s.scale;
          v[i] = turn_a ? x * sn[i] + y * cs[i] : y * s.scale;
        }
      }
      Vec<TO> w;
      pack(a, w);
      store_vec(out + u * s.out_stride[1] + ca, w);
      if (has_b) {
        pack(v, w);
        store_vec(out + u * s.out_stride[1] + cb, w);
      }
    }
    in += U * s.in_stride[1];
    out += U * s.out_stride[1];
  }
}

template <typename TQ, typename TK, typename TO, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads)
    rotary_kernel(Args p, int items, int per, int q_groups, long long tokens) {
  ptx::grid_dependency_wait();
  const long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  long long token, b, n;
  int item;
  if (tokens * items <= 0x7fffffffLL) {  // 32-bit divisions take a fifth of the time
    const uint32_t j = static_cast<uint32_t>(i), t = j / static_cast<uint32_t>(items);
    const uint32_t q = t / static_cast<uint32_t>(p.N);
    token = t;
    item = static_cast<int>(j - t * static_cast<uint32_t>(items));
    b = q;
    n = t - q * static_cast<uint32_t>(p.N);
  } else {
    token = i / items;
    item = static_cast<int>(i - token * items);
    b = token / p.N;
    n = token - b * p.N;
  }
  if (token >= tokens) return;
  const int g = blockIdx.y;
  // loads in flight per thread: 128 bytes
  if (g < q_groups) {
    const int h0 = g * per;
    rotate_heads<TQ, TO, sizeof(TQ) == sizeof(TO) ? 4 : 2, INTERLEAVED>(
        p, p.side[0], h0, min(h0 + per, p.side[0].heads), b, n, item);
  } else {
    const int h0 = (g - q_groups) * per;
    rotate_heads<TK, TO, 4, INTERLEAVED>(p, p.side[1], h0, min(h0 + per, p.side[1].heads), b, n,
                                         item);
  }
}

// Whether rows and strides are whole 16-byte groups of the output's type (and
// of the input's).
template <typename TO>
bool whole_groups(const Args& a) {
  constexpr int E = Vec<TO>::kElems;
  if (a.d % E != 0 || (a.interleaved ? 2 * a.half : a.half) % E != 0) return false;
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 3; ++j)
      if (a.side[i].heads > 0 &&
          (a.side[i].in_stride[j] % E != 0 || a.side[i].out_stride[j] % E != 0))
        return false;
  return true;
}

template <typename TQ, typename TK, typename TO>
int launch(const Args& a, cudaStream_t stream) {
  const int sms = sm_count() > 0 ? sm_count() : 1;
  const int heads = a.side[0].heads + a.side[1].heads;
  if (!whole_groups<TO>(a)) {
    const long long total = static_cast<long long>(a.B) * a.N * heads * (a.d - a.half);
    const long long want = (total + 255) / 256, cap = sms * 8LL;
    return launch_overlapped(rotary_any_kernel<TQ, TK, TO>,
                             dim3(static_cast<unsigned>(want < cap ? want : cap)), 256, 0, 0,
                             stream, a);
  }
  constexpr int E = Vec<TO>::kElems;
  const int items = a.interleaved ? (a.d + 2 * E - 1) / (2 * E)
                                  : a.half / E + (a.d - 2 * a.half + 2 * E - 1) / (2 * E);
  const long long tokens = static_cast<long long>(a.B) * a.N;
  const long long blocks = (tokens * items + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffffLL) return ATTN_ERR_TOO_LARGE;
  // heads per thread: as many as leave every SM a few blocks
  int per = 8;
  auto groups = [&](int i) { return (a.side[i].heads + per - 1) / per; };
  while (per > 1 && blocks * (groups(0) + groups(1)) < sms * 8LL) per /= 2;
  const int qg = groups(0), kg = groups(1);
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(qg + kg));
  return launch_overlapped(
      a.interleaved ? rotary_kernel<TQ, TK, TO, true> : rotary_kernel<TQ, TK, TO, false>, grid,
      kThreads, 0, 0, stream, a, items, per, qg, tokens);
}

// Checks shared by the two calls.
int check_geometry(const void* turns, const void* positions, long long pos_stride, int B, int H,
                   int H_kv, int N, int d, int rot, float magnitude) {
  if (B < 0 || H < 0 || H_kv < 0 || N < 0 || d <= 0 || rot < 0 || rot > d || rot % 2 != 0 ||
      pos_stride < 0 || !std::isfinite(magnitude))
    return ATTN_ERR_SHAPE;
  if (rot > 0 && turns == nullptr) return ATTN_ERR_NULL;
  if (!aligned16(turns) || (reinterpret_cast<uintptr_t>(positions) & 7u) != 0)
    return ATTN_ERR_ALIGN;
  const long long rows = static_cast<long long>(B) * N;
  if (rows >= (1LL << 40) || H > 65535 || H_kv > 65535 ||
      rows * (static_cast<long long>(H) + H_kv) >= (1LL << 40) / d)
    return ATTN_ERR_TOO_LARGE;
  return ATTN_OK;
}

// Strides of one tensor: given ones (non-negative, the last element's offset
// below 2^40; an output's not 0, where elements would share a place) or those
// of a contiguous [B, heads, N, d]. A dimension of one element has stride 0.
int set_strides(long long (&to)[3], const long long* from, bool output, int B, int heads, int N,
                int d) {
  const long long dense[3] = {static_cast<long long>(heads) * N * d,
                              static_cast<long long>(N) * d, d};
  const long long count[3] = {B, heads, N};
  const bool empty = B == 0 || heads == 0 || N == 0;
  long long last = d;
  for (int i = 0; i < 3; ++i) {
    const long long s = from != nullptr ? from[i] : dense[i];
    if (s < 0 || (output && s == 0 && count[i] > 1 && !empty)) return ATTN_ERR_SHAPE;
    to[i] = 0;
    if (count[i] > 1) {
      if (s >= (1LL << 40) / (count[i] - 1)) return ATTN_ERR_TOO_LARGE;
      last += s * (count[i] - 1);
      to[i] = s;
    }
  }
  return last >= (1LL << 40) ? ATTN_ERR_TOO_LARGE : ATTN_OK;
}

}  // namespace rotary
}  // namespace attn

using namespace attn;

extern "C" int attn_rotary_frequencies(unsigned long long* turns, float* magnitude, int rot,
                                       double base, int scaling, double factor,
                                       int original_length, double low_turns, double high_turns) {
  if (!turns || !magnitude) return ATTN_ERR_NULL;
  if (rot < 0 || rot % 2 != 0 || !std::isfinite(base) || base < 1.0) return ATTN_ERR_SHAPE;
  if (scaling < ATTN_ROTARY_PLAIN || scaling > ATTN_ROTARY_RAMP) return ATTN_ERR_SHAPE;
  if (scaling != ATTN_ROTARY_PLAIN && (!std::isfinite(factor) || factor < 1.0))
    return ATTN_ERR_SHAPE;
  if (scaling == ATTN_ROTARY_RAMP &&
      (original_length <= 0 || !std::isfinite(low_turns) || !std::isfinite(high_turns) ||
       low_turns < 0.0 || high_turns <= low_turns))
    return ATTN_ERR_SHAPE;
  const double two_pi = 6.283185307179586476925286766559;
  if (scaling == ATTN_ROTARY_BASE && rot > 2) base *= std::pow(factor, rot / (rot - 2.0));
  for (int i = 0; i < rot / 2; ++i) {
    double w = std::pow(base, -2.0 * i / rot);  // radians per position
    if (scaling == ATTN_ROTARY_LINEAR) w /= factor;
    if (scaling == ATTN_ROTARY_RAMP) {
      const double turned = original_length * w / two_pi;
      double keep = (turned - low_turns) / (high_turns - low_turns);
      keep = keep < 0.0 ? 0.0 : (keep > 1.0 ? 1.0 : keep);
      w = w * keep + w / factor * (1.0 - keep);
    }
    // w <= 1 radian, so the fraction stays below 2^62
    turns[i] = static_cast<unsigned long long>(std::nearbyint(w / two_pi * 18446744073709551616.0));
  }
  *magnitude =
      scaling == ATTN_ROTARY_RAMP ? static_cast<float>(1.0 + 0.1 * std::log(factor)) : 1.0f;
  return ATTN_OK;
}

extern "C" int attn_rotary(const void* q, const void* k, void* q_out, void* k_out,
                           const unsigned long long* turns, const long long* positions,
                           long long pos_stride, int B, int H, int H_kv, int N, int d, int rot,
                           float magnitude, int interleaved, int adjoint, int dtype,
                           const long long* strides, void* stream) {
  if (B > 0 && N > 0 && ((H > 0 && (!q || !q_out)) || (H_kv > 0 && (!k || !k_out))))
    return ATTN_ERR_NULL;
  int rc = rotary::check_geometry(turns, positions, pos_stride, B, H, H_kv, N, d, rot, magnitude);
  if (rc != ATTN_OK) return rc;
  if (!known_dtype(dtype)) return ATTN_ERR_SHAPE;
  if (!aligned16(q) || !aligned16(k) || !aligned16(q_out) || !aligned16(k_out))
    return ATTN_ERR_ALIGN;
  rotary::Args a{};
  const void* in[2] = {q, k};
  void* out[2] = {q_out, k_out};
  const int heads[2] = {H, H_kv};
  for (int i = 0; i < 2; ++i) {
    a.side[i].in = in[i];
    a.side[i].out = out[i];
    a.side[i].heads = heads[i];
    a.side[i].scale = 1.0f;
    rc = rotary::set_strides(a.side[i].in_stride, strides ? strides + 3 * i : nullptr, false, B,
                             heads[i], N, d);
    if (rc != ATTN_OK) return rc;
    rc = rotary::set_strides(a.side[i].out_stride, strides ? strides + 6 + 3 * i : nullptr, true,
                             B, heads[i], N, d);
    if (rc != ATTN_OK) return rc;
  }
  a.turns = turns;
  a.positions = positions;
  a.pos_stride = pos_stride;
  a.B = B;
  a.N = N;
  a.d = d;
  a.half = rot / 2;
  a.magnitude = magnitude;
  a.sign = adjoint ? -1.0f : 1.0f;
  a.interleaved = interleaved != 0;
  if (B == 0 || N == 0 || H + H_kv == 0) return ATTN_OK;
  return with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    return rotary::launch<T, T, T>(a, as_stream(stream));
  });
}

extern "C" int attn_bwd_finalize_rotary(const float* dq_accum, void* dq, const void* dk,
                                        void* dk_out, float scale, const unsigned long long* turns,
                                        const long long* positions, long long pos_stride, int B,
                                        int H, int H_kv, int N, int d, int rot, float magnitude,
                                        int interleaved, const long long* strides, void* stream) {
  if (B > 0 && N > 0 && ((H > 0 && (!dq_accum || !dq)) || (H_kv > 0 && (!dk || !dk_out))))
    return ATTN_ERR_NULL;
  int rc = rotary::check_geometry(turns, positions, pos_stride, B, H, H_kv, N, d, rot, magnitude);
  if (rc != ATTN_OK) return rc;
  if (!std::isfinite(scale)) return ATTN_ERR_SHAPE;
  if (!aligned16(dq_accum) || !aligned16(dq) || !aligned16(dk) || !aligned16(dk_out))
    return ATTN_ERR_ALIGN;
  rotary::Args a{};
  const void* in[2] = {dq_accum, dk};
  void* out[2] = {dq, dk_out};
  const int heads[2] = {H, H_kv};
  for (int i = 0; i < 2; ++i) {
    a.side[i].in = in[i];
    a.side[i].out = out[i];
    a.side[i].heads = heads[i];
    a.side[i].scale = i == 0 ? scale : 1.0f;
    rc = rotary::set_strides(a.side[i].in_stride, nullptr, false, B, heads[i], N, d);
    if (rc != ATTN_OK) return rc;
    rc = rotary::set_strides(a.side[i].out_stride, strides ? strides + 3 * i : nullptr, true, B,
                             heads[i], N, d);
    if (rc != ATTN_OK) return rc;
  }
  a.turns = turns;
  a.positions = positions;
  a.pos_stride = pos_stride;
  a.B = B;
  a.N = N;
  a.d = d;
  a.half = rot / 2;
  a.magnitude = magnitude;
  a.sign = -1.0f;
  a.interleaved = interleaved != 0;
  if (B == 0 || N == 0 || H + H_kv == 0) return ATTN_OK;
  return rotary::launch<float, __nv_bfloat16, __nv_bfloat16>(a, as_stream(stream));
}
