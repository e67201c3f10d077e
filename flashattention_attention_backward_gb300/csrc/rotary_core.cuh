// The rotation of one row's heads in registers, shared by the rotary kernels and
// the append to a paged cache.
#pragma once

#include <cstdint>

#include "element.cuh"

namespace attn {
namespace rotary {

// What a row's rotation needs besides its position: turns [half] per position,
// the row's d columns (2 half of them turn), the factor on cosine and sine, the
// direction (+1, or -1 for the adjoint) and a factor on every element.
struct Turn {
  const unsigned long long* turns;
  int d, half;
  float magnitude, sign, scale;
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
template <typename TI, typename TO, int U, bool INTERLEAVED, typename Position>
__device__ __forceinline__ void rotate_row_heads(const Turn& p, const TI* in, long long in_head,
                                                 TO* out, long long out_head, int heads,
                                                 int item, Position position) {
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
  float cs[E], sn[E];
  bool ready = false;
  for (int h = 0; h < heads; h += U) {
    Group<TI, E> ga[U], gb[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (h + u < heads) {
        ga[u].load(in + u * in_head + ca);
        if (has_b) gb[u].load(in + u * in_head + cb);
      }
    }
    if (!ready) {  // behind the first loads, so that their latency covers it
      ready = true;
      if (turn_a) {
        const long long pos = position();
        const float m = p.magnitude * p.scale, ms = m * p.sign;
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
      if (h + u >= heads) continue;
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
            a[i] *= p.scale;
            a[i + 1] *= p.scale;
          }
          if (turn_b) {
            const float x = v[i], y = v[i + 1];
            v[i] = x * cs[(E + i) / 2] - y * sn[(E + i) / 2];
            v[i + 1] = x * sn[(E + i) / 2] + y * cs[(E + i) / 2];
          } else {
            v[i] *= p.scale;
            v[i + 1] *= p.scale;
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const float x = a[i], y = v[i];
          a[i] = turn_a ? x * cs[i] - y * sn[i] : x * p.scale;
          v[i] = turn_a ? x * sn[i] + y * cs[i] : y * p.scale;
        }
      }
      Vec<TO> w;
      pack(a, w);
      store_vec(out + u * out_head + ca, w);
      if (has_b) {
        pack(v, w);
        store_vec(out + u * out_head + cb, w);
      }
    }
    in += U * in_head;
    out += U * out_head;
  }
}

}  // namespace rotary
}  // namespace attn
