// The router's choice of experts by scores, its gradient, and the balance
// bias's update.
//
//   score = softmax(x) or 1 / (1 + e^-x);  choice = score + bias (or x)
//   a group's value = its largest choice or the sum of its two largest
//   picks = the k largest choices of the best groups;  w = scale * score / sum
//
// LPT lanes share a token.  Its experts go to them group by group: P = LPT /
// (groups rounded up to a power of two) lanes a group, each with W consecutive
// ids, all in registers (V is what they hold), so a token's logits are read once
// and an equal choice of a lower id is one of a lower lane or slot.
//
// Few tokens wait for a launch and its code, many for the steps of the choice,
// each of which needs the one before; their bytes take less.  16 tokens of 256
// experts in 8 groups take 5.2 us, 16384 of them 15.7 (17.8 MB: 3.2 at the rate of
// a copy) and 16384 of 128 experts without groups 9.4.  The second would take 10.5
// without the counts (every workgroup's atomics on the same lines, one after the
// other) and without the tokens that fp32 leaves open, some 20, for which a wave
// each goes on alone; with either it takes 15.0, since the two overlap.  All
// choices in 64 bits took 127, 32 bits and a search for the largest by a whole wave
// 27 .. 36.
#include <type_traits>
#include <utility>

#include "common.h"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kNoId = 0x7fffffff;

MOE_DEV float neg_inf() { return -__builtin_inff(); }
MOE_DEV double neg_inf64() { return -__builtin_inf(); }

template <typename T>
MOE_DEV float logit_of(T v) {
  if constexpr (std::is_same_v<T, float>) return v;
  else return bf16_to_f32(v);
}

// Where a token's experts are: E experts in n_groups runs of Eg, P = 2^lgP
// lanes a run, W ids a lane.
struct Layout {
  int E, Eg, n_groups, P, lgP, W;
  int lgPw, Ww;        // P and W if a whole wave takes the token
  int full;            // every lane has V experts
  int vec, vec_bias;   // rows, the bias can be read vec_of(V) values at a time
};
struct Place {
  int group, id0, n;   // the lane's run, its first id and how many it has
};
MOE_DEV Place place_of(const Layout& l, int lane, int lgP, int W) {
  Place p;
  p.group = lane >> lgP;
  const int at = (lane & ((1 << lgP) - 1)) * W;
  p.id0 = p.group * l.Eg + at;
  p.n = p.group < l.n_groups && at < l.Eg ? (l.Eg - at < W ? l.Eg - at : W) : 0;
  return p;
}
MOE_DEV Place place_of(const Layout& l, int lane) { return place_of(l, lane, l.lgP, l.W); }

// The lane's V values of a row, 0 .. n - 1 of them its own and the others any
// of the row's: a load behind a condition would be waited for before the next.
constexpr int vec_of(int V) { return V < 4 ? V : 4; }   // values of a load
template <int V, typename T>
MOE_DEV void load_row(const T* row, bool vec, const Place& p, float (&x)[V]) {
  constexpr int N = vec_of(V);
  static_assert(V % N == 0, "whole vectors");
  if (vec) {   // n is a multiple of N
    typedef T Vec __attribute__((ext_vector_type(N)));
#pragma unroll
    for (int i = 0; i < V; i += N) {
      const Vec f = *reinterpret_cast<const Vec*>(row + static_cast<uint32_t>(i < p.n ? p.id0 + i : 0));
#pragma unroll
      for (int j = 0; j < N; ++j) x[i + j] = logit_of(static_cast<T>(f[j]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = logit_of(row[static_cast<uint32_t>(i < p.n ? p.id0 + i : 0)]);
  }
}
// The lane's own values of a row.  (vec: n is a multiple of N; the LDS rows are
// made of whole vectors.)
template <int V, typename T>
MOE_DEV void store_row(T* row, bool vec, const Place& p, const float (&x)[V]) {
  constexpr int N = vec_of(V);
  auto put = [](float f) {
    if constexpr (std::is_same_v<T, float>) return f;
    else return static_cast<T>(pack_bf16x2(f, 0.0f));
  };
  if (vec) {
    typedef T Vec __attribute__((ext_vector_type(N)));
#pragma unroll
    for (int i = 0; i < V; i += N) {
      Vec f;
#pragma unroll
      for (int j = 0; j < N; ++j) f[j] = put(x[i + j]);
      if (i < p.n) *reinterpret_cast<Vec*>(row + p.id0 + i) = f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < p.n) row[p.id0 + i] = put(x[i]);
  }
}
// The lane's logits; slots without an expert and ruled-out ones are -infinity.
template <int V, typename T>
MOE_DEV void load_logits(const T* row, const Layout& l, const Place& p, float (&x)[V]) {
  load_row<V>(row, l.vec, p, x);
  if (!l.full) {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = i < p.n ? x[i] : neg_inf();
  }
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = fmaxf(x[i], neg_inf());   // NaN too
}

template <int CTRL>
MOE_DEV uint32_t dpp(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xF, 0xF, false));
}
// f(other): one step over P lanes after another, other(v) the value that v has in
// the lanes across.
template <typename F>
MOE_DEV void lane_steps(int P, F&& f) {
  if (P > 1) f([](uint32_t v) { return dpp<0xB1>(v); });    // quad_perm: lane ^ 1
  if (P > 2) f([](uint32_t v) { return dpp<0x4E>(v); });    // quad_perm: lane ^ 2
  if (P > 4) f([](uint32_t v) { return dpp<0x141>(v); });   // row_half_mirror: the other quad of 8
  if (P > 8) f([](uint32_t v) { return dpp<0x140>(v); });   // row_mirror: the other 8
  if (P > 16)
    f([](uint32_t v) {
      const auto s = __builtin_amdgcn_permlane16_swap(v, v, false, false);
      return threadIdx.x & 16 ? static_cast<uint32_t>(s[0]) : static_cast<uint32_t>(s[1]);
    });
  if (P > 32)
    f([](uint32_t v) {
      const auto s = __builtin_amdgcn_permlane32_swap(v, v, false, false);
      return threadIdx.x & 32 ? static_cast<uint32_t>(s[0]) : static_cast<uint32_t>(s[1]);
    });
}
template <int LPT, typename T, typename F>
MOE_DEV T over_lanes(T v, F&& f) {
  if constexpr (sizeof(T) == 8) {
#pragma unroll
    for (int o = 1; o < LPT; o <<= 1) v = f(v, __shfl_xor(v, o, kWave));
  } else {
    auto bits = [&] { return __builtin_bit_cast(uint32_t, v); };
    lane_steps(LPT < 16 ? LPT : 16, [&](auto other) { v = f(v, __builtin_bit_cast(T, other(bits()))); });
    if constexpr (LPT == 64) {   // both of the swapped words
      const auto a = __builtin_amdgcn_permlane16_swap(bits(), bits(), false, false);
      v = f(__builtin_bit_cast(T, static_cast<uint32_t>(a[0])), __builtin_bit_cast(T, static_cast<uint32_t>(a[1])));
      const auto b = __builtin_amdgcn_permlane32_swap(bits(), bits(), false, false);
      v = f(__builtin_bit_cast(T, static_cast<uint32_t>(b[0])), __builtin_bit_cast(T, static_cast<uint32_t>(b[1])));
    }
  }
  return v;
}
template <int LPT>
MOE_DEV float max_lanes(float v) {
  return over_lanes<LPT>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int LPT>
MOE_DEV uint32_t max_lanes(uint32_t v) {
  return over_lanes<LPT>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
template <int LPT, typename T>
MOE_DEV T sum_lanes(T v) {
  return over_lanes<LPT>(v, [](T a, T b) { return a + b; });
}

// x - m, 0 for the largest itself (an infinite one too).
MOE_DEV float below(float x, float m) { return x == m ? 0.0f : x - m; }

struct GateP {
  const void* logits;
  const float* bias;
  const uint8_t* mask;
  int32_t* idx;
  float* probs;
  int32_t* counts;
  int64_t ld;
  int T, k;
  float scale;
  Layout l;
  uint8_t sigmoid, top, stay, renorm;   // top: 0 without groups
};

// 1 / (1 + e^-x), which keeps its bits for large -x.
MOE_DEV float sigmoid_of(float x) {
  const float e = expf(-fabsf(x));
  return (x < 0.0f ? e : 1.0f) / (1.0f + e);
}

// The lane's weight share: its pick's score over the sum of the token's, which
// its first kMaxTopK lanes hold.  Scores so small that they, or their share of a
// small sum, would lose bits as subnormal numbers are taken times a factor that
// keeps the token's largest in range, with a sum of such ones.
MOE_DEV float renormed(bool sigmoid, bool live, float x) {
  static_assert(kMaxTopK == 8, "sums over 8 lanes");
  float s = 0.0f, z = 0.0f;
  if (sigmoid) {
    s = live ? sigmoid_of(x) : 0.0f;
    z = sum_lanes<8>(s);
  }
  const bool small = live && !(s > 1e-30f);   // (all, without a sigmoid)
  if (__ballot(small)) {
    const float top = max_lanes<8>(live ? x : neg_inf());
    float r = expf(below(x, top));
    if (sigmoid) r = top < 0.0f ? r / (1.0f + expf(x)) : sigmoid_of(x);
    r = live ? r : 0.0f;
    const float y = sum_lanes<8>(r);
    if (small) {
      s = r;
      z = y;
    }
  }
  return live ? s / z : 0.0f;
}

// ---- the choice in 32 bits ----
// What fp32 arithmetic leaves open, two neighbours in the order nearer than the
// sum of both errors or groups so, is decided by picks64.
//
// Errors of fp32 scores against exact ones.  Sigmoid: the exponential, off by
// (1.5 |x| + 2) 2^-24 of itself, changes s by s (1 - s) times that, at most
// 2^-24; the sum with 1, the reciprocal and the sum with a bias add 2^-24 (3 +
// |c|): in all 2^-22 (1 + |c|).  Softmax: the same of exponentials, and a sum of
// up to 1024 terms over 32 additions and 6 exchanges: under 2^-18 (1 + |c|).
MOE_DEV float score_error(bool sigmoid) { return sigmoid ? 0x1p-22f : 0x1p-18f; }

// A float's bits with the order of its value (that of -0 is below that of +0, so
// logits come with + 0.0f, which makes one of the other); 0 is left for no choice.
MOE_DEV uint32_t key_of(float f) {
  const uint32_t u = __float_as_uint(f);
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
MOE_DEV float value_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

// The lane's choices, those of groups that stay; e: exponentials over the
// largest logit m, of their sum 1 / rz (softmax).  open: two groups are too near.
template <int LPT, int V>
MOE_DEV void choices32(const GateP& g, const Place& p, int lane, const float (&x)[V], const float (&bias)[V], const float (&e)[V], float m,
                       float rz, float (&c)[V], bool& open) {
  const float err = score_error(g.sigmoid);
  auto score = [&](float v, float ev) { return g.sigmoid ? __builtin_amdgcn_rcpf(1.0f + __expf(-v)) : ev * rz; };
  if (g.bias) {
    if (g.sigmoid) {   // (a choice inside the loop would part the exponentials)
#pragma unroll
      for (int i = 0; i < V; ++i) c[i] = __builtin_amdgcn_rcpf(1.0f + __expf(-x[i]));
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) c[i] = e[i] * rz;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      c[i] = fmaxf(c[i] + bias[i], neg_inf());
      c[i] = x[i] > neg_inf() ? c[i] : neg_inf();
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = x[i];
  }
  if (!g.top) return;
  float a = neg_inf(), b = neg_inf();   // the two largest of the group
#pragma unroll
  for (int i = 0; i < V; ++i) {
    b = fmaxf(b, fminf(a, c[i]));
    a = fmaxf(a, c[i]);
  }
  lane_steps(g.l.P, [&](auto other) {
    const float a2 = __uint_as_float(other(__float_as_uint(a))), b2 = __uint_as_float(other(__float_as_uint(b)));
    b = fmaxf(fminf(a, a2), fmaxf(b, b2));
    a = fmaxf(a, a2);
  });
  if (g.top == 2 && !g.bias) {   // choices are logits, sums are of scores
    b = b > neg_inf() ? score(b, __expf(below(b, m))) : neg_inf();
    a = a > neg_inf() ? score(a, __expf(below(a, m))) : neg_inf();
  }
  // errors of two groups' values, each of one or two terms and their sum
  // (a single logit has none)
  const float both = g.top == 2 || g.bias ? 3.0f * err * max_lanes<LPT>(a > neg_inf() ? 2.0f + fabsf(a) + (b > neg_inf() ? fabsf(b) : 0.0f) : 0.0f) : -1.0f;
  if (g.top == 2 && b > neg_inf()) a += b;
  // a group's P lanes compare it with P others at a time
  const int first = threadIdx.x & (kWave - 1) & ~(LPT - 1), sub = lane & (g.l.P - 1);
  int rank = 0;
  for (int o = sub; o - sub < g.l.n_groups; o += g.l.P) {
    const bool in = o < g.l.n_groups;
    const float v = __shfl(a, first + ((in ? o : 0) << g.l.lgP), kWave);
    const bool better = in && (v > a || (v == a && o < p.group));
    open |= in && o != p.group && p.group < g.l.n_groups && v > neg_inf() && a > neg_inf() && fabsf(v - a) <= both;
    rank += __popcll(__ballot(better) >> (first + (p.group << g.l.lgP)) & ((1ull << g.l.P) - 1));
  }
  if (rank >= g.stay) {
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = neg_inf();
  }
}

// The want largest keys of a wave (0: none): put(place, i) for the lane's key i,
// places from 0 on, lower ids first among equal keys; returns how many there
// are above the least key taken if more than these have it, else want.
//
// The threshold that just want keys reach is searched bit by bit, each step a
// comparison of all keys and a count of the lanes: for a token of 256 experts
// half the instructions of taking the largest nine times.
template <int V, typename F>
MOE_DEV int take_largest(const uint32_t (&k)[V], int want, F&& put) {
  uint32_t top = k[0];
#pragma unroll
  for (int i = 1; i < V; ++i) top = k[i] > top ? k[i] : top;
  top = __builtin_amdgcn_readfirstlane(max_lanes<kWave>(top));
  auto reach = [&](uint32_t t) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) n += __popcll(__ballot(k[i] >= t));
    return n;
  };
  // the largest's leading bits, fewer until enough share them (the best of
  // choices of one sign are mostly within an eighth of the largest)
  int b = 20;
  uint32_t t = top >> b << b;
  int n = reach(t > 0 ? t : 1);
  while (n < want) {
    ++b;
    t = b < 32 ? top >> b << b : 0;
    n = reach(t > 0 ? t : 1);
  }
  while (n > want && b > 0) {
    --b;
    const uint32_t u = t | 1u << b;
    const int r = reach(u);
    if (r >= want) {
      t = u;
      n = r;
    }
  }
  // (n > want: t is the last one's key itself, and more have it)
  int at = 0;
  auto take = [&](auto has) {
    uint32_t pos = at;
    bool mine[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      mine[i] = has(k[i]);
      const uint64_t w = __ballot(mine[i]);
      pos = __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(w >> 32), __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(w), pos));
      at += __popcll(w);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (mine[i] && static_cast<int>(pos) < want) put(pos, i);
      pos += mine[i];
    }
  };
  const uint32_t least = n > want ? t + 1 : t > 0 ? t : 1;
  take([&](uint32_t v) { return v >= least; });
  const int above = at;
  if (n > want) take([&](uint32_t v) { return v == t; });
  asm volatile("" ::: "memory");
  __builtin_amdgcn_wave_barrier();   // LDS operations of one wave complete in order
  return n > want ? above : want;
}
template <int V>
MOE_DEV int count_keys(const uint32_t (&k)[V]) {
  int n = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) n += __popcll(__ballot(k[i] != 0));
  return n;
}

// A wave's token: the k + 1 largest go to a lane each and are ranked there.
// room: the wave's 32 words.
template <int V>
MOE_DEV void picks_of_wave(const GateP& g, const Place& p, int lane, const float (&c)[V], int* room, int* own, bool& open) {
  uint32_t k[V];
#pragma unroll
  for (int i = 0; i < V; ++i) k[i] = c[i] > neg_inf() ? key_of(c[i]) : 0;
  const int valid = count_keys<V>(k), want = valid < g.k + 1 ? valid : g.k + 1;
  take_largest<V>(k, want, [&](uint32_t pos, int i) {
    room[pos] = static_cast<int>(k[i]);
    room[16 + pos] = p.id0 + i;
  });
  const bool has = lane < want;
  uint32_t key = has ? static_cast<uint32_t>(room[lane]) : 0;
  const int id = has ? room[16 + lane] : -1;
  int rank = has ? 0 : lane;
  for (int i = 0; i < want; ++i) {
    const uint32_t v = __builtin_amdgcn_readlane(key, i);
    rank += has && (v > key || (v == key && i < lane));
  }
  if (rank < g.k) own[rank] = id;
  if (g.bias) {   // (without one keys are the logits themselves)
    key = __builtin_amdgcn_ds_permute(4 * rank, key);
    const float hi = value_of(key), lo = value_of(dpp<0x101>(key));   // row_shl: the next lane's
    open |= lane + 1 < want && hi - lo <= 2.0f * score_error(g.sigmoid) * (1.0f + fmaxf(fabsf(hi), fabsf(lo)));
  }
}

// The picks of a token by 64-bit choices, by a whole wave, V of them a lane:
// ids to own[0 .. k - 1].  Few tokens come here, and wait for this code to be
// loaded, so it is short: the long steps are loops over choices in LDS.
struct Room64 {
  uint64_t key[16];
  int id[16];
};
template <int V, typename T>
MOE_DEV void picks64(const GateP& g, const T* row, double* choice, Room64* room, int* own) {
  const int lane = threadIdx.x & (kWave - 1);
  const Place p = place_of(g.l, lane, g.l.lgPw, g.l.Ww);
  choice += lane;   // choice i at 64 i
  float x[V], bias[V] = {};
  if (g.bias) load_row<V>(g.bias, false, p, bias);
  load_row<V>(row, false, p, x);
  float m = neg_inf();
#pragma unroll
  for (int i = 0; i < V; ++i) {
    x[i] = fmaxf(i < p.n ? x[i] : neg_inf(), neg_inf()) + 0.0f;   // (-0 too)
    m = fmaxf(m, x[i]);
    choice[kWave * i] = x[i];
  }
  if (!g.sigmoid) m = max_lanes<kWave>(m);
  double z = g.sigmoid ? 1.0 : 0.0;
#pragma unroll 1
  for (int i = 0; i < V; ++i) {
    const double v = choice[kWave * i];
    double s = exp(g.sigmoid ? -v : v == m ? 0.0 : v - m);
    if (g.sigmoid) s = 1.0 / (1.0 + s);
    else z += s = v > neg_inf64() ? s : 0.0;
    choice[kWave * i] = s;
  }
  if (!g.sigmoid) z = sum_lanes<kWave>(z);
  double a = neg_inf64(), b = neg_inf64();   // the lane's two largest
#pragma unroll 1
  for (int i = 0; i < V; ++i) choice[kWave * i] /= z;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    double c = choice[kWave * i] + static_cast<double>(bias[i]);
    c = x[i] > neg_inf() && c > neg_inf64() ? c : neg_inf64();
    // a group's largest choice is a logit without a bias (scores of different logits
    // may be equal), two of them are added as scores
    const double by = g.bias || g.top == 2 ? c : x[i];
    b = fmax(b, fmin(a, by));
    a = fmax(a, by);
    choice[kWave * i] = c;
  }
  bool stays = true;
  if (g.top) {
#pragma unroll 1
    for (int o = 1; o < 1 << g.l.lgPw; o <<= 1) {
      const double a2 = __shfl_xor(a, o, kWave), b2 = __shfl_xor(b, o, kWave);
      b = fmax(fmin(a, a2), fmax(b, b2));
      a = fmax(a, a2);
    }
    if (g.top == 2 && b > neg_inf64()) a += b;
    int rank = 0;
#pragma unroll 1
    for (int o = 0; o < g.l.n_groups; ++o) {
      const double v = __shfl(a, o << g.l.lgPw, kWave);
      rank += v > a || (v == a && o < p.group);
    }
    stays = rank < g.stay;
  }
  // keys in the order of the choices (without a bias of the logits): their
  // upper halves choose 16, whole ones order these
  uint32_t k[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    double c = choice[kWave * i];
    const bool in = stays && c > neg_inf64();
    if (!g.bias && in) c = x[i];
    const uint64_t u = __builtin_bit_cast(uint64_t, c);
    const uint64_t key = in ? u ^ (static_cast<uint64_t>(static_cast<int64_t>(u) >> 63) | 1ull << 63) : 0;
    choice[kWave * i] = __builtin_bit_cast(double, key);
    k[i] = static_cast<uint32_t>(key >> 32);
  }
  const int valid = count_keys<V>(k), want = valid < 16 ? valid : 16;
  const int sure = take_largest<V>(k, want, [&](uint32_t pos, int i) {
    room->key[pos] = __builtin_bit_cast(uint64_t, choice[kWave * i]);
    room->id[pos] = p.id0 + i;
  });
  if (sure >= g.k || sure == want) {
    const bool has = lane < want;
    const uint64_t key = has ? room->key[lane] : 0;
    int rank = 0;
#pragma unroll 1
    for (int i = 0; i < want; ++i) {
      const uint64_t v = room->key[i];
      rank += v > key || (v == key && room->id[i] < room->id[lane & 15]);
    }
    if (has && rank < g.k) own[rank] = room->id[lane];
    if (lane >= want && lane < g.k) own[lane] = -1;
  } else {   // many equal upper halves: the largest, k times
#pragma unroll 1
    for (int j = 0; j < g.k; ++j) {
      uint64_t v = 0;
      int id = kNoId;
#pragma unroll 1
      for (int i = 0; i < V; ++i) {
        const uint64_t u = __builtin_bit_cast(uint64_t, choice[kWave * i]);
        if (u > v) {
          v = u;
          id = p.id0 + i;
        }
      }
#pragma unroll 1
      for (int o = 1; o < kWave; o <<= 1) {
        const uint64_t v2 = __shfl_xor(v, o, kWave);
        const int id2 = __shfl_xor(id, o, kWave);
        const bool take = v2 > v || (v2 == v && id2 < id);
        v = take ? v2 : v;
        id = take ? id2 : id;
      }
      if (lane == 0) own[j] = id == kNoId ? -1 : id;
      if (id >= p.id0 && id < p.id0 + p.n) choice[kWave * (id - p.id0)] = 0.0;
    }
  }
  asm volatile("" ::: "memory");
  __builtin_amdgcn_wave_barrier();
}

// LPT < 64 lanes a token, with their keys sorted; a pick is the largest head of
// the token's lists, of the lowest lane among equal ones, and leaves its list.  The
// low bits of a key are its slot in the lane, a lower id the larger, so two
// choices that differ there only are open, unless all of them have zeros there,
// as logits that were bf16.
template <int V>
MOE_DEV void sort_keys(uint32_t (&k)[V]) {   // descending: Batcher's odd-even merge sort
#pragma unroll
  for (int p = 1; p < V; p *= 2)
#pragma unroll
    for (int q = p; q >= 1; q /= 2)
#pragma unroll
      for (int j = q % p; j + q < V; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i)
          if (i + j + q < V && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
            const uint32_t a = k[i + j], b = k[i + j + q];
            k[i + j] = a > b ? a : b;
            k[i + j + q] = a > b ? b : a;
          }
}
// The first of the list's kList keys leaves it.  (A loop over i would be made
// one over a vector with an index, by compares of every element.)
template <int kList, int V, int... I>
MOE_DEV void pop(uint32_t (&k)[V], bool win, std::integer_sequence<int, I...>) {
  ((k[I] = win ? k[I + 1] : k[I]), ...);
  if (kList == V) k[kList - 1] = win ? 0 : k[kList - 1];   // (no key is 0)
}
// room: 16 pairs of words for the token.
template <int LPT, int V>
MOE_DEV void picks_of_lanes(const GateP& g, const Place& p, int lane, const float (&c)[V], uint2* room, int* own, bool& open) {
  constexpr uint32_t kLow = V - 1, kNone = 0x00800000u;   // (keys of -infinity are below kNone)
  constexpr int kList = V < kMaxTopK + 1 ? V : kMaxTopK + 1;
  uint32_t k[V];
#pragma unroll
  for (int i = 0; i < V; ++i) k[i] = (key_of(c[i]) & ~kLow) | (kLow - i);
  sort_keys<V>(k);
  const int at = threadIdx.x & (kWave - 1) & ~(LPT - 1);   // the token's first lane
  // (rolled: a launch waits for its code)
#pragma unroll 1
  for (int j = 0; j <= g.k; ++j) {
    const uint32_t head = k[0] & ~kLow, top = max_lanes<LPT>(head);
    bool win = head == top;
    const uint64_t with = __ballot(win);
    if (__popcll(with) != kWave / LPT) {   // equal ones: the token's lowest lane
      asm volatile("");   // (a branch: the selects of both ways cost more)
      const uint32_t half = at & 32 ? static_cast<uint32_t>(with >> 32) : static_cast<uint32_t>(with);
      win = lane == __builtin_ctz(half >> (at & 31));
    }
    if (win) room[j] = uint2{k[0], static_cast<uint32_t>(p.id0 + static_cast<int>(kLow - (k[0] & kLow)))};
    pop<kList, V>(k, win, std::make_integer_sequence<int, kList - 1>{});
  }
  asm volatile("" ::: "memory");
  __builtin_amdgcn_wave_barrier();   // LDS operations of one wave complete in order
  // neighbours in the order
  bool near = false;
  for (int j = lane; j < g.k; j += LPT) {
    const uint2 a = room[j], b = room[j + 1];
    own[j] = a.x >= kNone ? static_cast<int>(a.y) : -1;
    if (b.x < kNone) continue;
    if (g.bias) {
      const float hi = value_of(a.x | kLow), lo = value_of(b.x | kLow);
      const float big = fmaxf(fabsf(hi), fabsf(lo));
      // either key's low bits, of a 23-bit mantissa, and either's error
      near |= hi - lo <= static_cast<float>(V) * 0x1p-22f * big + 2.0f * score_error(g.sigmoid) * (1.0f + big);
    } else {
      near |= (a.x ^ b.x) <= kLow;
    }
  }
  if (!g.bias && __ballot(near)) {   // (equal leading bits decide if the others are zeros)
    uint32_t lost = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) lost |= c[i] > neg_inf() ? __float_as_uint(c[i]) & kLow : 0;
    if (!__ballot(lost != 0)) near = false;
  }
  open |= near;
}

template <int LPT, int V, typename T>
MOE_DEV void gate_token(const GateP& g, const T* row, const Place& p, int lane, int64_t t, bool kept, const float (&x)[V], const float (&bias)[V],
                        int* own, int* room, double* choice, Room64* room64, int* s_count) {
  // softmax: the largest logit, the exponentials and their sum
  float e[V] = {}, m = 0.0f, z = 1.0f;
  if (!g.sigmoid && (!g.renorm || g.bias || g.top == 2)) {
    m = x[0];
#pragma unroll
    for (int i = 1; i < V; ++i) m = fmaxf(m, x[i]);
    m = max_lanes<LPT>(m);
    z = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      e[i] = x[i] > neg_inf() ? expf(below(x[i], m)) : 0.0f;
      z += e[i];
    }
    z = sum_lanes<LPT>(z);
  }
  float c[V];
  bool open = false;
  choices32<LPT, V>(g, p, lane, x, bias, e, m, z > 0.0f ? 1.0f / z : 0.0f, c, open);
  if constexpr (LPT == kWave) picks_of_wave<V>(g, p, lane, c, room, own, open);
  else picks_of_lanes<LPT, V>(g, p, lane, c, reinterpret_cast<uint2*>(room), own, open);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_wave_barrier();
  // the tokens left open, one after the other
  for (uint64_t left = __ballot(open && kept); left;) {
    const int first = __builtin_ctzll(left) & ~(LPT - 1);   // the token's first lane
    left &= ~((LPT == kWave ? ~uint64_t{0} : (uint64_t{1} << (LPT & 63)) - 1) << first);
    const int64_t token = __builtin_amdgcn_readlane(static_cast<int>(t), first);
    picks64<(LPT * V + kWave - 1) / kWave, T>(g, static_cast<const T*>(g.logits) + token * g.ld, choice, room64,
                                              own - (threadIdx.x & (kWave - 1)) / LPT * kMaxTopK + first / LPT * kMaxTopK);
  }
  const int id = kept && lane < g.k ? own[lane] : -1;
  const bool live = id >= 0;
  const float xi = live ? logit_of(row[id]) : neg_inf();
  float w;
  if (g.renorm) w = renormed(g.sigmoid, live, xi);
  else w = g.sigmoid ? sigmoid_of(xi) : expf(below(xi, m)) / z;
  if (lane < g.k && t < g.T) {
    g.idx[t * g.k + lane] = id;
    g.probs[t * g.k + lane] = live ? g.scale * w : 0.0f;
    if (live && g.counts) atomicAdd(s_count + id, 1);
  }
}

// Workgroups of kThreads, or larger ones where these leave no CU free: what a
// workgroup counts goes to counts in one pass.
constexpr int gate_threads(int V) { return V > 16 ? 2 * kThreads : 4 * kThreads; }

template <int LPT, int V, typename T>
__global__ __launch_bounds__(gate_threads(V)) void gate_kernel(const GateP g) {
  constexpr int kTokens = gate_threads(V) / LPT, kWaves = gate_threads(V) / kWave, kWide = (LPT * V + kWave - 1) / kWave;
  __shared__ int s_id[kTokens][kMaxTopK];
  __shared__ __attribute__((aligned(8))) int s_room[kTokens][32];
  __shared__ int s_count[kMaxExperts];
  __shared__ double s_choice[kWaves][kWave * kWide];
  __shared__ Room64 s_room64[kWaves];
  const int threads = blockDim.x, lane = threadIdx.x & (LPT - 1);
  // (a wave's token is the same for all lanes, which the compiler does not see)
  const int in_wg = LPT == kWave ? __builtin_amdgcn_readfirstlane(threadIdx.x / LPT) : threadIdx.x / LPT;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (threads / LPT) + in_wg;
  const Place p = place_of(g.l, lane);
  const int64_t tl = t < g.T ? t : g.T - 1;   // (a token past the last one loads its row)
  const T* row = static_cast<const T*>(g.logits) + tl * g.ld;
  const bool kept = t < g.T && (!g.mask || g.mask[tl] != 0);
  float x[V], bias[V] = {};
  if (g.bias) load_row<V>(g.bias, g.l.vec_bias, p, bias);
  load_logits<V>(row, g.l, p, x);
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] += 0.0f;   // -0 becomes +0
  if (g.counts) {
    for (int e = threadIdx.x; e < g.l.E; e += threads) s_count[e] = 0;
    __syncthreads();
  }
  // (all lanes of a wave stay: a token's exact choice is made by all of them)
  if (__ballot(t < g.T))
    gate_token<LPT, V, T>(g, row, p, lane, t, kept, x, bias, s_id[in_wg], s_room[in_wg], s_choice[threadIdx.x / kWave],
                          s_room64 + threadIdx.x / kWave, s_count);
  if (g.counts) {
    __syncthreads();
    // (each from a place of its own: where all workgroups begin with the same
    // line, 512 of them take 5 us longer)
    int e = (threadIdx.x + blockIdx.x * kWave) % g.l.E;
    for (int i = threadIdx.x; i < g.l.E; i += threads) {
      if (s_count[e]) atomicAdd(g.counts + e, s_count[e]);
      e = (e + threads) % g.l.E;
    }
  }
}

struct GateBwdP {
  const void* logits;
  const int32_t* idx;
  const float* dprobs;
  void* dlogits;
  int64_t ld, ld_d;
  int T, E, k;
  float scale;
  Layout l;
  uint8_t sigmoid, renorm, accumulate, vec_d;
};

// The gradient reads the logits (where every one has a part in it) and writes as
// many: bound by these bytes for many tokens, by the launch for few.  A wave for a
// token from 65 experts on (16384 x 256, 35 MB: 8.5 us, with 16 lanes 10.9; 256 x
// 8 takes 4.2).  Rows go out through LDS of their own, where the picks' terms are
// added to them.
template <int LPT, int V, typename T>
__global__ __launch_bounds__(kThreads) void gate_bwd_kernel(const GateBwdP g) {
  __shared__ __attribute__((aligned(16))) float s_row[kThreads * V];
  const int lane = threadIdx.x & (LPT - 1);
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kThreads / LPT) + threadIdx.x / LPT;
  if (t >= g.T) return;
  float* own = s_row + threadIdx.x / LPT * (LPT * V);
  const T* row = static_cast<const T*>(g.logits) + t * g.ld;
  const Place p = place_of(g.l, lane);
  const bool full = !g.sigmoid && !g.renorm;   // every logit has a gradient
  // (loads not behind conditions: a lane without a pick has the first one's)
  const int64_t slot = t * g.k + (lane < g.k ? lane : 0);
  const int id = lane < g.k ? g.idx[slot] : -1;
  const float dp = g.dprobs[slot];
  bool live = id >= 0 && id < g.E;
  float x[V] = {};
  float term, dot = 0.0f;
  if (full) {
    load_logits<V>(row, g.l, p, x);
    float m = neg_inf();
#pragma unroll
    for (int i = 0; i < V; ++i) m = fmaxf(m, x[i]);
    m = max_lanes<LPT>(m);
    float z = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      x[i] = x[i] > neg_inf() ? expf(below(x[i], m)) : 0.0f;
      z += x[i];
    }
    z = sum_lanes<LPT>(z);
    const float r = z > 0.0f ? 1.0f / z : 0.0f;
    store_row<V>(own, true, p, x);   // the picks' scores come from there
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();   // LDS operations of one wave complete in order
    // (a ruled-out pick's is 0, and its gradient too, whatever its dprobs is)
    const float e = live ? own[id] : 0.0f;
    live = e > 0.0f;
    term = live ? e * r * (g.scale * dp) : 0.0f;
    dot = sum_lanes<LPT>(term) * r;
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] *= -dot;
  } else {
    const float xi = live ? logit_of(row[id]) : neg_inf();
    live = live && xi > neg_inf();
    const float d = live ? g.scale * dp : 0.0f;
    if (g.renorm) {
      const float w = renormed(g.sigmoid, live, xi);
      const float mean = sum_lanes<LPT>(w * d);
      term = live ? w * (d - mean) : 0.0f;
      if (g.sigmoid) term *= sigmoid_of(-xi);
    } else {
      const float e = expf(-fabsf(xi));   // s (1 - s), either sign
      term = live ? d * (e / ((1.0f + e) * (1.0f + e))) : 0.0f;
    }
  }
  asm volatile("" ::: "memory");
  __builtin_amdgcn_wave_barrier();
  store_row<V>(own, true, p, x);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_wave_barrier();
  if (live) atomicAdd(own + id, term);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_wave_barrier();
  T* out = static_cast<T*>(g.dlogits) + t * g.ld_d;
  load_row<V>(own, true, p, x);
  if (g.accumulate) {
    float before[V];
    load_row<V>(out, g.vec_d, p, before);
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] += before[i];
  }
  store_row<V>(out, g.vec_d, p, x);
}

constexpr int kBiasThreads = 1024;
static_assert(kBiasThreads >= kMaxExperts, "a thread for every expert");
__global__ __launch_bounds__(kBiasThreads) void bias_update_kernel(int E, float rate, int reset, int32_t* counts, float* bias) {
  __shared__ int64_t s_sum[kBiasThreads / kWave];
  const int e = threadIdx.x;
  const int64_t n = e < E ? counts[e] : 0;
  int64_t total = n;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) total += __shfl_xor(total, o, kWave);
  if ((e & (kWave - 1)) == 0) s_sum[e / kWave] = total;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int w = 0; w < kBiasThreads / kWave; ++w) total += s_sum[w];
  if (e >= E) return;
  if (n * E != total) bias[e] += n * E < total ? rate : -rate;
  if (reset) counts[e] = 0;
}

int next_pow2(int v) {
  int p = 1;
  while (p < v) p <<= 1;
  return p;
}

// Lanes a token takes and logits a lane holds: the first that hold it of those
// up to 16 lanes, or of a wave's.  A wave shortens the way of one token, more of
// them share the instructions of 16 lanes each: 256 experts in 8 groups take 5.2
// us (wave) or 8.4 for 16 tokens, 27 .. 36 or 15.7 for 16384; a wave it is up to
// 4 tokens a CU, one for each of its SIMDs.
struct Shape {
  int lanes, values;
};
constexpr Shape kShapes[] = {{8, 4}, {16, 4}, {16, 8}, {16, 16}, {64, 2}, {64, 4}, {64, 8}, {64, 16}, {64, 32}};
constexpr int kLaneShapes = 4, kAllShapes = 9;
int shape_for(int E, int n_groups, bool wave, Layout* l) {
  l->E = E;
  l->n_groups = n_groups;
  l->Eg = E / n_groups;
  const int g2 = next_pow2(n_groups);
  for (int i = wave ? kLaneShapes : 0; i < kAllShapes; ++i) {
    if (kShapes[i].lanes < g2) continue;
    l->P = kShapes[i].lanes / g2;
    l->lgP = 0;
    while (1 << l->lgP < l->P) ++l->lgP;
    const int n = vec_of(kShapes[i].values);
    l->W = ((l->Eg + l->P - 1) / l->P + n - 1) / n * n;
    l->lgPw = 0;
    while (1 << l->lgPw < kWave / g2) ++l->lgPw;
    l->Ww = (l->Eg + kWave / g2 - 1) / (kWave / g2);
    l->full = l->Eg == l->P * kShapes[i].values && n_groups == g2;
    if (l->W <= kShapes[i].values) return i;
  }
  return -1;
}

bool can_vec(const Layout& l, int shape, const void* p, int64_t ld, int bytes) {
  const int n = vec_of(kShapes[shape].values);
  return l.Eg % n == 0 && ld % n == 0 && reinterpret_cast<uintptr_t>(p) % (n * bytes) == 0;
}

template <typename F>
void with_shape(int i, F&& f) {
  auto go = [&](auto at) {
    constexpr Shape k = kShapes[decltype(at)::value];
    f(std::integral_constant<int, k.lanes>{}, std::integral_constant<int, k.values>{});
  };
  switch (i) {
    case 0: go(std::integral_constant<int, 0>{}); break;
    case 1: go(std::integral_constant<int, 1>{}); break;
    case 2: go(std::integral_constant<int, 2>{}); break;
    case 3: go(std::integral_constant<int, 3>{}); break;
    case 4: go(std::integral_constant<int, 4>{}); break;
    case 5: go(std::integral_constant<int, 5>{}); break;
    case 6: go(std::integral_constant<int, 6>{}); break;
    case 7: go(std::integral_constant<int, 7>{}); break;
    default: go(std::integral_constant<int, 8>{}); break;
  }
}

}  // namespace

hipError_t launch_router_gate(const moe_gate_args& a, int cu, hipStream_t s) {
  GateP g{};
  g.logits = a.logits;
  g.bias = a.bias;
  g.mask = a.token_mask;
  g.idx = a.expert_idx;
  g.probs = a.probs;
  g.counts = a.counts;
  g.ld = a.ld ? a.ld : a.E;
  g.T = a.T;
  g.k = a.k;
  g.scale = a.scale;
  g.sigmoid = a.score == MOE_SCORE_SIGMOID;
  const int groups = a.n_groups > 1 && a.topk_groups < a.n_groups ? a.n_groups : 1;   // all stay: no groups
  g.top = groups > 1 ? static_cast<uint8_t>(a.group_top) : 0;
  g.stay = groups > 1 ? static_cast<uint8_t>(a.topk_groups) : 1;
  g.renorm = a.renorm != 0;
  const int shape = shape_for(a.E, groups, a.E > 64 && a.T <= 4 * cu, &g.l);
  if (shape < 0) return hipErrorInvalidValue;   // (every E <= 1024 with up to 64 groups has one)
  const bool f32 = a.logits_type == MOE_TYPE_F32;
  g.l.vec = can_vec(g.l, shape, a.logits, g.ld, f32 ? 4 : 2);
  g.l.vec_bias = can_vec(g.l, shape, a.bias, 0, 4);
  with_shape(shape, [&](auto lpt, auto v) {
    constexpr int L = decltype(lpt)::value, V = decltype(v)::value;
    const int64_t all = static_cast<int64_t>(a.T) * L;
    const int threads = all > static_cast<int64_t>(kThreads) * cu ? gate_threads(V) : kThreads;
    const uint32_t blocks = static_cast<uint32_t>((all + threads - 1) / threads);
    if (f32) gate_kernel<L, V, float><<<blocks, threads, 0, s>>>(g);
    else gate_kernel<L, V, bf16_t><<<blocks, threads, 0, s>>>(g);
  });
  return hipGetLastError();
}

hipError_t launch_router_gate_bwd(const moe_gate_bwd_args& a, hipStream_t s) {
  GateBwdP g{};
  g.logits = a.logits;
  g.idx = a.expert_idx;
  g.dprobs = a.dprobs;
  g.dlogits = a.dlogits;
  g.ld = a.ld ? a.ld : a.E;
  g.ld_d = a.ld_d ? a.ld_d : a.E;
  g.T = a.T;
  g.E = a.E;
  g.k = a.k;
  g.scale = a.scale;
  g.sigmoid = a.score == MOE_SCORE_SIGMOID;
  g.renorm = a.renorm != 0;
  g.accumulate = a.accumulate != 0;
  const int shape = shape_for(a.E, 1, a.E > 64, &g.l);   // (as measured above)
  if (shape < 0) return hipErrorInvalidValue;
  const bool f32 = a.logits_type == MOE_TYPE_F32;
  g.l.vec = can_vec(g.l, shape, a.logits, g.ld, f32 ? 4 : 2);
  g.vec_d = can_vec(g.l, shape, a.dlogits, g.ld_d, f32 ? 4 : 2);
  with_shape(shape, [&](auto lpt, auto v) {
    constexpr int L = decltype(lpt)::value, V = decltype(v)::value;
    const int64_t blocks = (static_cast<int64_t>(a.T) * L + kThreads - 1) / kThreads;
    if (f32) gate_bwd_kernel<L, V, float><<<static_cast<uint32_t>(blocks), kThreads, 0, s>>>(g);
    else gate_bwd_kernel<L, V, bf16_t><<<static_cast<uint32_t>(blocks), kThreads, 0, s>>>(g);
  });
  return hipGetLastError();
}

hipError_t launch_bias_update(const moe_bias_update_args& a, hipStream_t s) {
  bias_update_kernel<<<1, kBiasThreads, 0, s>>>(a.E, a.rate, a.reset, a.counts, a.bias);
  return hipGetLastError();
}

}  // namespace moe
