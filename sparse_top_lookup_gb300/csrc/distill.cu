// Distillation from a teacher's top logits: the loss and its gradient.
//
// Per row b of student logits z [V], with the teacher's list (idx_j, t_j),
// j < k, and a temperature T:
//   p = softmax(t / T) over the list, q = softmax(z / T) over all V,
//   loss = T^2 sum_j p_j (log p_j - log q[idx_j])
//   dz   = dloss * T * (P q - sum_j p_j [idx_j])      P = sum_j p_j (1, or 0
//                                                     for an empty list)
// An entry with a negative idx, or a t of -inf, is absent.
//
// Bound by HBM: the logits are read once and (with a gradient) dz is written
// once.  A row is held in shared memory between its sum and its gradient.  It
// is cut into slices, one for each CTA of a cluster, which exchange (maximum,
// sum); short rows are held in the registers of a warp each.
//
// Softmax arithmetic is in powers of two: with c = log2(e) / T and the
// largest logit m, the terms are 2^((z - m) c).  Where |m c| < 2^24 the sums
// form them as 2^(z c - r), r = rn(m c), one instruction less, and 2^(r - m c)
// at the end, within 2^(1/2) of 1; further out (masked stretches, tiny T) what
// r leaves of m c grows to powers that overflow, and the difference comes first.
//
// Measured, GB/s of logits read and dz written (a copy reaches 6802), ten calls in a graph: training
// step fp32 4096 x 65536 6650 (98 %), bf16 4096 x 131072 with lists of 64 6440 (95 %), loss alone,
// bf16 4096 x 131072 6840 (101 %), backward pass bf16 4096 x 131072 6490 (95 %).
#include <cuda_bf16.h>
#include <math.h>
#include <stdint.h>

#include "num_common.cuh"
#include "pkm_internal.cuh"
#include "tc_common.cuh"

namespace pkm {
namespace {

using tc::cluster_ctarank;
using tc::mapa_shared;
using tc::smem_u32;

constexpr int DTHREADS = 256;
constexpr int DWARPS = DTHREADS / 32;
constexpr int kMaxLsh = 3, kMaxSlices = 1 << kMaxLsh;  // CTAs of a cluster (the portable limit)
constexpr int kWarpMaxK = 128;   // longest list of the warp-per-row form (its shared memory)

enum Mode { kFwd, kBwd, kTrain };

// Set-up before this may run before the launch before this one has ended (programmatic dependent
// launch); no memory is read or written until it has.
__device__ __forceinline__ void after_earlier_work() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <typename E>
struct El;
template <>
struct El<float> {
  static constexpr int kPerVec = 4;
  static constexpr uint32_t kNegInf = 0xff800000u;
  __device__ static float get(float v) { return v; }
  __device__ static void put(float* p, float v) { *p = v; }
  __device__ static float get(const uint4& d, int i) {
    return __uint_as_float(i == 0 ? d.x : i == 1 ? d.y : i == 2 ? d.z : d.w);
  }
  // the largest value of several vectors (NaNs are passed over)
  struct Max {
    float m = -INFINITY;
    __device__ void add(const uint4& d) {
      m = fmaxf(m, fmaxf(fmaxf(get(d, 0), get(d, 1)), fmaxf(get(d, 2), get(d, 3))));
    }
    __device__ float value() const { return m; }
  };
};
template <>
struct El<__nv_bfloat16> {
  static constexpr int kPerVec = 8;
  static constexpr uint32_t kNegInf = 0xff80ff80u;
  __device__ static float get(__nv_bfloat16 v) { return __bfloat162float(v); }
  __device__ static void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
  __device__ static float get(const uint4& d, int i) {
    const uint32_t w = i < 2 ? d.x : i < 4 ? d.y : i < 6 ? d.z : d.w;
    return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
  }
  struct Max {
    uint32_t w = kNegInf;
    __device__ void add(const uint4& d) {
      auto h = [](const uint32_t& v) { return *reinterpret_cast<const __nv_bfloat162*>(&v); };
      const __nv_bfloat162 m =
          __hmax2(__hmax2(h(w), __hmax2(h(d.x), h(d.y))), __hmax2(h(d.z), h(d.w)));
      w = *reinterpret_cast<const uint32_t*>(&m);
    }
    __device__ float value() const {
      return fmaxf(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
  };
};

// Two fp32 operations in one instruction, each rounded as by itself (the loss of 4096 x 131072 bf16:
// 167 us one by one, 159 so, when that was chosen).
struct Two {
  unsigned long long v;
  __device__ Two(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
  __device__ float2 get() const {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
  }
};
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(a.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return a;
}
__device__ __forceinline__ Two add2(Two a, Two b) {
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(a.v) : "l"(a.v), "l"(b.v));
  return a;
}

// A positive s as f 2^e, f in [0.75, 1.5): its log is e log 2 + logf(f), to about 1e-8 when the
// two are added in 64 bits.
struct Split {
  int e;
  float f;
};
__device__ __forceinline__ Split split(float s) {
  Split r;
  r.f = frexpf(s, &r.e);  // [0.5, 1)
  if (r.f < 0.75f) r.f *= 2.0f, --r.e;
  return r;
}

// s * exp(m / T), s in the order of 1 (m = -inf: nothing yet, s is 0 or NaN).
struct Sum {
  float m, s;
};
// The sum over groups of kLanes lanes of a warp (a power of two; every group has the same), on
// every lane.
template <int kLanes>
__device__ __forceinline__ Sum lanes_join(Sum a, float c) {
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(a.m));
  float s = m == -INFINITY ? a.s : a.s * ex2((a.m - m) * c);
#pragma unroll
  for (int o = kLanes / 2; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return Sum{m, s};
}

struct DistillArgs {
  const void* z;
  void* dz;
  int64_t ld, ld_d;
  int B, V, k, kpad;  // kpad: k rounded up to 4
  int lsh;            // log2 of a row's slices: the cluster's CTAs, or (kBwd) separate units
  int slots, chunk;   // ring of the CTA-per-slice form: slots of `chunk` 16-byte vectors
  float T;
  double inv_t, t2;   // 1 / T, T^2
  const int64_t* idx;
  const float *teacher, *dloss;
  float *loss, *lse;  // kBwd reads lse
  int* status;        // may be NULL
};

// What calls without a status word report into (looked up by the kernels: the address costs the
// host 0.3 us a call).
__device__ int g_distill_status;
__device__ __forceinline__ int* status_of(const DistillArgs& a) {
  return a.status ? a.status : &g_distill_status;
}

// A row as whole 16-byte vectors, and the few elements before and after them (slice 0's); the
// vectors [v0, v1) are one slice's.
template <typename E>
struct Row {
  const E* z;
  const uint4* vec;
  int head, nvec, v0, v1, extra;  // extra: this thread's element outside the vectors, or -1
  __device__ Row(const DistillArgs& a, int64_t b, int slice, int lsh, int tid) {
    constexpr int kPer = El<E>::kPerVec;
    z = static_cast<const E*>(a.z) + b * a.ld;
    const int off = (int)((reinterpret_cast<uintptr_t>(z) & 15u) / sizeof(E));
    head = min((kPer - off) % kPer, a.V);
    nvec = (a.V - head) / kPer;
    vec = reinterpret_cast<const uint4*>(z + head);
    const int per = (nvec + (1 << lsh) - 1) >> lsh;
    v0 = min(slice * per, nvec), v1 = min(v0 + per, nvec);
    extra = slice == 0 && tid < a.V - nvec * kPer ? (tid < head ? tid : nvec * kPer + tid) : -1;
  }
  // whether column `at` is this slice's
  __device__ bool mine(int at, int slice) const {
    constexpr int kPer = El<E>::kPerVec;
    if (at < head || at >= head + nvec * kPer) return slice == 0;
    const int v = (at - head) / kPer;
    return v >= v0 && v < v1;
  }
};

// The teacher's list of one row in shared memory.
struct List {
  int* idx;    // column, -1: absent
  float* t;
  float* z;    // the student's logit there
  float* p;    // softmax over the list (0 where absent)
  float* dz;   // the column's gradient (list_grad())
  __device__ List(unsigned char* base, int kpad)
      : idx(reinterpret_cast<int*>(base)),
        t(reinterpret_cast<float*>(base) + kpad),
        z(reinterpret_cast<float*>(base) + 2 * kpad),
        p(reinterpret_cast<float*>(base) + 3 * kpad),
        dz(reinterpret_cast<float*>(base) + 4 * kpad) {}
  // By one warp: whether a column occurs twice among those of the first n that count(column), through
  // a table of 2 n columns' hashes in t's place.
  template <typename F>
  __device__ bool twice(int n, int lane, F&& count) const {
    constexpr unsigned short kNone = 0xffff;
    unsigned short* seen = reinterpret_cast<unsigned short*>(t);
    for (int j = lane; j < 2 * n; j += 32) seen[j] = kNone;
    __syncwarp();
    bool found = false;
    for (int j0 = 0; j0 < n; j0 += 32) {
      const int j = j0 + lane, at = j < n ? idx[j] : -1;
      uint32_t slot = __umulhi((uint32_t)at * 0x9E3779B1u, 2u * n);
      for (bool open = at >= 0 && count(at); __any_sync(0xffffffffu, open);) {
        if (!open) continue;
        const unsigned short other = atomicCAS(seen + slot, kNone, (unsigned short)j);
        if (other == kNone)
          open = false;
        else if (idx[other] == at)
          found = true, open = false;
        else if (++slot == 2u * n)
          slot = 0;
      }
    }
    return __any_sync(0xffffffffu, found);
  }
};
constexpr int kListBytes = 16;      // per entry
constexpr int kGradListBytes = 20;  // with dz

// One warp's loader of lists, whose loads from memory take as long as a few units of work: begin()
// asks for a row's first 64 entries, ask() (some time later) for the student's logits there, end()
// (later again) puts the list together and loads the rest of a longer one, kBatch * 32 at a time
// (more cost registers, which lists of up to 64 pay for too: training step 4096 x 131072 bf16, k = 64 and 128,
// with 1, 2, 4 and 8: 338 and 421, 340 and 404, 342 and 438, 385 and 527 us).
template <typename E, int kBatch = 2>
struct ListLoader {
  int64_t raw[2];  // what begin() asked for
  float raw_t[2];
  int at[2];       // what ask() made of it
  float t[2], z[2];
  __device__ void begin(const DistillArgs& a, int64_t b, int lane) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int j = h * 32 + lane;
      raw[h] = -1, raw_t[h] = -INFINITY;
      if (j < a.k) raw[h] = a.idx[b * a.k + j], raw_t[h] = a.teacher[b * a.k + j];
    }
  }
  // The column, -1 if the entry is absent, and the student's logit there; only in this slice unless
  // `all`, 0 elsewhere.
  __device__ static int column(const DistillArgs& a, int64_t i, float t, bool report) {
    if (i >= a.V && report) atomicExch(status_of(a), PKM_ERR_BAD_INDEX);
    return i >= 0 && i < a.V && t != -INFINITY ? (int)i : -1;
  }
  __device__ static float logit(const Row<E>& row, int slice, bool all, int at) {
    return at >= 0 && (all || row.mine(at, slice)) ? El<E>::get(row.z[at]) : 0.0f;
  }
  __device__ void ask(const DistillArgs& a, const Row<E>& row, int slice, bool all, bool report) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      at[h] = column(a, raw[h], raw_t[h], report), t[h] = raw_t[h];
      z[h] = logit(row, slice, all, at[h]);
    }
  }
  // Forms p; returns the largest t (-inf for an empty list) and the sum of exp((t - largest) / T).
  __device__ Sum end(const List& l, const DistillArgs& a, int64_t b, int slice, int lsh, bool all,
                     bool report, float c, int lane) {
    float tm = -INFINITY;
    auto entry = [&](int j, int aj, float tj, float zj) {
      if (j >= a.kpad) return;
      l.idx[j] = aj, l.t[j] = tj, l.z[j] = zj;
      if (aj >= 0) tm = tj > tm || isnan(tj) ? tj : tm;
    };
    entry(lane, at[0], t[0], z[0]);
    entry(32 + lane, at[1], t[1], z[1]);
    if (a.kpad > 64) {
      const Row<E> row(a, b, slice, lsh, 0);
      for (int j0 = 64; j0 < a.kpad; j0 += 32 * kBatch) {
        int64_t i[kBatch];
        float tj[kBatch], zj[kBatch];
#pragma unroll
        for (int h = 0; h < kBatch; ++h) {
          const int j = j0 + 32 * h + lane;
          i[h] = -1, tj[h] = -INFINITY;
          if (j < a.k) i[h] = a.idx[b * a.k + j], tj[h] = a.teacher[b * a.k + j];
        }
#pragma unroll
        for (int h = 0; h < kBatch; ++h) {
          i[h] = column(a, i[h], tj[h], report);
          zj[h] = logit(row, slice, all, (int)i[h]);
        }
#pragma unroll
        for (int h = 0; h < kBatch; ++h) entry(j0 + 32 * h + lane, (int)i[h], tj[h], zj[h]);
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const float v = __shfl_xor_sync(0xffffffffu, tm, o);
      tm = v > tm || isnan(v) ? v : tm;
    }
    auto term = [&](int aj, float tj) { return aj >= 0 ? ex2((tj - tm) * c) : 0.0f; };
    const float e0 = term(at[0], t[0]), e1 = term(at[1], t[1]);
    float total = e0 + e1;
    for (int j = 64 + lane; j < a.kpad; j += 32) total += l.p[j] = term(l.idx[j], l.t[j]);
#pragma unroll
    for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    const float inv = total > 0.0f || isnan(total) ? 1.0f / total : 0.0f;
    if (lane < a.kpad) l.p[lane] = e0 * inv;
    if (32 + lane < a.kpad) l.p[32 + lane] = e1 * inv;
    for (int j = 64 + lane; j < a.kpad; j += 32) l.p[j] *= inv;
    __syncwarp();
    return Sum{tm, total};
  }
};
// By one warp: loss and lse of row b from its sum and its list (ls: what loading it returned).
//   log p_j - log q_j = ((t_j - tm) - (z_j - m)) / T + log(sum of q's terms / sum of p's)
// The loss is a small difference of large logits, so each is taken from its maximum first; what is
// left is good to fp32, and the logs and the last sums are in 64 bits (few of them: the GPU does
// two 64-bit operations per SM and cycle, and with whole rows of terms in 64 bits they took
// longer than rows of 2000 columns).
__device__ void put_loss(const DistillArgs& a, int64_t b, const Sum& sum, const List& list,
                         const Sum& ls, int lane) {
  float d = 0.0f;
  if (ls.m != -INFINITY)
    for (int j = lane; j < a.k; j += 32) {
      const float p = list.p[j];
      if (p != 0.0f)  // (a NaN counts)
        d += list.z[j] == -INFINITY ? INFINITY : p * ((list.t[j] - ls.m) - (list.z[j] - sum.m));
    }
#pragma unroll
  for (int o = 16; o; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
  if (lane == 0) {
    constexpr double kLn2 = 0.6931471805599453;
    const Split q = split(sum.s), p = split(ls.s);
    const float log_q = logf(q.f);
    double loss = 0.0;
    if (ls.m != -INFINITY)
      loss = sum.s == 0.0f ? (double)INFINITY
                           : a.t2 * (d * a.inv_t + ((q.e - p.e) * kLn2 + (double)(log_q - logf(p.f))));
    a.loss[b] = (float)loss;
    if (a.lse)
      a.lse[b] = sum.s == 0.0f ? -INFINITY : (float)(sum.m * a.inv_t + (q.e * kLn2 + log_q));
  }
}

// The fast forms of a gradient take the row's reference in the exponent of 2^(z c + off), off of
// magnitude below this (a limit of 2^24 would do for fp32, where only the rest of off's rounding
// matters; the difference first costs one instruction more per logit).
constexpr float kFastOff = 1024.0f;

// g q(z) of a row, from its sum; every q is 0 when every logit is -inf.  With the factor
// 2^(z c + off) ahead of `scale` the difference z - ref costs no instruction; what the rounding of
// off leaves is in scale_fast.  For bf16 the factor |scale| goes into the exponent too (off_all,
// rounded by 2^-14 / 2 at most below kFastOff, where dz is rounded to 2^-8), and its sign into the
// packed result.  Rows further out (masked stretches, a common offset, tiny T) are `far` and take
// the difference first.
struct Grad {
  float c, ref, scale, scale_fast, off, off_all;
  bool far;
  Grad() = default;
  __device__ Grad(float c, float ref, float scale) : c(c), ref(ref), scale(scale) {
    off = -ref * c;
    scale_fast = scale * ex2(fmaf(-ref, c, -off));
    off_all = off + log2f(fabsf(scale_fast));
    far = !(fabsf(off) < kFastOff && fabsf(off_all) < kFastOff);
  }
  __device__ float operator()(float z) const { return ex2((z - ref) * c) * scale; }
  __device__ float fast(float z) const { return ex2(fmaf(z, c, off)) * scale_fast; }
};
__device__ __forceinline__ Grad grad_of(const Sum& sum, float g, float c) {
  const float ref = sum.m == -INFINITY ? 0.0f : sum.m;
  return Grad(c, ref, sum.s == 0.0f ? 0.0f : __fdividef(g, sum.s));
}
// From an lse in fp32: q = exp(z / T - lse).  The forms are Grad's.  Far rows keep q within [0, 1],
// which an lse so rounded says no more about (from 10^5 T on; at a mask's value of -10^9 it holds
// the row's maximum alone): off is a quarter there, so that any lse has one, and off_all what its
// rounding leaves.
struct GradLse {
  float c, scale, off, off_all;
  bool far;
  __device__ GradLse(float lse, float g, float c) : c(c) {
    // (a row whose lse is NaN or +inf has no gradient)
    scale = lse < INFINITY ? g : NAN;
    if (lse == -INFINITY) lse = 0.0f;  // every logit is -inf, or beyond fp32: q is 0
    off = -lse * kLog2e;
    const float scale_fast = scale * ex2(fmaf(-lse, kLog2e, -off));
    off_all = off + log2f(fabsf(scale_fast));
    far = !(fabsf(off) < kFastOff && fabsf(off_all) < kFastOff);
    if (far) {
      off = -lse * (0.25f * kLog2e);
      off_all = fmaf(-lse, 0.25f * kLog2e, -off);
    } else {
      scale = scale_fast;
    }
  }
  __device__ float operator()(float z) const {
    if (!far) return fast(z);
    const float e = 4.0f * (fmaf(z, 0.25f * c, off) + off_all);
    return ex2(e > 0.0f ? 0.0f : e) * scale;
  }
  __device__ float fast(float z) const { return ex2(fmaf(z, c, off)) * scale; }
};

// By kThreads threads (whole warps): the gradients of the listed columns, from z as it was (dz may be
// z).  sum: a column may be there twice; four threads to an entry share the search for its others.
template <int kThreads, typename G>
__device__ __forceinline__ void list_grad(const List& list, const DistillArgs& a, bool sum,
                                          const G& q, float g, int tid) {
  if (!sum) {
    for (int j = tid; j < a.k; j += kThreads)
      if (list.idx[j] >= 0) list.dz[j] = fmaf(-g, list.p[j], q(list.z[j]));
    return;
  }
  const int part = tid & 3;
  for (int j0 = 0; j0 < a.kpad; j0 += kThreads / 4) {
    const int j = j0 + (tid >> 2);
    if (j0 + ((tid & ~31) >> 2) >= a.kpad) break;  // (a whole warp)
    const int at = j < a.kpad ? list.idx[j] : -1;
    float p = 0.0f;
    if (at >= 0)
      for (int l = 4 * part; l < a.kpad; l += 16) {
        const int4 i4 = *reinterpret_cast<const int4*>(list.idx + l);
        const float4 p4 = *reinterpret_cast<const float4*>(list.p + l);
        p += (i4.x == at ? p4.x : 0.0f) + (i4.y == at ? p4.y : 0.0f) +
             (i4.z == at ? p4.z : 0.0f) + (i4.w == at ? p4.w : 0.0f);
      }
    p += __shfl_xor_sync(0xffffffffu, p, 1);
    p += __shfl_xor_sync(0xffffffffu, p, 2);
    if (at >= 0 && part == 0) list.dz[j] = fmaf(-g, p, q(list.z[j]));
  }
}

// By one warp: the listed columns of a row's slice, whose values replace those that the row's q alone
// gave them (z as it was is in the list: dz may be z).  The list is used up: the slice's entries
// move to its front.
template <typename E, typename G>
__device__ __forceinline__ void put_listed(const DistillArgs& a, const Row<E>& row, int slice,
                                           E* out, const List& list, const G& q, float g,
                                           int lane) {
  int n = 0;
  for (int j0 = 0; j0 < a.kpad; j0 += 32) {
    const int j = j0 + lane;
    const int at = j < a.kpad ? list.idx[j] : -1;
    const bool mine = at >= 0 && row.mine(at, slice);
    const float p = mine ? list.p[j] : 0.0f, z = mine ? list.z[j] : 0.0f;
    const uint32_t all = __ballot_sync(0xffffffffu, mine);  // (every lane has read)
    const int to = n + __popc(all & ((1u << lane) - 1u));
    if (mine) list.idx[to] = at, list.p[to] = p, list.z[to] = z;
    n += __popc(all);
  }
  if (n + lane < (n + 3) / 4 * 4) list.idx[n + lane] = -1, list.p[n + lane] = 0.0f;
  __syncwarp();
  // A column's entries are summed.  More than 64 are looked through for one that occurs twice first:
  // every entry against every other takes n^2 / 128 steps of the warp.
  const bool sum = n <= 64 || list.twice(n, lane, [](int) { return true; });
  for (int j = lane; j < n; j += 32) {
    const int at = list.idx[j];
    float p = sum ? 0.0f : list.p[j];
    if (sum)
      for (int l = 0; l < n; l += 4) {
        const int4 i4 = *reinterpret_cast<const int4*>(list.idx + l);
        const float4 p4 = *reinterpret_cast<const float4*>(list.p + l);
        p += (i4.x == at ? p4.x : 0.0f) + (i4.y == at ? p4.y : 0.0f) +
             (i4.z == at ? p4.z : 0.0f) + (i4.w == at ? p4.w : 0.0f);
      }
    El<E>::put(out + at, fmaf(-g, p, q(list.z[j])));
  }
}

// Elements from p to the next 16-byte boundary.
template <typename E>
__device__ __forceinline__ int shift_of(const E* p) {
  return (int)(((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / sizeof(E));
}

// 16 bytes from byte kBytes on of w and the vector behind it.
template <int kBytes>
__device__ __forceinline__ uint4 window(const uint32_t (&c)[8]) {
  constexpr int i = kBytes / 4;
  if constexpr (kBytes % 4 == 0)
    return make_uint4(c[i], c[i + 1], c[i + 2], c[i + 3]);
  else
    return make_uint4(__funnelshift_r(c[i], c[i + 1], 16), __funnelshift_r(c[i + 1], c[i + 2], 16),
                      __funnelshift_r(c[i + 2], c[i + 3], 16),
                      __funnelshift_r(c[i + 3], c[i + 4], 16));
}

// One vector of dz per lane: vector v (< end) of the row's body, from z's vector d.  shift: from the
// body to the next 16-byte boundary; where it is not 0 a lane stores the 16 aligned bytes that begin
// in its vector and end in the next lane's, and the warp's first and last elements go singly.
enum Form { kZero, kFast, kSlow };
template <Form kForm>
struct FormOf {
  static constexpr Form value = kForm;
};
template <typename E, Form kForm, typename G>
__device__ __forceinline__ void put_vector(E* body, int v, int end, const uint4& d, const G& q,
                                           int shift, int lane) {
  constexpr int kPer = El<E>::kPerVec;
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kForm == kZero) {
      w[i] = 0;
    } else if constexpr (kPer == 4) {
      const float z = El<E>::get(d, i);
      w[i] = __float_as_uint(kForm == kFast ? q.fast(z) : q(z));
    } else {
      const float z0 = El<E>::get(d, 2 * i), z1 = El<E>::get(d, 2 * i + 1);
      if constexpr (kForm == kFast)
        w[i] = pack2(ex2(fmaf(z0, q.c, q.off_all)), ex2(fmaf(z1, q.c, q.off_all))) ^
               (q.scale < 0.0f ? 0x80008000u : 0u);
      else
        w[i] = pack2(q(z0), q(z1));
    }
  }
  if (shift == 0) {
    if (v < end) __stcs(reinterpret_cast<uint4*>(body) + v, make_uint4(w[0], w[1], w[2], w[3]));
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) w[4 + i] = __shfl_down_sync(0xffffffffu, w[i], 1);
  const int last = min(32, end - (v - lane)) - 1;  // the warp's last vector, may be below 0
  E* o = body + (int64_t)v * kPer;
  if (lane < last) {
    uint4 x;
    if constexpr (kPer == 4)
      x = shift == 1 ? window<4>(w) : shift == 2 ? window<8>(w) : window<12>(w);
    else
      switch (shift) {
        case 1: x = window<2>(w); break;
        case 2: x = window<4>(w); break;
        case 3: x = window<6>(w); break;
        case 4: x = window<8>(w); break;
        case 5: x = window<10>(w); break;
        case 6: x = window<12>(w); break;
        default: x = window<14>(w); break;
      }
    __stcs(reinterpret_cast<uint4*>(o + shift), x);
  }
#pragma unroll
  for (int e = 0; e < kPer; ++e)
    if ((lane == 0 && last >= 0 && e < shift) || (lane == last && e >= shift)) {
      if constexpr (kPer == 4)
        o[e] = __uint_as_float(w[e]);
      else
        reinterpret_cast<unsigned short*>(o)[e] = (unsigned short)(w[e / 2] >> (16 * (e & 1)));
    }
}

// sum joined with the terms of vectors d, by one thread: 2^((z - m) c).
template <typename E, int kNV>
__device__ __forceinline__ void add_vectors(Sum& sum, const uint4 (&d)[kNV], float c) {
  constexpr int kPer = El<E>::kPerVec;
  typename El<E>::Max most;
#pragma unroll
  for (int j = 0; j < kNV; ++j) most.add(d[j]);
  const float m = fmaxf(sum.m, most.value());
  const float ref = m == -INFINITY ? 0.0f : m;
  Two s0(m == -INFINITY ? sum.s : sum.s * ex2((sum.m - ref) * c), 0.0f), s1(0.0f, 0.0f);
  const Two less(-ref, -ref);
  auto terms = [&](const uint4& v, int i) {
    const float2 t = add2(Two(El<E>::get(v, i), El<E>::get(v, i + 1)), less).get();
    return Two(ex2(t.x * c), ex2(t.y * c));
  };
#pragma unroll
  for (int j = 0; j < kNV; ++j)
#pragma unroll
    for (int i = 0; i < kPer; i += 4) s0 = add2(s0, terms(d[j], i)), s1 = add2(s1, terms(d[j], i + 2));
  const float2 sa = s0.get(), sb = s1.get();
  sum = Sum{m, (sa.x + sa.y) + (sb.x + sb.y)};
}
// The same for `count` vectors in shared memory, kThreads apart, as 2^(z c - r), r = rn(m c),
// and one factor 2^(r - m c) for them all; one by one in the form above from |m c| = 2^24 on, where
// r is off by more than half.
template <typename E, int kThreads>
__device__ __forceinline__ void add_shared(Sum& sum, const uint4* src, int count, float c) {
  constexpr int kPer = El<E>::kPerVec;
  typename El<E>::Max most;
#pragma unroll 4
  for (int j = 0; j < count; ++j) most.add(src[j * kThreads]);
  const float m = fmaxf(sum.m, most.value());
  const float r = m * c;
  if (!(fabsf(r) < 16777216.0f)) {
#pragma unroll 1
    for (int j = 0; j < count; ++j) {
      const uint4 one[1] = {src[j * kThreads]};
      add_vectors<E>(sum, one, c);
    }
    return;
  }
  Two s0(0.0f, 0.0f), s1(0.0f, 0.0f);
  const Two cc(c, c), rr(-r, -r);
  auto terms = [&](const uint4& d, int i) {
    const float2 t = fma2(Two(El<E>::get(d, i), El<E>::get(d, i + 1)), cc, rr).get();
    return Two(ex2(t.x), ex2(t.y));
  };
#pragma unroll 4
  for (int j = 0; j < count; ++j) {
    const uint4 d = src[j * kThreads];
#pragma unroll
    for (int i = 0; i < kPer; i += 4) s0 = add2(s0, terms(d, i)), s1 = add2(s1, terms(d, i + 2));
  }
  const float2 sa = s0.get(), sb = s1.get();
  const float before = sum.m == -INFINITY ? sum.s : sum.s * ex2((sum.m - m) * c);
  sum = Sum{m, fmaf((sa.x + sa.y) + (sb.x + sb.y), ex2(fmaf(-m, c, r)), before)};
}
__device__ __forceinline__ void add_one(Sum& sum, float x, float c) {
  const float m = fmaxf(sum.m, x);
  const float ref = m == -INFINITY ? 0.0f : m;
  sum = Sum{m, (m == -INFINITY ? sum.s : sum.s * ex2((sum.m - ref) * c)) + ex2((x - ref) * c)};
}

template <typename E>
__device__ __forceinline__ uint4 masked_vector() {
  return make_uint4(El<E>::kNegInf, El<E>::kNegInf, El<E>::kNegInf, El<E>::kNegInf);
}

// Short rows: a warp each, which keeps the row in registers, kNV vectors per lane, between its
// sum and its gradient.  Bound by the lists and the loss's logs more than by the logits: training
// step bf16 8192 x 2000 31 us with lists of 64 (65 MB), 26 with lists of 4.
template <typename E, int kNV, int kMode>
__global__ void __launch_bounds__(DTHREADS, kNV == 2 ? 4 : 3)
distill_warp_kernel(const DistillArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float c = kLog2e / a.T;
  const List list(smem + (size_t)warp * kListBytes * a.kpad, a.kpad);
  const int64_t step = (int64_t)gridDim.x * DWARPS;
  int64_t b = (int64_t)blockIdx.x * DWARPS + warp;
  after_earlier_work();
  ListLoader<E, 1> loader;
  if (b < a.B) loader.begin(a, b, lane);
  for (; b < a.B; b += step) {
    const Row<E> row(a, b, 0, 0, lane);
    loader.ask(a, row, 0, true, true);
    uint4 d[kNV];
#pragma unroll
    for (int j = 0; j < kNV; ++j)
      d[j] = j * 32 + lane < row.nvec ? __ldcs(row.vec + j * 32 + lane) : masked_vector<E>();
    const float x = row.extra >= 0 ? El<E>::get(row.z[row.extra]) : -INFINITY;
    const float g = kMode == kFwd ? 0.0f : a.dloss[b] * a.T;
    const float lse = kMode == kBwd ? a.lse[b] : 0.0f;
    const Sum ls = loader.end(list, a, b, 0, 0, true, true, c, lane);
    if (b + step < a.B) loader.begin(a, b + step, lane);
    Sum sum{-INFINITY, 0.0f};
    if constexpr (kMode != kBwd) {
      add_vectors<E>(sum, d, c);
      add_one(sum, x, c);
      sum = lanes_join<32>(sum, c);
    }
    __syncwarp();
    if constexpr (kMode != kBwd) put_loss(a, b, sum, list, ls, lane);
    if constexpr (kMode != kFwd) {
      const bool zero = g == 0.0f || ls.m == -INFINITY;  // no gradient, whatever z holds
      const auto q = [&] {
        if constexpr (kMode == kBwd) return GradLse(lse, g, c);
        else return grad_of(sum, g, c);
      }();
      E* out = static_cast<E*>(a.dz) + b * a.ld_d;
      const int shift = shift_of(out + row.head);
#pragma unroll
      for (int j = 0; j < kNV; ++j) {
        const int v = j * 32 + lane;
        if (zero)
          put_vector<E, kZero>(out + row.head, v, row.nvec, d[j], q, shift, lane);
        else
          put_vector<E, kSlow>(out + row.head, v, row.nvec, d[j], q, shift, lane);
      }
      if (row.extra >= 0) El<E>::put(out + row.extra, zero ? 0.0f : q(x));
      __syncwarp();  // the listed columns come after the row
      if (!zero) put_listed(a, row, 0, out, list, q, g, lane);
    }
    __syncwarp();
  }
}

// kBwd: units of 8 vectors per data thread, each by itself, in registers.  A list warp is a unit
// ahead with the lists (two copies: a unit's is in use until the next unit's barrier).  lse is
// known, so nothing is exchanged and units need no ring: loads of 8 vectors per thread and three
// CTAs per SM cover HBM's latency.  fp32 1500 x 50257 97 us (6220 GB/s, 92 %), bf16 4096 x 131072
// with lists of 64 337 (6380), with lists of 4 333.
constexpr int kBwdVecs = 8;
template <typename E>
__global__ void __launch_bounds__(DTHREADS + 32, 3)
distill_backward_kernel(const DistillArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ Sum s_ls[2];
  __shared__ bool s_sum[2];  // a column may occur twice in the list
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float c = kLog2e / a.T;
  const int64_t units = (int64_t)a.B << a.lsh;
  auto list_at = [&](int i) { return List(smem + (size_t)i * kGradListBytes * a.kpad, a.kpad); };
  auto slice_of = [&](int64_t unit) { return (int)(unit & ((1 << a.lsh) - 1)); };
  if (warp == DWARPS) {
    ListLoader<E> loader;
    loader.begin(a, blockIdx.x >> a.lsh, lane);
    int par = 0;
    for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x, par ^= 1) {
      const int slice = slice_of(unit);
      const bool report = slice == 0;
      const Row<E> row(a, unit >> a.lsh, slice, a.lsh, 0);
      loader.ask(a, row, slice, false, report);
      const Sum ls = loader.end(list_at(par), a, unit >> a.lsh, slice, a.lsh, false, report, c, lane);
      const bool sum = a.kpad <= 64 || list_at(par).twice(a.kpad, lane, [&](int at) {
        return row.mine(at, slice);
      });
      if (lane == 0) s_ls[par] = ls, s_sum[par] = sum;
      if (unit + gridDim.x < units) loader.begin(a, (unit + gridDim.x) >> a.lsh, lane);
      __syncthreads();
    }
    return;
  }
  int par = 0;
  for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x, par ^= 1) {
    const int64_t b = unit >> a.lsh;
    const int slice = slice_of(unit);
    const Row<E> row(a, b, slice, a.lsh, tid);
    uint4 d[kBwdVecs];
#pragma unroll
    for (int j = 0; j < kBwdVecs; ++j) {
      const int v = row.v0 + j * DTHREADS + tid;
      d[j] = v < row.v1 ? __ldcs(row.vec + v) : masked_vector<E>();
    }
    const float x = row.extra >= 0 ? El<E>::get(row.z[row.extra]) : -INFINITY;
    const float g = a.dloss[b] * a.T;
    const GradLse q(a.lse[b], g, c);
    __syncthreads();  // the unit's list
    const List list = list_at(par);
    const bool zero = g == 0.0f || s_ls[par].m == -INFINITY;
    if (!zero) list_grad<DTHREADS>(list, a, s_sum[par], q, g, tid);
    E* out = static_cast<E*>(a.dz) + b * a.ld_d;
    const int shift = shift_of(out + row.head);
    auto put = [&](auto form) {
#pragma unroll
      for (int j = 0; j < kBwdVecs; ++j) {
        const int v = row.v0 + j * DTHREADS + tid;
        if (v - lane >= row.v1) break;
        put_vector<E, decltype(form)::value>(out + row.head, v, row.v1, d[j], q, shift, lane);
      }
    };
    if (zero)
      put(FormOf<kZero>());
    else if (q.far)
      put(FormOf<kSlow>());
    else
      put(FormOf<kFast>());
    if (row.extra >= 0) El<E>::put(out + row.extra, zero ? 0.0f : q(x));
    // the listed columns' values replace those of the row
    asm volatile("bar.sync 2, %0;" ::"n"(DTHREADS) : "memory");
    if (!zero)
      for (int j = tid; j < a.k; j += DTHREADS) {
        const int at = list.idx[j];
        if (at >= 0 && row.mine(at, slice)) El<E>::put(out + at, list.dz[j]);
      }
  }
}

// kFwd and kTrain: a CTA per slice of a row, a cluster per row.
//   data warps  each chunk of the slice: maximum and sum (first pass); then (kTrain) each chunk
//               again: the gradient, written out (second pass).  A vector is always the same
//               warp's, so the warps need no barrier among themselves;
//   list warps  (a row each in turn) join the data warps' sums and send them to the cluster's CTAs
//               (st.async to shared memory), form what the second pass needs from what comes back,
//               and do the rows' lists: p, the listed columns, the loss (by the slices in turn);
//   copy warp   the slices' chunks by bulk copies into a ring of slots.
// The data warps have 8 vectors each of a 32 KB slice, in which every instruction per row counts:
// with the sums' joining, the gradient's constants and the lists among their work, 4096 x 131072
// bf16 took 396 us with lists of 64 and 369 with lists of 4, without it 343 and 334.  The lists take a
// warp longer than the data warps need for a row: two list warps 397 us, three 342, four 344 (and
// fewer registers).
// A row's second pass comes after the next row's first, so the exchange costs no waiting, and
// in kTrain a slot is free when its gradient is written: the ring holds up to three rows'
// slices, one in each pass and one on its way.
//
// Order (kTrain).  A data warp: first pass of i + 1, local(i + 1), wait grad(i), second pass of i.
// A list warp, for every L-th row (L list warps): wait local(i), send i, wait sums(i), grad(i), the
// listed columns of i - L, list i + L, loss of i.  local(i): every data warp's sum of row i is
// written; sums(i): every slice's sum of row i has come; grad(i): what the second pass of i needs is
// there.  So
// - local(i + L) says that row i's second pass is over: its listed columns replace what that wrote,
//   after which its list may go (local(count) and later ones are for these alone);
// - dz may be z: row i is written after sums(i), so after every CTA has read list i;
// - with 2 L copies, a warp's sum i + 2 L is written after grad(i + L), and another CTA sends
//   i + 2 L after its grad(i + L), for which this CTA has sent i + L: both come after all that
//   the list warp of row i does for it but its listed columns, which need its own copies only.
// In kFwd, without second passes, data warps wait for sums(i - L) before they write their sum i.
//
// Giving up.  A warp whose wait runs out, or that sees that another's did, sends and writes nothing
// more.  A list warp leaves when its last row's sums have come from every CTA, which is the last that
// any sends to it; one that gave up ends at a barrier of the cluster instead, so that its CTA's memory
// stays while another may send to it (threads that have left count as arrived).  What it has sent
// itself has landed by then: it waits for that row's sums, whose senders wait for its own in turn, or
// until that wait has run out too.  With the barrier on every path 4096 x 131072 bf16 took 336 us, so 333.
constexpr int kListWarps = 3;
constexpr int kCopies = 2 * kListWarps;
constexpr int kMaxSlots = 16;
constexpr int kChunkVecs = 2048;        // 32 KB
constexpr size_t kDynamic = 216 * 1024;  // dynamic shared memory at most
constexpr int kTrainChunks = 2;  // of a slice, at most: two slices fit beside the longest lists
static_assert(2 * kTrainChunks * 16 * kChunkVecs + kCopies * kListBytes * PKM_DISTILL_MAX_K <=
                  kDynamic,
              "ring of the longest slices");

// What the data warps need of a row, written by the copy warp before the row's first chunk.
template <typename E>
struct Geo {
  E* body;   // dz at the slice's first vector
  const E* z;
  float g;   // dloss * T
  int n;     // vectors of the slice
  int head, nvec, v0, ends;  // as in Row; ends: elements outside the vectors (slice 0: else 0)
  int shift;  // elements from dz's body to the next 16-byte boundary
};

// What the second pass needs of a row, by its list warp.
struct RowGrad {
  Grad q;
  float g;    // dloss * T
  bool zero;  // no gradient, whatever z holds
};

constexpr int kData = DWARPS;
constexpr int kStreamThreads = 32 * (kData + kListWarps + 1);
template <typename E, int kMode>
__global__ void __launch_bounds__(kStreamThreads, 3)
distill_stream_kernel(const DistillArgs a) {
  using namespace tc;
  constexpr int kThreads = kData * 32, kPer = El<E>::kPerVec;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ Sum s_warp[kCopies][kData];
  __shared__ __align__(8) Sum s_slice[kCopies][kMaxSlices];
  __shared__ __align__(16) RowGrad s_grad[kCopies];
  __shared__ __align__(16) Geo<E> s_geo[kCopies];
  __shared__ __align__(8) uint64_t s_bars[2 * kMaxSlots + 3 * kCopies];
  __shared__ int s_abort;
  const int tid = (int)threadIdx.x - 32 * (kListWarps + 1);  // of the data threads
  const int lane = threadIdx.x & 31, warp = (int)(threadIdx.x >> 5) - (kListWarps + 1);
  const float c = kLog2e / a.T;
  const int lsh = a.lsh, slices = 1 << lsh;
  const int slots = a.slots, chunk = a.chunk;
  uint4* ring = reinterpret_cast<uint4*>(smem);
  unsigned char* lists = smem + (size_t)slots * chunk * 16;
  auto list_at = [&](int i) { return List(lists + (size_t)i * kListBytes * a.kpad, a.kpad); };
  const uint32_t bar0 = smem_u32(s_bars);
  auto bar_full = [&](int s) { return bar0 + 8u * s; };
  auto bar_empty = [&](int s) { return bar0 + 8u * (kMaxSlots + s); };
  auto bar_sums = [&](int i) { return bar0 + 8u * (2 * kMaxSlots + i % kCopies); };
  auto bar_local = [&](int i) { return bar0 + 8u * (2 * kMaxSlots + kCopies + i % kCopies); };
  auto bar_grad = [&](int i) { return bar0 + 8u * (2 * kMaxSlots + 2 * kCopies + i % kCopies); };
  if (threadIdx.x == 0) {
    for (int s = 0; s < slots; ++s) {
      mbar_init(bar_full(s), 1);
      mbar_init(bar_empty(s), kData);
    }
    for (int i = 0; i < kCopies; ++i) {
      mbar_init(bar_sums(i), 1);
      mbar_init(bar_local(i), kData);
      mbar_init(bar_grad(i), 1);
    }
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  cluster_sync();  // every CTA's barriers exist before its memory is written
  after_earlier_work();
  const Ctl ctl{&s_abort, status_of(a)};

  // this CTA's slice (consecutive CTAs, a cluster's, have those of one row) of rows first + i *
  // every, i < count
  const int slice = (int)(blockIdx.x & (slices - 1));
  const int64_t first = blockIdx.x >> lsh, every = gridDim.x >> lsh;
  const int count = (int)((a.B - first + every - 1) / every);
  auto row_at = [&](int i) { return first + i * every; };
  if (warp == -1) {
    // ---------------------------------------------------------------- copies
    if (lane == 0) {
      int s = 0, issued = 0;
      uint32_t ph = 1;
      bool ok = true;
      for (int i = 0; ok && i < count; ++i) {
        const int64_t b = row_at(i);
        const Row<E> row(a, b, slice, lsh, 0);
        Geo<E> geo;
        E* out = static_cast<E*>(a.dz) + b * a.ld_d + row.head;
        geo.body = out + (int64_t)row.v0 * kPer;
        geo.z = row.z;
        geo.g = kMode == kTrain ? a.dloss[b] * a.T : 0.0f;
        geo.n = row.v1 - row.v0;
        geo.head = row.head, geo.nvec = row.nvec, geo.v0 = row.v0;
        geo.ends = slice == 0 ? a.V - row.nvec * kPer : 0;
        geo.shift = shift_of(out);
        int v = 0;
        do {  // (a slice without vectors is one empty chunk)
          if (!(ok = wait_phase(bar_empty(s), ph, ctl))) break;
          // the slot is free, so its row's predecessors up to kCopies back are done with
          if (v == 0) s_geo[i % kCopies] = geo;
          const uint32_t bytes = 16u * min(chunk, geo.n - v);
          if (bytes) {
            mbar_expect_tx(bar_full(s), bytes);
            bulk_load(smem_u32(ring + (size_t)s * chunk), row.vec + row.v0 + v, bytes, bar_full(s));
          } else {
            mbar_arrive(bar_full(s));
          }
          if (issued < slots) ++issued;
          if (++s == slots) s = 0, ph ^= 1u;
          v += chunk;
        } while (v < geo.n);
      }
      // (normally the data warps have waited for them all) no copy outlives the CTA
      for (int i = 0; i < issued; ++i) {
        if (--s < 0) s = slots - 1, ph ^= 1u;
        wait_phase_drain(bar_full(s), ph ^ 1u);
      }
    }
    return;
  }
  // Waits of a whole warp; false: gave up.  wait_sums: every slice's sum of row i has come.
  auto all = [](bool ok) { return __all_sync(0xffffffffu, ok) != 0; };
  auto wait_sums = [&](int i) {
    return all(wait_phase_cluster(bar_sums(i), (uint32_t)(i / kCopies) & 1u, ctl));
  };
  auto sum_of = [&](int i) {
    return lanes_join<kMaxSlices>(lane % kMaxSlices < slices
                                      ? s_slice[i % kCopies][lane % kMaxSlices]
                                      : Sum{-INFINITY, 0.0f}, c);
  };
  if (warp < 0) {
    // ---------------------------------------------------------------- lists, sums, losses
    auto my_loss = [&](int i) { return (i / kListWarps & (slices - 1)) == slice; };
    // (kFwd needs a row's list for its loss alone)
    auto wanted = [&](int i) { return i < count && (kMode == kTrain || my_loss(i)); };
    ListLoader<E> loader;
    Sum ls_next{-INFINITY, 0.0f};
    auto ask = [&](int i) {  // for its logits, and for the next one's list
      if (wanted(i)) {
        const Row<E> row(a, row_at(i), slice, lsh, 0);
        loader.ask(a, row, slice, my_loss(i), my_loss(i));
      }
      if (wanted(i + kListWarps)) loader.begin(a, row_at(i + kListWarps), lane);
    };
    auto load = [&](int i) {  // what was asked for
      if (wanted(i))
        ls_next = loader.end(list_at(i % kCopies), a, row_at(i), slice, lsh, my_loss(i),
                             my_loss(i), c, lane);
      ask(i + kListWarps);
    };
    const int h = warp + kListWarps + 1;
    if (wanted(h)) loader.begin(a, row_at(h), lane);
    ask(h);
    load(h);
    int sent = -1;  // the last row whose sum was sent
    // (kTrain: as many rows more, for the listed columns of the last)
    for (int i = h; i < count + (kMode == kTrain ? kListWarps : 0); i += kListWarps) {
      const Sum ls = ls_next;
      if (!all(wait_phase(bar_local(i), (uint32_t)(i / kCopies) & 1u, ctl))) break;
      if (i < count) {
        sent = i;
        const Sum sum = lanes_join<kData>(s_warp[i % kCopies][lane & (kData - 1)], c);
        // to every CTA of the cluster (this one too), completing on the receiver's barrier
        if (lane == 0) mbar_expect_tx(bar_sums(i), 8u * slices);
        if (lane < slices)
          asm volatile(
              "st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];" ::
                  "r"(mapa_shared(smem_u32(&s_slice[i % kCopies][slice]), lane)),
              "r"(__float_as_uint(sum.m)), "r"(__float_as_uint(sum.s)),
              "r"(mapa_shared(bar_sums(i), lane))
              : "memory");
      }
      if (kMode == kTrain && i < count) {
        const float g = s_geo[i % kCopies].g;
        if (!wait_sums(i)) break;
        const Grad q = grad_of(sum_of(i), g, c);
        if (lane == 0) {
          s_grad[i % kCopies] = RowGrad{q, g, g == 0.0f || ls.m == -INFINITY};
          mbar_arrive(bar_grad(i));
        }
      }
      // an earlier row is written but for its listed columns
      if (kMode == kTrain && i >= kListWarps && !s_grad[(i - kListWarps) % kCopies].zero) {
        const RowGrad last = s_grad[(i - kListWarps) % kCopies];
        const int64_t b = row_at(i - kListWarps);
        const List list = list_at((i - kListWarps) % kCopies);
        put_listed(a, Row<E>(a, b, slice, lsh, 0), slice, static_cast<E*>(a.dz) + b * a.ld_d, list,
                   last.q, last.g, lane);
      }
      __syncwarp();
      load(i + kListWarps);
      if (i < count && my_loss(i)) {
        if (!wait_sums(i)) break;
        put_loss(a, row_at(i), sum_of(i), list_at(i % kCopies), ls, lane);
      }
    }
    // Once its last row's sums have come from every CTA, none sends to this warp's barriers again
    // (earlier rows' came before that row's were sent).
    const bool done = sent < 0 ? h >= count : sent + kListWarps >= count && wait_sums(sent);
    if (!done) {
      if (sent >= 0) wait_phase_drain(bar_sums(sent), (uint32_t)(sent / kCopies) & 1u);
      __syncwarp();
      if (slices > 1) cluster_sync();
    }
    return;
  }
  // ------------------------------------------------------------------ data
  int s1 = 0, s2 = 0;  // next slot of the first and the second pass
  uint32_t ph = 0;     // its parity in the first
  float x = -INFINITY, x_last;  // this thread's element outside the vectors
  for (int i = 0; i <= count; ++i) {
    x_last = x;
    if (i < count) {
      Sum sum{-INFINITY, 0.0f};
      if (!all(wait_phase(bar_full(s1), ph, ctl))) return;  // (gave up)
      const Geo<E>& geo = s_geo[i % kCopies];
      const int total = geo.n;
      x = -INFINITY;
      if (tid < geo.ends) x = El<E>::get(geo.z[tid < geo.head ? tid : geo.nvec * kPer + tid]);
      for (int v = 0;;) {
        const uint4* src = ring + (size_t)s1 * chunk + tid;
        const int n = min(chunk, total - v);
        add_shared<E, kThreads>(sum, src, max(0, n - tid + kThreads - 1) / kThreads, c);
        if constexpr (kMode == kFwd) {
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_empty(s1));
        }
        if (++s1 == slots) s1 = 0, ph ^= 1u;
        if ((v += chunk) >= total) break;
        if (!all(wait_phase(bar_full(s1), ph, ctl))) return;
      }
      if (geo.ends) add_one(sum, x, c);
      sum = lanes_join<32>(sum, c);
      if (kMode == kFwd && i >= kListWarps && !wait_sums(i - kListWarps)) return;
      if (lane == 0) {
        s_warp[i % kCopies][warp] = sum;
        mbar_arrive(bar_local(i));
      }
    } else if (kMode == kTrain && lane == 0) {
      mbar_arrive(bar_local(i));
    }
    if (kMode == kTrain && i > 0) {
      const Geo<E>& geo = s_geo[(i - 1) % kCopies];
      if (!all(wait_phase(bar_grad(i - 1), (uint32_t)((i - 1) / kCopies) & 1u, ctl))) return;
      const bool zero = s_grad[(i - 1) % kCopies].zero;
      const Grad q = s_grad[(i - 1) % kCopies].q;
      E* body = geo.body;
      const int total = geo.n;
      const int shift = geo.shift;
      for (int v = 0; v < total || v == 0; v += chunk) {
        const uint4* src = ring + (size_t)s2 * chunk;
        const int n = min(chunk, total - v);
        E* out = body + (int64_t)v * kPer;
        auto put = [&](auto form) {
          constexpr Form kForm = decltype(form)::value;
          if (shift == 0) {
#pragma unroll 4
            for (int at = tid; at < n; at += kThreads)
              put_vector<E, kForm>(out, at, n, src[at], q, 0, lane);
          } else {
            for (int at = tid; at - lane < n; at += kThreads)
              put_vector<E, kForm>(out, at, n, at < n ? src[at] : masked_vector<E>(), q, shift,
                                   lane);
          }
        };
        if (zero)
          put(FormOf<kZero>());
        else if (q.far)
          put(FormOf<kSlow>());
        else
          put(FormOf<kFast>());
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_empty(s2));
        if (++s2 == slots) s2 = 0;
      }
      E* out = body - ((int64_t)geo.v0 * kPer + geo.head);
      if (tid < geo.ends)
        El<E>::put(out + (tid < geo.head ? tid : geo.nvec * kPer + tid), zero ? 0.0f : q(x_last));
    }
  }
  if (kMode == kTrain && lane == 0)
    for (int i = 1; i < kListWarps; ++i) mbar_arrive(bar_local(count + i));
}

// CTAs that run at one time at most, for a grid that leaves no second round to a few.
template <typename K>
cudaError_t resident_ctas(int* out, K kernel, int threads, size_t smem) {
  if (*out) return cudaSuccess;
  int n = 0;
  cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem);
  if (e != cudaSuccess) return e;
  if (n < 1) return cudaErrorInvalidConfiguration;
  *out = n * tc::sm_count();
  return cudaSuccess;
}

struct Launch {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg;
  Launch(unsigned grid, int threads, size_t smem, int cluster, cudaStream_t stream) : cfg{} {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
  }
  Launch(const Launch&) = delete;
};

// Vectors of a row at most (V up to the largest int).
template <typename E>
int64_t vectors_of(int V) {
  return ((int64_t)V + El<E>::kPerVec - 1) / El<E>::kPerVec;
}

template <typename E, int kNV, int kMode>
cudaError_t launch_warps(const DistillArgs& a, cudaStream_t stream) {
  static int most = 0;
  auto kernel = distill_warp_kernel<E, kNV, kMode>;
  cudaError_t e = resident_ctas(&most, kernel, DTHREADS, (size_t)DWARPS * kWarpMaxK * kListBytes);
  if (e != cudaSuccess) return e;
  const int64_t ctas = ((int64_t)a.B + DWARPS - 1) / DWARPS;
  const Launch l((unsigned)(ctas < most ? ctas : most), DTHREADS, (size_t)DWARPS * kListBytes * a.kpad, 1,
                 stream);
  return cudaLaunchKernelEx(&l.cfg, kernel, a);
}

template <typename E>
cudaError_t launch_backward(DistillArgs& a, cudaStream_t stream) {
  const int64_t nvec = vectors_of<E>(a.V);
  while (nvec > (int64_t)kBwdVecs * DTHREADS << a.lsh) ++a.lsh;
  static int most = 0;
  auto kernel = distill_backward_kernel<E>;
  cudaError_t e =
      resident_ctas(&most, kernel, DTHREADS + 32, (size_t)2 * PKM_DISTILL_MAX_K * kGradListBytes);
  if (e != cudaSuccess) return e;
  const int64_t units = (int64_t)a.B << a.lsh;
  kernel<<<(unsigned)(units < most ? units : most), DTHREADS + 32,
           (size_t)2 * kGradListBytes * a.kpad, stream>>>(a);
  return cudaGetLastError();
}

template <typename E, int kMode>
cudaError_t launch_stream(const DistillArgs& a, cudaStream_t stream) {
  auto kernel = distill_stream_kernel<E, kMode>;
  const int slices = 1 << a.lsh;
  const size_t smem = (size_t)a.slots * a.chunk * 16 + (size_t)kCopies * kListBytes * a.kpad;
  Launch l(0, kStreamThreads, smem, slices, stream);
  // clusters that run at one time, by their size and shared memory (in steps of 4 KB)
  constexpr size_t kStep = 4096;
  static int most[kMaxLsh + 1][kDynamic / kStep + 1];
  const size_t step = (smem + kStep - 1) / kStep;
  int& n = most[a.lsh][step];
  if (!n) {
    static bool attr_set = false;
    if (!attr_set) {
      cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           kDynamic);
      if (e != cudaSuccess) return e;
      attr_set = true;
    }
    Launch most_of(slices * tc::sm_count(), kStreamThreads, step * kStep, slices, stream);
    most_of.cfg.numAttrs = 1;
    int got = 0;
    cudaError_t e = cudaOccupancyMaxActiveClusters(&got, kernel, &most_of.cfg);
    if (e != cudaSuccess) return e;
    if (got < 1) return cudaErrorInvalidConfiguration;
    n = got;
  }
  l.cfg.gridDim = dim3((unsigned)(a.B < n ? a.B : n) * slices);
  // Not before the launch before it has ended where larger clusters fill the GPU: placed as SMs
  // become free one after the other, fewer of them run at one time (kTrain, a row of calls: 8 slices,
  // 4096 x 131072 bf16, 381 us against 340; 4 slices, 2000 x 60000, 98 against 95; 2 slices, 4096 x 32000,
  // 98 against 101; kFwd, 4 slices, 2000 x 50257, 40 against 42).
  if (kMode == kTrain && slices > 2) l.cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&l.cfg, kernel, a);
}

template <typename E, int kMode>
cudaError_t dispatch_stream(DistillArgs& a, cudaStream_t stream) {
  const int64_t nvec = vectors_of<E>(a.V);
  // slices of at most 32 KB; more and smaller ones while CTAs are few
  while (a.lsh < kMaxLsh && nvec > (int64_t)kChunkVecs << a.lsh) ++a.lsh;
  while (a.lsh < kMaxLsh && ((int64_t)a.B << a.lsh) * 2 <= tc::sm_count() &&
         nvec > 2 * DTHREADS << a.lsh)
    ++a.lsh;
  const int64_t per = (nvec + (1 << a.lsh) - 1) >> a.lsh;
  // chunks of up to 32 KB in steps of 1 KB, and three slices of them in the ring (kFwd: two
  // chunks)
  a.chunk = per >= kChunkVecs ? kChunkVecs : (int)((per + 63) / 64 * 64);
  if (a.chunk < 64) a.chunk = 64;
  const int64_t chunks = per ? (per + a.chunk - 1) / a.chunk : 1;
  const int64_t room =
      (kDynamic - (size_t)kCopies * kListBytes * a.kpad) / ((size_t)a.chunk * 16);
  a.slots = kMode == kFwd ? 2 : (int)(chunks * 3 < room ? chunks * 3 : room);
  if (a.slots > kMaxSlots) a.slots = kMaxSlots;
  return launch_stream<E, kMode>(a, stream);
}

template <typename E, int kMode>
cudaError_t dispatch(DistillArgs& a, cudaStream_t stream) {
  a.kpad = (a.k + 3) / 4 * 4;
  a.lsh = 0;
  // rows of up to 4 KB, when there are enough of them to fill the GPU: a warp each
  const int64_t nvec = vectors_of<E>(a.V);
  if (nvec <= 32 * 8 && a.k <= kWarpMaxK && a.B >= 4 * tc::sm_count())
    return nvec <= 32 * 2 ? launch_warps<E, 2, kMode>(a, stream)
                          : launch_warps<E, 8, kMode>(a, stream);
  if constexpr (kMode == kBwd)
    return launch_backward<E>(a, stream);
  else
    return dispatch_stream<E, kMode>(a, stream);
}

template <int kMode>
cudaError_t dispatch_type(DistillArgs& a, int dtype, cudaStream_t stream) {
  return dtype == PKM_BF16 ? dispatch<__nv_bfloat16, kMode>(a, stream)
                           : dispatch<float, kMode>(a, stream);
}

DistillArgs args_of(const void* z, int64_t ld, int B, int V, const int64_t* idx,
                    const float* teacher, int k, float T, int* status) {
  DistillArgs a = {};
  a.z = z, a.ld = ld, a.B = B, a.V = V, a.idx = idx, a.teacher = teacher, a.k = k, a.T = T;
  a.inv_t = 1.0 / (double)T, a.t2 = (double)T * T;
  a.status = status;
  return a;
}

}  // namespace

cudaError_t launch_distill(const void* z, int dtype, int64_t ld, int B, int V, const int64_t* idx,
                           const float* teacher, int k, float T, float* loss, float* lse,
                           int* status, cudaStream_t stream) {
  DistillArgs a = args_of(z, ld, B, V, idx, teacher, k, T, status);
  a.loss = loss, a.lse = lse;
  return dispatch_type<kFwd>(a, dtype, stream);
}

cudaError_t launch_distill_backward(const void* z, int dtype, int64_t ld, int B, int V,
                                    const int64_t* idx, const float* teacher, int k, float T,
                                    const float* lse, const float* dloss, void* dz, int64_t ld_d,
                                    int* status, cudaStream_t stream) {
  DistillArgs a = args_of(z, ld, B, V, idx, teacher, k, T, status);
  a.lse = const_cast<float*>(lse), a.dloss = dloss, a.dz = dz, a.ld_d = ld_d;
  return dispatch_type<kBwd>(a, dtype, stream);
}

cudaError_t launch_distill_train(const void* z, int dtype, int64_t ld, int B, int V,
                                 const int64_t* idx, const float* teacher, int k, float T,
                                 const float* dloss, float* loss, float* lse, void* dz,
                                 int64_t ld_d, int* status, cudaStream_t stream) {
  // a row that a cluster's rings hold; longer ones are read twice
  const int64_t most = (int64_t)kMaxSlices * kTrainChunks * kChunkVecs * (dtype == PKM_BF16 ? 8 : 4);
  if (V > most) {
    cudaError_t e =
        launch_distill(z, dtype, ld, B, V, idx, teacher, k, T, loss, lse, status, stream);
    return e != cudaSuccess ? e
                            : launch_distill_backward(z, dtype, ld, B, V, idx, teacher, k, T, lse,
                                                      dloss, dz, ld_d, status, stream);
  }
  DistillArgs a = args_of(z, ld, B, V, idx, teacher, k, T, status);
  a.loss = loss, a.lse = lse, a.dloss = dloss, a.dz = dz, a.ld_d = ld_d;
  return dispatch_type<kTrain>(a, dtype, stream);
}

}  // namespace pkm

namespace {

int distill_check(int dtype, int64_t ld, int B, int V, int k, float T) {
  if (B < 0 || V < 1 || k < 1 || !(T >= 1e-30f) || isinf(T)) return PKM_ERR_INVALID;
  if (dtype != PKM_F32 && dtype != PKM_BF16) return PKM_ERR_UNSUPPORTED;
  if (k > PKM_DISTILL_MAX_K) return PKM_ERR_UNSUPPORTED;
  if (ld < V) return PKM_ERR_RANGE;
  return PKM_OK;
}

// Pointers to whole elements: what CUDA's own types ask for.
bool whole(const void* p, uintptr_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}
// (those that a call has none of are NULL)
bool distill_aligned(int dtype, const void* logits, const void* dlogits, const int64_t* idx,
                     const float* teacher, const float* loss, const float* lse,
                     const float* dloss, const int* status) {
  const uintptr_t e = dtype == PKM_BF16 ? 2 : 4;
  return whole(logits, e) && whole(dlogits, e) && whole(idx, 8) && whole(teacher, 4) &&
         whole(loss, 4) && whole(lse, 4) && whole(dloss, 4) && whole(status, 4);
}

}  // namespace

extern "C" int pkm_distill(const void* logits, int logit_dtype, int64_t ld, int B, int V,
                           const int64_t* idx, const float* teacher, int k, float temperature,
                           float* loss, float* lse, int* status, void* stream) {
  int rc = distill_check(logit_dtype, ld, B, V, k, temperature);
  if (rc || B == 0) return rc;
  if (!logits || !idx || !teacher || !loss) return PKM_ERR_INVALID;
  if (!distill_aligned(logit_dtype, logits, nullptr, idx, teacher, loss, lse, nullptr, status))
    return PKM_ERR_ALIGN;
  return pkm::launch_distill(logits, logit_dtype, ld, B, V, idx, teacher, k, temperature, loss,
                             lse, status, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? PKM_OK
             : PKM_ERR_CUDA;
}

extern "C" int pkm_distill_backward(const void* logits, int logit_dtype, int64_t ld, int B, int V,
                                    const int64_t* idx, const float* teacher, int k,
                                    float temperature, const float* lse, const float* dloss,
                                    void* dlogits, int64_t ld_d, int* status, void* stream) {
  int rc = distill_check(logit_dtype, ld, B, V, k, temperature);
  if (rc) return rc;
  if (ld_d < V || (logits == dlogits && ld != ld_d)) return PKM_ERR_RANGE;
  if (B == 0) return PKM_OK;
  if (!logits || !idx || !teacher || !lse || !dloss || !dlogits) return PKM_ERR_INVALID;
  if (!distill_aligned(logit_dtype, logits, dlogits, idx, teacher, nullptr, lse, dloss, status))
    return PKM_ERR_ALIGN;
  return pkm::launch_distill_backward(logits, logit_dtype, ld, B, V, idx, teacher, k, temperature,
                                      lse, dloss, dlogits, ld_d, status,
                                      static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? PKM_OK
             : PKM_ERR_CUDA;
}

extern "C" int pkm_distill_train(const void* logits, int logit_dtype, int64_t ld, int B, int V,
                                 const int64_t* idx, const float* teacher, int k,
                                 float temperature, const float* dloss, float* loss, float* lse,
                                 void* dlogits, int64_t ld_d, int* status, void* stream) {
  int rc = distill_check(logit_dtype, ld, B, V, k, temperature);
  if (rc) return rc;
  if (ld_d < V || (logits == dlogits && ld != ld_d)) return PKM_ERR_RANGE;
  if (B == 0) return PKM_OK;
  if (!logits || !idx || !teacher || !dloss || !loss || !lse || !dlogits) return PKM_ERR_INVALID;
  if (!distill_aligned(logit_dtype, logits, dlogits, idx, teacher, loss, lse, dloss, status))
    return PKM_ERR_ALIGN;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return pkm::launch_distill_train(logits, logit_dtype, ld, B, V, idx, teacher, k, temperature,
                                   dloss, loss, lse, dlogits, ld_d, status, s) == cudaSuccess
             ? PKM_OK
             : PKM_ERR_CUDA;
}
