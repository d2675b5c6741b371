// A whole mixture-of-experts layer for a few tokens (1..16) in one kernel.
//
//   l = x Wr^T + b;  ids = top-k;  w = softmax;  h_e = silu(Wg_e x) * (Wu_e x);
//   out[t] = bf16( sum_j w_j Wd_{ids_j} h_{ids_j} + Wd_s h_s )
//
// For a few tokens the layer is one read of the selected experts' weights: every weight
// meets at most 16 rows, so HBM bounds it, and what a chain of kernels adds to that read
// (launches, ramps and tails of each, the permutation) is what this kernel takes out.
// One cooperative launch, one CTA per SM, in three phases separated by two grid barriers:
//
//   1. router: eight experts and a split of K a CTA, on warp-wide MMAs with the fp32 weights
//      in three bf16 parts (7 MB of weights at most).  FP8: x is quantised per 1x128 group
//      here.
//   2. every CTA selects the experts of all tokens itself (a warp a token; reading T * E
//      logits from L2 is cheaper than another barrier), then gate/up over the distinct
//      experts that some token selected: a tile is 128 features, their 128 gate rows and 128
//      up rows of one expert, and multiplies all tokens at once, since a product's rows are
//      there whether used or not; only the routed ones are kept, so no permutation.
//   3. down: a tile is 256 output columns, its K axis the concatenated h of every selected
//      expert, accumulated with the routing weights; so the combine is the K loop itself,
//      and nothing is left to add up after it.
//
// Weights arrive through the ring of weight_stream.cuh, whose producer runs ahead through
// the barriers: the shared expert's gate/up rows load during the router phase, and the
// first down rows while the CTAs meet after gate/up, though not before the CTA's own part
// of h is made.  h lies in rows [expert slot][token], so that the tokens of an expert are
// one TMA box.  With bf16 weights it keeps 16 bits of fraction as two bf16 parts, rows of
// the same product, which costs nothing (a third part would be rows that the promoters' lanes
// do not reach; the outputs' bf16 has 8 bits, and their distance to 64-bit results is that of
// an fp32 h to five digits); with FP8 it is quantised per 1x128 group, a tile's features.  Every sum is fp32 and in an order fixed
// by the shapes and the routing.
//
// Measured: one token through 3 of 48 experts and the shared one (882 MB of bf16 weights) in
// 144 us, 6100 GB/s; through 8 of 256 and the shared one (404 MB of e4m3) in 78 us, 5200 GB/s;
// 16 rows of a padded batch through 46 experts and the shared one (4.1 GB of bf16) in 640 us,
// 6500 GB/s.  These are after a rest, called or replayed alike; under lasting load the card's
// power limit takes clocks from 1965 to 1170-1580 MHz, and they take 160, 86 and 740 us.
// 13 rows, 11 of them tokens, through 15 of 40 small experts and the shared one (61 MB of
// e4m3, 9.3 us at HBM's rate) in 37 us: 8 are the router and selection, 6 the second meeting
// and the first h after it, 4 the last tiles; both phases stream in the other 19, of which bytes
// account for 9.  Nothing but latencies: 16 tokens through 8 experts of 200 KB take 25 us.
#include <cudaTypedefs.h>

#include "weight_stream.cuh"

namespace moe {
namespace {

constexpr int kShared = kFewSlots;                    // slot of the shared expert

constexpr int kTokens = MOE_FEW_TOKENS_MAX;           // rows of every product
constexpr int kSelected = 4;                          // named barrier: workers arrive, promoters wait

template <bool FP8>
struct FewSmem {
  static constexpr int kParts = FP8 ? 1 : 2;          // of h
  WsSmem<FP8, kParts * kTokens, kTokens, FP8 ? 6 : 5> ws;
  float w[kTokens][kMaxTopK];                         // routing weights
  int ids[kTokens][kMaxTopK];                         // routed experts, -1 in padding rows
  short active[kFewSlots];                            // the distinct experts, ascending
  signed char pick[kFewSlots + 1][kTokens];           // j with ids[t][j] = active[slot], or -1
  unsigned int bitmap[kMaxExperts / 32];
  // router's weights read; x quantised; selection made; this CTA's part of h made; h complete
  uint64_t scored, ready, routed, drained, met;
  int flag;
};

struct FewMaps {
  CUtensorMap gate_up, down, shared_gate_up, shared_down, x, h;
};

__device__ __forceinline__ uint32_t two_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// a and b as two bf16 parts, high + low, each the nearest bf16 of what is left: 16 bits of
// fraction.  An infinite value is its high part alone, and a finite one past bf16's largest has
// that as its high part.
__device__ __forceinline__ void two_parts(float a, float b, uint32_t* high, uint32_t* low) {
  const auto top = [](float v) {
    return fabsf(v) > 0x1.FEp127f && !isinf(v) ? copysignf(0x1.FEp127f, v) : v;
  };
  const uint32_t hi = two_bf16(top(a), top(b));
  *high = hi;
  *low = two_bf16(isinf(a) ? 0.f : a - __uint_as_float(hi << 16),
                  isinf(b) ? 0.f : b - __uint_as_float(hi & 0xffff0000u));
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// logits[t * E + e] = the sum of at most SPLITS splits' values, N of them a thread at a time.
template <int N, int SPLITS>
__device__ __forceinline__ void sum_logits(const FewArgs& p, int tid, float* logits) {
  const int n = p.T * p.E;
#pragma unroll 1
  for (int i = tid; i < n; i += N * kWsThreads) {
    float part[N][SPLITS];
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
      for (int sp = 0; sp < SPLITS; ++sp)
        part[j][sp] = sp < p.router_splits && i + j * kWsThreads < n
                          ? __ldcg(p.logits + (size_t)sp * kTokens * p.E + i + j * kWsThreads)
                          : 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      float l = part[j][0];
#pragma unroll
      for (int sp = 1; sp < SPLITS; ++sp) l += part[j][sp];
      if (i + j * kWsThreads < n) logits[i + j * kWsThreads] = l;
    }
  }
}

// The experts and weights of token t, by a warp; N: experts a lane, E <= 32 N.
template <int N, bool FP8>
__device__ __forceinline__ void select(FewSmem<FP8>& s, const FewArgs& p, const float* logits, int t) {
  const int lane = threadIdx.x & 31, cta = blockIdx.x;
  const bool real = p.valid == nullptr || p.valid[t];
  // Logits as keys of their order (larger float, larger key; -0 as +0; at least 1, and 0 once
  // taken), so that a round is two warp reductions: the largest key, then the lowest expert
  // that has it.  The rounds are a loop, not unrolled: every launch fetches this code anew,
  // and it runs once (unrolled, the selection took 11000 clocks for 8 experts, as a loop
  // 3000).
  float v[N];
  uint32_t key[N];
#pragma unroll
  for (int i = 0; i < N; ++i)
    v[i] = lane + 32 * i < p.E ? logits[t * p.E + lane + 32 * i] : 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = lane + 32 * i;
    key[i] = 0;
    if (e < p.E) {
      const uint32_t u = __float_as_uint(v[i] + 0.f);
      key[i] = max(u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u), 1u);
      if (cta == 0 && p.logits_out != nullptr)
        p.logits_out[(size_t)t * p.E + e] = real ? v[i] : 0.f;
    }
  }
  int mine_e = -1;                                  // lane j: the j-th expert and its logit
  float mine_v = 0.f;
  if (real) {
#pragma unroll 1
    for (int j = 0; j < p.k; ++j) {
      uint32_t best = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) best = max(best, key[i]);
      best = __reduce_max_sync(0xffffffffu, best);
      int e = kMaxExperts;
#pragma unroll
      for (int i = N - 1; i >= 0; --i)
        if (key[i] == best) e = lane + 32 * i;
      e = __reduce_min_sync(0xffffffffu, e);
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (e == lane + 32 * i) key[i] = 0;
      if (lane == j) {
        mine_e = e;
        mine_v = __uint_as_float(best ^ ((best >> 31) ? 0x80000000u : 0xffffffffu));
      }
    }
  }
  const float top = __shfl_sync(0xffffffffu, mine_v, 0);
  const float ex = real && lane < p.k ? expf(mine_v - top) : 0.f;
  float z = ex;
  if (!p.renorm) {
    z = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (lane + 32 * i < p.E) z += expf(v[i] - top);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) z += __shfl_xor_sync(0xffffffffu, z, off);
  if (lane < p.k) {
    const float w = real ? ex / z : 0.f;
    s.ids[t][lane] = mine_e;
    s.w[t][lane] = w;
    if (real) atomicOr(&s.bitmap[mine_e >> 5], 1u << (mine_e & 31));
    if (cta == 0 && p.ids_out != nullptr) p.ids_out[t * p.k + lane] = mine_e;
    if (cta == 0 && p.w_out != nullptr) p.w_out[t * p.k + lane] = w;
  }
}

// A token's place in the tiles of a slot (an expert's, or the shared one's).
template <bool FP8>
__device__ __forceinline__ bool few_on(const FewSmem<FP8>& s, const FewArgs& p, int slot, int t) {
  return t < p.T && s.pick[slot][t] >= 0;
}
template <bool FP8>
__device__ __forceinline__ int few_active(const FewSmem<FP8>& s) {   // distinct experts
  int n = 0;
#pragma unroll
  for (int i = 0; i < kMaxExperts / 32; ++i) n += __popc(s.bitmap[i]);
  return n;
}

// The promoters' part.
template <bool FP8>
__device__ __forceinline__ void few_promote(FewSmem<FP8>& s, const FewArgs& p, int ch_h, int ch_i,
                                            int ch_s) {
  using S = decltype(s.ws);
  const int lane = threadIdx.x & 31, t_lane = lane & (kTokens - 1);
  WsPromoter<S> sum(s.ws, WsRole{p.wait_limit_ns, p.status, p.timeout_bit});
  auto done = [&]() {
    ws_tile_free();
    sum.park(kTokens);
    ws_tile_ready();
  };
  // at the shared expert while the workers still select the routed ones
  int A = 0;
#pragma unroll 1                                      // one copy of the code
  for (int routed = 0; routed < 2; ++routed) {
    if (routed) {
      named_bar_sync(kSelected, kWsThreads + 128);
      A = few_active(s);
    }
    const int tiles = routed ? A * (p.I / 128) : p.S * (p.Is / 128);
    ws_each_run(WsSplit(tiles, ch_h, gridDim.x), ch_h, [&](int, int c0, int c1, int) {
      sum.clear();
      // bf16: one buffer takes the whole run
      for (int c = FP8 ? c0 : c1 - 1; c < c1; ++c) sum.add(1.f, lane < p.T);
      done();
    });
  }
  if (A == 0) return;
  const int per = ch_s + A * ch_i;
  ws_each_run(WsSplit((p.H + kWsRows - 1) / kWsRows, per, gridDim.x), per,
              [&](int, int c0, int c1, int) {
    sum.clear();
    for (int c = c0; c < c1;) {
      // the run of stages of one slot
      const int slot = c < ch_s ? kShared : (c - ch_s) / ch_i;
      const int first = slot == kShared ? 0 : ch_s + slot * ch_i;
      const int end = min(c1, first + (slot == kShared ? ch_s : ch_i));
      // a token that did not select this expert takes nothing from it, not even 0 * inf
      const bool take = (!FP8 || lane < kTokens) && few_on(s, p, slot, t_lane);
      const float f = take && slot != kShared ? s.w[t_lane][(int)s.pick[slot][t_lane]] : 1.f;
      if (FP8) {
        for (; c < end; ++c) sum.add(f, take);
      } else {
        sum.add(f, take);
        c = end;
      }
    }
    if (!FP8) {                                       // high and low part of h
#pragma unroll
      for (int i = 0; i < kWsCols; ++i)
        sum.acc[i] += __shfl_down_sync(0xffffffffu, sum.acc[i], kTokens);
    }
    done();
  });
}

// The workers' part.
template <bool FP8>
__device__ __forceinline__ void few_work(FewSmem<FP8>& s, const FewArgs& p, int ch_h, int ch_i,
                                         int ch_s) {
  constexpr int EB = FP8 ? 1 : 2;
  constexpr int kParts = FewSmem<FP8>::kParts;
  const int tid = ws_worker_thread(), warp = tid >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x, ctas = gridDim.x;
  const int kb_h = p.H / 128, kb_i = p.imax / 128;
  WsRole role{p.wait_limit_ns, p.status, p.timeout_bit};
  float* const down_parts = p.part + (size_t)2 * kWsCtas * p.T * kWsRows;

  // All CTAs meet: `arrive`, then `meet`, after which what they stored before is visible.
  bool met = false;                                   // thread 0's
  auto arrive = [&](unsigned int* counter) {
    ws_workers_sync();
    if (tid == 0) met = atomic_add_acq_rel(counter) + 1 >= (unsigned int)ctas;
  };
  auto meet = [&](unsigned int* counter) {
    if (tid == 0) {
      const uint64_t t0 = global_timer_ns();
      while (!met) {
        met = ld_acquire_gpu(counter) >= (unsigned int)ctas;
        if (!met && global_timer_ns() - t0 >= p.wait_limit_ns) {
          atomicOr(p.status, p.timeout_bit);
          break;
        }
      }
      s.flag = met;
    }
    ws_workers_sync();
    if (!s.flag) role.ok = false;
  };

  {
    // ---- 1. router logits: eight experts and a part of K a CTA, on m16n8k16 products with the
    // fp32 weights split exactly into three bf16 parts (each the nearest bf16 of what is
    // left), so the sums are the fp32 sums with the full weights.  Few instructions, as for
    // the selection below: every launch fetches this code anew.  (As an unrolled loop of
    // fp32 FMAs, sixteen tokens took 32000 clocks.)
    const int groups = (p.E + 7) / 8, chunks = p.H / 32;
    // FP8: x per 1x128 group, a warp a group, codes of x / s, s = amax / 448; loaded before the
    // router's products, which take the first CTAs, and stored after them
    const auto x_group = [&](int i) {
      const int t = i / kb_h, kb = i - t * kb_h;
      return t < p.T ? *reinterpret_cast<const uint2*>(p.x + (size_t)t * p.H + kb * 128 + lane * 4)
                     : make_uint2(0, 0);
    };
    int xi = (ctas - 1 - cta) * kWsWorkers + warp;
    uint2 xv = make_uint2(0, 0);
    if (FP8) xv = x_group(xi);
    if (cta < groups * p.router_splits) {
      const int split = cta / groups, e0 = (cta - split * groups) * 8;
      const int g = lane >> 2, q = lane & 3;
      const int end = chunks * (split + 1) / p.router_splits;
      const float* wr = p.router_w + (size_t)min(e0 + g, p.E - 1) * p.H + 8 * q;
      const __nv_bfloat16* x0 = p.x + (size_t)g * p.H + 8 * q;
      const __nv_bfloat16* x1 = x0 + (size_t)8 * p.H;
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
      for (int c = chunks * split / p.router_splits + warp; c < end; c += 4 * kWsWorkers) {
        float4 w[4][2];                               // the loads of four chunks go out together
        uint4 a[4][2];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int cj = c + j * kWsWorkers;
          w[j][0] = w[j][1] = make_float4(0.f, 0.f, 0.f, 0.f);
          a[j][0] = a[j][1] = make_uint4(0, 0, 0, 0);
          if (cj < end) {
            w[j][0] = __ldg(reinterpret_cast<const float4*>(wr + cj * 32));
            w[j][1] = __ldg(reinterpret_cast<const float4*>(wr + cj * 32) + 1);
            if (g < p.T) a[j][0] = __ldg(reinterpret_cast<const uint4*>(x0 + cj * 32));
            if (g + 8 < p.T) a[j][1] = __ldg(reinterpret_cast<const uint4*>(x1 + cj * 32));
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float f[8] = {w[j][0].x, w[j][0].y, w[j][0].z, w[j][0].w,
                        w[j][1].x, w[j][1].y, w[j][1].z, w[j][1].w};
#pragma unroll
          for (int part = 0; part < 3; ++part) {
            uint32_t b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              b[i] = two_bf16(f[2 * i], f[2 * i + 1]);
              f[2 * i] -= __uint_as_float(b[i] << 16);
              f[2 * i + 1] -= __uint_as_float(b[i] & 0xffff0000u);
            }
            mma_bf16(acc, a[j][0].x, a[j][1].x, a[j][0].y, a[j][1].y, b[0], b[1]);
            mma_bf16(acc, a[j][0].z, a[j][1].z, a[j][0].w, a[j][1].w, b[2], b[3]);
          }
        }
      }
      if (lane == 0) mbar_arrive(smem_u32(&s.scored));
      // the warps' sums meet where tiles will lie later
      auto* sums = reinterpret_cast<float(*)[kTokens][8]>(&s.ws.tile[0][0]);
#pragma unroll
      for (int i = 0; i < 4; ++i) sums[warp][g + 8 * (i >> 1)][2 * q + (i & 1)] = acc[i];
      ws_workers_sync();
      const int t = tid >> 3, e = e0 + (tid & 7);
      if (t < p.T && e < p.E) {
        float l = split == 0 && p.router_b != nullptr ? p.router_b[e] : 0.f;
#pragma unroll
        for (int w = 0; w < kWsWorkers; ++w) l += sums[w][t][tid & 7];
        p.logits[((size_t)split * kTokens + t) * p.E + e] = l;
      }
    } else if (lane == 0) {
      mbar_arrive(smem_u32(&s.scored));
    }
    // partial tiles of gate/up: of the shared expert, of the routed ones
    if (p.S) ws_clear_partial(ws_partial(p.part, p.T, cta, false), p.T);
    ws_clear_partial(ws_partial(p.part, p.T, cta, true), p.T);
    if (FP8) {
      for (; xi < p.T * kb_h; xi += ctas * kWsWorkers) {
        const int t = xi / kb_h, kb = xi - t * kb_h;
        const uint2 v = xv;
        xv = x_group(xi + ctas * kWsWorkers);
        if (p.valid != nullptr && !p.valid[t]) continue;
        const float f[4] = {__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u),
                            __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u)};
        float sc;
        const uint32_t codes = quantize_group_lane(f, &sc);
        *reinterpret_cast<uint32_t*>(p.xq + (size_t)t * p.H + kb * 128 + lane * 4) = codes;
        if (lane == 0) p.sx[(size_t)t * kb_h + kb] = sc;
      }
    }
    if (FP8) fence_proxy_async();                       // the codes are read by TMA
    arrive(p.bar);

    meet(p.bar);
    if (FP8 && tid == 0) mbar_arrive(smem_u32(&s.ready));

    // ---- 2a. the experts of every token, by every CTA for itself; first the logits of all
    // splits, with as many loads on their way as there are (behind the ring's loads each
    // round trip takes up to 4 us)
    float* const logits = &s.ws.tile[0][0];
    if (p.router_splits <= 4)
      sum_logits<8, 4>(p, tid, logits);
    else
      sum_logits<2, kFewRouterSplits>(p, tid, logits);
    ws_workers_sync();
    for (int t = warp; t < p.T; t += kWsWorkers) {
      if (p.E <= 32)
        select<1>(s, p, logits, t);
      else if (p.E <= 64)
        select<2>(s, p, logits, t);
      else
        select<8>(s, p, logits, t);
    }
    ws_workers_sync();
    auto rank_of = [&](int e) {
      int r = __popc(s.bitmap[e >> 5] & ((1u << (e & 31)) - 1u));
#pragma unroll
      for (int i = 0; i < kMaxExperts / 32 - 1; ++i)
        if (i < (e >> 5)) r += __popc(s.bitmap[i]);
      return r;
    };
    if (tid < p.E && ((s.bitmap[tid >> 5] >> (tid & 31)) & 1u)) s.active[rank_of(tid)] = (short)tid;
    if (tid < p.T * p.k) {
      const int t = tid / p.k, j = tid - t * p.k, e = s.ids[t][j];
      if (e >= 0) s.pick[rank_of(e)][t] = (signed char)j;
    }
    if (tid < p.T && s.ids[tid][0] >= 0) s.pick[kShared][tid] = 0;
    ws_workers_sync();
    if (tid == 0) mbar_arrive(smem_u32(&s.routed));
    // the promoters learn of it without waiting for what the workers do next (a tile of the shared
    // expert that other CTAs share takes them up to 6 us beside full rings)
    asm volatile("bar.arrive %0, %1;" ::"n"(kSelected), "n"(kWsThreads + 128) : "memory");
    ws_clear_partial(ws_partial(down_parts, p.T, cta, false), p.T);
    ws_clear_partial(ws_partial(down_parts, p.T, cta, true), p.T);
  }

  auto h_row = [&](int slot, int t) {                 // its high part; the low one kTokens below
    return (size_t)((slot == kShared ? 0 : slot + p.S) * kParts * kTokens + t);
  };

  // Finished tiles: gate/up of the shared expert, of the routed ones, down.
  int A = 0;
#pragma unroll 1                                      // one copy of the code
  for (int step = 0; step < 3; ++step) {
    const bool routed = step == 1, down = step == 2;
    if (routed) A = few_active(s);
    if (down) {
      fence_proxy_async();                            // h is read by TMA
      if (tid == 0) mbar_arrive(smem_u32(&s.drained));
      arrive(p.bar + 1);
      meet(p.bar + 1);
      if (tid == 0) mbar_arrive(smem_u32(&s.met));
      if (A == 0) {                                   // every row is padding
        const int n = p.T * p.H / 8;
        for (int i = cta * kWsThreads + tid; i < n; i += ctas * kWsThreads)
          reinterpret_cast<uint4*>(p.out)[i] = make_uint4(0, 0, 0, 0);
        return;
      }
    }
    const int I = routed ? p.I : p.Is, ft = I / 128;
    const int per = down ? ch_s + A * ch_i : ch_h;
    const int tiles = down ? (p.H + kWsRows - 1) / kWsRows : routed ? A * ft : p.S * ft;
    float* const parts = down ? down_parts : ws_partial(p.part, p.T, 0, routed);
    const WsSplit split(tiles, per, ctas);
    ws_each_run(split, per, [&](int tile, int, int, int t0) {
      ws_tile_free();
      ws_tile_ready();
      const WsShare share(split, t0, per);
      // ---- 3. down and combine
      if (down) {
        const int n = share.finishers();
        if (share.b0 != share.b1 && (cta == share.b1 || n > 1))
          ws_store_partial(s.ws.tile, ws_partial(parts, p.T, cta, cta == share.b0), p.T);
        if (share.b0 != share.b1 && cta == share.b1) return;
        // an n-th of the columns, four a thread
        const int q0 = (kWsRows / 4) * (cta - share.b0) / n, q1 = (kWsRows / 4) * (cta - share.b0 + 1) / n;
#pragma unroll 1
        for (int i = tid; i < p.T * (q1 - q0); i += kWsThreads) {
          const int t = i / (q1 - q0), col = 4 * (q0 + i - t * (q1 - q0));
          if (tile * kWsRows + col >= p.H) continue;
          float v[4];
          ws_tile_values(s.ws.tile[t], parts, p.T, share, t, col, role, v);
          const bool real = s.ids[t][0] >= 0;
          *reinterpret_cast<uint2*>(p.out + (size_t)t * p.H + tile * kWsRows + col) =
              make_uint2(real ? two_bf16(v[0], v[1]) : 0u, real ? two_bf16(v[2], v[3]) : 0u);
        }
        return;
      }
      // ---- 2b. gate/up: columns 0 .. 127 of a tile are gate values, 128 .. 255 up values; the
      // first of its CTAs finishes a shared tile
      const int slot = routed ? tile / ft : kShared, f = (routed ? tile - slot * ft : tile) * 128;
      if (cta != share.b0) {
        ws_store_partial(s.ws.tile, ws_partial(parts, p.T, cta, false), p.T);
        return;
      }
      // a warp a token, four features a lane
#pragma unroll 1
      for (int t = warp; t < p.T; t += kWsWorkers) {
        if (!few_on(s, p, slot, t)) continue;
        float v[8], h[4];
        ws_tile_values<8, 4, 128>(s.ws.tile[t], parts, p.T, share, t, 4 * lane, role, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = v[i] / (1.0f + expf(-v[i])) * v[4 + i];
        const size_t row = h_row(slot, t), at = row * p.imax + f + 4 * lane;
        if (FP8) {                                    // the tile's 128 features are a group
          float sc;
          *reinterpret_cast<uint32_t*>(p.h + at) = quantize_group_lane(h, &sc);
          if (lane == 0) p.sh[row * kb_i + f / 128] = sc;
        } else {
          uint32_t hi0, hi1, lo0, lo1;
          two_parts(h[0], h[1], &hi0, &lo0);
          two_parts(h[2], h[3], &hi1, &lo1);
          uint8_t* o = p.h + at * EB;
          *reinterpret_cast<uint2*>(o) = make_uint2(hi0, hi1);
          *reinterpret_cast<uint2*>(o + (size_t)kTokens * p.imax * EB) = make_uint2(lo0, lo1);
        }
      }
    });
  }
}

template <bool FP8>
__global__ void __launch_bounds__(kWsBlock, 1) few_kernel(const __grid_constant__ FewMaps maps,
                                                          const FewArgs p) {
  extern __shared__ uint8_t smem_raw[];
  FewSmem<FP8>& s = *reinterpret_cast<FewSmem<FP8>*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  using S = decltype(s.ws);
  constexpr int EB = FP8 ? 1 : 2;                     // bytes of a weight
  const int warp = warp_index();
  const int ch_h = p.H * EB / kWsBytes;               // stages of a gate/up tile
  const int ch_i = p.I * EB / kWsBytes;               // stages of a slot of a down tile
  const int ch_s = p.S ? p.Is * EB / kWsBytes : 0;
  const int tiles_s = p.S * (p.Is / 128);
  const int down_tiles = (p.H + kWsRows - 1) / kWsRows;

  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&s.scored), kWsWorkers);
    mbar_init(smem_u32(&s.ready), 1);
    mbar_init(smem_u32(&s.routed), 1);
    mbar_init(smem_u32(&s.drained), 1);
    mbar_init(smem_u32(&s.met), 1);
  }
  if (threadIdx.x < kMaxExperts / 32) s.bitmap[threadIdx.x] = 0;
  for (int i = threadIdx.x; i < (kFewSlots + 1) * kTokens; i += kWsBlock) (&s.pick[0][0])[i] = -1;
  ws_setup(s.ws);

  const WsRole role{p.wait_limit_ns, p.status, p.timeout_bit};
  // stage c of a down tile: the slot it reads, and the stage within the slot
  auto down_slot = [&](int c, int* ci) {
    if (c < ch_s) {
      *ci = c;
      return kShared;
    }
    const int slot = (c - ch_s) / ch_i;
    *ci = c - ch_s - slot * ch_i;
    return slot;
  };

  if (warp == 1) {
    // ------------------------------------------------------------- weight producer
    WsWeights<S> out(s.ws, role);
    auto gate_up = [&](const CUtensorMap* m, int I, int tiles, bool routed) {
      const int ft = I / 128;
      ws_each_unit(tiles, ch_h, [&](int tile, int c, bool, bool) {
        const int slot = routed ? tile / ft : 0, f = (routed ? tile - slot * ft : tile) * 128;
        const int row = (routed ? s.active[slot] * 2 * I : 0) + f;
        out.load(m, row, row + I, c * kWsBytes);
      });
    };
    // the router's few loads first: behind a ring's worth of weights they would wait 4 us
    out.role.wait(&s.scored, 0);
    gate_up(&maps.shared_gate_up, p.Is, tiles_s, false);
    if (out.role.wait(&s.routed, 0)) {
      const int A = few_active(s);
      gate_up(&maps.gate_up, p.I, A * (p.I / 128), true);
      // what the last tiles still need from other CTAs would wait behind a ring's worth of
      // weights
      if (A > 0 && out.role.wait(&s.drained, 0)) {
        const int per = ch_s + A * ch_i;
        ws_each_unit(down_tiles, per, [&](int tile, int c, bool, bool) {
          int ci;
          const int slot = down_slot(c, &ci), r = tile * kWsRows;
          const int row = (slot == kShared ? 0 : s.active[slot] * p.H) + r;
          out.load(slot == kShared ? &maps.shared_down : &maps.down, row,
                   r + kWsBoxRows < p.H ? row + kWsBoxRows : -1, ci * kWsBytes);
        });
      }
    }
    out.drain();
  } else if (warp == 2) {
    // ------------------------------------------------------------------ MMA issuer
    WsMma<S> mma(s.ws, role);
    auto gate_up = [&](int tiles) {
      ws_each_unit(tiles, ch_h, [&](int, int, bool first, bool last) {
        mma.stage(FP8 || first, FP8 || last);
      });
    };
    gate_up(tiles_s);
    if (mma.role.wait(&s.routed, 0)) {
      const int A = few_active(s);
      gate_up(A * (p.I / 128));
      if (A > 0) {
        const int per = ch_s + A * ch_i;
        ws_each_unit(down_tiles, per, [&](int, int c, bool first, bool last) {
          int ci;
          const bool shared = down_slot(c, &ci) == kShared;
          mma.stage(FP8 || first || ci == 0, FP8 || last || ci + 1 == (shared ? ch_s : ch_i));
        });
      }
    }
    mma.drain();
  } else if (warp == 3) {
    // --------------------------------------------------------- activation producer
    WsActivations<S> out(s.ws, role);
    const int lane = threadIdx.x & 31, kb_h = p.H / 128;
    auto gate_up = [&](int I, int experts, bool routed) {
      const int ft = I / 128;
      ws_each_unit(experts * ft, ch_h, [&](int tile, int c, bool, bool) {
        const float *sx = nullptr, *sw = nullptr;
        if (FP8) {
          const int slot = routed ? tile / ft : 0, f = routed ? tile - slot * ft : tile;
          if (lane < p.T) sx = p.sx + (size_t)lane * kb_h + c;
          if (lane < 2)
            sw = (routed ? p.s_gate_up + (size_t)s.active[slot] * 2 * ft * kb_h : p.ss_gate_up) +
                 (size_t)(f + lane * ft) * kb_h + c;
        }
        out.load(&maps.x, 0, c * kWsBytes, kTokens, sx, sw);
      });
    };
    if (FP8 && out.role.wait(&s.ready, 0)) fence_proxy_async();
    gate_up(p.Is, p.S, false);
    if (out.role.wait(&s.routed, 0)) {
      const int A = few_active(s);
      gate_up(p.I, A, true);
      if (A > 0 && out.role.wait(&s.met, 0)) {
        fence_proxy_async();
        const int per = ch_s + A * ch_i, kb_i = p.imax / 128;
        ws_each_unit(down_tiles, per, [&](int tile, int c, bool, bool) {
          int ci;
          const int slot = down_slot(c, &ci), place = slot == kShared ? 0 : slot + p.S;
          const float *sx = nullptr, *sw = nullptr;
          if (FP8) {
            const int kbs = (slot == kShared ? p.Is : p.I) / 128;
            if (lane < p.T) sx = p.sh + (size_t)(place * kTokens + lane) * kb_i + ci;
            // past the end of H the last block, whose sums are not used
            if (lane < 2)
              sw = (slot == kShared ? p.ss_down : p.s_down + (size_t)s.active[slot] * kb_h * kbs) +
                   (size_t)min(2 * tile + lane, kb_h - 1) * kbs + ci;
          }
          out.load(&maps.h, place * S::ROWS, ci * kWsBytes, S::ROWS, sx, sw);
        });
      }
    }
    out.drain();
  } else {
    if (ws_is_promoter())
      few_promote<FP8>(s, p, ch_h, ch_i, ch_s);
    else
      few_work<FP8>(s, p, ch_h, ch_i, ch_s);
  }
  ws_teardown(s.ws);
}

template <bool FP8>
cudaError_t launch(const FewMaps& m, const FewArgs& a, int ctas, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, 1, 1);
  cfg.blockDim = dim3(kWsBlock, 1, 1);
  cfg.dynamicSmemBytes = sizeof(FewSmem<FP8>) + 1024;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];                        // the CTAs wait for one another
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, few_kernel<FP8>, m, a);
}

template <bool FP8>
cudaError_t prepare() {
  static_assert(sizeof(FewSmem<FP8>) + 1024 <= 227 * 1024, "shared memory of one CTA");
  return cudaFuncSetAttribute(few_kernel<FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)sizeof(FewSmem<FP8>) + 1024);
}

}  // namespace

bool ws_map_nd(CUtensorMap* m, const void* w, int rank, const uint64_t* dims,
               const uint64_t* strides, const uint32_t* box) {
  static const auto encode = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }();
  if (encode == nullptr) return false;
  cuuint64_t d[5], st[5];
  cuuint32_t b[5], one[5];
  for (int i = 0; i < rank; ++i) {
    d[i] = dims[i];
    b[i] = box[i];
    one[i] = 1;
    if (i + 1 < rank) st[i] = strides[i];
  }
  return encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, (cuuint32_t)rank, const_cast<void*>(w), d, st, b,
                one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool ws_map(CUtensorMap* m, const void* w, uint64_t row_bytes, uint64_t rows, int box_rows) {
  const uint64_t dims[2] = {row_bytes, rows};
  const uint32_t box[2] = {128, (uint32_t)box_rows};
  return ws_map_nd(m, w, 2, dims, &row_bytes, box);
}

cudaError_t prepare_few_kernels() {
  const cudaError_t e = prepare<false>();
  return e == cudaSuccess ? prepare<true>() : e;
}

cudaError_t launch_few(FewArgs a, bool fp8, int num_sms, cudaStream_t st) {
  const int ctas = num_sms < kWsCtas ? num_sms : kWsCtas;
  // eight experts a CTA; with CTAs left over K is cut too, a chunk of 32 a warp at least
  const int groups = (a.E + 7) / 8;
  const int most = a.H / 32 / kWsWorkers < kFewRouterSplits ? a.H / 32 / kWsWorkers : kFewRouterSplits;
  a.router_splits = ctas / groups < most ? ctas / groups : most;
  if (a.router_splits < 1) a.router_splits = 1;
  const uint64_t eb = fp8 ? 1 : 2, E = a.E, H = a.H, I = a.I, Is = a.Is;
  FewMaps m;
  if (!ws_map(&m.gate_up, a.w_gate_up, H * eb, E * 2 * I, kWsBoxRows) ||
      !ws_map(&m.down, a.w_down, I * eb, E * H, kWsBoxRows) ||
      !ws_map(&m.x, fp8 ? (const void*)a.xq : a.x, H * eb, a.T, kTokens) ||
      !ws_map(&m.h, a.h, (uint64_t)a.imax * eb, (uint64_t)a.h_slots * kTokens * (fp8 ? 1 : 2),
              kTokens * (fp8 ? 1 : 2)))
    return cudaErrorInvalidValue;
  if (a.S == 0) {
    m.shared_gate_up = m.gate_up;      // not used
    m.shared_down = m.down;
  } else if (!ws_map(&m.shared_gate_up, a.ws_gate_up, H * eb, 2 * Is, kWsBoxRows) ||
             !ws_map(&m.shared_down, a.ws_down, Is * eb, H, kWsBoxRows)) {
    return cudaErrorInvalidValue;
  }
  return fp8 ? launch<true>(m, a, ctas, st) : launch<false>(m, a, ctas, st);
}

}  // namespace moe
