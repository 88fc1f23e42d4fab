// experts8.cu -- the routed experts' step over 8-bit weights, from given ids
// and weights.
//
// Few rows (decode, verify): two kernels that stream the union's weights
// once, by bulk copies through a ring of shared-memory stages that a warp of
// its own keeps full, so that HBM is read without a pause between a CTA's
// tiles.  A stage is a few whole weight rows, contiguous in memory.
// Every row is a column of the m16n8 tiles, whether it chose the expert or
// not, so no row lists are built.
//   gate_up  persistent; an item is 8 channels of one expert (its 8 gate and
//            8 up rows are one M = 16 tile); four teams of four warps take
//            the items in turn, a team shares out an item's k blocks, its
//            sums are met by a warp of its own; writes h in fp32
//   down     a CTA per 16 output rows over all experts of the union, the
//            (expert, two k blocks) items shared out over 16 warps; it
//            quantises h while its weights arrive; sums meet in a fixed order
// An item's chain of wait, loads, MMAs and arrival takes a warp some 1000
// cycles, in which HBM brings 23 KB to an SM: so several items are worked on
// at once, and two k blocks' MMAs are interleaved.
// One row, 8 of 128 experts, 2048 x 768, 38 MB: 13.2 us back to back; four
// rows, 39 of 512 experts, 2048 x 512, 123 MB: 30.  By time stamps in the
// latter: union 1.1, gate_up's sums until 17 (13 without MMAs and loads: HBM),
// down's start, union and tables until 20, gate_up's end seen at 21, h ready
// at 24 (80 KB loaded and quantised by every CTA), products and sums until 31.
//
// Many rows: the entries are grouped by expert (count, scan), x is quantised
// once per row and written to its entries' places, mm8_tc computes h8 and
// the outputs y, and a last kernel sums a row's weighted outputs in the
// order of its entries.  4096 rows, 10 of 512 experts by Zipf(1.1), 2048 x
// 512, alone: count 7, scatter 19 (101 MB), gate_up 205 (1.16 GB from HBM, 5.7
// TB/s; L2 15.6), down 154 (559 MB read, 288 of 336 written, 5.5 TB/s), sum 60
// us (336 MB read, 5.8 TB/s); 446 in a graph.
#include <cuda_runtime.h>

#include "fp8.cuh"
#include "tc05.cuh"

namespace moe {
namespace {

constexpr unsigned FULLM = 0xffffffffu;
constexpr int kWarps = 8, kThreads = 32 * kWarps;  // many rows

// One k block of 128: 16 weight rows (eight from lo, eight from hi on, ld
// bytes apart) times eight rows of x or h.  Lane (g, q) = (lane / 4, lane %
// 4) takes the bytes 32q .. 32q + 31 of weight rows g and g + 8 and of row g
// of x (`col`): the k order inside a block is permuted alike on both sides.
// (Rows are a multiple of 128 bytes apart, so two rows of a load meet in a
// bank.  Loads without such conflicts, odd rows exchanging two pieces after
// them, took 35.5 us instead of 33.4 for 4 rows through 39 experts, and rows
// of x and h a piece further apart 33.4: the MMAs take longer than the loads.
// Converting the weights to f16 by hand, by the conversion instruction or by
// integer operations, was 10 to 25% slower than the 8-bit MMA.)
struct Block {
  uint4 a0, a1, a2, a3, b0, b1;
};
__device__ __forceinline__ void load_block(Block &x, const uint8_t *lo, const uint8_t *hi, int ld, int g, int q,
                                           const uint8_t *col, bool have) {
  const uint8_t *r0 = lo + g * ld + 32 * q, *r1 = hi + g * ld + 32 * q;
  x.b0 = x.b1 = make_uint4(0, 0, 0, 0);
  if (have) x.b0 = *reinterpret_cast<const uint4 *>(col), x.b1 = *reinterpret_cast<const uint4 *>(col + 16);
  x.a0 = *reinterpret_cast<const uint4 *>(r0), x.a2 = *reinterpret_cast<const uint4 *>(r0 + 16);
  x.a1 = *reinterpret_cast<const uint4 *>(r1), x.a3 = *reinterpret_cast<const uint4 *>(r1 + 16);
}
// the MMAs of two blocks, in turn
__device__ __forceinline__ void mma_blocks(float (&d)[4], const Block &x, float (&e)[4], const Block &y) {
  mma_e4m3(d, x.a0.x, x.a1.x, x.a0.y, x.a1.y, x.b0.x, x.b0.y);
  mma_e4m3(e, y.a0.x, y.a1.x, y.a0.y, y.a1.y, y.b0.x, y.b0.y);
  mma_e4m3(d, x.a0.z, x.a1.z, x.a0.w, x.a1.w, x.b0.z, x.b0.w);
  mma_e4m3(e, y.a0.z, y.a1.z, y.a0.w, y.a1.w, y.b0.z, y.b0.w);
  mma_e4m3(d, x.a2.x, x.a3.x, x.a2.y, x.a3.y, x.b1.x, x.b1.y);
  mma_e4m3(e, y.a2.x, y.a3.x, y.a2.y, y.a3.y, y.b1.x, y.b1.y);
  mma_e4m3(d, x.a2.z, x.a3.z, x.a2.w, x.a3.w, x.b1.z, x.b1.w);
  mma_e4m3(e, y.a2.z, y.a3.z, y.a2.w, y.a3.w, y.b1.z, y.b1.w);
}

// acc += d scaled: columns 2q (x0) and 2q + 1 (x1), gate rows (fg), up rows (fu)
__device__ __forceinline__ void add_scaled(float4 &acc, const float (&d)[4], float x0, float x1, float fg, float fu) {
  const float p[4] = {x0 * fg, x1 * fg, x0 * fu, x1 * fu};
  if (scales_hold(p)) {
    acc.x += d[0] * p[0], acc.y += d[1] * p[1], acc.z += d[2] * p[2], acc.w += d[3] * p[3];
  } else {
    acc.x += by_scales(d[0], x0, fg), acc.y += by_scales(d[1], x1, fg);
    acc.z += by_scales(d[2], x0, fu), acc.w += by_scales(d[3], x1, fu);
  }
}
// acc += w * (d scaled by a and b), two sums: a weight meets the scaled
// product, as in the definition
__device__ __forceinline__ void add_weighted(float &acc0, float &acc1, float d0, float d1, float a, float b, float w) {
  const float p[1] = {a * b};
  if (scales_hold(p)) acc0 += d0 * p[0] * w, acc1 += d1 * p[0] * w;
  else acc0 += d0 * a * b * w, acc1 += d1 * a * b * w;
}

// bounded wait on an mbarrier phase, of a thread and of a warp; false (and
// the status) once the limit passes
__device__ bool thread_wait(uint64_t *bar, uint32_t par, const Ex8P &P) {
  if (mbar_try_wait(bar, par)) return true;
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait(bar, par))
    if (globaltimer() - t0 > P.timeout_ns) {
      atomicCAS(P.status, 0, kStatusTimeout);
      return false;
    }
  return true;
}
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t par, const Ex8P &P) {
  if (__all_sync(FULLM, mbar_try_wait(bar, par))) return true;
  return __all_sync(FULLM, thread_wait(bar, par, P));
}

// eight consecutive values of x
template <bool BF16>
__device__ __forceinline__ void load_x8(const void *x, int64_t i, float (&v)[8]) {
  if (BF16) {
    const uint4 u = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(x) + i);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; j++) v[2 * j] = bf16lo(w[j]), v[2 * j + 1] = bf16hi(w[j]);
  } else {
    const float4 a = *reinterpret_cast<const float4 *>(static_cast<const float *>(x) + i);
    const float4 b = *reinterpret_cast<const float4 *>(static_cast<const float *>(x) + i + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
}

// Half a warp: the 128 values its lanes hold eight each of -> e4m3, scale byte
__device__ __forceinline__ uint2 quant128(const float (&v)[8], uint32_t &e) {
  uint32_t w[2];
  quant_block<8>(v, w, e);
  return make_uint2(w[0], w[1]);
}

// ------------------------------------------------------------ few rows

constexpr int kMaxEntries = kEx8SmallRows * 32;
constexpr int kMaxStages = 24;  // at most a lane each
constexpr int kDownWarps = 16;
constexpr size_t kSmemCap = 226 * 1024;

// The union of the rows' experts, as each kernel builds it for itself (in
// the order of the id table; ids below E, once each).
struct Union {
  uint32_t *ids, *ex;                // [n entries], the experts
  float *wt;                         // [n entries]
  float (*w)[kEx8SmallRows];         // [experts] sum of a row's weights for the expert
  short (*ent)[kEx8SmallRows];       // a row's first entry with that expert, or -1
  uint8_t *own;                      // [n entries] is a row's first entry with its expert
  uint32_t *seen;                    // a bit an expert
  int *n;
};
__host__ __device__ constexpr size_t union_bytes(int n) { return (size_t)n * (4 + 4 + 4 + 4 * 8 + 2 * 8 + 1) + 16 + 128 + 15; }
__device__ __forceinline__ Union union_at(void *p, int n) {
  Union U;
  U.n = static_cast<int *>(p);
  U.seen = reinterpret_cast<uint32_t *>(U.n + 4), U.ids = U.seen + 32, U.ex = U.ids + n;
  U.wt = reinterpret_cast<float *>(U.ex + n);
  U.w = reinterpret_cast<float(*)[kEx8SmallRows]>(U.wt + n);
  U.ent = reinterpret_cast<short(*)[kEx8SmallRows]>(U.w + n);
  U.own = reinterpret_cast<uint8_t *>(U.ent + n);
  return U;
}

// One warp: ids, ex and n.  32 entries at a time: the first of each id among
// them by a match, those of earlier groups by the experts' bits.
__device__ void union_warp(const Union &U, const Ex8P &P) {
  const int lane = threadIdx.x & 31, n = P.t * P.K;
  uint32_t id[kMaxEntries / 32];
  float wt[kMaxEntries / 32];
#pragma unroll
  for (int i = 0; i < kMaxEntries / 32; i++) {
    id[i] = 32 * i + lane < n ? P.idx[32 * i + lane] : 0xffffffffu;
    wt[i] = 32 * i + lane < n ? P.w[32 * i + lane] : 0.f;
  }
  int cnt = 0;
  U.seen[lane] = 0;  // E <= 1024
  __syncwarp();
#pragma unroll
  for (int i = 0; i < kMaxEntries / 32; i++) {
    if (32 * i >= n) break;
    if (32 * i + lane < n) U.ids[32 * i + lane] = id[i], U.wt[32 * i + lane] = wt[i], U.own[32 * i + lane] = 0;
    bool first = __ffs(__match_any_sync(FULLM, id[i])) - 1 == lane && id[i] < (uint32_t)P.E;
    if (first) first = !(atomicOr(&U.seen[id[i] >> 5], 1u << (id[i] & 31)) >> (id[i] & 31) & 1u);
    const unsigned bal = __ballot_sync(FULLM, first);
    if (first) U.ex[cnt + __popc(bal & ((1u << lane) - 1u))] = id[i];
    cnt += __popc(bal);
    __syncwarp();
  }
  if (lane == 0) *U.n = cnt;
  __syncwarp();
}
// Threads tid of count: ent, w and own, once the union is there.
__device__ void union_rows(const Union &U, const Ex8P &P, int tid, int count) {
  for (int i = tid; i < *U.n * kEx8SmallRows; i += count) {
    const int u = i / kEx8SmallRows, r = i - u * kEx8SmallRows;
    const uint32_t ex = U.ex[u];
    int at = -1;
    float s = 0.f;
    if (r < P.t)
      for (int j = r * P.K; j < (r + 1) * P.K; j++)
        if (U.ids[j] == ex) {
          if (at < 0) at = j;
          s += U.wt[j];
        }
    U.ent[u][r] = (short)at, U.w[u][r] = s;
    if (at >= 0) U.own[at] = 1;
  }
}

// One warp: n copies of `bytes` each, from src(f), into the ring of ns stages.
// A lane looks after a stage, so that the copies of free stages are issued
// together.  For down's many short copies: one thread issuing all of them
// took 0.24 us a copy, 9 us for the 39 of a CTA, more than HBM.  (gate_up's
// long ones come at HBM's rate from one thread, in the order of their use;
// all at once, they arrive together: 33.4 us instead of 32.4 for 4 rows
// through 39 experts.)
template <class Src>
__device__ void produce(uint64_t *full, uint64_t *empty, uint8_t *ring, int ns, int bytes, int n, const Ex8P &P, Src src) {
  const int lane = threadIdx.x & 31;
  int f = lane;
  uint32_t ph = 0;  // of the stage's next copy
  unsigned long long t0 = 0;
  bool on = lane < ns && f < n;
  while (__any_sync(FULLM, on)) {
    if (on) {
      if (mbar_test_wait(&empty[lane], ph ^ 1)) {
        mbar_expect_tx(&full[lane], (uint32_t)bytes);
        bulk_g2s(ring + (size_t)lane * bytes, src(f), (uint32_t)bytes, &full[lane]);
        f += ns, ph ^= 1, t0 = 0;
        on = f < n;
      } else if (t0 == 0) {
        t0 = globaltimer();
      } else if (globaltimer() - t0 > P.timeout_ns) {
        atomicCAS(P.status, 0, kStatusTimeout);
        on = false;
      }
    }
  }
  // the copy still in flight lands before the CTA ends
  if (lane < ns && f >= ns) thread_wait(&full[lane], ph ^ 1, P);
}

// ---- gate_up: dynamic shared memory: ring | x rows | their scales | sums | union
constexpr int kTeams = 4, kTeam = 4, kGuWarps = kTeams * kTeam, kGuThreads = 32 * (kGuWarps + 2);
GuLay gu_layout(int H, int t, int K) {
  GuLay l{};
  l.stage = 8 * H;
  const size_t xs = (size_t)t * H, sx = ((size_t)t * (H / 128) * 4 + 15) / 16 * 16, red = 2 * kGuWarps * 512;  // two of each team
  const size_t rest = xs + sx + red + union_bytes(t * K);
  const size_t room = kSmemCap > rest ? (kSmemCap - rest) / l.stage : 0;
  const int fit = (int)(room < kMaxStages ? room : kMaxStages);
  l.teams = fit >= 2 * kTeams ? kTeams : (fit >= 4 ? 2 : 1);
  l.ns = fit / (2 * l.teams) * (2 * l.teams);
  l.xs = (size_t)l.ns * l.stage, l.sx = l.xs + xs, l.red = l.sx + sx, l.un = l.red + red;
  l.total = (size_t)l.ns * l.stage + rest;
  return l;
}

// The warps' steps over the items are counted, not divided: an item costs a
// warp some 150 instructions, and HBM brings one in 1400 cycles.
template <bool BF16>
__global__ void __launch_bounds__(kGuThreads, 1) ex8_gate_up(const __grid_constant__ Ex8P P) {
  extern __shared__ __align__(128) uint8_t sm[];
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], red_full[kTeams][2], red_empty[kTeams][2];
  const GuLay L = P.gl;
  uint8_t *xs = sm + L.xs;
  float *sx = reinterpret_cast<float *>(sm + L.sx);
  float4 *red = reinterpret_cast<float4 *>(sm + L.red);
  const Union U = union_at(sm + L.un, P.t * P.K);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
  const int H = P.H, I = P.I, nk = H / 128, nct = I / 8;
  // first item of CTA b: a CTA's items follow one another, so that it reads
  // few experts' pages (with every 152nd item each copy was another page, and
  // the misses in the address translation bound the kernel)
  auto share = [&](int items, unsigned b) { return (int)((int64_t)items * b / gridDim.x); };
  // everything before this call; only the launch itself is hidden.  The next
  // kernel may start from here on, not sooner: it reads the ids before it
  // waits for this one
  pdl_wait_prev();
  pdl_launch_next();

  if (warp == kGuWarps) {
    // ---- the union, then the producer: gate rows, up rows of every item
    if (lane < L.ns) mbar_init(&full[lane], 1), mbar_init(&empty[lane], kTeam);
    if (lane < 2 * kTeams) mbar_init(&red_full[0][lane], kTeam), mbar_init(&red_empty[0][lane], 1);
    fence_mbar_init();
    if (lane == 0 && blockIdx.x == 0) *P.status = 0;
    union_warp(U, P);
    tc05::named_arrive(3, kGuThreads);  // the union and the barriers are there
    if (lane == 0) {
      int f = 0, s = 0;
      uint32_t ph = 0;
      bool ok = true;
      const int items = *U.n * nct, end = share(items, blockIdx.x + 1);
      for (int it = share(items, blockIdx.x); it < end && ok; it++) {
        const int u = it / nct, ct = it - u * nct;
        const uint8_t *src = P.gu + ((size_t)U.ex[u] * 2 * I + ct * 8) * H;
        for (int h = 0; h < 2; h++) {
          ok = thread_wait(&empty[s], ph ^ 1, P);
          if (!ok) break;
          mbar_expect_tx(&full[s], (uint32_t)L.stage);
          bulk_g2s(sm + (size_t)s * L.stage, src + (size_t)h * I * H, (uint32_t)L.stage, &full[s]);
          f++;
          if (++s == L.ns) s = 0, ph ^= 1;
        }
      }
      // copies still in flight land before the CTA ends
      for (int i = f > L.ns ? f - L.ns : 0; i < f; i++) thread_wait(&full[i % L.ns], (uint32_t)((i / L.ns) & 1), P);
    }
    return;
  }
  if (warp == kGuWarps + 1) {
    // ---- sums: lane (c, q) adds the warps' parts of channel c, columns 2q
    // and 2q + 1, in the order of the warps
    tc05::named_sync(3, kGuThreads);
    const int items = *U.n * nct, end = share(items, blockIdx.x + 1);
    int team = 0, turn = 0;
    uint32_t ph = 0;
    for (int it = share(items, blockIdx.x); it < end; it++) {
      const int u = it / nct, ct = it - u * nct;
      // the columns' entries: a row's first with this expert
      int e0 = -1, e1 = -1;
      for (int r = 0; r < P.t; r++) {
        const unsigned m = __ballot_sync(FULLM, lane < P.K && U.ids[r * P.K + min(lane, P.K - 1)] == U.ex[u]);
        const int e = m ? r * P.K + __ffs(m) - 1 : -1;
        if (r == 2 * q) e0 = e;
        if (r == 2 * q + 1) e1 = e;
      }
      if (!warp_wait(&red_full[team][turn], ph, P)) break;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kTeam; w++) {
        const float4 p = red[((team * 2 + turn) * kTeam + w) * 32 + lane];
        v.x += p.x, v.y += p.y, v.z += p.z, v.w += p.w;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&red_empty[team][turn]);
      if (++team == L.teams) {
        team = 0, turn ^= 1;
        if (turn == 0) ph ^= 1;
      }
      const size_t c = (size_t)ct * 8 + g;
      if (e0 >= 0) P.h32[(size_t)e0 * I + c] = v.x / (1.f + expf(-v.x)) * v.z;
      if (e1 >= 0) P.h32[(size_t)e1 * I + c] = v.y / (1.f + expf(-v.y)) * v.w;
    }
    return;
  }
  // ---- the rows of x in e4m3, half a warp a block, the loads
  // of two rounds together
  for (int b = warp * 2; b < P.t * nk; b += 4 * kGuWarps) {
    float v[2][8];
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const int bb = b + 2 * kGuWarps * i + (lane >> 4);
#pragma unroll
      for (int j = 0; j < 8; j++) v[i][j] = 0.f;
      if (bb < P.t * nk) load_x8<BF16>(P.x, (int64_t)bb * 128 + (lane & 15) * 8, v[i]);
    }
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const int bb = b + 2 * kGuWarps * i + (lane >> 4), r = bb / nk;
      if (b + 2 * kGuWarps * i >= P.t * nk) break;  // warp-uniform
      uint32_t e;
      const uint2 w = quant128(v[i], e);
      if (bb < P.t * nk) {
        *reinterpret_cast<uint2 *>(xs + (size_t)r * H + (bb - r * nk) * 128 + (lane & 15) * 8) = w;
        if ((lane & 15) == 0) sx[bb] = e8m0_f(e);
      }
    }
  }
  tc05::named_sync(3, kGuThreads);
  tc05::named_sync(1, 32 * kGuWarps);
  const int team = warp / kTeam, tw = warp - team * kTeam;  // the warp within its team
  if (team >= L.teams) return;
  const int all = *U.n * nct, items = share(all, blockIdx.x + 1), step = L.teams, step_u = step / nct,
            step_c = step - step_u * nct;
  const bool have = g < P.t, have0 = 2 * q < P.t, have1 = 2 * q + 1 < P.t;
  const uint8_t *col = xs + (size_t)(have ? g : 0) * H + q * 32;
  const float *sx0 = sx + (have0 ? 2 * q : 0) * nk, *sx1 = sx + (have1 ? 2 * q + 1 : 0) * nk;
  const size_t up_s = (size_t)(I / 128) * nk;  // from a gate scale to its up scale
  int it = share(all, blockIdx.x) + team;
  int u = it / nct, ct = it - u * nct;
  // the weight scales of the warp's first four k blocks, a byte each, loaded
  // an item ahead
  uint32_t ng = 0, nu = 0;
  auto prefetch = [&](int uu, int cc) {
    const uint8_t *sg = P.gus + ((size_t)U.ex[uu] * (2 * I / 128) + cc / 16) * nk + tw;
    uint32_t a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      a[i] = tw + kTeam * i < nk ? sg[kTeam * i] : 0u;
      b[i] = tw + kTeam * i < nk ? sg[up_s + kTeam * i] : 0u;
    }
    ng = a[0] | a[1] << 8 | a[2] << 16 | a[3] << 24, nu = b[0] | b[1] << 8 | b[2] << 16 | b[3] << 24;
  };
  if (it < items) prefetch(u, ct);
  int s = 2 * team, turn = 0;
  uint32_t ph = 0, rph = 0;
  for (; it < items; it += step) {
    const int u0 = u, ct0 = ct;
    uint32_t wg = ng, wu = nu;
    u += step_u, ct += step_c;
    if (ct >= nct) ct -= nct, u++;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (!warp_wait(&full[s], ph, P) || !warp_wait(&full[s + 1], ph, P)) break;
    if (it + step < items) prefetch(u, ct);
    const uint8_t *gr = sm + (size_t)s * L.stage, *ur = gr + L.stage;
    for (int kb = tw; kb < nk; kb += 2 * kTeam) {
      // two blocks; past the end the second is the first again, unscaled
      const bool two = kb + kTeam < nk;
      const int k2 = two ? kb + kTeam : kb;
      Block x, y;
      load_block(x, gr + kb * 128, ur + kb * 128, H, g, q, col + kb * 128, have);
      load_block(y, gr + k2 * 128, ur + k2 * 128, H, g, q, col + k2 * 128, have);
      float d[4] = {0.f, 0.f, 0.f, 0.f}, e[4] = {0.f, 0.f, 0.f, 0.f};
      mma_blocks(d, x, e, y);
      if (kb >= 4 * kTeam) {
        const uint8_t *sg = P.gus + ((size_t)U.ex[u0] * (2 * I / 128) + ct0 / 16) * nk;
        wg = sg[kb] | (uint32_t)sg[k2] << 8, wu = sg[up_s + kb] | (uint32_t)sg[up_s + k2] << 8;
      }
      const float fg = e8m0_f(wg & 255u), fu = e8m0_f(wu & 255u), x0 = have0 ? sx0[kb] : 1.f, x1 = have1 ? sx1[kb] : 1.f;
      add_scaled(acc, d, x0, x1, fg, fu);
      if (two) {
        const float hg = e8m0_f(wg >> 8 & 255u), hu = e8m0_f(wu >> 8 & 255u);
        const float y0 = have0 ? sx0[k2] : 1.f, y1 = have1 ? sx1[k2] : 1.f;
        add_scaled(acc, e, y0, y1, hg, hu);
      }
      wg >>= 16, wu >>= 16;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[s]), mbar_arrive(&empty[s + 1]);
    s += 2 * L.teams;
    if (s >= L.ns) s -= L.ns, ph ^= 1;
    if (!warp_wait(&red_empty[team][turn], rph ^ 1, P)) break;
    red[((team * 2 + turn) * kTeam + tw) * 32 + lane] = acc;
    __syncwarp();
    if (lane == 0) mbar_arrive(&red_full[team][turn]);
    turn ^= 1;
    if (turn == 0) rph ^= 1;
  }
}

// ---- down: dynamic shared memory: ring | h rows | their scales | weight scales | union | sums
DnLay dn_layout(int I, int n) {
  DnLay l{};
  const int nk = I / 128;
  l.stage = 16 * I;
  const size_t hs = (size_t)n * I, sh = ((size_t)n * nk * 4 + 15) / 16 * 16, red = kDownWarps * 16 * 9 * 4;
  const size_t un = union_bytes(n) / 16 * 16, rest = hs + 2 * sh + un + red;
  const size_t room = kSmemCap > rest ? (kSmemCap - rest) / l.stage : 0;
  const int fit = (int)(room < kMaxStages ? room : kMaxStages), np = (nk + 1) / 2;
  for (int ns = fit; ns >= 1 && 2 * ns >= fit; ns--) {
    int w = kDownWarps;
    while (ns * np % w) w--;
    if (w > l.warps) l.warps = w, l.ns = ns;
  }
  l.hs = (size_t)l.ns * l.stage, l.sh = l.hs + hs, l.sd = l.sh + sh, l.un = l.sd + sh, l.red = l.un + un;
  l.total = (size_t)l.ns * l.stage + rest;
  return l;
}

template <bool BF16>
__global__ void __launch_bounds__(32 * kDownWarps + 32, 1) ex8_down(const __grid_constant__ Ex8P P) {
  extern __shared__ __align__(128) uint8_t sm[];
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages];
  const int n = P.t * P.K;
  const DnLay L = P.dl;
  uint8_t *hs = sm + L.hs;
  float *sh = reinterpret_cast<float *>(sm + L.sh), *sd = reinterpret_cast<float *>(sm + L.sd);
  float *red = reinterpret_cast<float *>(sm + L.red);
  const Union U = union_at(sm + L.un, n);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
  const int H = P.H, I = P.I, nk = I / 128, n0 = blockIdx.x * 16;
  if (warp == kDownWarps) {
    // ---- the union, then the producer: this CTA's rows of every expert
    if (lane < L.ns) mbar_init(&full[lane], 1), mbar_init(&empty[lane], (uint32_t)(nk + 1) / 2);
    fence_mbar_init();
    union_warp(U, P);
    tc05::named_arrive(3, 32 * kDownWarps + 32);
    produce(full, empty, sm, L.ns, L.stage, *U.n, P, [&](int u) { return P.dn + ((size_t)U.ex[u] * H + n0) * I; });
    return;
  }
  tc05::named_sync(3, 32 * kDownWarps + 32);
  const int items = *U.n * nk;  // (expert, k block), k fastest
  auto scale = [&](int i) { return P.dns[((size_t)U.ex[i / nk] * (H / 128) + (n0 >> 7)) * nk + i % nk]; };
  const uint32_t first = tid < items ? scale(tid) : 0u;  // on its way while the tables are made
  union_rows(U, P, tid, 32 * kDownWarps);
  if (tid < items) sd[tid] = e8m0_f(first);
  for (int i = tid + 32 * kDownWarps; i < items; i += 32 * kDownWarps) sd[i] = e8m0_f(scale(i));
  tc05::named_sync(1, 32 * kDownWarps);
  pdl_wait_prev();  // h is the previous kernel's; the weights on their way are not
  // h of every entry that has one (of an expert twice in a row: the first) ->
  // e4m3, half a warp a block, the loads of six rounds together
  constexpr int R = 6;
  for (int b = warp * 2; b < n * nk; b += 2 * R * kDownWarps) {
    float v[R][8];
#pragma unroll
    for (int i = 0; i < R; i++) {
      const int bb = b + 2 * kDownWarps * i + (lane >> 4), e = bb / nk;
#pragma unroll
      for (int j = 0; j < 8; j++) v[i][j] = 0.f;
      if (bb < n * nk && U.own[e]) load_x8<false>(P.h32, (int64_t)bb * 128 + (lane & 15) * 8, v[i]);
    }
#pragma unroll
    for (int i = 0; i < R; i++) {
      const int bb = b + 2 * kDownWarps * i + (lane >> 4), e = bb / nk;
      if (b + 2 * kDownWarps * i >= n * nk) break;  // warp-uniform
      uint32_t x;
      const uint2 w = quant128(v[i], x);
      if (bb < n * nk) {
        *reinterpret_cast<uint2 *>(hs + (size_t)e * I + (bb - e * nk) * 128 + (lane & 15) * 8) = w;
        if ((lane & 15) == 0) sh[bb] = e8m0_f(x);
      }
    }
  }
  tc05::named_sync(1, 32 * kDownWarps);
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  const int np = (nk + 1) / 2, pairs = *U.n * np, step_u = L.warps / np, step_p = L.warps - step_u * np;
  int u = warp / np, pr = warp - u * np, s = u;
  uint32_t ph = 0;
  while (s >= L.ns) s -= L.ns, ph ^= 1;
  for (int it = warp; it < pairs && warp < L.warps; it += L.warps) {
    // two blocks; past the end the second is the first again, unscaled
    const int kb = 2 * pr, k2 = kb + 1 < nk ? kb + 1 : kb;
    const int e = U.ent[u][g], e0 = U.ent[u][2 * q], e1 = U.ent[u][2 * q + 1];
    const uint8_t *col = hs + (size_t)max(e, 0) * I + q * 32;
    if (!warp_wait(&full[s], ph, P)) break;
    const uint8_t *wr = sm + (size_t)s * L.stage;
    Block x, y;
    load_block(x, wr + kb * 128, wr + 8 * I + kb * 128, I, g, q, col + kb * 128, e >= 0);
    load_block(y, wr + k2 * 128, wr + 8 * I + k2 * 128, I, g, q, col + k2 * 128, e >= 0);
    float d[4] = {0.f, 0.f, 0.f, 0.f}, f[4] = {0.f, 0.f, 0.f, 0.f};
    mma_blocks(d, x, f, y);
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[s]);
    // a column whose row did not choose the expert adds nothing, whatever
    // the product is (a NaN weight times zero)
    const float w1 = sd[u * nk + kb], w2 = k2 > kb ? sd[u * nk + k2] : 0.f;
    if (e0 >= 0) {
      add_weighted(acc[0], acc[2], d[0], d[2], sh[e0 * nk + kb], w1, U.w[u][2 * q]);
      if (k2 > kb) add_weighted(acc[0], acc[2], f[0], f[2], sh[e0 * nk + k2], w2, U.w[u][2 * q]);
    }
    if (e1 >= 0) {
      add_weighted(acc[1], acc[3], d[1], d[3], sh[e1 * nk + kb], w1, U.w[u][2 * q + 1]);
      if (k2 > kb) add_weighted(acc[1], acc[3], f[1], f[3], sh[e1 * nk + k2], w2, U.w[u][2 * q + 1]);
    }
    int du = step_u;
    pr += step_p;
    if (pr >= np) pr -= np, du++;
    u += du, s += du;
    while (s >= L.ns) s -= L.ns, ph ^= 1;
  }
#pragma unroll
  for (int i = 0; i < 4; i++) red[(warp * 16 + g + 8 * (i >> 1)) * 9 + 2 * q + (i & 1)] = acc[i];
  tc05::named_sync(1, 32 * kDownWarps);
  if (tid < 128) {
    const int row = tid & 15, r = tid >> 4;
    if (r < P.t) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kDownWarps; w++) v += red[(w * 16 + row) * 9 + r];
      const size_t o = (size_t)r * H + n0 + row;
      if (BF16) {
        uint16_t b;
        asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(b) : "f"(v));
        static_cast<uint16_t *>(P.out)[o] = b;
      } else {
        static_cast<float *>(P.out)[o] = v;
      }
    }
  }
}

// ------------------------------------------------------------ many rows

constexpr int kCountThreads = 1024, kCountEntries = 4 * kCountThreads;  // of a block

// Exclusive scan of the E counts into offs, by one block (E <= kCountThreads).
__device__ void scan_counts(const Ex8P &P, int c, int *part) {
  const int tid = threadIdx.x, lane = tid & 31;
  int x = c;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(FULLM, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) part[tid >> 5] = x;
  __syncthreads();
  if (tid < 32) {
    int p = part[tid];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(FULLM, p, o);
      if (lane >= o) p += y;
    }
    part[tid] = p;
  }
  __syncthreads();
  const int base = x - c + (tid >= 32 ? part[(tid >> 5) - 1] : 0);
  if (tid < P.E) P.offs[tid] = base;
  if (tid == kCountThreads - 1) P.offs[P.E] = base + c;
}

// Place of every entry within its expert's rows.  A block counts its entries
// in shared memory; one block alone is done then, several take runs of places
// from global counters (zeroed before), and the last to finish scans them.
// Which places an entry gets depends on the order of the atomics, its results
// do not.
__global__ void __launch_bounds__(kCountThreads) ex8_count(const __grid_constant__ Ex8P P) {
  pdl_wait_prev();
  pdl_launch_next();  // behind the wait: the next kernel reads x before its own
  extern __shared__ int hist[];  // [E]
  __shared__ int last, part[32];
  const int tid = threadIdx.x, n = P.t * P.K, E = P.E;
  if (blockIdx.x == 0 && tid == 0) *P.status = 0;
  uint32_t ex[4];
  int rank[4];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int j = blockIdx.x * kCountEntries + i * kCountThreads + tid;
    ex[i] = j < n ? P.idx[j] : 0xffffffffu;
  }
  if (tid < E) hist[tid] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; i++) rank[i] = ex[i] < (uint32_t)E ? atomicAdd(&hist[ex[i]], 1) : 0;
  __syncthreads();
  const int mine = tid < E ? hist[tid] : 0;
  if (gridDim.x > 1) {
    if (tid < E) hist[tid] = mine ? atomicAdd(&P.counts[tid], mine) : 0;
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int j = blockIdx.x * kCountEntries + i * kCountThreads + tid;
    if (j < n) P.place[j] = ex[i] < (uint32_t)E ? (gridDim.x > 1 ? hist[ex[i]] : 0) + rank[i] : -1;
  }
  if (gridDim.x == 1) {
    scan_counts(P, mine, part);
    return;
  }
  __threadfence();
  __syncthreads();
  if (tid == 0) last = atomicAdd(&P.counts[E], 1) == (int)gridDim.x - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  scan_counts(P, tid < E ? __ldcg(&P.counts[tid]) : 0, part);
}

// x rows -> e4m3, written to the places of their entries: a warp per row,
// 16 values a lane (eight lanes a block), 16-byte stores.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) ex8_scatter(const __grid_constant__ Ex8P P) {
  pdl_launch_next();
  const int row = blockIdx.x * kWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (row >= P.t) return;
  const int K = P.K, H = P.H;
  float v[2][16];
  auto load = [&](float (&x)[16], int c) {
#pragma unroll
    for (int j = 0; j < 16; j++) x[j] = 0.f;
    if (c < H) {
      float lo[8], hi[8];
      load_x8<BF16>(P.x, (int64_t)row * H + c, lo);
      load_x8<BF16>(P.x, (int64_t)row * H + c + 8, hi);
#pragma unroll
      for (int j = 0; j < 8; j++) x[j] = lo[j], x[8 + j] = hi[j];
    }
  };
  load(v[0], lane * 16);  // x is older than the previous kernel, the places are its
  pdl_wait_prev();
  int at = -1;
  if (lane < K) {
    const int j = row * K + lane, pl = P.place[j];
    if (pl >= 0) at = P.offs[P.idx[j]] + pl;
    P.place[j] = at;  // from here on: the entry's row
  }
  for (int c0 = 0; c0 < H; c0 += 1024) {
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const int c = c0 + 512 * i + lane * 16;
      load(v[i ^ 1], c + 512);
      uint32_t w[4], e;
      quant_block<16>(v[i], w, e);
      for (int j = 0; j < K; j++) {
        const int to = __shfl_sync(FULLM, at, j);
        if (to >= 0 && c < H) {
          *reinterpret_cast<uint4 *>(P.x8 + (size_t)to * H + c) = make_uint4(w[0], w[1], w[2], w[3]);
          if ((lane & 7) == 0) P.x8s[(size_t)to * P.ldh + c / 128] = (uint8_t)e;
        }
      }
    }
  }
}

// out[row] = sum over the row's entries, in order, of weight * y: a warp per
// row and 256 columns, eight a lane.  The outputs y are in 32 bits whatever
// out's type, so that the sum is rounded once, for many rows as for few (y in
// bf16 halved its traffic, 395 us instead of 445 for the 4096 rows above in a
// graph, and its rounding left 1.4 times the error of the last one).
// U entries' loads are in flight at once: one or two where many warps hide
// the latency (five took 54 us instead of 35 at 4096 x 10 rows of 2048, then
// in bf16, for want of warps), eight where there are few.
template <bool BF16, int U>
__global__ void __launch_bounds__(256) ex8_combine(const __grid_constant__ Ex8P P) {
  pdl_wait_prev();
  const int lane = threadIdx.x & 31, K = P.K, H = P.H, segs = (H + 255) / 256;
  const int64_t total = (int64_t)P.t * segs, step = (int64_t)gridDim.x * 8;
  for (int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); i < total; i += step) {
    const int row = (int)(i / segs), c = (int)(i - (int64_t)row * segs) * 256 + lane * 8;
    const int at = lane < K ? P.place[(size_t)row * K + lane] : -1;
    const float wt = lane < K ? P.w[(size_t)row * K + lane] : 0.f;
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if constexpr (U > 1) {
      for (int j0 = 0; j0 < K; j0 += U) {
        float v[U][8], w[U];
  #pragma unroll
        for (int j = 0; j < U; j++) {
          const int a = __shfl_sync(FULLM, at, (j0 + j) & 31);
          w[j] = __shfl_sync(FULLM, wt, (j0 + j) & 31);
          const bool on = j0 + j < K && a >= 0 && c < H;
          if (on) load_x8<false>(P.y, (int64_t)a * H + c, v[j]);
          if (!on) {
            w[j] = 0.f;
  #pragma unroll
            for (int k = 0; k < 8; k++) v[j][k] = 0.f;
          }
        }
  #pragma unroll
        for (int j = 0; j < U; j++)
  #pragma unroll
          for (int k = 0; k < 8; k++) s[k] += w[j] * v[j][k];
      }
    } else {
#pragma unroll 2
      for (int j = 0; j < K; j++) {
        const int a = __shfl_sync(FULLM, at, j);
        const float w = __shfl_sync(FULLM, wt, j);
        if (a < 0 || c >= H) continue;
        float v[8];
        load_x8<false>(P.y, (int64_t)a * H + c, v);
#pragma unroll
        for (int k = 0; k < 8; k++) s[k] += w * v[k];
      }
    }
    if (c >= H) continue;
    if (BF16) {
      uint32_t u[4];
#pragma unroll
      for (int k = 0; k < 4; k++) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u[k]) : "f"(s[2 * k + 1]), "f"(s[2 * k]));
      *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(P.out) + (size_t)row * H + c) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
      float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(P.out) + (size_t)row * H + c);
      o[0] = make_float4(s[0], s[1], s[2], s[3]);
      o[1] = make_float4(s[4], s[5], s[6], s[7]);
    }
  }
}

size_t al(size_t n) { return (n + 1023) & ~(size_t)1023; }

}  // namespace

bool ex8_small(int H, int I, int t, int K) {
  // an item is two of gate_up's stages
  return t <= kEx8SmallRows && gu_layout(H, t, K).ns >= 2 && dn_layout(I, t * K).ns >= 2;
}

Ex8Sizes ex8_sizes(int H, int E, int I, int t, int K) {
  const size_t n = (size_t)t * K;
  const size_t ldi = (size_t)(I / 128 + 3) / 4 * 4, ldh = (size_t)(H / 128 + 3) / 4 * 4;
  Ex8Sizes s{};
  if (ex8_small(H, I, t, K)) {
    s.total = s.h32 = al(n * I * 4);
    return s;
  }
  s.h8 = al(n * I), s.h8s = al(n * ldi);
  s.x8 = al(n * H), s.x8s = al(n * ldh);
  s.counts = al((size_t)(E + 1) * 4), s.offs = al((size_t)(E + 1) * 4), s.place = al(n * 4);
  s.y = al(n * H * 4);
  s.total = s.h8 + s.h8s + s.x8 + s.x8s + s.counts + s.offs + s.place + s.y;
  return s;
}

cudaError_t launch_ex8_small(Ex8P &p, int n_sms, cudaStream_t st) {
  const GuLay l = p.gl = gu_layout(p.H, p.t, p.K);
  const DnLay d = p.dl = dn_layout(p.I, p.t * p.K);
  auto f = p.x_bf16 ? ex8_gate_up<true> : ex8_gate_up<false>;
  auto h = p.out_bf16 ? ex8_down<true> : ex8_down<false>;
  // the most any launch asks for (another host thread may launch them too)
  cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemCap);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(h, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemCap);
  if (e != cudaSuccess) return e;
  const int items = p.t * p.K * (p.I / 8);
  e = launch_pdl(f, dim3((unsigned)(items < n_sms ? items : n_sms)), kGuThreads, l.total, st, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(h, dim3((unsigned)(p.H / 16)), 32 * kDownWarps + 32, d.total, st, p);
}

cudaError_t launch_ex8_group(const Ex8P &p, cudaStream_t st) {
  const int n = p.t * p.K, blocks = (n + kCountEntries - 1) / kCountEntries;
  if (blocks > 1) {
    const cudaError_t e = cudaMemsetAsync(p.counts, 0, (size_t)(p.E + 1) * 4, st);
    if (e != cudaSuccess) return e;
  }
  const cudaError_t e = launch_pdl(ex8_count, dim3((unsigned)blocks), kCountThreads, (size_t)p.E * 4, st, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(p.x_bf16 ? ex8_scatter<true> : ex8_scatter<false>, dim3((unsigned)((p.t + kWarps - 1) / kWarps)), kThreads,
                    0, st, p);
}

cudaError_t launch_ex8_combine(const Ex8P &p, int n_sms, cudaStream_t st) {
  const int64_t need = ((int64_t)p.t * ((p.H + 255) / 256) + 7) / 8, cap = (int64_t)n_sms * 8;
  const bool few = need <= 2 * n_sms;
  auto f = p.out_bf16 ? (few ? ex8_combine<true, 8> : ex8_combine<true, 1>)
                      : (few ? ex8_combine<false, 8> : ex8_combine<false, 1>);
  return launch_pdl(f, dim3((unsigned)(need < cap ? need : cap)), 256, 0, st, p);
}

}  // namespace moe
