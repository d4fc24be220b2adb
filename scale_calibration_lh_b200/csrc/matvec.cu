// Products of up to 8 tokens with one layer's packed NVFP4 weights, or of routed slots with their experts'.
//
// y_{i,r} = g_e * sum_c (q_{e,r,c} v_{e,r,c/16}) x_{i,c}, with e the slot's expert.
//
// The weights are read once and everything else is small, so the kernel is a stream of 4-bit
// weights through the tensor cores' m16n8k16 (fp16 in, fp32 out): 16 rows of W by 8 tokens. Every
// q * v is exact in fp16 (E2M1 times E4M3: 6 significant bits between 2^-10 and 2688), so decoding
// is one conversion a pair and one multiplication by the block's scale.
//
// Activations become fp16 in registers: E4M3 is exact; bf16 is scaled per token and 128 channels
// by the power of two that brings the block's largest magnitude to [2^14, 2^15), exact for all
// elements down to 2^-29 of it. The scale (or the E4M3 scale) multiplies the 128 channels' fp32
// sum. Since the order of channels in a dot product is free, a lane takes 16 consecutive bytes (32
// weights, two blocks) of its row and the same channels of its token, with no shuffles.
//
// One or two tokens fill a quarter of the columns. There a token has four columns, one for each
// lane of a row's quad, whose activations are zero in the other lanes: the sums come apart by
// scale block, and the scales multiply 8 sums a lane in place of 64 weights.
//
// One CTA an SM takes an equal, contiguous range of all rows (of the experts hit, one after the
// other). One warp copies them, 16 rows at a time, into a ring of stages in shared memory (bulk
// copies, an mbarrier a stage), as far ahead as the ring goes and across experts. The other warps
// split the channels, 256 to a warp and pass, and hold their activations while the rows go by;
// their sums meet in shared memory in a fixed order, a block of rows at a time.
//
// Measured (us): 1 x 1280 x 2560 4.3, 1 x 4096 x 4096 5.9, 1 x 65536 x 4096 29.3 (5.2 TB/s), 1 x 467200 x 2560 114
// (5.9 TB/s), 4 x 12288 x 4096 E4M3 9.6 (3.0 TB/s), routed 1 x 10 of 512 experts 1280 x 2560 10.4, 8 x 10
// 33 (4.2 TB/s), 64 x 10 136 (5.0 TB/s). Bound by HBM where the rows are many; else by instructions (16
// for 8 weights of a lane, 20 where an entry has more than two slots, 4 of them conversions; before the last step a tile took a warp 1450 cycles, of which 940 issued)
// and by what comes first: 1200 cycles until the shares are known (routed 3000), 2000 to 3000 for the
// activations, while the ring fills. All loads of a tile go before its products (1 x 467200 x 2560: 121 ->
// 114, 4 x 12288 x 4096 10.1 -> 9.5).
#include "common.cuh"
#include "matvec.cuh"
#include "matvec_plan.cuh"

namespace lhcal {
namespace {

using Plan = MatvecPlan;

template <int N>
struct Int {
  static constexpr int value = N;
};

struct KernelArgs {
  MatvecArgs m;
  Plan p;
};

// Both addresses and the size are multiples of 16 bytes.
__device__ __forceinline__ void bulk_copy(uint32_t dst, const uint8_t* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// 32 bf16 activations of a token (a lane's of 128; the quad holds the rest) to fp16 in place, and
// the power of two that they were divided by.
__device__ __forceinline__ float bf16_to_f16(uint32_t (&u)[16]) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) top = max_bf16x2(top, u[i]);
  top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
  uint32_t up;
  float down;
  fp16_range(top, up, down);
#pragma unroll
  for (int i = 0; i < 16; ++i) u[i] = bf16x2_to_f16(u[i], up);
  return down;
}

// The work of a row of an entry, in quarters of that with one or two slots (measured at 1280 rows by
// 2560 channels: 0.77, 1.0 and 1.1 us a tile).
__device__ __forceinline__ uint32_t work_of(int slots) { return slots <= 2 ? 4 : slots <= 4 ? 5 : 6; }

// Entries: up to 8 slots of one expert, bits 0 to 15: the expert, 16 to 27: where its slots begin in
// `order`, 28 to 31: how many slots. The same list in every CTA: by expert, slots in order.
__device__ int plan_entries(const MatvecArgs& m, int* ids, uint32_t* hist, uint32_t* entries, uint32_t* sums, int2* scan) {
  const int tid = threadIdx.x, threads = blockDim.x, lane = tid & 31, warp = tid >> 5, warps = threads / 32;
  for (int i = tid; i < m.groups / 2 + 1; i += threads) hist[i] = 0;
  __syncthreads();
  for (int i = tid; i < m.slots; i += threads) {
    int e = __ldg(m.experts + i);
    if (e < 0 || e >= m.groups) e = -1;
    ids[i] = e;
    if (e >= 0) atomicAdd(hist + (e >> 1), e & 1 ? 0x10000u : 1u);
  }
  __syncthreads();
  const int per = (m.groups + threads - 1) / threads, e0 = tid * per, e1 = min(e0 + per, m.groups);
  auto slots_of = [&](int e) { return static_cast<int>(hist[e >> 1] >> (16 * (e & 1)) & 0xffffu); };
  int n = 0, work = 0;  // entries, and slots << 16, of this thread's experts; their work
  for (int e = e0; e < e1; ++e) {
    const int c = slots_of(e);
    n += (c + kTokens - 1) / kTokens + (c << 16);
    for (int k = 0; k < c; k += kTokens) work += work_of(min(c - k, kTokens));
  }
  int n_upto = n, work_upto = work;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, n_upto, o), u = __shfl_up_sync(0xffffffffu, work_upto, o);
    if (lane >= o) {
      n_upto += v;
      work_upto += u;
    }
  }
  if (lane == 31) scan[warp] = make_int2(n_upto, work_upto);
  __syncthreads();
  int2 mine = lane < warps ? scan[lane] : make_int2(0, 0);
  int at = __reduce_add_sync(0xffffffffu, lane < warp ? mine.x : 0) + n_upto - n;
  int work_at = __reduce_add_sync(0xffffffffu, lane < warp ? mine.y : 0) + work_upto - work;
  const int n_entries = __reduce_add_sync(0xffffffffu, mine.x) & 0xffff;
  const int all = __reduce_add_sync(0xffffffffu, mine.y);
  for (int e = e0; e < e1; ++e) {
    const int c = slots_of(e);
    for (int k = 0; k < c; k += kTokens) {
      entries[at & 0xffff] = static_cast<uint32_t>(e) | static_cast<uint32_t>((at >> 16) + k) << 16 |
                             static_cast<uint32_t>(min(c - k, kTokens)) << 28;
      sums[at & 0xffff] = work_at;
      work_at += work_of(min(c - k, kTokens));
      ++at;
    }
    at += c << 16;
  }
  if (tid == 0) sums[n_entries] = all;
  __syncthreads();
  return n_entries;
}

// The slots of the experts of entries [from, to], in order, a warp an expert (its entries lie
// together).
__device__ void order_slots(const MatvecArgs& m, const int* ids, const uint32_t* entries, int* order, int from, int to,
                            int warps) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  while (from > 0 && (entries[from - 1] & 0xffff) == (entries[from] & 0xffff)) --from;
  for (int k = from + warp; k <= to; k += warps) {
    const uint32_t v = entries[k];
    const int e = v & 0xffff;
    if (k > from && static_cast<int>(entries[k - 1] & 0xffff) == e) continue;
    int seen = v >> 16 & 0xfff;
    for (int i = 0; i < m.slots; i += 32) {
      const bool hit = i + lane < m.slots && ids[i + lane] == e;
      const uint32_t mask = __ballot_sync(0xffffffffu, hit);
      if (hit) order[seen + __popc(mask & ((1u << lane) - 1))] = i + lane;
      seen += __popc(mask);
    }
  }
}

// The few slots of a decoded token or three, by one warp: entries by first slot; how many, or -1 if an
// expert has more than 8.
__device__ int plan_few(const MatvecArgs& m, uint32_t* entries, uint32_t* sums, int* order) {
  const int lane = threadIdx.x & 31;
  int e = lane < m.slots ? __ldg(m.experts + lane) : -1;
  if (e < 0 || e >= m.groups) e = -1;
  const uint32_t same = __match_any_sync(0xffffffffu, e), before = (1u << lane) - 1;
  const bool first = e >= 0 && (same & before) == 0;
  const uint32_t firsts = __ballot_sync(0xffffffffu, first);
  const int n = first ? __popc(same) : 0;
  if (__any_sync(0xffffffffu, n > kTokens)) return -1;
  const uint32_t w = first ? work_of(n) : 0;
  uint32_t upto = static_cast<uint32_t>(n) << 16 | w;  // slots and work; at most 32 and 32 * 6
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += v;
  }
  const int at = static_cast<int>(upto >> 16) - n, begin = __shfl_sync(0xffffffffu, at, __ffs(same) - 1);
  if (first) {
    const int k = __popc(firsts & before);
    entries[k] = static_cast<uint32_t>(e) | static_cast<uint32_t>(begin) << 16 | static_cast<uint32_t>(n) << 28;
    sums[k] = (upto & 0xffff) - w;
  }
  if (e >= 0) order[begin + __popc(same & before)] = lane;
  if (lane == 31) sums[__popc(firsts)] = upto & 0xffff;
  __syncwarp();
  return __popc(firsts);
}

// The same value in every lane, so that what follows from it is computed once a warp.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// An entry's expert and slots: from where (in order), how many; floats of a row's sums: its slots,
// rounded up to pairs.
struct Entry {
  int expert, first, count, shift;  // pitch = 1 << shift
  __device__ __forceinline__ int pitch() const { return 1 << shift; }
};
template <bool ROUTED>
__device__ __forceinline__ Entry read_entry(const MatvecArgs& m, uint32_t entries, int k) {  // shared address
  Entry e;
  if (ROUTED) {
    const uint32_t v = static_cast<uint32_t>(uniform(static_cast<int>(lds32(entries + 4 * k))));
    e.expert = v & 0xffff;
    e.first = v >> 16 & 0xfff;
    e.count = v >> 28;
  } else {
    e.expert = e.first = 0;
    e.count = min(m.slots, kTokens);  // as it is; without the bound 1 x 467200 x 2560 takes 135 us in place of 114
  }
  e.shift = e.count <= 2 ? 1 : e.count <= 4 ? 2 : 3;
  return e;
}

// A block: consecutive rows of one entry, as many as the warps' sums have room for.
template <bool ROUTED>
struct Rows {
  int entry, row, n;
  int left;  // of the CTA, from here on

  __device__ __forceinline__ void clip(const MatvecArgs& m, uint32_t entries, int room) {
    n = min(min(static_cast<int>(m.rows) - row, left), room >> read_entry<ROUTED>(m, entries, entry).shift & ~(kTile - 1));
  }
  __device__ __forceinline__ void advance(const MatvecArgs& m, uint32_t entries, int room) {
    left -= n;
    row += n;
    if (left <= 0) return;
    if (row == static_cast<int>(m.rows)) {
      row = 0;
      ++entry;
    }
    clip(m, entries, room);
  }
};

// WARPS: at most, for the registers a thread may have.
template <bool WIDE, bool ROUTED, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, 1) matvec_kernel(const KernelArgs ka) {
  constexpr bool kAhead = WARPS <= 17;  // registers for a tile's loads of more than two slots before its products
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t barriers[2 * kMaxStages];
  __shared__ int failed, share[5];  // share: entry, row, rows, last entry; entries
  const MatvecArgs& m = ka.m;
  const Plan& p = ka.p;
  const int tid = threadIdx.x, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int warp = uniform(tid >> 5);
  const int wstride = static_cast<int>(m.cin / 2), cstride = static_cast<int>(m.cin / kBlock);
  // Routed: the slots in the entries' order, the entries, and (while they are made) the slots' experts.
  // `most` words each; and as many for the counts' scan, and the entries' work so far.
  const uint32_t most = max(m.slots + 31 & ~31, 64), order_at = p.list, entries_at = order_at + most * 4, ids_at = entries_at + most * 4;
  const uint32_t base = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
  const uint32_t bar = static_cast<uint32_t>(__cvta_generic_to_shared(barriers));  // a stage's: full, empty

  const uint32_t entries = base + entries_at, order = base + order_at;
  const int warps = p.wk * p.wr;  // that multiply
  const uint32_t failed_at = static_cast<uint32_t>(__cvta_generic_to_shared(&failed));

  const int my_k = warp % p.wk, my_r = warp / p.wk;
  auto channel_of = [&](int pass) { return (pass * p.wk + my_k) * kPieceK; };  // the warp's first in a pass
  const int n_k = static_cast<int>((m.cin + kXBlock - 1) / kXBlock);         // activation blocks
  uint32_t x[2][16];  // the lane's channels of token g in the two blocks, as fp16 pairs: 4 words a weight word
  float xs[2][2];     // the scales of the tokens of the lane's columns of the sums
  auto load_x = [&](const Entry& en, int pass) {
    const bool few = en.count <= 2;  // tokens past the last: columns that are not stored
    const int i = en.first + min(few ? g >> 2 : g, en.count - 1);
    const int64_t row = ROUTED ? static_cast<int>(lds32(order + 4 * i) * p.per_row >> 20) : i;
    const int k = channel_of(pass) + t * 32;
    float s[2] = {0.f, 0.f};
    if (m.xtype == LHCAL_E4M3) {
      uint4 v[2][2];
      const uint8_t* src = static_cast<const uint8_t*>(m.x) + row * m.ldx + k;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          v[j][h] = make_uint4(0u, 0u, 0u, 0u);
          if (k + j * kXBlock + h * 16 < m.cin) v[j][h] = __ldg(reinterpret_cast<const uint4*>(src + j * kXBlock + h * 16));
        }
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (channel_of(pass) + j * kXBlock < m.cin)
          s[j] = __ldg(m.x_scale + (m.scale_block ? row * n_k + k / kXBlock + j : row));
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t u[4] = {v[j][h].x, v[j][h].y, v[j][h].z, v[j][h].w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            x[j][h * 8 + q * 2] = e4m3x2_to_f16(u[q]);
            x[j][h * 8 + q * 2 + 1] = e4m3x2_to_f16(u[q] >> 16);
          }
        }
    } else {
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(m.x) + row * m.ldx + k;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (k + j * kXBlock + w * 8 < m.cin) v = __ldg(reinterpret_cast<const uint4*>(src + j * kXBlock + w * 8));
          x[j][w * 4] = v.x; x[j][w * 4 + 1] = v.y; x[j][w * 4 + 2] = v.z; x[j][w * 4 + 3] = v.w;
        }
#pragma unroll
      for (int j = 0; j < 2; ++j) s[j] = bf16_to_f16(x[j]);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      xs[j][0] = __shfl_sync(0xffffffffu, s[j], few ? t >> 1 << 4 : t * 8);
      xs[j][1] = __shfl_sync(0xffffffffu, s[j], t * 8 + 4);
      if (few && (g & 3) != t) {
#pragma unroll
        for (int w = 0; w < 16; ++w) x[j][w] = 0;
      }
    }
  };

  int n_entries = 1;  // one layer
  int held = -1;  // whose activations x holds
  if (tid == 0) {
    failed = 0;
    for (int s = 0; s < p.stages; ++s) {
      barrier_init(bar + s * 16, 1);
      barrier_init(bar + s * 16 + 8, p.wk);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  // The CTA's share: equal shares of the work. Any cut does that is monotone and the same for
  // neighbours. Routed: one warp makes the cuts (and the plan of few slots).
  Rows<ROUTED> here;
  int last;  // the CTA's last entry
  bool few_slots = true;
  const int rows = static_cast<int>(m.rows);
  auto cut = [&](uint64_t total, uint32_t i) { return i == gridDim.x ? total : __umul64hi(total, i * p.per_cta); };
  if (ROUTED) {
    uint32_t* list = reinterpret_cast<uint32_t*>(smem + entries_at);
    int* ids = reinterpret_cast<int*>(smem + ids_at);
    uint32_t* sums = reinterpret_cast<uint32_t*>(ids) + 2 * most;
    auto share_out = [&](int n) {
      const uint64_t total = static_cast<uint64_t>(sums[n]) * rows;
      const uint64_t at[2] = {cut(total, blockIdx.x), cut(total, blockIdx.x + 1)};
      int found[2] = {0, 0}, row[2];  // entries that begin at or before
      for (int k = lane; k < n; k += 32) {
        const uint64_t from = static_cast<uint64_t>(sums[k]) * rows;
        found[0] += from <= at[0];
        found[1] += from <= at[1];
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        found[c] = __reduce_add_sync(0xffffffffu, found[c]) - 1;
        // Into the entry by a rounded, but monotone, quotient.
        const uint32_t begin = sums[found[c]], w = sums[found[c] + 1] - begin;
        const float into = __ull2float_rn(at[c] - static_cast<uint64_t>(begin) * rows) * (w == 4 ? 1.f / 4 : w == 5 ? 1.f / 5 : 1.f / 6);
        row[c] = blockIdx.x + c == gridDim.x ? rows : min(rows, __float2int_rd(into));
        if (row[c] == rows) {
          row[c] = 0;
          ++found[c];
        }
      }
      if (lane == 0) {
        share[0] = found[0];
        share[1] = row[0];
        share[2] = static_cast<int>(static_cast<int64_t>(found[1] - found[0]) * rows + row[1] - row[0]);
        share[3] = row[1] > 0 ? found[1] : found[1] - 1;
      }
    };
    few_slots = m.slots <= 32;
    if (few_slots) {
      if (warp == 0) {
        n_entries = plan_few(m, list, sums, reinterpret_cast<int*>(smem + order_at));
        if (n_entries > 0) share_out(n_entries);
        if (lane == 0) share[4] = n_entries;
      }
      __syncthreads();
      n_entries = share[4];
      few_slots = n_entries >= 0;
    }
    if (!few_slots) {
      n_entries = plan_entries(m, ids, reinterpret_cast<uint32_t*>(smem), list, sums, reinterpret_cast<int2*>(ids + most));
      if (warp == 0 && n_entries > 0) share_out(n_entries);
      __syncthreads();
    }
    if (n_entries == 0) return;
    here.entry = share[0];
    here.row = share[1];
    here.left = share[2];
    last = share[3];
  } else {
    const uint64_t begin = cut(rows, blockIdx.x), end = cut(rows, blockIdx.x + 1);
    here.entry = last = 0;
    here.row = static_cast<int>(begin);
    here.left = static_cast<int>(end - begin);
  }
  if (here.left <= 0) return;
  here.clip(m, entries, p.room);
  int stage = 0;
  uint32_t phase = 0;

  if (warp == warps) {
    // The copies, by one lane: of a tile's rows whole where all channels go in one pass, else row by
    // row. They begin and end on 16-byte boundaries around the bytes; the readers know where those
    // lie in them.
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the plan's counts lay where the stages do
    const int64_t rows_all = static_cast<int64_t>(m.groups) * m.rows;
    const bool codes16 = m.cin % kPieceK == 0 && (reinterpret_cast<uintptr_t>(m.codes) & 15) == 0;
    const uint8_t *const w_end = m.packed + rows_all * wstride, *const c_end = m.codes + rows_all * cstride;
    // The size of the copy of `bytes` from src on that starts at its 16-byte boundary. Not past the
    // end of the tensor: its last bytes go by themselves.
    auto size_of = [](const uint8_t* src, int bytes, const uint8_t* src_end) {
      const int head = static_cast<int>(reinterpret_cast<uintptr_t>(src) & 15), size = (head + bytes + 15) & ~15;
      return src_end - (src - head) < size ? size - 16 : size;
    };
    auto copy = [](uint32_t to, const uint8_t* src, int bytes, int size, uint32_t full) {
      const int head = static_cast<int>(reinterpret_cast<uintptr_t>(src) & 15);
      if (size > 0) bulk_copy(to, src - head, size, full);
    };
    auto copy_last = [](uint32_t to, const uint8_t* src, int bytes, int size) {
      const int head = static_cast<int>(reinterpret_cast<uintptr_t>(src) & 15);
      for (int i = max(size, head); i < head + bytes; ++i)
        asm volatile("st.shared.u8 [%0], %1;" ::"r"(to + i), "r"(static_cast<uint32_t>(__ldg(src - head + i))) : "memory");
    };
    // The CTA, and its shared memory, last until its copies are in, even if the others gave up.
    auto drain = [&]() {
      for (int s = lane; s < p.stages; s += 32)
        for (int i = 0; i < kDrainLimit && !barrier_poll(bar + s * 16, s < stage ? phase : phase ^ 1); ++i) {}
    };
    for (; here.left > 0; here.advance(m, entries, p.room)) {
      for (int pass = 0; pass < p.passes; ++pass) {
        const int k0 = pass * p.wk * kPieceK, k1 = static_cast<int>(imin64(m.cin, k0 + p.wk * kPieceK));
        const int wb = (k1 - k0) / 2, cb = (k1 - k0) / kBlock;  // bytes of a row
        const int64_t row = read_entry<ROUTED>(m, entries, here.entry).expert * m.rows + here.row;
        const uint8_t *w = m.packed + row * wstride + k0 / 2, *c = m.codes + row * cstride + k0 / kBlock;
        for (int r = 0; r < here.n; r += kTile, w += kTile * wstride, c += kTile * cstride) {
          const int n = min(kTile, here.n - r);
          const uint32_t full = bar + stage * 16, w_to = base + stage * p.stage, c_to = w_to + p.codes_at;
          bool free = lane != 0 || barrier_wait(full + 8, phase ^ 1, &failed);
          // Warps free a stage whose wait ran out, too. What has not come in after kWaitLimit polls will not; but
          // waits that give up at once leave copies in flight, which no other may follow. (In every build this
          // would cost 1 x 467200 x 2560 121 us in place of 114.)
          if (kImpatient && lane == 0) free = free && lds32(failed_at) == 0;
          if (!__all_sync(0xffffffffu, free)) return drain();
          if (lane != 0) {
          } else if (p.passes == 1) {
            const int ws = size_of(w, n * wb, w_end), cs = size_of(c, n * cb, c_end);
            copy_last(w_to, w, n * wb, ws);
            copy_last(c_to, c, n * cb, cs);
            barrier_expect(full, ws + cs);
            copy(w_to, w, n * wb, ws, full);
            copy(c_to, c, n * cb, cs, full);
          } else if (WIDE && codes16) {  // rows are whole 16-byte units
            barrier_expect(full, n * (wb + cb));
            for (int i = 0; i < n; ++i) {
              bulk_copy(w_to + i * p.w_pitch, w + i * wstride, wb, full);
              bulk_copy(c_to + i * p.c_pitch, c + i * cstride, cb, full);
            }
          } else {
            uint32_t all = 0;
            for (int i = 0; i < n; ++i) {
              const int ws = size_of(w + i * wstride, wb, w_end), cs = size_of(c + i * cstride, cb, c_end);
              copy_last(w_to + i * p.w_pitch, w + i * wstride, wb, ws);
              copy_last(c_to + i * p.c_pitch, c + i * cstride, cb, cs);
              all += ws + cs;
            }
            barrier_expect(full, all);
            for (int i = 0; i < n; ++i) {
              copy(w_to + i * p.w_pitch, w + i * wstride, wb, size_of(w + i * wstride, wb, w_end), full);
              copy(c_to + i * p.c_pitch, c + i * cstride, cb, size_of(c + i * cstride, cb, c_end), full);
            }
          }
          __syncwarp();
          if (++stage == p.stages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
    }
    return drain();
  }

  if (ROUTED && !few_slots) {
    order_slots(m, reinterpret_cast<int*>(smem + ids_at), reinterpret_cast<uint32_t*>(smem + entries_at),
                reinterpret_cast<int*>(smem + order_at), here.entry, last, warps);
    asm volatile("bar.sync 1, %0;" ::"r"(32 * warps) : "memory");
  }
  int buffer = 0;
  const int step = p.wr * kTile;
  for (; here.left > 0; here.advance(m, entries, p.room), buffer ^= 1) {
    const Entry en = read_entry<ROUTED>(m, entries, here.entry);
    const int pitch = en.pitch(), n_tiles = (here.n + kTile - 1) / kTile;
    if (ROUTED) asm volatile("prefetch.global.L1 [%0];" ::"l"(m.g + en.expert));
    const uint32_t sums = base + p.red + buffer * (p.wk * p.room * 4);
    for (int pass = 0; pass < p.passes; ++pass) {
      if (held != here.entry * p.passes + pass) load_x(en, pass);
      held = here.entry * p.passes + pass;
      const int k0 = channel_of(pass), kp = pass * p.wk * kPieceK;
      // Where the lane's rows begin in a stage; the same for every tile, since 16 rows are whole
      // 16-byte units of weights and of codes.
      uint32_t w_at[2], c_at[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = g + h * 8;
        // A tile copied whole begins with its first row, else every row by itself.
        const int64_t row = en.expert * m.rows + here.row + (p.passes == 1 ? 0 : r);
        w_at[h] = base + r * p.w_pitch + my_k * (kPieceK / 2) + t * 16;
        if (!WIDE) w_at[h] += static_cast<uint32_t>(reinterpret_cast<uintptr_t>(m.packed) + row * wstride + kp / 2) & 15;
        c_at[h] = base + p.codes_at + r * p.c_pitch + my_k * (kPieceK / kBlock) +
                  (static_cast<uint32_t>(reinterpret_cast<uintptr_t>(m.codes) + row * cstride + kp / kBlock) & 15);
      }
      uint32_t to = sums + (my_k * p.room + (my_r * kTile + g) * pitch) * 4;  // this warp's sums of the lane's rows
      // This warp's tiles' stages, from the pass's first on.
      int at = stage + my_r;
      uint32_t at_phase = phase;
      if (at >= p.stages) {
        at -= p.stages;
        at_phase ^= 1;
      }
      uint32_t off = 0;
      auto arrive = [&]() {
        barrier_wait(bar + at * 16, at_phase, &failed);
        __syncwarp();
        off = at * p.stage;
      };
      auto leave = [&]() {
        __syncwarp();
        if (lane == 0) barrier_arrive(bar + at * 16 + 8);
        at += p.wr;
        if (at >= p.stages) {
          at -= p.stages;
          at_phase ^= 1;
        }
      };
      auto weights = [&](int j, uint32_t (&wv)[2][4]) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t from = w_at[h] + off + j * (kXBlock / 2);
          if (WIDE) {
            const uint4 v = lds128(from);
            wv[h][0] = v.x; wv[h][1] = v.y; wv[h][2] = v.z; wv[h][3] = v.w;
          } else {
            const uint2 v = lds64(from), u = lds64(from + 8);
            wv[h][0] = v.x; wv[h][1] = v.y; wv[h][2] = u.x; wv[h][3] = u.y;
          }
        }
      };
      // N codes of row g + 8 h from block b of the piece.
      auto codes = [&](int h, int b, auto n) -> uint32_t {
        constexpr int N = decltype(n)::value;
        const uint32_t from = c_at[h] + off + b;
        if (WIDE) return N == 4 ? lds32(from) : lds16(from);
        return N == 4 ? lds8(from) | lds8(from + 1) << 8 | lds8(from + 2) << 16 | lds8(from + 3) << 24
                      : lds8(from) | lds8(from + 1) << 8;
      };
      // What of the lane's codes is cin's, by the piece's halves; past them lie other bytes.
      const int have = cstride - k0 / kBlock, lane_blocks = pitch == 2 ? 4 : 2;
      const int first = pitch == 2 ? (t & 1) * 4 : t * 2;
      uint32_t within[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int k = have - j * 8 - first;
        within[j] = k >= lane_blocks ? 0xffffffffu : k <= 0 ? 0u : (1u << 8 * k) - 1;
      }
      if (pitch == 2) {
        for (int i = my_r; i < n_tiles; i += p.wr, to += step * 2 * 4) {
          arrive();
          float acc[2] = {0.f, 0.f};
          uint32_t wv[2][2][4], c[2][2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            weights(j, wv[j]);
#pragma unroll
            for (int h = 0; h < 2; ++h) c[j][h] = codes(h, j * 8 + first, Int<4>()) & within[j];  // of lanes 2 (t & 1) and the next
          }
          leave();
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float sum[2][4];  // by the lanes' first and second blocks; columns: lanes 2 (t & 1) and the next
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              uint32_t q[2][4];
              e2m1x8_to_f16(wv[j][0][w], q[0]);
              e2m1x8_to_f16(wv[j][1][w], q[1]);
              const uint32_t* xw = x[j] + w * 4;
              if (w % 2 == 0)
                mma16816_first(sum[w / 2], q[0][0], q[1][0], q[0][1], q[1][1], xw[0], xw[1]);
              else
                mma16816(sum[w / 2], q[0][0], q[1][0], q[0][1], q[1][1], xw[0], xw[1]);
              mma16816(sum[w / 2], q[0][2], q[1][2], q[0][3], q[1][3], xw[2], xw[3]);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float2 s0 = f16x2_to_float2(e4m3x2_to_f16(c[j][h])), s1 = f16x2_to_float2(e4m3x2_to_f16(c[j][h] >> 16));
              float v = s0.x * sum[0][2 * h];
              v = fmaf(s0.y, sum[1][2 * h], v);
              v = fmaf(s1.x, sum[0][2 * h + 1], v);
              v = fmaf(s1.y, sum[1][2 * h + 1], v);
              acc[h] = fmaf(xs[j][0], v, acc[h]);
            }
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float v = acc[h] + __shfl_xor_sync(0xffffffffu, acc[h], 1);
            const uint32_t o = to + (h * 16 + (t >> 1)) * 4;
            if ((t & 1) == 0) sts_float(o, pass > 0 ? __uint_as_float(lds32(o)) + v : v);
          }
        }
      } else {
        for (int i = my_r; i < n_tiles; i += p.wr, to += step * pitch * 4) {
          arrive();
          float acc[4] = {0.f, 0.f, 0.f, 0.f};
          uint32_t both[2][2][4], c[2][2];
          auto load = [&](int j) {
            weights(j, both[j]);
#pragma unroll
            for (int h = 0; h < 2; ++h) c[j][h] = codes(h, j * 8 + first, Int<2>()) & within[j];
          };
          if (kAhead) {
            load(0);
            load(1);
            leave();
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (!kAhead) load(j);
            float sum[2][4];
            uint32_t s2[2];
            const auto& wv = both[j];
#pragma unroll
            for (int h = 0; h < 2; ++h) s2[h] = e4m3x2_to_f16(c[j][h]);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              uint32_t q[2][4];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                e2m1x8_to_f16(wv[h][w], q[h]);
                const uint32_t s = __byte_perm(s2[h], 0, w < 2 ? 0x1010 : 0x3232);
#pragma unroll
                for (int v = 0; v < 4; ++v) q[h][v] = hmul2(q[h][v], s);
              }
              const uint32_t* xw = x[j] + w * 4;
              if (w == 0) {  // two chains of sums
                mma16816_first(sum[0], q[0][0], q[1][0], q[0][1], q[1][1], xw[0], xw[1]);
                mma16816_first(sum[1], q[0][2], q[1][2], q[0][3], q[1][3], xw[2], xw[3]);
              } else {
                mma16816(sum[0], q[0][0], q[1][0], q[0][1], q[1][1], xw[0], xw[1]);
                mma16816(sum[1], q[0][2], q[1][2], q[0][3], q[1][3], xw[2], xw[3]);
              }
            }
#pragma unroll
            for (int v = 0; v < 4; ++v) acc[v] = fmaf(xs[j][v & 1], sum[0][v] + sum[1][v], acc[v]);
          }
          if (!kAhead) leave();
          if (2 * t < pitch) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t o = to + (h * 8 * pitch + 2 * t) * 4;
              float2 v = make_float2(acc[2 * h], acc[2 * h + 1]);
              if (pass > 0) {
                const uint2 u = lds64(o);
                v = make_float2(__uint_as_float(u.x) + v.x, __uint_as_float(u.y) + v.y);
              }
              sts_float(o, v.x);
              sts_float(o + 4, v.y);
            }
          }
        }
      }
      stage += n_tiles % p.stages;  // past the pass's stages
      phase ^= n_tiles / p.stages & 1;
      if (stage >= p.stages) {
        stage -= p.stages;
        phase ^= 1;
      }
    }
    // The warps that multiply; the other buffer is free again once every one is here.
    asm volatile("bar.sync 1, %0;" ::"r"(32 * warps) : "memory");
    const Entry joined = read_entry<ROUTED>(m, entries, here.entry);
    const float gs = __ldg(m.g + joined.expert);
    for (int o = tid; o < here.n * pitch; o += 32 * warps) {
      const int n = o & (pitch - 1), r = o >> joined.shift;
      if (n >= joined.count) continue;
      // 0, or NaN from the block on in which a wait ran out: it set `failed` before its warp came to the barrier
      // above, and a wait can pass for an earlier lap of its stage only after that.
      float v = __uint_as_float(lds32(failed_at));
      for (int k = 0; k < p.wk; ++k) v += __uint_as_float(lds32(sums + (k * p.room + o) * 4));
      const int64_t y = (ROUTED ? static_cast<int>(lds32(order + 4 * (joined.first + n))) : joined.first + n) * m.ldy + here.row + r;
      if (m.ytype == LHCAL_F32)
        static_cast<float*>(m.y)[y] = v * gs;
      else
        static_cast<__nv_bfloat16*>(m.y)[y] = __float2bfloat16(v * gs);
    }
  }
}

Plan make_plan(const MatvecArgs& m) {
  return make_matvec_plan({m.experts != nullptr, m.cin % 64 == 0 && aligned(m.packed, 16) && aligned(m.codes, 4), m.slots,
                           m.per_row, m.groups, m.rows, m.cin, kNumSms});
}

template <bool WIDE, bool ROUTED, int WARPS>
lhcal_status launch(const KernelArgs& ka, cudaStream_t stream) {
  auto* fn = matvec_kernel<WIDE, ROUTED, WARPS>;
  const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             kMaxSmem - kStaticSmem);  // of any plan: calls may run at once
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail(LHCAL_ERR_CUDA, "matvec: %s", cudaGetErrorString(e));
  }
  void* args[] = {const_cast<KernelArgs*>(&ka)};
  // 0.2 us less on the host than the launch syntax.
  cudaLaunchKernel(reinterpret_cast<const void*>(fn), dim3(ka.p.grid), dim3(32 * (ka.p.wk * ka.p.wr + 1)), args, ka.p.smem, stream);
  return check_launch("matvec");
}

template <bool WIDE, bool ROUTED>
lhcal_status launch_warps(const KernelArgs& ka, cudaStream_t stream) {
  // 17: up to 4096 channels. With a bound of 20 warps in its place 1 x 65536 x 4096 took 31.2 us in place of 29.3.
  const int warps = ka.p.wk * ka.p.wr + 1;
  return warps <= 16 ? launch<WIDE, ROUTED, 16>(ka, stream)
         : warps <= 17 ? launch<WIDE, ROUTED, 17>(ka, stream)
                       : launch<WIDE, ROUTED, kMaxWarps + 1>(ka, stream);
}

}  // namespace

lhcal_status launch_matvec(const MatvecArgs& m, cudaStream_t stream) {
  // One layer with more than 8 tokens: decoding each weight once for all of them wins (16 x 4096 x 4096: 8.4
  // against 13.4 us, 64: 16.5 against 31, 17 x 4096 x 12288: 17.5 against 35). Fewer tokens would fill half of its
  // columns (8 x 4096 x 4096: 8.2 against 7.2 us), but where the warps do not hold all channels at once, the
  // kernel here comes back to each block of rows with other activations, and its clusters split the channels
  // instead: better for small layers (1 x 4096 x 12288 12.4 against 14.0, 8 14.5 against 15.1, 1 x 1280 x 40960 18.9
  // against 24.2), not for large ones, which are several waves of clusters (1 x 8192 x 8192 19.2 against 16.9, 1 x
  // 16384 x 12288 46.7 against 38.6, 8 48.4 against 43.0). 56 Mi weights part most of the sizes measured (a few lie up
  // to 9% on the wrong side: 8 x 24576 x 6144 38.0 against 41.1, 1 x 2560 x 20480 20.0 against 18.3).
  const bool passes = m.cin > kMaxWarps * kPieceK;
  if (m.experts == nullptr && (m.slots > kTokens || (passes && m.rows * m.cin < int64_t{56} << 20))) return launch_matvec_batch(m, stream);
  const KernelArgs ka = {m, make_plan(m)};
  const bool routed = m.experts != nullptr;
  if (ka.p.wide) return routed ? launch_warps<true, true>(ka, stream) : launch_warps<true, false>(ka, stream);
  return routed ? launch_warps<false, true>(ka, stream) : launch_warps<false, false>(ka, stream);
}

}  // namespace lhcal
