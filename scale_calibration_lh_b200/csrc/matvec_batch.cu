// Products of a batch of tokens (up to 64) with one layer's packed NVFP4 weights, or of few tokens
// with many channels and not many rows: y_{i,r} = g * sum_c (q_{r,c} v_{r,c/16}) x_{i,c}.
//
// Decoding is what costs here, so each weight is decoded once for all tokens: to fp16 (q v is exact),
// a row a lane, into tensor memory, where tcgen05.mma takes its 128 x 128 operand from. The
// activations are the other operand, N = 16 to 64 tokens in shared memory: fp16 with a power of two (or
// the E4M3 scale) per token and 128 channels beside them. So the product of 128 channels is read
// back and added to fp32 sums in registers with its scale.
//
// A cluster of up to 8 CTAs takes tiles of 128 rows and splits the channels, so that a CTA's
// activations lie in shared memory, converted once, while its rows go by. Four warpgroups take the
// CTA's blocks of 128 channels in turn, each with operands of its own (64 columns decoded, N of
// sums): while one's product runs, the others decode. Each warp copies its rows' weights into a ring
// of its own (cp.async), a block ahead. Sums meet at a tile's end in a fixed order: the warpgroups'
// through tensor memory, the cluster's through its shared memory.
//
// Measured (us): 17 x 4096 x 12288 E4M3 17.5, 16 x 4096 x 4096 8.5, 32 x 12288 x 4096 22, 64 x 4096 x 4096
// 16.1, 64 x 12288 x 4096 32 (22, 11.0, 29.5, 27.5 and 64 with m16n8k16 products and each weight decoded
// once a warp). Bound by latency: 64 x 12288 x 4096 takes 64 000 cycles with 48% of the issue slots used,
// 12 000 of them until the first activations are there and converted, 24 blocks of 128 channels at 1250,
// and 6 000 to join a tile's sums. Two operands of 64 channels a warpgroup, the next decoded while the
// last is multiplied, gave 18.4 and 33 us: twice the barriers, and the others decode in the meantime anyway.
// Five warpgroups up to N = 32: 19.2 against 17.3 us (a pass of 12 blocks takes them three turns as well).
#include <cooperative_groups.h>

#include "common.cuh"
#include "matvec.cuh"

namespace lhcal {
namespace {

namespace cg = cooperative_groups;

constexpr int kGroups = 4;                 // warpgroups
constexpr int kWarps = 4 * kGroups;
constexpr int kTile = 128;                 // rows of a product: a lane of tensor memory each
constexpr int kChunk = LHCAL_SCALE_BLOCK;  // channels of a product
constexpr int kStepK = 16;                 // of an instruction
constexpr int kColumns = 512;              // of tensor memory, all of it
constexpr int kDecoded = kChunk / 2;       // columns of decoded weights, then N of sums
constexpr int kMaxSmem = 227 * 1024 - 1024;

constexpr int kSlots = 2;                  // blocks of a warp's ring

// A ring slot: weights of a warp's 32 rows (64 bytes each, their 16-byte units exchanged against bank
// conflicts), then their scale codes: 8 bytes a row, or (not WIDE) the 3 words that hold them.
constexpr int kCodesAt = 32 * 64;
__host__ __device__ constexpr int slot_bytes(bool wide) { return kCodesAt + 32 * (wide ? 8 : 12); }

struct Plan {
  int wide, split;          // split: CTAs of a cluster, over the channels
  int tiles, clusters;
  int y_bytes, each;        // of an element of y; tokens of a warp that a CTA of a cluster adds up
  int pass_blocks, passes;  // a pass: the blocks of 128 channels whose activations lie in shared memory
  uint32_t per_block;       // 2^20 / pass_blocks, rounded up: quotients of fewer than 64 pass_blocks are exact
  uint32_t ring, sx;        // bytes: where the rings and the activations' scales begin
};

struct KernelArgs {
  MatvecArgs m;
  Plan p;
};

__device__ __forceinline__ void tmem_store32(uint32_t at, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t at, const float* f) {
  uint32_t r[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(f[i]);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Complete on return.
__device__ __forceinline__ void tmem_load16(uint32_t at, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_load4x4(uint32_t at, uint32_t apart, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%16];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%4, %5, %6, %7}, [%17];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%8, %9, %10, %11}, [%18];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%12, %13, %14, %15}, [%19];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at), "r"(at + apart), "r"(at + 2 * apart), "r"(at + 3 * apart)
      : "memory");
}
__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// d = a b^T, or d += where `add`: a 128 x 16 fp16 in tensor memory, b N x 16 in shared memory.
__device__ __forceinline__ void product(uint32_t d, uint32_t a, uint64_t b, uint32_t shape, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(shape), "r"(static_cast<uint32_t>(add))
      : "memory");
}

// The barrier is arrived at once the products that this thread has issued have ended.
__device__ __forceinline__ void commit_products(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// Into the same place of another CTA's shared memory.
__device__ __forceinline__ void store_cluster(uint32_t at, int rank, float v) {
  asm volatile("{\n\t.reg .b32 there;\n\tmapa.shared::cluster.u32 there, %0, %1;\n\tst.shared::cluster.f32 [there], %2;\n\t}" ::"r"(at),
               "r"(rank), "f"(v)
               : "memory");
}

__device__ __forceinline__ void store_cluster4(uint32_t at, int rank, const float (&v)[4]) {
  asm volatile(
      "{\n\t.reg .b32 there;\n\tmapa.shared::cluster.u32 there, %0, %1;\n\tst.shared::cluster.v4.f32 [there], {%2, %3, %4, %5};\n\t}" ::"r"(at),
      "r"(rank), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3])
      : "memory");
}

// N: tokens, a multiple of 16 at or above their number.
template <int N, bool WIDE>
__global__ void __launch_bounds__(32 * kWarps, 1) matvec_batch_kernel(const KernelArgs ka) {
  constexpr int kSlot = slot_bytes(WIDE);
  constexpr uint32_t kSlab = N * 128;  // bytes of 64 channels of the activations: rows of 128 bytes, swizzled
  // fp32 sums of fp16 products, both operands with their channels consecutive.
  constexpr uint32_t kShape = 1u << 4 | N / 8 << 17 | kTile / 16 << 24;
  // The operand's layout: 128-byte swizzle, 8 rows every 1024 bytes.
  constexpr uint64_t kLayout = 2ull << 61 | 1ull << 46 | static_cast<uint64_t>(1024 / 16) << 32 | 1ull << 16;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t barriers[2 * kGroups];  // a warpgroup's: a product's end, the last ones' where a wait ran out
  __shared__ uint32_t tmem_at;
  __shared__ int failed;
  const MatvecArgs& m = ka.m;
  const Plan& p = ka.p;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0), group = warp >> 2, quarter = warp & 3;  // of the tile's rows
  const int cin = static_cast<int>(m.cin), wstride = cin / 2, cstride = cin / kBlock, blocks = (cin + kChunk - 1) / kChunk;
  const int rank = static_cast<int>(blockIdx.x) % p.split, cluster = static_cast<int>(blockIdx.x) / p.split;
  const int block0 = blocks * rank / p.split, block1 = blocks * (rank + 1) / p.split;
  // Swizzling goes by the address: the activations begin on a 1024-byte boundary.
  const uint32_t raw = static_cast<uint32_t>(__cvta_generic_to_shared(smem_raw)), base = (raw + 1023) & ~1023u;
  const uint32_t ring = base + p.ring + warp * (kSlots * kSlot);
  const uint32_t bar = static_cast<uint32_t>(__cvta_generic_to_shared(barriers + group));
  const uint32_t failed_at = static_cast<uint32_t>(__cvta_generic_to_shared(&failed));
  const uint8_t* const codes_end = m.codes + m.rows * cstride;

  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(&tmem_at))),
                 "n"(kColumns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 0) {
    failed = 0;
    for (int i = 0; i < 2 * kGroups; ++i) barrier_init(static_cast<uint32_t>(__cvta_generic_to_shared(barriers + i)), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }

  // x of a pass to fp16: a half-warp a block of 128 channels of a token, a lane 8 channels.
  constexpr int halves = 2 * kWarps;
  const int v = lane & 15;
  auto stage_x = [&](int pass) {
    constexpr int kAtOnce = 2;
    const int k0 = (block0 + pass * p.pass_blocks) * kChunk, end = min(cin, block1 * kChunk), jobs = m.slots * p.pass_blocks;
    for (int j0 = warp * 2; j0 < jobs; j0 += kAtOnce * halves) {  // converged
      uint4 u[kAtOnce];
      float s[kAtOnce];
      uint32_t at[kAtOnce], s_at[kAtOnce];  // at: 0 where there is nothing
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const int j = j0 + (lane >> 4) + i * halves, n = j * p.per_block >> 20, blk = j - n * p.pass_blocks, k = k0 + blk * kChunk;
        u[i] = make_uint4(0u, 0u, 0u, 0u);
        at[i] = 0;
        if (j >= jobs) continue;
        at[i] = base + (blk * 2 + (v >> 3)) * kSlab + n * 128 + ((v ^ n) & 7) * 16;
        s_at[i] = base + p.sx + (blk * N + n) * 4;
        if (k + v * 8 >= end) continue;
        const int64_t from = n * m.ldx + k + v * 8;
        if (m.xtype == LHCAL_E4M3) {
          const uint2 b = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(m.x) + from));
          u[i].x = b.x;
          u[i].y = b.y;
          if (v == 0) s[i] = __ldg(m.x_scale + (m.scale_block ? static_cast<int64_t>(n) * blocks + k / kChunk : n));
        } else {
          u[i] = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(m.x) + from));
        }
      }
      if (m.xtype == LHCAL_E4M3) {
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
          u[i] = make_uint4(e4m3x2_to_f16(u[i].x), e4m3x2_to_f16(u[i].x >> 16), e4m3x2_to_f16(u[i].y), e4m3x2_to_f16(u[i].y >> 16));
      } else {
        uint32_t top[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
          top[i] = max_bf16x2(max_bf16x2(max_bf16x2(max_bf16x2(0, u[i].x), u[i].y), u[i].z), u[i].w);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1)
#pragma unroll
          for (int i = 0; i < kAtOnce; ++i) top[i] = __vmaxu2(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
          uint32_t up;
          fp16_range(top[i], up, s[i]);
          u[i] = make_uint4(bf16x2_to_f16(u[i].x, up), bf16x2_to_f16(u[i].y, up), bf16x2_to_f16(u[i].z, up),
                            bf16x2_to_f16(u[i].w, up));
        }
      }
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        if (at[i] == 0) continue;
        sts128(at[i], u[i]);
        if (v == 0) sts_float(s_at[i], s[i]);
      }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the products read them
  };

  // The weights of the warp's rows, block by block: the next to copy. A lane copies 16 bytes of each
  // 8th row, and (WIDE) 4 codes of each 16th.
  int next_tile = cluster, next_pass = 0, next_c = group;
  uint32_t to = ring;  // its slot
  const uint8_t* const w_lane = m.packed + static_cast<int64_t>(quarter * 32 + (lane >> 2)) * wstride + (lane & 3) * 16;
  const uint8_t* const c_lane = m.codes + static_cast<int64_t>(quarter * 32 + (lane >> 1)) * cstride + (lane & 1) * 4;
  const uint32_t w_at = (lane >> 2) * 64 + ((lane ^ lane >> 3) & 3) * 16;
  auto copy_next = [&]() {
    __syncwarp();  // every lane has read the slot
    const int q = block0 + next_pass * p.pass_blocks + next_c;
    if (next_tile < p.tiles && next_c < p.pass_blocks && q < block1) {
      const int64_t row = static_cast<int64_t>(next_tile) * kTile;
      const int rows = static_cast<int>(imin64(m.rows - row - quarter * 32, 32)), room = cin - q * kChunk;  // of the warp, of the block on
      const uint8_t *w = w_lane + row * wstride + q * (kChunk / 2), *c = c_lane + row * cstride + q * (kChunk / kBlock);
      if (WIDE && rows == 32 && room >= kChunk) {
#pragma unroll
        for (int i = 0; i < 4; ++i) copy_async<16>(to + w_at + i * 512, w + i * (8 * wstride));
#pragma unroll
        for (int i = 0; i < 2; ++i) copy_word_async(to + kCodesAt + i * 128 + lane * 4, c + i * (16 * cstride));
      } else {
        for (int i = 0; i < 4; ++i, w += 8 * wstride) {
          if ((lane >> 2) + 8 * i >= rows) break;
          const uint32_t w_to = to + w_at + i * 512;
          if (WIDE) {
            if ((lane & 3) * 32 < room) copy_async<16>(w_to, w);
          } else {
            if ((lane & 3) * 32 < room) copy_async<8>(w_to, w);
            if ((lane & 3) * 32 + 16 < room) copy_async<8>(w_to + 8, w + 8);
          }
        }
        if (WIDE) {
          for (int i = 0; i < 2; ++i) {
            const bool on = (lane >> 1) + 16 * i < rows && (lane & 1) * 64 < room;
            copy_word_async(to + kCodesAt + i * 128 + lane * 4, on ? c + i * (16 * cstride) : m.codes, on ? 4 : 0);
          }
        } else {
          // The three aligned words of a row's 8 codes, from the first that holds one of them; no byte
          // past the codes' end is read.
          c = m.codes + (row + quarter * 32) * cstride + q * (kChunk / kBlock);
          for (int i = 0; i < 3; ++i) {
            const int j = i * 32 + lane, r = j / 3;
            const uint8_t* from = c + static_cast<int64_t>(r) * cstride;
            from += (j - r * 3) * 4 - static_cast<int>(reinterpret_cast<uintptr_t>(from) & 3);
            const int64_t valid = codes_end - from;
            const bool on = r < rows && valid > 0;
            copy_word_async(to + kCodesAt + j * 4, on ? from : m.packed, on ? static_cast<int>(imin64(4, valid)) : 0);
          }
        }
      }
    }
    commit_copies();
    to = to + kSlot == ring + kSlots * kSlot ? ring : to + kSlot;
    next_c += kGroups;
    if (next_c >= p.pass_blocks) {
      next_c = group;
      if (++next_pass == p.passes) {
        next_pass = 0;
        next_tile += p.clusters;
      }
    }
  };

  for (int d = 0; d < kSlots - 1; ++d) copy_next();
  uint32_t at = ring, phase = 0, tmem = 0;  // the slot to use; the next product's parity; the warp's lanes of tensor memory
  for (int tile = cluster; tile < p.tiles; tile += p.clusters) {
    float acc[N];
#pragma unroll
    for (int n = 0; n < N; ++n) acc[n] = 0.f;
    for (int pass = 0; pass < p.passes; ++pass) {
      if (tile == cluster || p.passes > 1) {
        if (tile != cluster || pass > 0) __syncthreads();  // the last activations are read
        stage_x(pass);
        tmem_fence_before();
        __syncthreads();
        tmem_fence_after();
        tmem = tmem_at + (quarter * 32 << 16);
      }
      const uint32_t decoded = tmem + group * (kColumns / kGroups), sums = decoded + kDecoded;
      const uint32_t x = base + p.sx;
      int pending = -1;  // the block whose product runs
      for (int c = group;; c += kGroups) {
        const bool in = c < p.pass_blocks, on = in && block0 + pass * p.pass_blocks + c < block1;
        uint32_t codes[2] = {};  // the row's 8
        auto decode = [&](int h) {  // 64 channels
          uint32_t a[32];
          const uint32_t s[2] = {e4m3x2_to_f16(codes[h]), e4m3x2_to_f16(codes[h] >> 16)};
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint4 w4 = lds128(at + lane * 64 + ((h * 2 + u) ^ (lane >> 1 & 3)) * 16);
            const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t f[4];
              e2m1x8_to_f16(w[i], f);
              const uint32_t by = __byte_perm(s[u], 0, i < 2 ? 0x1010 : 0x3232);
#pragma unroll
              for (int k = 0; k < 4; ++k) a[u * 16 + i * 4 + k] = hmul2(f[k], by);
            }
          }
          tmem_store32(decoded + h * 32, a);
        };
        auto multiply = [&]() {
          tmem_store_wait();
          tmem_fence_before();
          asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory");
          if (quarter == 0 && lane == 0) {
            tmem_fence_after();
            const uint32_t from = base + c * 2 * kSlab;
#pragma unroll
            for (int k = 0; k < kChunk / kStepK; ++k)
              product(sums, decoded + k * (kStepK / 2), kLayout | (from + k / 4 * kSlab + k % 4 * (kStepK * 2)) >> 4, kShape, k > 0);
            commit_products(bar);
          }
          __syncwarp();
        };
        if (in) {
          wait_copies<kSlots - 2>();  // this block's
          __syncwarp();               // every lane's copies
        }
        if (on) {
          if (WIDE) {
            const uint2 u = lds64(at + kCodesAt + lane * 8);
            codes[0] = u.x;
            codes[1] = u.y;
          } else {
            const int q = block0 + pass * p.pass_blocks + c;
            const int64_t row = static_cast<int64_t>(tile) * kTile + quarter * 32 + lane;
            const uint32_t shift = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(m.codes) + row * cstride + q * (kChunk / kBlock)) % 4 * 8;
            const uint32_t from = at + kCodesAt + lane * 12, u0 = lds32(from), u1 = lds32(from + 4), u2 = lds32(from + 8);
            codes[0] = __funnelshift_r(u0, u1, shift);
            codes[1] = __funnelshift_r(u1, u2, shift);
            const int have = cstride - q * (kChunk / kBlock);  // past cin lie other rows' codes, or none
            if (have < 4) codes[0] &= (1u << 8 * have) - 1;
            if (have < 8) codes[1] = have <= 4 ? 0u : codes[1] & ((1u << 8 * (have - 4)) - 1);
          }
        }
        if (pending >= 0) {
          barrier_wait(bar, phase ^ 1, &failed);
          __syncwarp();
          tmem_fence_after();
#pragma unroll
          for (int n = 0; n < N; n += 16) {
            uint32_t r[16];
            tmem_load16(sums + n, r);
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              const uint4 s = lds128(x + (pending * N + n + i) * 4);
              acc[n + i] = fmaf(__uint_as_float(s.x), __uint_as_float(r[i]), acc[n + i]);
              acc[n + i + 1] = fmaf(__uint_as_float(s.y), __uint_as_float(r[i + 1]), acc[n + i + 1]);
              acc[n + i + 2] = fmaf(__uint_as_float(s.z), __uint_as_float(r[i + 2]), acc[n + i + 2]);
              acc[n + i + 3] = fmaf(__uint_as_float(s.w), __uint_as_float(r[i + 3]), acc[n + i + 3]);
            }
          }
          pending = -1;
        }
        if (!in) break;
        if (on) {
          decode(0);
          decode(1);
        }
        copy_next();
        if (on) {
          multiply();
          pending = c;
          phase ^= 1;
        }
        at = at + kSlot == ring + kSlots * kSlot ? ring : at + kSlot;
      }
    }
    // Join the warpgroups' sums through tensor memory: a warp adds up N / 4 tokens of its 32 rows.
    // Then the cluster's: the warps of the same place exchange tokens through the ring slot that each
    // read last, and each rank adds up some of the warp's tokens.
    const uint32_t mine = tmem + kDecoded, free_slot = (at == ring ? ring + kSlots * kSlot : at) - kSlot;
#pragma unroll
    for (int n = 0; n < N; n += 16) tmem_store16(mine + group * (kColumns / kGroups) + n, acc + n);
    tmem_store_wait();
    tmem_fence_before();
    if (p.split > 1)
      cg::this_cluster().sync();
    else
      __syncthreads();
    tmem_fence_after();
    const float gs = __ldg(m.g);
    const float lost = __uint_as_float(lds32(failed_at));  // 0, or NaN for good once a wait of the CTA ran out
    const int64_t row = static_cast<int64_t>(tile) * kTile + quarter * 32 + lane;
    uint8_t* const y_lane = static_cast<uint8_t*>(m.y) + (group * 4 * m.ldy + row) * p.y_bytes;
    auto put = [&](int j, float sum) {  // the warp's token j
      const int n = (j >> 2) * 16 + (j & 3);
      if (n + group * 4 >= m.slots || row >= m.rows) return;
      uint8_t* const y = y_lane + n * (m.ldy * p.y_bytes);
      if (p.y_bytes == 4)
        *reinterpret_cast<float*>(y) = sum * gs;
      else
        *reinterpret_cast<__nv_bfloat16*>(y) = __float2bfloat16(sum * gs);
    };
    const int each = p.each;  // tokens that a rank adds up
    int to_rank = 0, place = 0;
#pragma unroll
    for (int n = 0; n < N; n += 16) {
      uint32_t r[16];
      float sum[4];
      tmem_load4x4(mine + n + group * 4, kColumns / kGroups, r);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        sum[i] = ((__uint_as_float(r[i]) + __uint_as_float(r[4 + i])) + (__uint_as_float(r[8 + i]) + __uint_as_float(r[12 + i]))) + lost;
      if (p.split == 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) put(n / 4 + i, sum[i]);
      } else if (N == 64 && each >= 4) {  // whole to one rank
        store_cluster4(free_slot + ((rank * each + place) * 32 + lane * 4) * 4, to_rank, sum);
        place += 4;
        if (place == each) place = 0, ++to_rank;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          store_cluster(free_slot + ((rank * each + place) * 32 + lane) * 4, to_rank, sum[i]);
          if (++place == each) place = 0, ++to_rank;
        }
      }
    }
    tmem_fence_before();
    if (p.split > 1) {
      cg::this_cluster().sync();
      const int have = min(each, N / 4 - rank * each);
      for (int k = 0; k < have; ++k) {
        const uint32_t from = free_slot + (N == 64 && each >= 4 ? (k & ~3) * 128 + lane * 16 + (k & 3) * 4 : k * 128 + lane * 4);
        float part[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) part[i] = i < p.split ? __uint_as_float(lds32(from + i * each * 128)) : 0.f;
        put(rank * each + k, ((part[0] + part[1]) + (part[2] + part[3])) + ((part[4] + part[5]) + (part[6] + part[7])));
      }
      __syncwarp();  // before the next copies
    } else {
      __syncthreads();
    }
    tmem_fence_after();
  }
  // Products that no wait saw end still read the CTA's shared memory and write its tensor memory.
  if (lds32(failed_at) != 0) {
    if (quarter == 0 && lane == 0) {
      commit_products(bar + 8 * kGroups);
      for (int i = 0; i < kDrainLimit && !barrier_poll(bar + 8 * kGroups, 0); ++i) {}
    }
    __syncwarp();
    __syncthreads();
  }
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_at), "n"(kColumns) : "memory");
}

template <int N>
Plan make_plan(const MatvecArgs& m) {
  Plan best = {};
  double best_cost = 0;
  const bool wide = m.cin % 64 == 0 && aligned(m.packed, 16) && aligned(m.codes, 4);
  const int blocks = static_cast<int>(ceil_div(m.cin, kChunk)), tiles = static_cast<int>(ceil_div(m.rows, kTile));
  for (int split = 1; split <= 8 && split <= blocks; split *= 2) {
    Plan p = {};
    p.wide = wide;
    p.split = split;
    p.tiles = tiles;
    p.y_bytes = m.ytype == LHCAL_F32 ? 4 : 2;
    p.each = static_cast<int>(ceil_div(N / 4, split));
    // Clusters that are resident at once (a GPC's SMs are not a multiple of 8): 15, 33 and 74 were.
    const int resident = split == 8 ? 15 : split == 4 ? 32 : split == 2 ? 74 : kNumSms;
    p.clusters = tiles < resident ? tiles : resident;
    const int own = static_cast<int>(ceil_div(blocks, split)), each = static_cast<int>(ceil_div(tiles, p.clusters));
    const int ring = kWarps * kSlots * slot_bytes(wide);
    const int room = (kMaxSmem - 1024 - ring) / (N * (kChunk * 2 + 4));
    p.passes = static_cast<int>(ceil_div(own, room));
    p.pass_blocks = static_cast<int>(ceil_div(own, p.passes));
    p.ring = static_cast<uint32_t>(p.pass_blocks * N * kChunk * 2);
    p.sx = p.ring + static_cast<uint32_t>(ring);
    p.per_block = (1u << 20) / static_cast<uint32_t>(p.pass_blocks) + 1;
    // In products of a block: the CTA's blocks, its activations' conversion and a tile's join. 32 x 12288 x
    // 4096 takes 21.8 us with the 4 CTAs that it finds, 25.5 with fewer; 64 x 4096 x 4096 16.5 and 8 CTAs
    // would be 15 clusters for 32 tiles.
    const double cost = static_cast<double>(each) * own + 0.008 * N * own * (p.passes > 1 ? each : 1) + (split > 1 ? 2. * each : 0.);
    if (best.tiles == 0 || cost < best_cost) {
      best = p;
      best_cost = cost;
    }
  }
  return best;
}

template <int N, bool WIDE>
lhcal_status launch(const KernelArgs& ka, cudaStream_t stream) {
  auto* fn = matvec_batch_kernel<N, WIDE>;
  const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail(LHCAL_ERR_CUDA, "matvec: %s", cudaGetErrorString(e));
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ka.p.clusters * ka.p.split));
  cfg.blockDim = dim3(32 * kWarps);
  // All of it, so that no SM holds two CTAs that use tensor memory: clusters that each hold a part of
  // what the other waits for would wait for good.
  cfg.dynamicSmemBytes = kMaxSmem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = static_cast<unsigned>(ka.p.split);
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t launched = cudaLaunchKernelEx(&cfg, fn, ka);
  if (launched != cudaSuccess) {
    cudaGetLastError();
    return fail(LHCAL_ERR_CUDA, "matvec: %s", cudaGetErrorString(launched));
  }
  return check_launch("matvec");
}

template <int N>
lhcal_status launch_n(const MatvecArgs& m, cudaStream_t stream) {
  const KernelArgs ka = {m, make_plan<N>(m)};
  return ka.p.wide ? launch<N, true>(ka, stream) : launch<N, false>(ka, stream);
}

}  // namespace

lhcal_status launch_matvec_batch(const MatvecArgs& m, cudaStream_t stream) {
  switch ((m.slots + 15) / 16) {
    case 1: return launch_n<16>(m, stream);
    case 2: return launch_n<32>(m, stream);
    case 3: return launch_n<48>(m, stream);
    default: return launch_n<64>(m, stream);
  }
}

}  // namespace lhcal
