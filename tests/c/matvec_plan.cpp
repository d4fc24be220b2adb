// Checks the layout of lhcal_matvec's products over the sizes that it takes, without a GPU: prints the first
// sizes that break each property, and how many did. With arguments (routed slots groups rows cin, in turn):
// prints the layout of each.
#include <cstdio>
#include <cstdlib>
#include <map>
#include <string>

#include "matvec_plan.cuh"

using namespace lhcal;

namespace {

std::map<std::string, long> broken;

void expect(bool ok, const char* what, const MatvecSizes& m, const MatvecPlan& p) {
  if (ok || broken[what]++ > 0) return;
  std::printf("%s: slots %d groups %d rows %lld cin %lld routed %d: wk %d wr %d stages %d room %d list %u smem %u\n", what,
              m.slots, m.groups, (long long)m.rows, (long long)m.cin, m.routed, p.wk, p.wr, p.stages, p.room, p.list, p.smem);
}

void check(const MatvecSizes& m) {
  const MatvecPlan p = make_matvec_plan(m);
  expect(p.wk >= 1 && p.wr >= 1 && p.wk * p.wr <= kMaxWarps, "warps", m, p);
  expect(p.wk * p.passes * int64_t{kPieceK} >= m.cin, "channels", m, p);
  expect(p.passes == 1 || p.wr == 1, "passes", m, p);
  expect(p.stages >= 2 && p.stages <= kMaxStages && p.wr <= p.stages, "stages", m, p);
  expect(p.stages % p.wr == 0, "stage owners", m, p);
  expect(p.smem <= uint32_t{kMaxSmem - kStaticSmem}, "shared memory", m, p);
  expect(p.room >= kTile * kTokens, "room", m, p);
  // Copies start on 16-byte boundaries; reads of the last stage's last row stay inside.
  expect(p.stage % 128 == 0 && p.codes_at % 16 == 0, "stage alignment", m, p);
  const uint32_t last = (p.stages - 1) * p.stage, k = p.wk - 1;
  expect(last + 15 * p.w_pitch + k * (kPieceK / 2) + 3 * 16 + kXBlock / 2 + 16 + 8 <= p.smem, "weights read", m, p);
  expect(last + p.codes_at + 15 * p.c_pitch + k * (kPieceK / LHCAL_BLOCK) + 15 + 16 <= p.smem, "codes read", m, p);
  expect(p.red % 16 == 0, "sums", m, p);
  // The slots' order, the entries, the experts, the counts' scan (8-byte pairs) and the work: `most` words each.
  const uint32_t most = m.slots < 64 ? 64 : (m.slots + 31) & ~31u;
  expect(!m.routed || p.list % 16 == 0, "list alignment", m, p);
  expect(!m.routed || (p.list + 3 * most * 4) % 8 == 0, "scan alignment", m, p);
  expect(!m.routed || p.list >= (m.groups / 2u + 1) * 4, "counts", m, p);
  expect(!m.routed || p.list >= p.red + 2u * p.wk * p.room * 4, "sums below the lists", m, p);
  expect(!m.routed || p.smem >= p.list + (5 * most + 1) * 4, "lists", m, p);
}

}  // namespace

int main(int argc, char** argv) {
  if (argc > 1) {
    for (int i = 1; i + 4 < argc; i += 5) {
      const int64_t rows = std::atoll(argv[i + 3]), cin = std::atoll(argv[i + 4]);
      const MatvecPlan p = make_matvec_plan(
          {std::atoi(argv[i]) != 0, cin % 64 == 0, std::atoi(argv[i + 1]), 1, std::atoi(argv[i + 2]), rows, cin, 148});
      std::printf("%d %d %d\n", p.wk, p.wr, p.stages);
    }
    return 0;
  }
  const int64_t cins[] = {16, 32, 48, 64, 96, 128, 256, 272, 512, 768, 784, 1024, 1040, 1296, 1536, 2080, 2448, 2560, 2576,
                          4096, 5120, 5136, 6144, 12288, 20000, 262144, 1048560};
  const int64_t many_rows[] = {1, 2, 7, 16, 32, 64, 100, 128, 1280, 5000, 40000, 467200, 2147483647};
  const int32_t many_slots[] = {1, 2, 8, 9, 32, 33, 37, 64, 65, 80, 500, 640, 1023, 1024};
  long n = 0;
  for (int64_t cin : cins)
    for (int64_t rows : many_rows) {
      for (int32_t slots = 1; slots <= kTokens; ++slots, ++n) check({false, cin % 64 == 0, slots, 1, 1, rows, cin, 148});
      for (int32_t slots : many_slots)
        for (int32_t groups = 1; groups <= 65535; groups += groups < 600 ? 1 : 997, ++n)
          check({true, cin % 64 == 0, slots, 1, groups, rows, cin, 148});
    }
  for (int64_t cin = 16; cin <= 6000; cin += 16)  // every channel count of one pass
    for (int64_t rows : many_rows)
      for (int32_t slots : {1, 8, 640}) {
        check({false, cin % 64 == 0, slots < 8 ? 1 : 8, 1, 1, rows, cin, 148});
        check({true, cin % 64 == 0, slots, 1, 512, rows, cin, 148});
        n += 2;
      }
  for (int32_t groups = 1; groups <= 65535; ++groups, ++n) check({true, true, 64, 1, groups, 32, 128, 148});  // every number of experts
  for (const auto& b : broken)
    if (b.second > 0) std::printf("%s: %ld of %ld\n", b.first.c_str(), b.second, n);
  std::printf("checked %ld\n", n);
  return 0;
}
