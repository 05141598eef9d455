"""What no run of the paged attention shows without an expired wait: the copies that its loading warps wait for before the CTA ends,
counted on the host with the code that the kernel counts with."""
import os
import re
import subprocess

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_attention_indexer_e4m3_gb300", "csrc")

# Loaders, each of which issues every kStep-th tile of blocks of kTiles and gives up before its n-th (chosen at random, none further
# ahead than the ring allows): what is waited for is the last tile of each place, in the phase that it fills.
RING = r"""
#include <cstdio>
#include <cstdlib>
#include <map>
#include "tile_ring.h"
template <uint32_t kRing, uint32_t kStep, uint32_t kTiles>
int check() {
  for (int turn = 0; turn < 20000; ++turn) {
    const uint32_t near = std::rand() % 40;
    uint32_t issued[kStep];
    std::map<uint32_t, uint32_t> want, got;
    for (uint32_t w = 0; w < kStep; ++w) {
      const uint32_t most = kRing / kStep + 1, n = near + std::rand() % most;
      dsa::TileRing<kRing, kStep> ring(w);
      for (uint32_t block = 0; ring.issued < n; ++block)
        for (uint32_t m = 0; m < kTiles && ring.issued < n; m += kStep) {
          const uint32_t tile = block * kTiles + m + w, place = tile % kRing;
          if (ring.at != place || ring.round != tile / kRing) return 1;
          if (want.count(place) == 0 || want[place] < tile) want[place] = tile;
          ring.next();
        }
      issued[w] = ring.issued;
    }
    bool twice = false;
    dsa::tiles_in_flight<kRing, kStep>(issued, [&](uint32_t place, uint32_t parity) { twice |= !got.emplace(place, parity).second; });
    for (auto& t : want) t.second = t.second / kRing & 1u;
    if (twice || got != want) return std::printf("ring %u step %u\n", kRing, kStep), 1;
  }
  return 0;
}
int main() { return check<8, 1, 1>() || check<5, 1, 1>() || check<5, 1, 2>() || check<9, 4, 4>() || check<9, 1, 4>(); }
"""


def test_copies_in_flight_are_counted(tmp_path):
    (tmp_path / "ring.cpp").write_text(RING)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", f"-I{SRC}", str(tmp_path / "ring.cpp"), "-o", str(tmp_path / "ring")], check=True)
    subprocess.run([str(tmp_path / "ring")], check=True)


def test_copies_land_before_the_end():
    """Each tile is counted behind its copies; all counts are written before the roles meet, and behind that, where some role gave
    up, the copies are waited for."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(SRC, "paged_attn_kernel.cuh")).read())
    load = text[text.index("} else if (warp >= kPgFirstLoad) {"):text.index("} else if (warp < 2) {")]
    tiles = load[load.index("for (int m0 = 0;"):]
    assert re.search(r"tma_load_2d_if\([^;]*;\s*\}\s*ring\.next\(\);", tiles) and load.count("ring.next()") == 1
    assert re.search(r"issued_s\[loader\] = ring\.issued;\s*if \(loader == 0\) issued_s\[L::kLoaders\] = nq;\s*\}\s*$", load)
    assert "return" not in load.replace("return __all_sync(", "")
    kernel = text[text.index("paged_attn_kernel("):text.index("paged_join_kernel(")]
    end = kernel[kernel.rindex("__syncthreads();"):]
    assert "if (*abort_flag != 0 && warp == kPgFirstLoad) {" in end and end.index("tiles_in_flight<") < end.index("tmem_dealloc")


def test_no_early_end_leaves_the_join_stale_entries():
    """A CTA that ends before the plan (its shared memory lies elsewhere than expected) has emptied its entry of the shared units,
    behind the stream's earlier work, which may still read the workspace."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(SRC, "paged_attn_kernel.cuh")).read())
    kernel = text[text.index("paged_attn_kernel("):text.index("paged_join_kernel(")]
    start = kernel[:kernel.index("mbar_init(")]
    assert start.count("return;") == 1
    early = start[start.index("1023u"):start.index("return;")]
    assert early.index("wait_stream();") < early.index("p.shared[blockIdx.x] = make_int4(0, 0, 0, 0);")
    assert "return;" not in kernel[kernel.index("mbar_init("):]
