"""How an eviction's selection shares a request's slots over the thread blocks
of a cluster, walked through on the host over lengths, regions that always stay
and cluster sizes: every access that the kernel derives from a share lies inside
the block's keys, sixteen bytes at a time.  No device."""
import ctypes
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mtp_self_speculative_gb300", "csrc")

# walk(lo, hi, table, out): lengths lo .. hi - 1 in a table of `table` slots; the number of faults, the first one in out
SOURCE = r"""
#include "mtp_kv_evict_range.h"
using namespace mtp;
extern "C" long long walk(int lo, int hi, int table, int most_cached, int* out) {
  const int sinks[] = {0, 1, 2, 3, 4, 5, 127, 128, 130, 700}, recents[] = {0, 1, 2, 3, 4, 5, 8, 100, 129, 1500};
  long long faults = 0;
  for (int C = 1; C <= 4; C *= 2) {
    // the keys that a block's shared memory holds, as the launch sizes them
    const long long part = evict_share(table, C) + 4;
    const int cached = (int)(part < most_cached ? part : most_cached) & ~3;
    for (int L = lo; L < hi; ++L)
      for (int sink : sinks)
        for (int recent : recents) {
          if (sink + recent >= L) continue;
          int slots = 0, candidates = 0;
          bool ok = true;
          for (int c = 0; c < C; ++c) {
            const EvictRange r = evict_range(L, sink, recent, C, c);
            ok &= r.s0 == slots && r.s1 >= r.s0;           // shares follow one another
            slots = r.s1;
            if (r.c0 < r.c1) {
              ok &= r.c0 == sink + candidates && r.c0 >= r.s0 && r.c1 <= r.s1;
              candidates += r.c1 - r.c0;
            }
            // the loops over fours: t = f0, f0 + 4, .. below c1
            if (r.f0 < r.c1) {
              ok &= r.f0 >= r.s0 && (r.f0 - r.s0) % 4 == 0 && r.f0 % 4 == 0 && r.f0 <= r.c0 && r.c0 < r.f0 + 4;
              const int last = r.f0 + (r.c1 - 1 - r.f0) / 4 * 4;
              if (cached < most_cached) ok &= last - r.s0 + 4 <= cached;
              ok &= (last + 3) / 16 == last / 16;          // four slots of one cache block
            }
          }
          ok &= slots == L && candidates == L - sink - recent;
          if (!ok && !faults++) { out[0] = C; out[1] = L; out[2] = sink; out[3] = recent; }
        }
  }
  return faults;
}
"""


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("range")
    (d / "walk.cpp").write_text(SOURCE)
    lib = str(d / "walk.so")
    subprocess.run([cxx, "-std=c++17", "-O2", "-shared", "-fPIC", "-I" + CSRC, str(d / "walk.cpp"), "-o", lib], check=True)
    f = ctypes.CDLL(lib).walk
    f.restype, f.argtypes = ctypes.c_longlong, [ctypes.c_int] * 4 + [ctypes.POINTER(ctypes.c_int)]
    return f


@pytest.mark.parametrize("lo,hi,table", [(1, 2600, 16384), (8000, 8300, 8304), (16300, 16385, 16384), (69900, 70100, 70112),
                                         (196000, 196400, 196608), (2 ** 30 - 40, 2 ** 30 + 1, 2 ** 30)])
def test_shares_of_a_cluster_stay_inside_their_keys(walk, lo, hi, table):
    out = (ctypes.c_int * 4)()
    n = walk(lo, hi, table, 49152, out)
    assert n == 0, "%d of them, the first: cluster %d, length %d, sink %d, recent %d" % ((n,) + tuple(out))
