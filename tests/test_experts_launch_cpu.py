"""How the experts' calls are cut into launches, seen through a stand-in for the CUDA
runtime that writes launches down. Nothing runs on a GPU."""

import os
import subprocess
import sys

import pytest

from latent_moe_output_gb300 import binding

FAKE_RUNTIME = r"""
#include <cuda_runtime_api.h>
#include <stdio.h>
#include <stdlib.h>
static unsigned cluster_of(const cudaLaunchConfig_t* c) {
  for (unsigned i = 0; i < c->numAttrs; ++i)
    if (c->attrs[i].id == cudaLaunchAttributeClusterDimension)
      return c->attrs[i].val.clusterDim.x;
  return 1;
}
static int accept_all(void) { return 0; }
cudaError_t cudaGetDevice(int* d) { *d = 0; return 0; }
cudaError_t cudaDeviceGetAttribute(int* v, enum cudaDeviceAttr attr, int dev) {
  *v = attr == 75 ? 10 : attr == 76 ? 3 : attr == 16 ? 152 : attr == 97 ? 232448 : 0;
  return 0;
}
cudaError_t cudaGetSymbolAddress(void** p, const void* symbol) { *p = (void*)4096; return 0; }
cudaError_t cudaGetDriverEntryPointByVersion(const char* name, void** fn, unsigned v,
                                             unsigned long long flags,
                                             enum cudaDriverEntryPointQueryResult* result) {
  *fn = (void*)accept_all;
  *result = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void* fn, enum cudaFuncAttribute attr, int value) {
  return 0;
}
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void* fn, const cudaLaunchConfig_t* c) {
  /* of 2, 4, 6 and 8 CTAs */
  static const char* const names[] = {"CLUSTERS2", "CLUSTERS4", "CLUSTERS6", "CLUSTERS8"};
  *n = atoi(getenv(names[cluster_of(c) / 2 - 1]));
  return 0;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* fn, void** args) {
  fprintf(stderr, "launch %u %u %u %u\n", c->gridDim.x, cluster_of(c), c->blockDim.x,
          (unsigned)c->dynamicSmemBytes);
  return 0;
}
"""

CHILD = r"""
import ctypes, sys
lib = ctypes.CDLL(sys.argv[1])
a = [ctypes.c_void_p(0x1000000000 * (i + 1)) for i in range(8)]
null = ctypes.c_void_p(0)
for call in sys.argv[2:]:
    name, *n = call.split(",")
    n = [int(v) for v in n]
    if name == "weights":    # N, M, C: gradient of one matrix
        N, M, C = n
        st = lib.latent_tail_expert_matmul_backward(a[0], a[1], null, null, null, a[2], N, 1, M, C,
                                                    null)
    elif name == "gated":    # N, E, F, C, kind of kept projections
        N, E, F, C, kind = n
        st = lib.latent_tail_expert_gated(a[0], a[1], a[2], a[3], a[4] if kind else null,
                                          a[5] if kind == 2 else null, N, E, F, C, 0, kind, null)
    print(int(st))
"""

RESIDENT = (76, 36, 23, 15)  # a GB300's: clusters of 2, 4, 6 and 8 CTAs that are resident at once


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    from latent_moe_output_gb300 import build

    build.build()
    where = tmp_path_factory.mktemp("runtime")
    (where / "fake.c").write_text(FAKE_RUNTIME)
    fake = where / "fake.so"
    subprocess.run(["gcc", "-shared", "-fPIC", f"-I{build.cuda_home() / 'include'}", "-o",
                    str(fake), str(where / "fake.c")], check=True)

    def child(*calls, clusters=RESIDENT):
        """(grid, cluster, block, shared memory) of each launch"""
        env = dict(os.environ, LD_PRELOAD=str(fake),
                   **{f"CLUSTERS{2 * (i + 1)}": str(n) for i, n in enumerate(clusters)})
        r = subprocess.run([sys.executable, "-c", CHILD, str(binding.library_path()), *calls],
                           capture_output=True, text=True, env=env)
        assert r.returncode == 0, r.stderr
        assert r.stdout.split() == ["0"] * len(calls)
        return [tuple(int(v) for v in line.split()[1:]) for line in r.stderr.splitlines()
                if line.startswith("launch ")]

    return child


@pytest.mark.parametrize("N,M,C,tiles,resident4", [
    (65536, 512, 768, 12, 15), (65536, 256, 1920, 15, 15), (16384, 3840, 128, 15, 15),
    (65536, 256, 2048, 16, 16), (65536, 1024, 512, 16, 18), (16384, 4096, 128, 16, 19)])
def test_a_sum_over_many_rows_is_shared_as_it_was_cut(run, N, M, C, tiles, resident4):
    """Tiles of 256 x 128, each shared by four pairs: the ring holds the three other pairs'
    sums, 3 * 128 * 512 bytes, in its three stages of 64 KB."""
    grid, cluster, _, smem = run(f"weights,{N},{M},{C}", clusters=RESIDENT[:3] + (resident4,))[0]
    assert (cluster, grid) == (8, tiles * 8)
    assert smem >= 3 * 128 * 512


@pytest.mark.parametrize("N,F,C", [(100, 256, 2048), (128, 2048, 7168), (65, 512, 4096)])
def test_what_is_kept_does_not_change_the_order_of_a_sum(run, N, F, C):
    """The same pairs per sum whether projections are kept or not."""
    launches = run(*(f"gated,{N},1,{F},{C},{kind}" for kind in range(3)))
    assert len({launch[:2] for launch in launches}) == 1 and launches[0][1] > 2


@pytest.mark.parametrize("E,stages", [(1, 3), (254, 3), (256, 3), (297, 3), (298, 2), (1024, 2)])
def test_stages_beside_what_is_kept(run, E, stages):
    """64 KB per stage beside the chunk buffers of projections kept in bf16 and the table."""
    _, _, _, smem = run(f"gated,65536,{E},1024,2048,1")[0]
    table = ((E + 1) * 12 + 15) // 16 * 16
    assert smem == 1024 + stages * 65536 + 2 * 15360 + table
    assert smem + 512 <= 232448
