"""What a call sets up on its device, seen through a stand-in for the CUDA runtime.

A child process loads the library with a preloaded shared object that answers the
runtime's calls, writes down which kernels are configured and refuses the ones named in
its environment. Nothing runs on a GPU."""

import os
import subprocess
import sys

import pytest

from latent_moe_output_gb300 import binding

FAKE_RUNTIME = r"""
#define _GNU_SOURCE
#include <dlfcn.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>
static int accept_all(void) { return 0; }
int cudaGetDevice(int* d) { *d = 0; return 0; }
int cudaDeviceGetAttribute(int* v, int attr, int dev) {
  *v = attr == 75 ? 10 : attr == 76 ? 3 : attr == 16 ? 152 : attr == 97 ? 232448 : 0;
  return 0;
}
int cudaGetSymbolAddress(void** p, const void* symbol) { *p = (void*)4096; return 0; }
int cudaGetDriverEntryPointByVersion(const char* name, void** fn, unsigned v,
                                     unsigned long long flags, int* result) {
  *fn = (void*)accept_all;
  *result = 0;
  return 0;
}
int cudaLaunchKernelExC(const void* cfg, const void* fn, void** args) { return 0; }
int cudaMemsetAsync(void* p, int v, size_t n, void* stream) { return 0; }
int cudaFuncSetAttribute(const void* fn, int attr, int value) {
  Dl_info info;
  char at[32];
  const char* refused = getenv("REFUSED_KERNELS");
  dladdr(fn, &info);
  snprintf(at, sizeof at, "k%lx,", (unsigned long)((const char*)fn - (char*)info.dli_fbase));
  fprintf(stderr, "%s", at);
  return refused != NULL && strstr(refused, at) != NULL ? 1 : 0;
}
"""

CHILD = r"""
import ctypes, sys
lib = ctypes.CDLL(sys.argv[1])
F, S = ctypes.c_float, ctypes.c_size_t
a = [ctypes.c_void_p(0x10000000 + 0x4000000 * i) for i in range(13)]
calls = dict(
    tail=lambda: lib.latent_tail_forward(a[0], a[1], a[2], a[3], a[4], 1, 4, 64, 64, F(1e-6),
                                         a[5], S(1 << 20), None),
    dispatch=lambda: lib.latent_tail_dispatch(a[0], a[1], a[2], a[3], a[4], a[5], 1000, 4, 16, 64,
                                              a[6], S(1 << 20), None),
    combine=lambda: lib.latent_tail_combine(a[0], a[1], a[2], a[3], 10, 4, 64, None),
    matvec4=lambda: lib.latent_tail_expert_matvec4(a[0], a[1], a[2], a[3], a[4], 4, 4, 16, 64, 32,
                                                   None),
    norm=lambda: lib.latent_tail_residual_norm(a[0], a[1], a[2], a[3], a[4], a[5], a[6], 4, 64, 2,
                                               0, F(1), F(1e-6), None))
print(" ".join(str(calls[name]()) for name in sys.argv[2:]))
"""

OWN = ["tail", "dispatch", "matvec4", "norm"]  # combine needs nothing set up


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    from latent_moe_output_gb300 import build

    build.build()
    where = tmp_path_factory.mktemp("runtime")
    (where / "fake.c").write_text(FAKE_RUNTIME)
    fake = where / "fake.so"
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(fake), str(where / "fake.c"), "-ldl"],
                   check=True)

    def child(*names, refused=()):
        """(status of each call, kernels configured)"""
        env = dict(os.environ, LD_PRELOAD=str(fake), REFUSED_KERNELS="".join(refused))
        r = subprocess.run([sys.executable, "-c", CHILD, str(binding.library_path()), *names],
                           capture_output=True, text=True, env=env)
        assert r.returncode == 0, r.stderr
        return ([int(v) for v in r.stdout.split()],
                [k + "," for k in r.stderr.split(",") if k.startswith("k")])

    return child


def test_a_call_sets_up_the_kernels_of_its_own_operator(run):
    own = {}
    for name in OWN:
        statuses, kernels = run(name)
        assert statuses == [0] and kernels
        own[name] = set(kernels)
    for i, name in enumerate(OWN):
        for other in OWN[:i]:
            assert not own[name] & own[other], (name, other)
    assert run("combine") == ([0], [])


def test_kernels_are_set_up_once(run):
    _, once = run(*OWN)
    statuses, kernels = run(*OWN, *OWN)
    assert statuses == [0] * 8 and kernels == once


@pytest.mark.parametrize("broken", OWN)
def test_an_operator_that_cannot_be_set_up_refuses_no_other(run, broken):
    """... and is refused itself, every time."""
    _, kernels = run(broken)
    names = [broken] + OWN + ["combine"] + OWN
    statuses, _ = run(*names, refused=kernels[-1:])
    assert statuses == [5 if name == broken else 0 for name in names]
