"""gdn_paged_mass where its first launch fails, on the CPU: the library's objects linked against a stand-in for the CUDA runtime.
The join, which would read what no kernel wrote, is not launched then."""
import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p
FAKE, WS = P(0x10000), P(0x20000)  # never dereferenced


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    from chunked_recurrence_gb300 import build as b
    b.build()
    so = str(tmp_path_factory.mktemp("launch") / "failing_launch.so")
    cuda = os.path.join(os.path.dirname(os.path.dirname(b._nvcc())), "include")
    objects = [os.path.join(b.OUT_DIR, name + ".o") for name in ("paged_mass", "paged_mass_few", "paged_mass_tc", "paged_attn")]
    if not all(os.path.exists(o) for o in objects):
        b.build(force=True)
    # what is not called stays unresolved
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-Wl,-Bsymbolic,-z,lazy", "-I", cuda, "-o", so,
                    os.path.join(ROOT, "tests", "host_emulation", "failing_launch_host.cpp"), *objects], check=True)
    import chunked_recurrence_gb300 as crg
    lib = ctypes.CDLL(so, mode=os.RTLD_LAZY)
    for name in ("gdn_paged_mass", "gdn_paged_mass_workspace_bytes"):
        getattr(lib, name).argtypes, getattr(lib, name).restype = crg._SIGS[name]
    return lib


@pytest.mark.parametrize("dtype,D,new", [(0, 64, 3), (0, 250, 40), (1, 96, 3), (1, 128, 1), (1, 256, 2)])
def test_join_follows_a_launch_that_worked(lib, dtype, D, new):
    import chunked_recurrence_gb300 as crg
    sh = crg.GdnCacheShape(n_seqs=2, n_tok=2 * new, Hq=4, Hkv=2, D=D, dtype=dtype, page_size=16, n_pages=10, max_pages=5)
    nbytes = lib.gdn_paged_mass_workspace_bytes(ctypes.byref(sh))
    for fails, status, launches in ((0, crg.GDN_OK, 2), (1, 3, 1), (0, crg.GDN_OK, 2)):
        lib.fake_reset(fails)
        assert lib.gdn_paged_mass(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, ctypes.byref(sh), new, 0.1, 0, 1, 0, FAKE, 0, 0, 80, WS,
                                  nbytes, None) == status
        assert lib.fake_launches() == launches
