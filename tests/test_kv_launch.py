"""kv8_attend's launches on the host, against a stand-in for the CUDA runtime's calls (no GPU is used, even where
there is one): what a first failure leaves behind, and what every launch sets up."""
import os
import subprocess
import sys
import textwrap

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FAKE = r"""
static int attrs, launches, attr_fails, lookup_fails;
static int encode(void) { return 0; }
int cudaFuncSetAttribute(const void *f, int a, int v) {
    (void)f; (void)a; (void)v;
    ++attrs;
    return attr_fails > 0 && attr_fails-- ? 2 : 0;
}
int cudaLaunchKernelExC(const void *c, const void *f, void **a) {
    (void)c; (void)f; (void)a;
    ++launches;
    return 0;
}
int cudaGetDriverEntryPointByVersion(const char *s, void **p, unsigned v, unsigned long long o, int *q) {
    (void)s; (void)v; (void)o;
    *p = (void *)encode;
    *q = 0;
    return lookup_fails > 0 && lookup_fails-- ? 3 : 0;
}
int fake_attrs(void) { return attrs; }
int fake_launches(void) { return launches; }
void fake_fail(int attr, int lookup) { attr_fails = attr; lookup_fails = lookup; }
"""

SETUP = """
import ctypes, sys
fake = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
from speculative_decoding_hybrid_gb300 import binding as gs

def cache(**kw):
    d = dict(h_q=8, h_kv=2, d=128, page_tokens=64, window=0, num_pages=10, num_layers=2, sm_scale=0.1, kv=4096,
             page_stride=2 * 32768, layer_stride=32768, scale=4096, scale_page_stride=8, scale_layer_stride=4)
    d.update(kw)
    c = gs.kv8_cache()
    for k, v in d.items():
        setattr(c, k, v)
    return c

def attend(c, cap=4, q=64, k=64, v=64, o=64):
    return gs.lib.kv8_attend(ctypes.byref(c), 0, 1, cap, 64, 64, 64, 4, 4, q, 1024, k, 256, v, 256, o, 1024, None, 256,
                             4, 0, None, 0, None, None)

def append(c, cap=4, table=64, pages=4, k=64, v=64):
    return gs.lib.kv8_append(ctypes.byref(c), 0, 1, cap, 64, 64, table, pages, 4, k, 256, v, 256, None, 4, None, None)
"""


@pytest.fixture(scope="module")
def fake(tmp_path_factory):
    from speculative_decoding_hybrid_gb300 import build
    build.build()
    d = tmp_path_factory.mktemp("fake")
    src, lib = str(d / "fake.c"), str(d / "fake.so")
    with open(src, "w") as f:
        f.write(FAKE)
    subprocess.run(["gcc", "-shared", "-fPIC", "-O1", "-o", lib, src], check=True)
    return lib


def run(fake, code):
    r = subprocess.run([sys.executable, "-c", SETUP + textwrap.dedent(code), fake], cwd=ROOT, capture_output=True,
                       text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr


def test_shared_memory_limit_is_raised_for_every_launch(fake):
    """The attribute belongs to the device that is current at the launch."""
    run(fake, """
        c = cache()
        for n in (1, 2, 3):
            assert attend(c) == gs.GDN_OK
            assert fake.fake_launches() == n and fake.fake_attrs() == n
    """)


@pytest.mark.parametrize("what", ["1, 0", "0, 1"])
def test_a_first_failure_does_not_stay(fake, what):
    run(fake, """
        c = cache()
        fake.fake_fail(%s)
        assert attend(c) == gs.GDN_ERR_CUDA and fake.fake_launches() == 0
        assert attend(c) == gs.GDN_OK and fake.fake_launches() == 1
    """ % what)


def test_nothing_to_do_needs_no_rows(fake):
    """No rows in the whole batch (empty tensors have a null address): launched, for the device's checks of the
    lengths, and never a null pointer where there are rows."""
    run(fake, """
        c = cache()
        none = dict(cap=0, q=None, k=None, v=None, o=None)
        assert attend(c, **none) == gs.GDN_OK
        for name in ("q", "k", "v", "o"):
            assert attend(c, **{name: None}) == gs.GDN_ERR_NULL, name
        assert append(c, cap=0, k=None, v=None) == gs.GDN_OK
        assert append(c, cap=0, k=None, v=None, table=None, pages=0) == gs.GDN_OK
        assert append(c, table=None, pages=0) == gs.GDN_OK
        for kw in (dict(k=None), dict(v=None), dict(table=None)):
            assert append(c, **kw) == gs.GDN_ERR_NULL, kw
    """)
