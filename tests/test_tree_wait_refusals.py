"""bi_tree_attention_wait_test refuses what bi_tree_attention refuses, a missing status word and a limit out of range,
before any launch."""
import ctypes
import os
import subprocess
import sys

from test_tree_refusals import INVALID, SHAPE, UNSUPPORTED, F, i32, load_lib, tree_call


class WaitTest:
    def __init__(self, lib, limit=1000000, status=F):
        self.lib, self.limit, self.status = lib, limit, status

    def bi_tree_attention(self, *a):
        return self.lib.bi_tree_attention_wait_test(*a[:-2], ctypes.c_uint64(self.limit), i32(0), self.status, None)


def check():
    L = load_lib()
    for kw in (dict(B=-1), dict(nodes=0), dict(seq=65)):
        assert tree_call(WaitTest(L), **kw) == SHAPE, kw
    assert tree_call(WaitTest(L), Dh=96) == UNSUPPORTED
    assert tree_call(WaitTest(L), q=None) == INVALID
    assert tree_call(WaitTest(L, status=None)) == INVALID
    for limit in (0, 999999, 2000000001):
        assert tree_call(WaitTest(L, limit)) == INVALID


def test_c_abi_refuses():
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, os.path.abspath(__file__)], env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


if __name__ == "__main__":
    check()
