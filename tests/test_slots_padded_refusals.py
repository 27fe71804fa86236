"""bi_build_slots_padded refuses what bi_build_slots refuses, before any launch."""
import os
import subprocess
import sys

from test_tree_refusals import INVALID, M, SHAPE, load_lib, slots_call


class Padded:
    def __init__(self, lib):
        self.bi_build_slots = lib.bi_build_slots_padded


def check():
    L = Padded(load_lib())
    for kw in (dict(B=-1), dict(T=-1), dict(n_free=-1), dict(max_pages=0), dict(num_pages=1 << 27)):
        assert slots_call(L, **kw) == SHAPE, kw
    for kw in (dict(q_len=None), dict(pos0=None), dict(table=None), dict(free=None), dict(head=None), dict(head_out=None),
               dict(cu=None), dict(req=None), dict(pos=None), dict(slots=None), dict(depth=M), dict(slots=M)):
        assert slots_call(L, **kw) == INVALID, kw


def test_c_abi_refuses():
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, os.path.abspath(__file__)], env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


if __name__ == "__main__":
    check()
