"""bi_tree_attention refuses more KV heads than its grid has rows, before any launch."""
import os
import subprocess
import sys

from test_tree_refusals import OK, SHAPE, load_lib, tree_call


def check():
    L = load_lib()
    for H, Hkv in ((65536, 65536), (1 << 19, 1 << 16)):
        assert tree_call(L, H=H, Hkv=Hkv, num_pages=1) == SHAPE
    assert tree_call(L, H=65535, Hkv=65535, num_pages=1, T=0) == OK


def test_c_abi_refuses():
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    r = subprocess.run([sys.executable, os.path.abspath(__file__)], env=env, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


if __name__ == "__main__":
    check()
