"""How bi_tree_attention cuts a request's keys: the length of a segment changes smoothly with the request, the workspace
has room for every cut that a call may make.  Host functions only, in a child process that sees no GPU."""
import os
import subprocess
import sys

STEP, ROWS, MAX_NODES = 128, 128, 256
HEADS = [(32, 8), (4, 2), (8, 8), (16, 2), (3, 3), (8, 1), (64, 16), (12, 12), (1, 1), (128, 128)]


def host():
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    from invariant_fixed_order_gb300 import build
    build.build()
    from invariant_fixed_order_gb300 import bi
    return bi


def nodes_of(H, Hkv):
    """One node count for each number of tiles."""
    nt = ROWS // (H // Hkv)
    return range(1, MAX_NODES + 1, nt)


def case_smooth(bi):
    for H, Hkv in HEADS:
        for n in nodes_of(H, Hkv):
            last = 0
            for steps in list(range(2, 300)) + [1000, 4000, 100000]:
                seg = bi.tree_attention_segment(steps * STEP, min(n, steps * STEP), H, Hkv)
                assert seg % STEP == 0 and seg >= 2 * STEP
                s = seg // STEP
                # never shorter for a longer request, and for one step more longer by what 32 runs of the request's
                # tiles take of it, at most
                tiles = -(-n // (ROWS // (H // Hkv))) * Hkv
                assert s >= last and (steps > 300 or last == 0 or s <= last + -(-tiles // 32)), (H, Hkv, n, steps, s, last)
                last = s
                assert -(-steps // s) <= 32
                # all positions of a step belong to one cut
                for p in (steps * STEP - STEP + 1, steps * STEP - 60):
                    assert n > p or bi.tree_attention_segment(p, n, H, Hkv) == seg
    for bad in ((0, 1, 8, 8), (10, 0, 8, 8), (10, 257, 8, 8), (10, 11, 8, 8), (300, 2, 6, 4), (300, 2, 32, 2), (-5, 1, 8, 8)):
        assert bi.tree_attention_segment(*bad) == 0, bad
    assert bi.tree_attention_segment(2 ** 31 - 256, 256, 8, 8) > 0


def slots(bi, H, Hkv, max_seq):
    """Segments per tile that the workspace has room for: from the size for one tile of one node a KV head (32 rows)."""
    def parts(Dh):
        return bi.tree_attention_workspace_size(1, 1, H, Hkv, Dh, 1, max_seq)
    per = (parts(128) - parts(64)) // (64 * 4)          # tiles x segments x rows
    tiles = (1 // (ROWS // (H // Hkv)) + 1) * Hkv
    assert per % (tiles * 32) == 0
    return per // (tiles * 32)


def case_workspace(bi):
    for H, Hkv in HEADS:
        for max_steps in (1, 2, 3, 4, 7, 8, 9, 16, 17, 31, 32, 33, 64, 65, 127, 128, 129, 160, 161, 250, 256, 257, 300, 1000):
            have = slots(bi, H, Hkv, max_steps * STEP)
            most = 0
            for n in nodes_of(H, Hkv):
                for steps in range(1, max_steps + 1):
                    p = steps * STEP
                    most = max(most, -(-p // bi.tree_attention_segment(p, min(n, p), H, Hkv)))
            assert most <= have <= 32, (H, Hkv, max_steps, most, have)
            assert have <= max(2 * most, most + 2), (H, Hkv, max_steps, most, have)   # and not much more


def test_cut():
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    for case in ("smooth", "workspace"):
        r = subprocess.run([sys.executable, os.path.abspath(__file__), case], env=env, capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, case + r.stdout + r.stderr


if __name__ == "__main__":
    globals()["case_" + sys.argv[1]](host())
