"""What the header promises of the operators that serve a tree of drafted tokens, at the calls where it is easiest to
break: logits that are not finite alone in their segment, the two output types, token rows behind the last token."""
import numpy as np
import pytest
import torch

from test_gpu_tree import HEADS, INF, NAN, TREE_F32, TreeCase, close, i32, normal, same_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bi():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from invariant_fixed_order_gb300 import bi as b
    return b


# ---- a NaN logit without a finite one beside it -----------------------------------------------------------------------

def nan_rows(V):
    """Rows with a NaN in a segment of 4096 columns that has no finite logit; the last row has no NaN."""
    x = normal((5, V), 3, 2.0, dtype=torch.float32)
    x[0, 4096:] = -INF
    x[0, V - 1] = NAN
    x[1, 4096:] = NAN
    x[2] = -INF
    x[2, 0] = NAN
    x[3, :4096] = -INF
    x[3, 4095] = NAN
    x[4, 4096:] = -INF
    return x


@pytest.mark.parametrize("V", [4097, 9000, 128256])
@pytest.mark.parametrize("K", [0, 1, 9])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_nan_logit_makes_its_row_nan(bi, V, K, dtype):
    x = nan_rows(V).to(dtype)
    tokens = torch.tensor([[0, 7, V - 1]] * 5, dtype=torch.int32)
    lp, ent, ids, top = bi.token_logprobs(x.cuda(), tokens.cuda(), top_k=K)
    assert torch.isnan(lp[:4]).all() and torch.isnan(ent[:4]).all()
    assert torch.isfinite(lp[4, :2]).all() and torch.isfinite(ent[4])
    if K:
        assert torch.isnan(top[:4]).all() and torch.isfinite(top[4]).all()
        assert ids[:4, 0].cpu().tolist() == [V - 1, 4096, 0, 4095]


@pytest.mark.parametrize("V", [4097, 9000, 128256])
def test_log_softmax_of_a_nan_logit(bi, V):
    x = nan_rows(V)
    lp = bi.log_softmax(x.cuda()).cpu()
    assert torch.isnan(lp[:4]).all()
    want = torch.log_softmax(x[4].double(), -1)
    f = torch.isfinite(want)
    assert torch.equal(torch.isfinite(lp[4]), f) and (lp[4][f].double() - want[f]).abs().max() < 1e-5


# ---- the output types of the attention --------------------------------------------------------------------------------

@pytest.mark.parametrize("H,Hkv,Dh", HEADS)
@pytest.mark.parametrize("ctx,nodes", [([0, 3, 1], [1, 2, 5]), ([700, 0, 16, 1999], [7, 64, 33, 31]), ([5000, 40], [100, 256])])
def test_a_bf16_output_is_the_fp32_output_rounded(bi, H, Hkv, Dh, ctx, nodes):
    c = TreeCase(ctx, nodes, H, Hkv, Dh, 40 + H)
    f = c.run(bi, out_dtype=bi.F32)
    b = c.run(bi)
    close(f, c.ref(), torch.float32)
    assert b.dtype == torch.bfloat16 and same_bits(b, f.to(torch.bfloat16))
    # so it is off by its own rounding and what the fp32 output may be off by
    ref = c.ref()
    assert ((b.cpu().double() - ref).abs() <= TREE_F32 * (1 + 2.0 ** -8) + ref.abs() * 2.0 ** -8).all()


@pytest.mark.parametrize("H,Hkv,Dh", [(32, 8, 128), (8, 1, 64), (3, 3, 64)])
def test_bf16_outputs_repeat_over_many_short_requests(bi, H, Hkv, Dh):
    rng = np.random.default_rng(4)
    ctx, nodes = rng.integers(0, 500, 200), rng.integers(0, 5, 200) * rng.integers(0, 20, 200)
    c = TreeCase(ctx.tolist(), nodes.tolist(), H, Hkv, Dh, 41)
    st = bi.new_status()
    first = c.run(bi, status=st).clone()
    assert same_bits(first, c.run(bi, out_dtype=bi.F32, status=st).to(torch.bfloat16))
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(300):
        differ += (c.run(bi, status=st) != first).sum()
    assert int(differ) == 0
    bi.check_status(st)


# ---- calls on a stream of their own -----------------------------------------------------------------------------------

def test_a_call_with_a_stream_keeps_its_memory_while_the_current_stream_works(bi):
    """Blocks that the current stream has just let go, with writes to them still pending, and its allocations right
    after the call: neither may meet the call's workspace or outputs."""
    c = TreeCase([3000, 60, 500], [40, 12, 3], 32, 8, 128, 50)
    x = normal((64, 50257), 51, 3.0, dtype=torch.float32).cuda()
    tok = torch.randint(0, 50257, (64, 2), generator=torch.Generator().manual_seed(3), dtype=torch.int32).cuda()
    attend = lambda **kw: (c.run(bi, **kw),)
    score = lambda **kw: bi.token_logprobs(x, tok, top_k=5, **kw)
    sizes = [bi.tree_attention_workspace_size(3, 55, 32, 8, 128, c.max_nodes, c.max_seq),
             bi.token_logprobs_workspace_size(64, 50257, 5), c.q.numel() * 2, 64 * 5 * 4]
    want = [attend(), score()]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for call in (attend, score):
            torch.cuda._sleep(200_000)
            for n in sizes * 2:
                torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255)
            got.append((call(stream=s), want[len(got) % 2]))
            for n in sizes * 2:
                torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255)
    torch.cuda.current_stream().wait_stream(s)
    for outs, refs in got:
        for a, b in zip(outs, refs):
            assert same_bits(a, b)


# ---- token rows behind the last token ---------------------------------------------------------------------------------

@pytest.mark.parametrize("T", [64, 5000, 9000])
@pytest.mark.parametrize("in_place", [True, False])
def test_rows_past_the_last_token_are_padding(bi, T, in_place):
    q, p0 = [30, 0, 10], [3, 0, 0]
    junk = [torch.full((T,), 3, dtype=torch.int32, device="cuda") for _ in range(64)]
    del junk
    args = lambda: (i32(q), i32(p0), i32(np.full((3, 4), 19)), i32(range(9)), i32([0]), T, 20)
    out = None if in_place else i32([0])
    got = bi.build_slots(*args(), free_head_out=out)
    for x in got[1:]:
        assert (x[40:] == -1).all() and (x[:40] >= 0).all()
    # arrays of the caller's: left, unless asked for
    mine = [torch.full((T,), 5, dtype=torch.int32, device="cuda") for _ in range(3)]
    names = ("tok_req", "tok_pos", "slots")
    bi.build_slots(*args(), free_head_out=out, **dict(zip(names, mine)))
    for x, y in zip(mine, got[1:]):
        assert (x[40:] == 5).all() and torch.equal(x[:40], y[:40])
    bi.build_slots(*args(), free_head_out=out, pad=True, **dict(zip(names, mine)))
    for x, y in zip(mine, got[1:]):
        assert torch.equal(x, y)
    # a row past T is nobody's; more tokens than rows leave none to pad
    wide = [torch.full((T + 7,), 5, dtype=torch.int32, device="cuda") for _ in range(3)]
    bi.build_slots(*args(), free_head_out=out, pad=True, **{n: w[:T] for n, w in zip(names, wide)})
    assert all((w[T:] == 5).all() for w in wide)
    st = bi.new_status()
    a = args()
    few = bi.build_slots(*a[:5], 35, 20, status=st)
    assert int(st) == 0x202 and all(torch.equal(x, y[:35]) for x, y in zip(few[1:], got[1:]))


def test_a_replayed_step_of_a_fixed_size_stores_its_own_tokens_only(bi):
    """Slots and append captured for 48 tokens, replayed with fewer: what the earlier step stored stays."""
    H, Hkv, Dh, T, pool = 4, 2, 64, 48, 20
    qkv = normal((T, (H + 2 * Hkv) * Dh), 60, dtype=torch.float32).cuda()
    k = torch.zeros(pool, Hkv, 16, Dh, dtype=torch.bfloat16, device="cuda")
    v, q_out = torch.zeros_like(k), torch.zeros(T, H, Dh, dtype=torch.bfloat16, device="cuda")
    c, s = (x.cuda() for x in bi.rope_table(64, Dh, 500000.0))
    q_len, pos0, head, nxt, st = i32([40, 8]), i32([0, 0]), i32([0]), i32([0]), bi.new_status()
    table, free = i32(np.full((2, 4), 19)), i32(range(12))

    def step():
        cu, req, pos, slots = bi.build_slots(q_len, pos0, table, free, head, T, pool, free_head_out=nxt, status=st)
        bi.qk_norm_rope_append(qkv, None, None, pos, slots, c, s, q_out, k, v, H, Hkv, Dh, status=st)
        return slots

    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        slots = step()
    g.replay()
    bi.check_status(st)
    first, k1, v1 = slots.clone(), k.clone(), v.clone()
    assert (first >= 0).all()
    qkv += 1.0
    q_len.copy_(i32([3, 1])), pos0.copy_(i32([40, 8])), head.copy_(nxt)
    g.replay()
    bi.check_status(st)
    assert (slots[:4] >= 0).all() and (slots[4:] == -1).all()
    for now, was in ((k, k1), (v, v1)):
        changed = (now != was).any(-1).any(1).nonzero()
        assert sorted((changed[:, 0] * 16 + changed[:, 1]).tolist()) == sorted(slots[:4].tolist())


def test_a_padding_token_is_not_reported_and_a_bad_position_is(bi):
    H, Hkv, Dh = 4, 2, 64
    qkv = normal((2, (H + 2 * Hkv) * Dh), 61).cuda()
    c, s = (x.cuda() for x in bi.rope_table(64, Dh, 500000.0))
    for pos, slot, code in ((-1, -1, 0), (5, -1, 0), (-2, -1, 0x202), (64, -1, 0x202), (-1, 4, 0x202), (5, -2, 0x201),
                            (5, 48, 0x201)):
        k = torch.zeros(3, Hkv, 16, Dh, dtype=torch.bfloat16, device="cuda")
        v, st = torch.zeros_like(k), bi.new_status()
        q_out = torch.zeros(2, H, Dh, dtype=torch.bfloat16, device="cuda")
        bi.qk_norm_rope_append(qkv, None, None, i32([pos, 2]), i32([slot, 7]), c, s, q_out, k, v, H, Hkv, Dh, status=st)
        assert int(st) == code, (pos, slot)
        stored = (k != 0).any(-1).any(1).nonzero()
        assert stored.tolist() == [[0, 7]]


# ---- a wait that runs out ---------------------------------------------------------------------------------------------

@pytest.mark.parametrize("H,Hkv,Dh", [(32, 8, 128), (8, 1, 64)])
@pytest.mark.parametrize("item", [0, 1, 2, 4, 6])
@pytest.mark.parametrize("v", [0, 1])
@pytest.mark.parametrize("warp", [0, 1])
def test_a_wait_that_runs_out_is_reported_and_the_stream_recovers(bi, H, Hkv, Dh, item, v, warp):
    """Failure detection without a fault: one copy of K or V is withheld in every CTA, by either copying warp, so the
    waits for it give up after 2 ms; the kernel reports a timeout, waits for the copies and products in flight, frees
    tensor memory and returns.  Calls right after it, on the same memory, are right.  Pairs of tiles, odd ones and lone
    requests over enough steps that later fills of a stage are withheld too."""
    c = TreeCase([9000, 300, 12000, 5], [70, 5, 20, 100], H, Hkv, Dh, 70)
    want = c.run(bi, out_dtype=bi.F32).clone()
    st, st2 = bi.new_status(), bi.new_status()
    ws = torch.empty(bi.tree_attention_workspace_size(4, 195, H, Hkv, Dh, c.max_nodes, c.max_seq), dtype=torch.uint8,
                     device="cuda")
    out = torch.empty_like(want)
    bi.tree_attention_wait_test(c.q, c.cu, c.pos0, c.mask, c.k, c.v, c.table, c.max_nodes, max_seq_len=c.max_seq,
                                out_dtype=bi.F32, ws=ws, out=out, status=st, wait_limit_ns=2_000_000,
                                skip_copy=4 * item + 2 * v + warp)
    again = [c.run(bi, out_dtype=bi.F32, ws=ws, status=st2).clone() for _ in range(3)]
    with pytest.raises(bi.BIError) as e:
        bi.check_status(st)
    assert e.value.status == bi.BI_ERR_TIMEOUT
    bi.check_status(st2)
    assert all(same_bits(x, want) for x in again)
    # nothing withheld: an ordinary call within the limit
    bi.reset_status(st)
    bi.tree_attention_wait_test(c.q, c.cu, c.pos0, c.mask, c.k, c.v, c.table, c.max_nodes, max_seq_len=c.max_seq,
                                out_dtype=bi.F32, ws=ws, out=out, status=st, wait_limit_ns=100_000_000, skip_copy=-1)
    bi.check_status(st)
    assert same_bits(out, want)


# ---- the cut of a request's keys --------------------------------------------------------------------------------------

@pytest.mark.parametrize("H,Hkv,Dh", [(8, 1, 64), (16, 2, 128), (32, 8, 128), (16, 16, 64)])
@pytest.mark.parametrize("steps", [1, 2, 16, 17, 64, 65, 130])
def test_cuts_of_every_length_within_the_workspace(bi, H, Hkv, Dh, steps):
    """Requests that end on, before and after a step, on both sides of the cut's thresholds, in exactly the workspace
    that the call asks for; nothing behind it is written."""
    ends = [128 * steps - 127, 128 * steps - 1, 128 * steps]
    nodes = [min(n, e) for n, e in zip((1, 40, 9), ends)]
    c = TreeCase([e - n for e, n in zip(ends, nodes)], nodes, H, Hkv, Dh, 80 + steps)
    need = bi.tree_attention_workspace_size(3, sum(nodes), H, Hkv, Dh, c.max_nodes, c.max_seq)
    buf = torch.full((need + 4096,), 77, dtype=torch.uint8, device="cuda")
    st = bi.new_status()
    out = c.run(bi, out_dtype=bi.F32, ws=buf[:need], status=st)
    bi.check_status(st)
    close(out, c.ref(), torch.float32)
    assert (buf[need:] == 77).all()
