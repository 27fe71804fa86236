"""What the header promises of the operators that serve a tree of drafted tokens, at the calls where it is easiest to
break: logits that are not finite alone in their segment, the two output types, token rows behind the last token."""
import pytest
import torch

from test_gpu_tree import INF, NAN, normal

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
