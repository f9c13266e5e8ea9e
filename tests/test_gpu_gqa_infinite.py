"""Prompts whose queries or keys hold an infinity: a row whose scores are all minus infinity is NaN (the softmax of it is 0 / 0), like
every other row of an infinite query; only a row that sees no key gives zeros."""
import math

import pytest

from test_gpu_gqa import gen, packed_qkv, setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("dim,H", [(64, 2), (128, 6)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_infinite_queries(kind, dim, H, sign):
    """The infinity meets keys of one sign: the scores of all keys are plus, or minus, infinity."""
    torch, coli = setup()
    g = gen(torch, dim)
    q, kv = packed_qkv(torch, [40, 30], [40, 10], H, 2, dim, g, torch.bfloat16 if kind == "bf16" else torch.float32)
    kv[:, :2, 7] = kv[:, :2, 7].abs() + 0.5
    cu_q, cu_k = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 40, 70], [0, 40, 50]))

    def run(q, scale):
        out, lse = torch.full((70, H, dim), -5.0, device="cuda"), torch.full((70, H), -5.0, device="cuda")
        d = kv.cuda()
        coli.gqa_prefill(q.cuda(), d[:, :2], d[:, 2:4], cu_q, cu_k, scale, out, lse)
        coli.sync_check()
        return out.cpu(), lse.cpu()

    for scale in (0.1, -0.1):
        want, want_lse = run(q, scale)
        q2 = q.clone()
        rows = [0, 1, 17, 39, 45, 60, 69]                # 45 sees no key: zeros all the same
        q2[rows, 1, 7] = sign * math.inf
        got, lse = run(q2, scale)
        for r in rows:
            if r == 45:
                assert (got[r] == 0).all() and (lse[r] == -math.inf).all()
            else:
                assert torch.isnan(got[r, 1]).all() and torch.isnan(lse[r, 1])
        got[rows, 1], lse[rows, 1] = want[rows, 1], want_lse[rows, 1]
        assert torch.equal(got, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_infinite_keys(kind):
    """A first key that scores minus infinity: NaN for the row that sees it alone, no weight beside others."""
    torch, coli = setup()
    g = gen(torch, 3)
    q, kv = packed_qkv(torch, [20], [20], 2, 1, 64, g, torch.bfloat16 if kind == "bf16" else torch.float32)
    q[:, :, 2] = q[:, :, 2].abs() + 0.5
    cu = torch.tensor([0, 20], dtype=torch.int32, device="cuda")
    outs = []
    for x in (-math.inf, None):
        c = kv.clone()
        if x is not None:
            c[0, 0, 2] = x
        out, lse = torch.empty(20, 2, 64, device="cuda"), torch.empty(20, 2, device="cuda")
        d = c.cuda()
        coli.gqa_prefill(q.cuda(), d[:, :1], d[:, 1:2], cu, cu, 0.1, out, lse)
        coli.sync_check()
        outs.append((out.cpu(), lse.cpu()))
    out, lse = outs[0]
    assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all()
    assert torch.isfinite(out[1:]).all() and torch.isfinite(lse[1:]).all()
    assert torch.allclose(out[1], kv[1, 1].float(), rtol=2.0 ** -7, atol=0)   # the second key alone is left
