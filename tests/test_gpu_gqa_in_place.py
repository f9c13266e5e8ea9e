"""Steps without weights whose output is the query tensor itself: the bits of the same call with an output of its own."""
import pytest

from test_gpu_gqa import filled, gen, setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,n_q,H,K,columns", [([300, 1, 70], 1, 16, 4, 0), ([5000, 300], 3, 24, 2, 0), ([700] * 40, 1, 16, 2, 300), ([40, 9], 1, 8, 8, 4000)])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_step_in_place(lens, n_q, H, K, columns, kind):
    torch, coli = setup()
    g = gen(torch, len(lens) + H)
    s, table, _ = filled(torch, coli, lens, K, 16, 64, 32, g, columns=columns)
    q = torch.randn(len(lens), n_q, H, 64, generator=g).to(torch.bfloat16 if kind == "bf16" else torch.float32).cuda()
    table, n = table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    want = coli.gqa_attend(s.c, q, table, n, 0.1, torch.empty_like(q))
    got = q.clone()
    coli.gqa_attend(s.c, got, table, n, 0.1, got)
    coli.sync_check()
    assert torch.equal(got, want)
    with pytest.raises(coli.ColiError) as e:
        coli.gqa_attend(s.c, got, table, n, 0.1, got, weigh=True)
    assert e.value.code == coli.COLI_EINVAL
