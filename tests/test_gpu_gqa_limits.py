"""Magnitudes at the ends of the ranges that coli.h states: a power of two in the queries, and the inverse in the keys, changes no bit."""
import pytest

from test_gpu_gqa import filled, gen, packed_qkv, run_step, setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("by", [-100, 113])
def test_step_queries(kind, by):
    """|scale| times a query's magnitudes up to 2^116: 2^113 times randn (below 2^3) here."""
    torch, coli = setup()
    g = gen(torch, 5)
    lens = [300, 40]
    s, table, _ = filled(torch, coli, lens, 2, 16, 128, 32, g)
    q = torch.randn(2, 1, 8, 128, generator=g).to(torch.bfloat16 if kind == "bf16" else torch.float32)
    want, lse = run_step(torch, coli, s, table, lens, q, 0.25, "f32")
    s.ks.mul_(2.0 ** -by)
    got, lse2 = run_step(torch, coli, s, table, lens, q * 2.0 ** by, 0.25, "f32")
    assert torch.equal(got, want) and torch.equal(lse, lse2)


@pytest.mark.parametrize("size_q,size_k", [(107, -83), (-83, 110), (60, -96)])
def test_prompt_f32_scores(size_q, size_k):
    """|scale| times a query's magnitudes up to 2^112, keys down to 2^-99 (whose smallest elements may round the other way: a tolerance of
    2^-23 of a row's largest element in each product, as stated)."""
    torch, coli = setup()
    g = gen(torch, 8)
    q, kv = packed_qkv(torch, [70], [190], 4, 2, 64, g, torch.float32)
    cu = [torch.tensor([0, n], dtype=torch.int32, device="cuda") for n in (70, 190)]
    outs = []
    for a, b in ((0, 0), (size_q, size_k)):
        out = torch.empty(70, 4, 64, device="cuda")
        coli.gqa_prefill((q * 2.0 ** a).cuda(), (kv[:, :2] * 2.0 ** b).contiguous().cuda(), kv[:, 2:4].contiguous().cuda(), *cu, 2.0 ** (-3 - a - b), out)
        coli.sync_check()
        outs.append(out.cpu())
    if size_k >= -83:
        assert torch.equal(*outs)
    else:
        # scores move by 2 x 64 x 2^-24 max|q| max|k| / 8 = 2^-20 x 25 at most, outputs by twice that of values up to 5, and P may round the other way
        assert ((outs[0] - outs[1]).abs() <= 2 * 25 * 2.0 ** -20 * 5 + 2.0 ** -11 * kv.abs().max()).all()


@pytest.mark.parametrize("dim", [64, 128])
def test_prompt_bf16_values(dim):
    """bf16 values times the keys' number up to 2^119."""
    torch, coli = setup()
    g = gen(torch, 9)
    q, kv = packed_qkv(torch, [256], [256], 2, 1, dim, g, torch.bfloat16)
    cu = torch.tensor([0, 256], dtype=torch.int32, device="cuda")
    outs = []
    for by in (0, 108):                                   # 2^108 x randn x 256 keys
        out = torch.empty(256, 2, dim, device="cuda")
        d = kv.cuda()
        coli.gqa_prefill((q * 3).cuda(), d[:, :1], d[:, 1:2] * 2.0 ** by, cu, cu, 0.3, out)
        coli.sync_check()
        outs.append(out.cpu())
    assert torch.equal(outs[1], outs[0] * 2.0 ** 108)
