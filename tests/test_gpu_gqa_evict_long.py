"""Evictions from sequences longer than shared memory has room for (48000 tokens of a head), exact against the definition."""
import pytest

from test_gpu_gqa import gen, setup, stays

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,keep,recent,page", [([100000, 48001], 30000, 64, 64), ([52000], 50000, 0, 16), ([48000, 60001, 47999], 1, 0, 128)])
@pytest.mark.parametrize("values", ["random", "ties", "equal", "behind"])
def test_evict_long(lens, keep, recent, page, values):
    """Random weights; few different ones, so that the last that stay straddle the place where the room ends; all the same; all that stay behind
    that place."""
    torch, coli = setup()
    g = gen(torch, sum(lens))
    per, new = [-(-n // page) for n in lens], -(-keep // page)
    total = sum(per) + new * len(lens)
    order = torch.randperm(total, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(per)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
    dst = order[at:].view(len(lens), new).contiguous()
    K = 2
    k, v = (torch.randint(0, 256, (total, K, page, 32), generator=g, dtype=torch.uint8).cuda() for _ in "kv")
    ks, vs = (torch.rand(total, K, page, 1, generator=g).to(torch.bfloat16).cuda() for _ in "kv")
    w = torch.zeros(total, K, page)
    rows = []
    for b, n in enumerate(lens):
        x = torch.rand(K, per[b] * page, generator=g)
        if values == "ties":
            x = (x * 5).floor() / 4
        elif values == "equal":
            x = torch.full_like(x, 0.5)
        elif values == "behind":
            x[:, :48000] *= 0.25
            x[:, 48000:] += 0.5
        rows.append(x)
        w[table[b, :per[b]].long()] = x.view(K, per[b], page).transpose(0, 1)
    wd = w.cuda()
    cache = coli.GqaCache(k, v, ks, vs, weights=wd)
    kept, length = torch.full((len(lens), K, keep), 9, dtype=torch.int32, device="cuda"), torch.zeros(len(lens), dtype=torch.int32, device="cuda")
    before = [t.cpu() for t in (k, v, ks, vs)]
    coli.gqa_evict(cache, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), keep, recent, dst.cuda(), kept, length)
    coli.sync_check()
    assert length.tolist() == [min(n, keep) for n in lens]
    after, w2 = [t.cpu() for t in (k, v, ks, vs)], wd.cpu()
    for b, n in enumerate(lens):
        for h in range(K):
            ref = torch.tensor(stays(rows[b][h].tolist(), n, keep, recent))
            m = len(ref)
            assert torch.equal(kept[b, h, :m].cpu().long(), ref) and (kept[b, h, m:] == -1).all()
            sp, dp, i = table[b, ref // page].long(), dst[b, torch.arange(m) // page].long(), torch.arange(m) % page
            assert torch.equal(w2[dp, h, i], rows[b][h, ref])
            for x, y in zip(before, after):
                assert torch.equal(y[dp, h, i], x[sp, h, ref % page])
