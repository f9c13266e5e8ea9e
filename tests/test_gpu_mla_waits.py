"""The latent attention's bounded device-side waits: a wait that runs out ends the call with COLI_ETIMEOUT and leaves the
device usable; equal calls after it give the bits of those before it.

No kernel is broken for this: with a limit of a nanosecond an ordinary wait of some 10 us is too long.  The queries lie in
pinned host memory, which the kernels read with plain loads, so that the tensor-core warp waits for them that long."""
import pytest

from test_gpu_mla import filled, gen, setup

pytestmark = pytest.mark.gpu


@pytest.fixture
def limit():
    torch, coli = setup()
    coli.sync_check()
    yield coli.set_wait_limit
    torch.cuda.synchronize()
    coli.set_wait_limit(0)


def attend(torch, coli, c, ql, qr, table, lens):
    """Through the C entry, which takes any address the device can read: the binding wants CUDA tensors."""
    B, n_q, H, L = ql.shape
    out = torch.zeros(B, n_q, H, L, device="cuda")
    rc = coli._lib.coli_mla_attend(c._p, coli.COLI_F32, ql.data_ptr(), qr.data_ptr(), B, n_q, H, table.data_ptr(), table.shape[1],
                                   lens.data_ptr(), 0.06, coli.COLI_F32, out.data_ptr(), None, torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    return out


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("lens", [[3000, 500], [300] * 40])
def test_attend_wait_runs_out(limit, e4m3, lens):
    torch, coli = setup()
    g = gen(torch, 1)
    c, table = filled(torch, coli, e4m3, 512, 64, 64, lens, g)
    ql, qr = torch.randn(len(lens), 1, 128, 512, generator=g).pin_memory(), torch.randn(len(lens), 1, 128, 64, generator=g).pin_memory()
    table, n = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    good = attend(torch, coli, c, ql, qr, table, n)
    coli.sync_check()
    limit(1)
    attend(torch, coli, c, ql, qr, table, n)
    with pytest.raises(coli.ColiError) as e:
        coli.sync_check()
    assert e.value.code == coli.COLI_ETIMEOUT
    limit(0)
    assert torch.equal(attend(torch, coli, c, ql, qr, table, n), good)
    coli.sync_check()


def test_prefill_wait_runs_out(limit):
    """Finding the first unit among 20000 sequences takes long enough."""
    torch, coli = setup()
    g = gen(torch, 2)
    n, B = 100, 20000
    cu = torch.cat([torch.zeros(B - n, dtype=torch.int32), torch.arange(n + 1, dtype=torch.int32)]).cuda()
    q, kv = torch.randn(n, 1, 192, generator=g).to(torch.bfloat16).cuda(), torch.randn(n, 1, 256, generator=g).to(torch.bfloat16).cuda()
    kr = torch.randn(n, 64, generator=g).to(torch.bfloat16).cuda()

    def run():
        out = torch.zeros(n, 1, 128, device="cuda")
        coli.mla_prefill(q, kv, kr, cu, cu, 0.07, out)
        return out
    good = run()
    coli.sync_check()
    assert torch.equal(good[:, 0], kv[:, 0, 128:].float())       # one key each
    limit(1)
    run()
    with pytest.raises(coli.ColiError) as e:
        coli.sync_check()
    assert e.value.code == coli.COLI_ETIMEOUT
    limit(0)
    assert torch.equal(run(), good)
    coli.sync_check()


@pytest.mark.parametrize("e4m3", [False, True])
def test_attend_longer_than_the_limit(limit, e4m3):
    """The limit is one wait's: a call may take many times as long (here some 3 ms, 512 sequences on the same pages)."""
    torch, coli = setup()
    g = gen(torch, 3)
    c, table = filled(torch, coli, e4m3, 512, 64, 64, [12000], g)
    B = 512
    table, n = table.cuda().expand(B, -1).contiguous(), torch.full((B,), 12000, dtype=torch.int32).cuda()
    ql, qr = torch.randn(B, 1, 128, 512, device="cuda").to(torch.bfloat16), torch.randn(B, 1, 128, 64, device="cuda").to(torch.bfloat16)
    outs = []
    for ns in (0, 500000):
        out = torch.zeros_like(ql)
        limit(ns)
        coli.mla_attend(c, ql, qr, table, n, 0.06, out)
        coli.sync_check()
        outs.append(out)
    assert torch.equal(*outs)


@pytest.mark.parametrize("n_q,n_k,H", [(24000, 24000, 32), (100, 300000, 1)])
def test_prefill_longer_than_the_limit(limit, n_q, n_k, H):
    """Likewise: 4 ms of many units, and one unit of 3 ms whose second query tile is empty."""
    torch, coli = setup()
    q, kv = torch.randn(n_q, H, 192, device="cuda").to(torch.bfloat16), torch.randn(n_k, H, 256, device="cuda").to(torch.bfloat16)
    kr = torch.randn(n_k, 64, device="cuda").to(torch.bfloat16)
    cu_q, cu_k = (torch.tensor([0, n], dtype=torch.int32).cuda() for n in (n_q, n_k))
    outs = []
    for ns in (0, 1000000):
        out = torch.zeros(n_q, H, 128, device="cuda", dtype=torch.bfloat16)
        limit(ns)
        coli.mla_prefill(q, kv, kr, cu_q, cu_k, 0.07, out)
        coli.sync_check()
        outs.append(out)
    assert torch.equal(*outs)
