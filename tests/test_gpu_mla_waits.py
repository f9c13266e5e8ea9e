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
