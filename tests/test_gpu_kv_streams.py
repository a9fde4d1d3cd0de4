"""Page moves on a stream of their own, whose cache object ends while they wait
to run and whose memory is then used anew (GPU)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("given", [True, False])
@pytest.mark.parametrize("call", ["fork", "compact"])
def test_cache_object_goes_before_its_moves_run(call, given):
    import int4_weight_quantized_amd as w4

    pages, ps, D = 600, 16, 16
    k, v = (torch.randn((2, pages, 1, ps, D), device="cuda").bfloat16() for _ in range(2))
    c = w4.KVCache(k, v)
    used = torch.randperm(pages, generator=torch.Generator().manual_seed(1))[:300].int()
    t = torch.full((6, 100), -1, dtype=torch.int32)
    t[:3] = used.view(3, 100)
    refs = torch.zeros(pages, dtype=torch.int32)
    refs[used.long()] = 1
    t, refs = t.cuda(), refs.cuda()
    lens = torch.tensor([1595, 1600, 1590, 0, 0, 0], dtype=torch.int32, device="cuda")
    parents, children = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 2, 1], [3, 4, 5]))

    def move(c, t, lens, refs, **kw):
        if call == "fork":
            w4.kv_fork(c, t, lens, refs, parents, children, **kw)
        else:
            w4.kv_compact(c, t, refs, **kw)

    want = [x.clone() for x in (k, v, t, lens, refs)]
    move(w4.KVCache(*want[:2]), *want[2:])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)
        if not given:
            move(c, t, lens, refs)
    if given:
        move(c, t, lens, refs, stream=s)
    del c
    junk = [torch.full((n,), 3, dtype=torch.int32, device="cuda") for n in (2464, 1264, 100) for _ in range(20)]
    s.synchronize()
    for a, b in zip((k, v, t, lens, refs), want):
        assert torch.equal(a, b)
    del junk
