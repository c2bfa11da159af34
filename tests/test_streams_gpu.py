"""The convolution's calls on a stream of their own, with tensors that they make themselves (GPU)."""
import pytest
import torch

import depthwise_causal_short_gb300 as cc
from depthwise_causal_short_gb300 import _build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _build.build()
    yield
    assert cc.cconv_device_fault() == 0


@pytest.mark.parametrize("raw", [False, True])
def test_a_given_streams_calls_keep_their_memory_until_it_has_used_it(raw):
    # the calls wait on a busy stream while the current one takes and fills all the memory it is given
    gen = torch.Generator().manual_seed(1)
    B, T, D, W = 2, 600, 512, 4
    x, dy = (torch.randn(B, T, D, generator=gen).bfloat16().cuda() for _ in range(2))
    w, b = torch.rand(D, W, generator=gen).cuda(), torch.rand(D, generator=gen).cuda()
    x2, dy2 = x.view(-1, D), dy.view(-1, D)
    cu = torch.tensor([0, 500, 1200], dtype=torch.int32).cuda()
    init = torch.randn(2, D, W - 1, generator=gen).bfloat16().cuda()

    def calls(**kw):
        state = init.clone()
        torch.cuda.synchronize()
        if kw:
            with torch.cuda.stream(side):
                torch.cuda._sleep(200_000_000)  # some 0.1 s
        out = [cc.cconv_fwd(x, w, b, **kw), *cc.cconv_bwd(x, dy, w, b, **kw),
               *cc.cconv_fwd_varlen(x2, cu, w, b, initial_state=init, final_state=True, **kw)[:2],
               *cc.cconv_bwd_varlen(x2, dy2, cu, w, b, initial_state=init, **kw),
               *cc.cconv_fwd_multi([x, dy], [w, w], **kw), cc.cconv_update(x2[:2], state, w, b, **kw)[0]]
        dxs, dws, dbs = cc.cconv_bwd_multi([x, dy], [dy, x], [w, w], [b, b], **kw)
        return [*out, *dxs, *dws, *dbs, cc.cconv_update_ex(x2[:2], state, w, b, **kw)[0], state]

    sizes = [16, 512, 2048, 1 << 20, 2 << 20, 8 << 20, 20 << 20] * 6
    sizes += [cc.cconv_bwd_workspace_bytes(B, T, D, W), cc.cconv_bwd_varlen_workspace_bytes(B * T, D, W),
              cc.cconv_bwd_multi_workspace_bytes([D, D], B, T, W)] * 4

    def take():
        return [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes]

    want = calls()
    side = torch.cuda.Stream()
    stream = side.cuda_stream if raw else side
    for first in (True, False):  # the first time, memory comes from the device, which waits for the streams
        got = calls(stream=stream)
        fill = take()
        if first:
            torch.cuda.synchronize()
            del got, fill
    torch.cuda.current_stream().synchronize()
    assert not side.query()  # the calls are still to run
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert all(bool((t == 255).all()) for t in fill)


def test_the_default_stream_by_its_handles():
    x, w = torch.randn(1, 64, 64).bfloat16().cuda(), torch.rand(64, 4).cuda()
    want = cc.cconv_fwd(x, w)
    for handle in (0, 1, torch.cuda.default_stream()):
        assert torch.equal(cc.cconv_fwd(x, w, stream=handle), want)
        q = x.view(64, 1, 64)
        assert torch.equal(cc.cattn_qknorm_fwd(q, q, stream=handle)[0], cc.cattn_qknorm_fwd(q, q)[0])
