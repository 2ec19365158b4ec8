"""The streams of the language-model operators' calls: a workspace that a call makes for itself is
memory of the stream that the call runs on, which is one of the tensors' GPU."""
import pytest
import torch

import lm_plain as P
from compressed_adamw_state_amd import flashopt as F


def test_a_calls_own_workspace_is_of_its_stream(monkeypatch):
    seen, empty = [], torch.empty

    class Current:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            seen.append(self.stream)

        def __exit__(self, *_):
            seen.append("left")

    def noted(*a, **k):
        seen.append("empty")
        return empty(*a, **k)
    monkeypatch.setattr(torch.cuda, "stream", Current)
    monkeypatch.setattr(torch, "empty", noted)
    side = object()
    at, size, held = F._scratch(None, 512, torch.device("cpu"), side)
    assert seen == [side, "empty", "left"] and size == 512 and at == held.data_ptr()
    del seen[:]
    F._scratch(None, 512, torch.device("cpu"), None)
    assert seen == ["empty"]
    del seen[:]
    assert F._scratch(None, 0, torch.device("cpu"), side) == (None, 0, None) and seen == []


def test_a_stream_of_another_gpu_is_refused():
    class Stream:
        device, cuda_stream = torch.device("cuda", 1), 0
    with pytest.raises(ValueError, match="stream"):
        F._call("flashopt_logprob", torch.device("cuda", 0), Stream())


@pytest.mark.gpu
def test_a_call_on_a_side_stream_beside_a_busy_one():
    """The current stream still writes memory that it has freed while calls run on a side stream."""
    rows, vocab = 4, 200000
    g = torch.Generator().manual_seed(3)
    x = torch.randn(rows, vocab, generator=g)
    t = torch.randint(0, vocab, (rows,), generator=g)
    lp, lt, en, et = P.logprob(x, t, 1.0)
    xc, tc = x.cuda(), t.cuda()
    need = F.lib().flashopt_logprob_workspace_bytes(2, rows, vocab, 8)
    assert need > 0
    work = torch.randn(4096, 4096, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(4):
        a, b = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        tl = torch.empty(rows, 8, device="cuda")
        ti = torch.empty(rows, 8, dtype=torch.int64, device="cuda")
        torch.cuda.current_stream().synchronize()          # of these outputs' own former users
        freed = torch.empty(need, dtype=torch.uint8, device="cuda")
        for _ in range(4):
            work = (work @ work) * 1e-2
        freed.fill_(0xFF)
        del freed
        F.flashopt_logprob(xc, tc, 8, 1.0, a, b, None, tl, ti, stream=side)
        outs.append((a, b, ti))
    torch.cuda.synchronize()
    for a, b, ti in outs:
        assert bool(((a.cpu().double() - lp).abs() <= lt + P.U * lp.abs()).all())
        assert bool(((b.cpu().double() - en).abs() <= et + P.U * en.abs()).all())
        assert torch.equal(ti.cpu(), P.top(x, 8))
