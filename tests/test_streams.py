"""Calls on a stream that is given: what a call allocates itself comes from that stream's memory, so that nothing still
queued on the caller's stream can be using it, and is not handed on before the caller's stream is done with it."""
import contextlib

import pytest
import torch

from parity_util import need_gpu


# ------------------------------------------------------------------------------------------------ CPU
class _Tensor:
    """Stands for a tensor that a call made: the stream it was allocated on, and those it was recorded on."""

    def __init__(self, made_on):
        self.made_on, self.recorded = made_on, []

    def record_stream(self, stream):
        self.recorded.append(stream)

    def is_contiguous(self):
        return True

    def numel(self):
        return 64

    element_size = data_ptr = numel


@pytest.fixture
def streams(monkeypatch):
    """The allocator's view of a call without a GPU: "caller" is current, torch.cuda.stream changes it."""
    current = ["caller"]

    @contextlib.contextmanager
    def use(stream):
        current.append(stream)
        yield
        current.pop()

    monkeypatch.setattr(torch.cuda, "stream", use)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current[-1])
    for name in ("empty", "empty_like"):
        monkeypatch.setattr(torch, name, lambda *a, **kw: _Tensor(current[-1]))
    return current


def test_outputs_come_from_the_given_stream(streams):
    import exact_io_aware_17_gb300 as fa
    t = fa._output("o", None, (2,), torch.float32, "cuda:0", "side")
    assert t.made_on == "side" and t.recorded == ["caller"] and streams == ["caller"]
    t = fa._output("o", None, (2,), torch.float32, "cuda:0", None)
    assert t.made_on == "caller" and t.recorded == []


def test_the_workspace_comes_from_the_given_stream(streams):
    import exact_io_aware_17_gb300 as fa
    t = fa._check_workspace(None, 64, "cuda:0", "side")[0]
    assert t.made_on == "side" and t.recorded == []        # the caller's stream never uses it
    assert fa._check_workspace(None, 64, "cuda:0", None)[0].made_on == "caller"
    assert fa._check_workspace(None, 0, "cuda:0", "side") == (None, 0)


def test_the_square_calls_outputs_come_from_the_given_stream(streams, monkeypatch):
    """Every output and workspace of fa_fwd, fa_fwd_f32 and the two backward calls."""
    import exact_io_aware_17_gb300 as fa
    made = []

    def empty(*a, **kw):
        made.append(_Tensor(streams[-1]))
        return made[-1]

    class Library:
        def __getattr__(self, name):
            return lambda *a: 0

    for name in ("empty", "empty_like"):
        monkeypatch.setattr(torch, name, empty)
    monkeypatch.setattr(torch.cuda, "device", lambda dev: contextlib.nullcontext())
    for name, value in (("_check_tensor", lambda *a: None), ("_ptr", lambda t: None), ("_stream", lambda *a: None),
                        ("load_library", Library), ("fa_bwd_workspace_size", lambda *a: 64)):
        monkeypatch.setattr(fa, name, value)
    x = torch.zeros(1, 1, 1, 64)
    monkeypatch.setattr(_Tensor, "is_cuda", True, raising=False)
    monkeypatch.setattr(_Tensor, "device", x.device, raising=False)
    for call, outputs, others in ((lambda s: fa.fa_fwd(x, x, x, stream=s), 2, 0),
                                  (lambda s: fa.fa_fwd_f32(x, x, x, stream=s), 2, 0),
                                  (lambda s: fa.fa_fwd_stepnorm(x, x, x, stream=s), 2, 0),
                                  (lambda s: fa.fa_bwd(x, x, x, x, x, x, stream=s), 3, 1),
                                  (lambda s: fa.fa_bwd_noalloc(x, x, x, x, x, x, stream=s), 3, 0)):
        made.clear()
        call("side")
        assert [t.made_on for t in made] == ["side"] * (outputs + others)
        assert [t.recorded for t in made] == [["caller"]] * outputs + [[]] * others
        made.clear()
        call(None)
        assert [t.made_on for t in made] == ["caller"] * (outputs + others)


# ------------------------------------------------------------------------------------------------ GPU
def _apart(fa, call, sizes):
    """Runs call(stream=side) while blocks of `sizes` bytes, freed on the host, are still to be read on the caller's
    stream: nothing may write them before that, and the results are those of a call on the caller's stream."""
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    blocks = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes]
    copies = [torch.empty_like(b) for b in blocks]
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)              # about 10 ms, in which the call below is long done
    for c, b in zip(copies, blocks):
        c.copy_(b)
    blocks.clear()
    del b
    got = call(stream=side)
    side.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g, w)
    torch.cuda.synchronize()
    assert all(bool((c == 7).all()) for c in copies)
    fa.fa_check_status()


def _sizes(outputs, workspace):
    return [t.numel() * t.element_size() for t in outputs] + ([workspace] if workspace else [])


def _normal(*shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(len(shape) + sum(shape))).bfloat16().cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("Nq,Nk", [(1, 9001), (300, 9001)])
def test_cross_attention_on_another_stream(Nq, Nk):
    fa = need_gpu()
    q, k, v = _normal(4, 4, Nq, 64), _normal(4, 2, Nk, 64), _normal(4, 2, Nk, 64)
    o, lse = fa.fa_cross_fwd(q, k, v)
    ws = fa.fa_cross_fwd_workspace_size(4, 4, 2, Nq, Nk, 64)
    assert ws > 0
    _apart(fa, lambda **kw: fa.fa_cross_fwd(q, k, v, **kw), _sizes((o, lse), ws))
    do = torch.ones_like(q)
    ws = fa.fa_cross_bwd_workspace_size(4, 4, 2, Nq, Nk, 64)
    grads = fa.fa_cross_bwd(q, k, v, o, do, lse)
    _apart(fa, lambda **kw: fa.fa_cross_bwd(q, k, v, o, do, lse, **kw)[1:], _sizes(grads, ws))


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [1, 40])
def test_cache_calls_on_another_stream(rows):
    fa = need_gpu()
    B, Hk, bs, mb, d = 4, 2, 32, 160, 64
    kd, vd = (torch.randint(0, 120, (B * mb, Hk, bs, d), generator=torch.Generator().manual_seed(i), dtype=torch.uint8).cuda()
              .view(torch.float8_e4m3fn) for i in range(2))
    scale = torch.full((B * mb, Hk), 2.0 ** -8, device="cuda")
    table = torch.arange(B * mb, dtype=torch.int32, device="cuda").view(B, mb)
    lens = torch.tensor([5000, 0, 1, 300], dtype=torch.int32, device="cuda")
    q = _normal(B, Hk * rows, 1, d)
    ws = fa.fa_cache_fwd_workspace_size(B, Hk * rows, Hk, 1, d, bs, mb)
    assert ws > 0
    out = fa.fa_cache_fwd(q, kd, vd, scale, scale, table, lens)
    _apart(fa, lambda **kw: fa.fa_cache_fwd(q, kd, vd, scale, scale, table, lens, **kw), _sizes(out, ws))
    new = torch.full((B,), 200, dtype=torch.int32, device="cuda")
    free = torch.arange(B * mb, dtype=torch.int32, device="cuda")
    tables = [table.clone() for _ in range(3)]          # a call changes its own
    sizes = _sizes(fa.fa_cache_plan(lens, new, tables.pop(), free, bs, 1000), 0)
    _apart(fa, lambda **kw: fa.fa_cache_plan(lens, new, tables.pop(), free, bs, 1000, **kw), sizes)


@pytest.mark.gpu
def test_square_attention_on_another_stream():
    fa = need_gpu()
    q, k, v, do = (_normal(2, 3, 500, 64) + i for i in range(4))
    o, lse = fa.fa_fwd(q, k, v)
    _apart(fa, lambda **kw: fa.fa_fwd(q, k, v, **kw), _sizes((o, lse), 0))
    ws = fa.fa_bwd_workspace_size(2, 3, 500, 64)
    _apart(fa, lambda **kw: fa.fa_bwd(q, k, v, o, do, lse, **kw)[1:], _sizes((q, k, v), ws))
    _apart(fa, lambda **kw: fa.fa_bwd_noalloc(q, k, v, o, do, lse, **kw)[1:], _sizes((q, k, v), 0))
    q, k, v = (x.float() for x in (q, k, v))
    _apart(fa, lambda **kw: fa.fa_fwd_f32(q, k, v, **kw), _sizes(fa.fa_fwd_f32(q, k, v), 0))
