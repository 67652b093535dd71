"""What sg_logprobs, sg_distill and the layer norm refuse on the host, before
anything reaches a device."""
import pytest
import torch

from sampling_gnn_mini_gb300 import binding as sg
from test_training_refusals import A, INVALID, UNSUPPORTED, _call, _on_device

BIG = 1 << 20  # an aligned address past A, never dereferenced


@pytest.fixture(scope="module")
def lib():
    return sg.load()


def test_logprobs(lib):
    ok = dict(x=A, dt=0, n=4, d_n=None, c=9, ld=9, y=A, k=3, logp=A, ent=A, ids=A, top=A, s=None)
    for change, want in ((dict(dt=2), UNSUPPORTED), (dict(n=-1), INVALID), (dict(n=(1 << 27) + 1), INVALID), (dict(c=0), INVALID),
                         (dict(ld=8), INVALID), (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(logp=None), INVALID),
                         (dict(k=-1), INVALID), (dict(k=129), INVALID), (dict(ids=None), INVALID), (dict(top=None), INVALID),
                         (dict(k=0), INVALID), (dict(x=A + 2), INVALID), (dict(y=A + 1), INVALID), (dict(ent=A + 2), INVALID),
                         (dict(c=2147483647, ld=1 << 40), INVALID)):
        assert _call(lib.sg_logprobs, ok, **change) == want, change
        assert "sg_logprobs" in sg.sg_last_error()
    assert _call(lib.sg_logprobs, ok, n=0) == 0  # nothing to do


def test_distill(lib):
    need = lib.sg_distill_workspace(4, 9)
    assert need > 0 and lib.sg_distill_workspace(-1, 9) == 0 and lib.sg_distill_workspace(4, 0) == 0
    ok = dict(x=A, dt=0, n=4, d_n=None, c=9, ld=9, ids=A, v=A, k=3, T=1.0, mean=1, gs=1.0, loss=A, total=A, grad=BIG, ldg=9, ws=A,
              wsb=need, s=None)
    for change, want in ((dict(dt=7), UNSUPPORTED), (dict(n=-1), INVALID), (dict(n=(1 << 27) + 1), INVALID), (dict(c=0), INVALID),
                         (dict(ld=8), INVALID), (dict(ldg=8), INVALID), (dict(x=None), INVALID), (dict(ids=None), INVALID),
                         (dict(v=None), INVALID), (dict(loss=None), INVALID), (dict(k=0), INVALID), (dict(k=129), INVALID),
                         (dict(T=0.0), INVALID), (dict(T=-1.0), INVALID), (dict(T=float("nan")), INVALID),
                         (dict(T=float("inf")), INVALID), (dict(T=1e-4), INVALID), (dict(ws=None), INVALID),
                         (dict(ws=A + 8), INVALID), (dict(wsb=need - 1), INVALID), (dict(x=A + 1), INVALID),
                         (dict(grad=BIG + 2), INVALID), (dict(v=A + 2), INVALID), (dict(grad=A), INVALID)):
        assert _call(lib.sg_distill, ok, **change) == want, change
        assert "sg_distill" in sg.sg_last_error()


def test_layernorm(lib):
    ok = dict(x=A, dt=0, n=4, d_n=None, dim=8, ld=8, w=A, b=A, dtw=0, eps=1e-5, y=BIG, ldy=8, mean=A, rstd=A, s=None)
    for change, want in ((dict(dt=2), UNSUPPORTED), (dict(dtw=-1), UNSUPPORTED), (dict(n=-1), INVALID), (dict(dim=0), INVALID),
                         (dict(dim=16385, ld=20000, ldy=20000), INVALID), (dict(eps=0.0), INVALID), (dict(eps=-1.0), INVALID),
                         (dict(eps=float("nan")), INVALID), (dict(ld=7), INVALID), (dict(ldy=7), INVALID),
                         (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(x=A + 2), INVALID), (dict(w=A + 1), INVALID),
                         (dict(mean=A + 2), INVALID), (dict(y=A, ldy=9), INVALID)):
        assert _call(lib.sg_layernorm_fwd, ok, **change) == want, change
        assert "sg_layernorm_fwd" in sg.sg_last_error()
    assert _call(lib.sg_layernorm_fwd, ok, n=0) == 0
    need = lib.sg_layernorm_bwd_workspace(4, 8)
    assert need > 0
    for bad in ((-1, 8), (4, 0), (4, 16385)):
        assert lib.sg_layernorm_bwd_workspace(*bad) == 0
    ok = dict(g=A, x=A, dt=0, n=4, d_n=None, dim=8, ldg=8, ld=8, w=A, dtw=0, mean=A, rstd=A, dx=BIG, lddx=8, dw=A, db=A, ws=A,
              wsb=need, s=None)
    for change, want in ((dict(dt=2), UNSUPPORTED), (dict(dtw=3), UNSUPPORTED), (dict(n=-1), INVALID), (dict(dim=-4), INVALID),
                         (dict(ld=7), INVALID), (dict(ldg=7), INVALID), (dict(lddx=7), INVALID), (dict(g=None), INVALID),
                         (dict(x=None), INVALID), (dict(dx=None), INVALID), (dict(mean=None), INVALID), (dict(rstd=None), INVALID),
                         (dict(ws=None), INVALID), (dict(ws=A + 64), INVALID), (dict(wsb=need - 1), INVALID),
                         (dict(g=A + 2), INVALID), (dict(dw=A + 2), INVALID), (dict(rstd=A + 1), INVALID),
                         (dict(dx=A, lddx=9), INVALID)):
        assert _call(lib.sg_layernorm_bwd, ok, **change) == want, change
        assert "sg_layernorm_bwd" in sg.sg_last_error()


@pytest.mark.parametrize("dim", [1, 7, 64, 128, 1001, 4096, 8192, 16384])
def test_layernorm_workspace_grows_with_the_rows(lib, dim):
    need = [lib.sg_layernorm_bwd_workspace(n, dim) for n in list(range(0, 3000, 7)) + [10 ** 4, 10 ** 6, 1 << 27]]
    assert need[0] > 0 and all(a <= b for a, b in zip(need, need[1:]))


@pytest.mark.parametrize("dim", [1, 128, 250, 257, 500, 512, 513, 1000, 1024, 1025, 2048, 4096, 8192, 16384])
def test_layernorm_workspace_has_room_for_the_blocks(lib, dim):
    # a block for every row up to 768 threads an SM: 3 of 256 threads for rows up to 512,
    # longer ones by the smallest of 64 to 1024 threads with 16 values each (fp32 rows of
    # more than 252 already, as they need not start on 16 bytes)
    threads = 64
    while threads * 16 < dim:
        threads *= 2
    blocks = max(1, 768 // threads) * 148 // 8 * 8  # (148 SMs when there is no device)
    assert lib.sg_layernorm_bwd_workspace(1 << 20, dim) >= blocks * 2 * dim * 4


class _Refuses:  # the library is not reached
    def __getattr__(self, name):
        raise AssertionError("%s was called" % name)


def test_binding_checks_tensors(monkeypatch):
    monkeypatch.setattr(sg, "_lib", _Refuses())
    x, f, i = _on_device(4, 8), _on_device(4), _on_device(4, dtype=torch.int32)
    ids, v = _on_device(4, 3, dtype=torch.int32), _on_device(4, 3)
    ws, p = _on_device(1 << 16, dtype=torch.uint8), _on_device(8)
    h = torch.zeros
    calls = [
        lambda: sg.sg_logprobs(h(4, 8), i, 4, None, f, f, stream=0),
        lambda: sg.sg_logprobs(x, i, 4, None, None, f, stream=0),
        lambda: sg.sg_logprobs(x, None, 4, None, f, f, stream=0),
        lambda: sg.sg_logprobs(x, i, 5, None, f, f, stream=0),
        lambda: sg.sg_logprobs(x, i.long(), 4, None, f, f, stream=0),
        lambda: sg.sg_logprobs(x.double(), i, 4, None, f, f, stream=0),
        lambda: sg.sg_logprobs(x, i, 4, None, f, f, ids, None, stream=0),
        lambda: sg.sg_logprobs(x, i, 4, None, f, f, None, v, stream=0),
        lambda: sg.sg_logprobs(x, i, 4, None, f, f, ids[:, :2], v, stream=0),
        lambda: sg.sg_logprobs(x, i, 4, None, f, f, ids, _on_device(6, 2), stream=0),
        lambda: sg.sg_logprobs(x, i, 4, None, f, f, _on_device(4, 129, dtype=torch.int32), _on_device(4, 129), stream=0),
        lambda: sg.sg_logprobs(x.t(), i, 4, None, f, f, stream=0),
        lambda: sg.sg_distill(x, ids, v[:3], 4, None, f, None, None, ws, stream=0),
        lambda: sg.sg_distill(x, ids.long(), v, 4, None, f, None, None, ws, stream=0),
        lambda: sg.sg_distill(x, ids, _on_device(6, 2), 4, None, f, None, None, ws, stream=0),
        lambda: sg.sg_distill(x, ids, v.bfloat16(), 4, None, f, None, None, ws, stream=0),
        lambda: sg.sg_distill(x, ids, v, 4, None, f, None, _on_device(4, 8, dtype=torch.bfloat16), ws, stream=0),
        lambda: sg.sg_distill(x, ids, v, 4, None, f, None, _on_device(4, 7), ws, stream=0),
        lambda: sg.sg_distill(x, ids, v, 4, None, f, f[:1], None, ws, stream=0),
        lambda: sg.sg_distill(x, ids, v, 4, None, f, None, None, h(1 << 16), stream=0),
        lambda: sg.sg_distill(x, i, v, 4, None, f, None, None, ws, stream=0),
        lambda: sg.sg_layernorm_fwd(x, p, p.bfloat16(), 4, None, x, stream=0),
        lambda: sg.sg_layernorm_fwd(x, p.double(), None, 4, None, x, stream=0),
        lambda: sg.sg_layernorm_fwd(x, p[:7], None, 4, None, x, stream=0),
        lambda: sg.sg_layernorm_fwd(x, p, p, 4, None, _on_device(4, 8, dtype=torch.bfloat16), stream=0),
        lambda: sg.sg_layernorm_fwd(x, p, p, 5, None, x, stream=0),
        lambda: sg.sg_layernorm_fwd(x, p, p, 4, None, x, f[:3], f, stream=0),
        lambda: sg.sg_layernorm_bwd(x, x, p, f, f, 4, None, x, p.bfloat16(), p, ws, stream=0),
        lambda: sg.sg_layernorm_bwd(x, x, p, f, f[:2], 4, None, x, p, p, ws, stream=0),
        lambda: sg.sg_layernorm_bwd(x.bfloat16(), x, p, f, f, 4, None, x, p, p, ws, stream=0),
        lambda: sg.sg_layernorm_bwd(x, x, p, f, f, 4, None, x, p, p, None, stream=0),
        lambda: sg.sg_layernorm_bwd(x, x, p, None, f, 4, None, x, p, p, ws, stream=0),
    ]
    for k, call in enumerate(calls):
        with pytest.raises(sg.SgError) as e:
            call()
        assert e.value.status == INVALID, k


def test_binding_refuses_tensors_of_another_device(monkeypatch):
    monkeypatch.setattr(sg, "_lib", _Refuses())
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)  # the tensors are on 0
    x, f = _on_device(4, 8), _on_device(4)
    ids, v, ws = _on_device(4, 3, dtype=torch.int32), _on_device(4, 3), _on_device(4096, dtype=torch.uint8)
    for call in (lambda: sg.sg_logprobs(x, None, 4, None, None, f),
                 lambda: sg.sg_distill(x, ids, v, 4, None, f, None, None, ws),
                 lambda: sg.sg_layernorm_fwd(x, None, None, 4, None, x),
                 lambda: sg.sg_layernorm_bwd(x, x, None, f, f, 4, None, x, None, None, ws)):
        with pytest.raises(sg.SgError) as e:
            call()
        assert e.value.status == INVALID and "current device" in str(e.value)


def test_binding_refuses_a_stream_address_of_another_device(monkeypatch):
    monkeypatch.setattr(sg, "_lib", _Refuses())
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)  # the tensors are on 0
    x, f = _on_device(4, 8), _on_device(4)
    for call in (lambda: sg.sg_logprobs(x, None, 4, None, None, f, stream=0),
                 lambda: sg.sg_layernorm_fwd(x, None, None, 4, None, x, stream=0)):
        with pytest.raises(sg.SgError) as e:
            call()
        assert e.value.status == INVALID and "current device" in str(e.value)
