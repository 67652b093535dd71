"""What the training operators (embeddings, loss, orthogonalised updates)
refuse on the host, before anything reaches a device."""
import ctypes

import numpy as np
import pytest
import torch

from sampling_gnn_mini_gb300 import binding as sg

INVALID, UNSUPPORTED = sg.SG_ERR_INVALID_ARG, sg.SG_ERR_UNSUPPORTED
A = 4096  # an aligned, never dereferenced address


@pytest.fixture(scope="module")
def lib():
    return sg.load()


def _call(f, base, **change):
    args = dict(base, **change)
    return f(*args.values())


def test_embed_fwd(lib):
    ok = dict(table=A, dt=0, n_rows=10, dim=8, ld=8, ids=A, n_cap=4, d_n=None, scale=1.0, out=A, dto=0, ldo=8, s=None)
    for change, want in ((dict(dt=2), UNSUPPORTED), (dict(dto=-1), UNSUPPORTED), (dict(n_rows=-1), INVALID),
                         (dict(n_rows=1 << 31), INVALID), (dict(dim=0), INVALID), (dict(n_cap=-1), INVALID),
                         (dict(ld=7), INVALID), (dict(ldo=7), INVALID), (dict(table=None), INVALID),
                         (dict(ids=None), INVALID), (dict(out=None), INVALID), (dict(table=A + 2), INVALID),
                         (dict(out=A + 1), INVALID), (dict(ids=A + 2), INVALID)):
        assert _call(lib.sg_embed_fwd, ok, **change) == want, change
        assert "sg_embed_fwd" in sg.sg_last_error()
    assert _call(lib.sg_embed_fwd, ok, n_cap=0) == 0  # nothing to do


def test_embed_bwd(lib):
    need = lib.sg_embed_bwd_workspace(4, 10, 8, sg.SG_GRAD_DENSE)
    assert need > 0
    ok = dict(ids=A, n_cap=4, d_n=None, n_rows=10, g=A, dt=0, dim=8, ld=8, scale=1.0, mode=sg.SG_GRAD_DENSE, rows=None,
              n_out=None, grad=A, dto=0, ldo=8, ws=A, wsb=need, s=None)
    for change, want in ((dict(dt=5), UNSUPPORTED), (dict(dto=5), UNSUPPORTED), (dict(mode=3), INVALID),
                         (dict(mode=-1), INVALID), (dict(n_rows=0), INVALID), (dict(n_cap=-1), INVALID),
                         (dict(dim=0), INVALID), (dict(ld=7), INVALID), (dict(ldo=7), INVALID),
                         (dict(rows=A), INVALID), (dict(n_out=A), INVALID), (dict(mode=sg.SG_GRAD_ROWS), INVALID),
                         (dict(g=None), INVALID), (dict(grad=None), INVALID), (dict(ids=None), INVALID),
                         (dict(ws=None), INVALID), (dict(ws=A + 16), INVALID), (dict(wsb=need - 1), INVALID),
                         (dict(g=A + 2), INVALID), (dict(grad=A + 2), INVALID)):
        assert _call(lib.sg_embed_bwd, ok, **change) == want, change
        assert "sg_embed_bwd" in sg.sg_last_error()
    for bad in ((0, 10, 8, 0), (4, 0, 8, 0), (4, 10, 0, 0), (4, 10, 8, 3), (-1, 10, 8, 0)):
        assert lib.sg_embed_bwd_workspace(*bad) == 0


def test_xent(lib):
    need = lib.sg_xent_workspace(4, 9)
    assert need > 0 and lib.sg_xent_workspace(-1, 9) == 0 and lib.sg_xent_workspace(4, 0) == 0
    ok = dict(x=A, dt=0, n=4, d_n=None, c=9, ld=9, y=A, mean=1, gs=1.0, loss=A, total=A, grad=A, ldg=9, ws=A, wsb=need,
              s=None)
    for change, want in ((dict(dt=7), UNSUPPORTED), (dict(n=-1), INVALID), (dict(c=0), INVALID), (dict(ld=8), INVALID),
                         (dict(ldg=8), INVALID), (dict(x=None), INVALID), (dict(y=None), INVALID),
                         (dict(loss=None), INVALID), (dict(ws=None), INVALID), (dict(ws=A + 8), INVALID),
                         (dict(wsb=need - 1), INVALID), (dict(x=A + 1), INVALID), (dict(grad=A + 2), INVALID),
                         (dict(total=A + 2), INVALID), (dict(ldg=10), INVALID)):  # last: in place, other stride
        assert _call(lib.sg_xent, ok, **change) == want, change
        assert "sg_xent" in sg.sg_last_error()


def test_orthogonalise_and_muon(lib):
    need = lib.sg_orthogonalise_workspace(1, 20, 30)
    assert need > 0
    for bad in ((0, 20, 30), (1, 0, 30), (1, 20, 0), (1, 65537, 4), (1, 8193, 8193), (70000, 4, 4)):
        assert lib.sg_orthogonalise_workspace(*bad) == 0
    ok = dict(g=A, dt=0, count=1, rows=20, cols=30, ld=30, steps=5, coef=None, eps=1e-7, scale=1.0, out=A, ldo=30, ws=A,
              wsb=need, s=None)
    for change, want in ((dict(dt=3), UNSUPPORTED), (dict(count=-1), INVALID), (dict(rows=0), INVALID),
                         (dict(cols=70000), INVALID), (dict(ld=29), INVALID), (dict(ldo=29), INVALID),
                         (dict(steps=-1), INVALID), (dict(steps=17), INVALID), (dict(g=None), INVALID),
                         (dict(out=None), INVALID), (dict(ws=None), INVALID), (dict(ws=A + 64), INVALID),
                         (dict(wsb=need - 1), INVALID), (dict(g=A + 2), INVALID), (dict(ldo=31), INVALID)):
        assert _call(lib.sg_orthogonalise, ok, **change) == want, change
        assert "sg_orthogonalise" in sg.sg_last_error()
    assert _call(lib.sg_orthogonalise, ok, count=0) == 0
    ok = dict(w=A, dt=0, g=A, m=A, count=1, rows=20, cols=30, lr=0.1, mu=0.9, nest=1, wd=0.0, scale=1.0, steps=5,
              coef=None, eps=1e-7, w2=A, m2=A, ws=A, wsb=need, s=None)
    for change, want in ((dict(dt=3), UNSUPPORTED), (dict(rows=-2), INVALID), (dict(steps=99), INVALID),
                         (dict(w=None), INVALID), (dict(g=None), INVALID), (dict(m=None), INVALID),
                         (dict(w2=None), INVALID), (dict(m2=None), INVALID), (dict(wsb=0), INVALID),
                         (dict(w=A + 2), INVALID), (dict(m=A + 1), INVALID)):
        assert _call(lib.sg_muon_step, ok, **change) == want, change
        assert "sg_muon_step" in sg.sg_last_error()


def test_binding_checks_tensors():
    x = torch.zeros((4, 8))
    ids = torch.zeros(4, dtype=torch.int32)
    ws = torch.zeros(512, dtype=torch.uint8)
    for call in (lambda: sg.sg_embed_fwd(x, ids, 4, None, 1.0, x),             # not on a device
                 lambda: sg.sg_embed_bwd(ids, 4, None, 10, x, 1.0, x, sg.SG_GRAD_DENSE, ws),
                 lambda: sg.sg_xent(x, ids, 4, None, torch.zeros(4), None, None, ws),
                 lambda: sg.sg_orthogonalise(x, x, ws),
                 lambda: sg.sg_muon_step(x, x, x, x, x, ws, lr=0.1)):
        with pytest.raises(sg.SgError) as e:
            call()
        assert e.value.status == INVALID


def test_coefficients_are_checked():
    assert sg._coef(5, None) is None
    assert sg._coef(2, [(1, 2, 3), (4, 5, 6)]).tolist() == [1, 2, 3, 4, 5, 6]
    with pytest.raises(sg.SgError):
        sg._coef(2, np.zeros(5))
    assert ctypes.sizeof(ctypes.c_float) == 4


@pytest.mark.parametrize("dim", [1, 3, 8, 20, 32, 64, 100, 128, 256, 1000, 1024, 4096])
def test_embed_bwd_workspace_grows_with_the_list(lib, dim):
    # sized for the longest list, a workspace serves every shorter one
    sizes = list(range(1, 12000, 7)) + [s for k in range(1, 400) for s in (640 * k, 640 * k + 1)] + [1 << k for k in range(30)]
    need = [lib.sg_embed_bwd_workspace(n, 1000, dim, sg.SG_GRAD_ADD) for n in sorted(set(sizes))]
    assert need[0] > 0 and all(a <= b for a, b in zip(need, need[1:]))


class _OnDevice(torch.Tensor):
    """A host tensor that says it is on device 0, so that the binding's checks
    can be met one by one without a device."""
    def get_device(self):
        return 0


def _on_device(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(_OnDevice)


def test_binding_checks_the_workspace(monkeypatch):
    class Refuses:  # the library is not reached
        def __getattr__(self, name):
            raise AssertionError("%s was called" % name)
    monkeypatch.setattr(sg, "_lib", Refuses())
    x, y, one = _on_device(4, 8), _on_device(4, dtype=torch.int32), _on_device(4)
    table = _on_device(10, 8)
    base = torch.zeros(1 << 16, dtype=torch.uint8)
    for ws in (base,                                             # on the host
               base.as_subclass(_OnDevice)[::2],                 # with gaps
               None, base.numpy()):
        for call in (lambda: sg.sg_embed_bwd(y, 4, None, 10, x, 1.0, table, sg.SG_GRAD_DENSE, ws, stream=0),
                     lambda: sg.sg_xent(x, y, 4, None, one, None, None, ws, stream=0),
                     lambda: sg.sg_orthogonalise(x, x, ws, stream=0),
                     lambda: sg.sg_muon_step(x, x, x, x, x, ws, lr=0.1, stream=0)):
            with pytest.raises(sg.SgError) as e:
                call()
            assert e.value.status == INVALID and "workspace" in str(e.value)


def test_binding_passes_the_workspace_in_bytes(monkeypatch):
    seen = []

    class Records:
        def __getattr__(self, name):
            return lambda *args: seen.append(args) or 0
    monkeypatch.setattr(sg, "_lib", Records())
    for dtype, n in ((torch.uint8, 4096), (torch.float32, 1024), (torch.int64, 512)):
        ws = _on_device(n, dtype=dtype)
        sg.sg_orthogonalise(_on_device(4, 8), _on_device(4, 8), ws, stream=0)
        assert seen[-1][-3:-1] == (ws.data_ptr(), 4096)


def test_embed_bwd_workspace_has_room_for_the_passes(lib):
    # where a device takes no cluster for a list of some thousands, the sort goes
    # over it in passes: pairs in and out (16 bytes a position), counts of 256
    # digits in 4 passes (8 copies), and a word a digit and pass for every 2,048 positions
    for n in (3073, 5000, 8192, 16384, 32768, 32769, 100000):
        room = 16 * n + 8 * 4 * 256 * 4 + -(-n // 2048) * 256 * 4 * 4
        assert lib.sg_embed_bwd_workspace(n, 1 << 30, 1, sg.SG_GRAD_ADD) >= room
