"""Layer norm of arrays whose rows do not start alike within 16 bytes (each is
moved value by value then), and the weight's and bias's gradients in whole numbers.

Tolerances of the former: as in test_gpu_norm.py, whose chain of additions (16 values
a thread, ten halvings) is this form's as well.  The whole numbers are below 2^24 in all
partial sums, so every sum is exact and a row that is lost or counted twice shows."""
import pytest
import torch

from sampling_gnn_mini_gb300 import binding as sg
from test_gpu_norm import DT, _Guarded, _hold_bwd, _hold_fwd, _inputs, _ws

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sg.load()


class _Placed:
    """A matrix inside wider rows: `start` values before each row, `gap` behind it."""
    def __init__(self, t, start, gap):
        n, d = t.shape
        self.wide = torch.full((n * (start + d + gap) + 16,), 7.0, dtype=t.dtype, device="cuda")
        self.t = self.wide[: n * (start + d + gap)].view(n, start + d + gap)[:, start:start + d]
        self.t.copy_(t)

    def around(self, rows):
        """Whether nothing but the first rows was written."""
        self.t[:rows] = 7.0
        return bool((self.wide == 7).all())


# (start, gap) of x, g and what is written
APART = [((0, 8), (1, 0), (3, 5)), ((0, 0), (0, 1), (0, 2)), ((0, 8), (0, 8), (1, 7)), ((5, 0), (2, 3), (2, 3))]


@pytest.mark.parametrize("dt,dw", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
@pytest.mark.parametrize("d", [1, 7, 15, 16, 17, 33, 64, 100, 129, 255, 256, 257, 500, 513, 1001, 4097, 8200, 16384])
@pytest.mark.parametrize("at", range(len(APART)))
def test_rows_that_do_not_start_alike(d, at, dt, dw):
    for n in (1, 45, 700 if d > 1001 else 5003):
        x, g, w, b = _inputs(n, d, dt, dw, n + d)
        px, pg = _Placed(x, *APART[at][0]), _Placed(g, *APART[at][1])
        for count in ((n, n * 3 // 5) if n > 1 else (n,)):
            d_n = torch.tensor([count], dtype=torch.int32, device="cuda")
            py, pd = _Placed(torch.full_like(x, 7.0), *APART[at][2]), _Placed(torch.full_like(x, 7.0), *APART[at][2])
            m, r = torch.full((n,), 7.0, device="cuda"), torch.full((n,), 7.0, device="cuda")
            pw, pb = torch.full((d,), 7.0, device="cuda", dtype=DT[dw]), torch.full((d,), 7.0, device="cuda", dtype=DT[dw])
            guarded = _Guarded(n, d)
            sg.sg_layernorm_fwd(px.t, w, b, n, d_n, py.t, m, r)
            sg.sg_layernorm_bwd(pg.t, px.t, w, m, r, n, d_n, pd.t, pw, pb, guarded.ws)
            sg.sg_stream_check()
            guarded.check()
            _hold_fwd(x[:count], w, b, py.t[:count], m[:count], r[:count])
            _hold_bwd(g[:count], x[:count], w, m[:count], r[:count], pd.t[:count], pw, pb)
            assert bool((m[count:] == 7).all()) and bool((r[count:] == 7).all())
            assert py.around(count) and pd.around(count)
            # dx over g (where g starts like x, in the form of rows that start alike), without the sums
            over = _Placed(g, *APART[at][1])
            sg.sg_layernorm_bwd(over.t, px.t, w, m, r, n, d_n, over.t, None, None, _ws(n, d))
            sg.sg_stream_check()
            _hold_bwd(g[:count], x[:count], w, m[:count], r[:count], over.t[:count], None, None)
            assert torch.equal(over.t[count:], g[count:])


SUMS = [(200001, 64), (100000, 7), (60001, 128), (600001, 128), (30011, 1001), (9000, 4096), (3000, 8192), (2000, 16384), (133333, 300),
        (9746, 4104), (19526, 4097), (65, 64), (513, 128), (520, 128), (1024, 40), (3, 16384)]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,d", SUMS)
@pytest.mark.parametrize("apart", [False, True])
def test_sums_of_whole_numbers(n, d, apart, dt):
    # mean 0 and 1 / deviation 1: h = x
    gen = torch.Generator("cuda").manual_seed(d)
    x = torch.randint(-3, 4, (n, d), generator=gen, device="cuda", dtype=torch.int8)
    g = torch.randint(-2, 3, (n, d), generator=gen, device="cuda", dtype=torch.int8)
    m, r = torch.zeros(n, device="cuda"), torch.ones(n, device="cuda")
    px, pg = _Placed(x.to(DT[dt]), 0, 0), _Placed(g.to(DT[dt]), int(apart), 0)
    dx = torch.empty((n, d), device="cuda", dtype=DT[dt])
    for count in (n, n - n // 3):
        d_n = torch.tensor([count], dtype=torch.int32, device="cuda")
        dw, db = torch.full((d,), 7.0, device="cuda"), torch.full((d,), 7.0, device="cuda")
        sg.sg_layernorm_bwd(pg.t, px.t, None, m, r, n, d_n, dx, dw, db, _ws(n, d))
        sg.sg_stream_check()
        assert torch.equal(dw, (x[:count] * g[:count]).sum(0, dtype=torch.int64).float())
        assert torch.equal(db, g[:count].sum(0, dtype=torch.int64).float())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("d", [5, 64, 128, 300, 1001, 4096, 4104, 10000])
@pytest.mark.parametrize("size", [1e-20, 1e20])
def test_gradient_of_tiny_and_huge_rows(d, size, dt):
    # 1 / deviation squared is past fp32's range there, dx is not
    n = 40
    x, g, w, _ = _inputs(n, d, dt, "f32", d)
    x = (x.float() * size).to(DT[dt])
    m, r = torch.zeros(n, device="cuda"), torch.full((n,), 0.7 / size, device="cuda")
    for start in (0, 1):  # g like x, and not
        pg, dx = _Placed(g, start, 0), torch.full_like(x, 7.0)
        dw, db = torch.full((d,), 7.0, device="cuda"), torch.full((d,), 7.0, device="cuda")
        sg.sg_layernorm_bwd(pg.t, x, w, m, r, n, None, dx, dw, db, _ws(n, d))
        sg.sg_stream_check()
        _hold_bwd(g, x, w, m, r, dx, dw, db)
