"""GPU tests of layer norm on operands at odd places: the same bits as on aligned ones, whichever of the operands
and outputs is off 16 bytes."""
import pytest
import torch
from test_glr import DT, sliced
from test_glr_places import odd
from test_layer_norm import EPS, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,D", [(5, 48), (70, 200), (700, 512), (3, 1111), (700, 1024), (650, 2568), (1300, 2560),
                                    (620, 5128), (6, 8200), (3, 16390)])
def test_same_bits_at_odd_places(cuda_lib, dtype, rows, D):
    z = inputs(rows, D, DT[dtype])
    ins = (z["x"], z["w"], z["b"], z["res"], z["dy"])

    def run(x, w, b, res, dy, y=None, out=None, dx=None, dw=None, db=None):
        fwd = cuda_lib.gdn_layer_norm_fwd(x, w, b, res, y, out, eps=EPS)
        bwd = cuda_lib.gdn_layer_norm_bwd(dy, x, w, res, dx, dw, db, eps=EPS)
        for mine, got in zip((y, out, dx, dw, db), fwd + bwd):
            assert mine is None or mine.data_ptr() == got.data_ptr()
        return fwd + bwd

    want = run(*ins)

    def same(got):
        return all(torch.equal(a, b) for a, b in zip(got, want))

    for i in range(5):
        assert same(run(*(odd(t) if j == i else t for j, t in enumerate(ins)))), i
        assert same(run(*ins, *(odd(torch.empty_like(t)) if j == i else None for j, t in enumerate(want)))), i
    assert same(run(*map(odd, ins), *(odd(torch.empty_like(t)) for t in want)))
    assert same(run(sliced(z["x"], 1, 2), *ins[1:4], sliced(z["dy"], 8, 1)))
    # in place at odd places
    res = odd(z["res"])
    y, r = cuda_lib.gdn_layer_norm_fwd(z["x"], z["w"], z["b"], res, residual_out=res, eps=EPS)
    assert torch.equal(y, want[0]) and torch.equal(res, want[1])
    res = odd(z["res"])
    dx, _, _ = cuda_lib.gdn_layer_norm_bwd(z["dy"], z["x"], z["w"], res, dx=res, eps=EPS)
    assert torch.equal(dx, want[2])
