"""The norm of rows where a workgroup goes through several of them, and dropout inside it at every width that has kernels
of its own (GPU): the checks and the derived bounds are those of test_layer_norm_gpu.py."""
import pytest

from tests.test_layer_norm_gpu import IDS, TYPES, check_bwd, check_fwd, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
@pytest.mark.parametrize("types", TYPES, ids=IDS)
@pytest.mark.parametrize("rows,E", [(20000, 129), (9000, 767), (5000, 768), (3000, 4099), (200, 8200), (30000, 40), (9001, 512)])
def test_gradients_of_rows_in_turn(types, rows, E, rms):
    """Teams that take several rows: their sums over lanes in turn, dweight and dbias over all of them."""
    print("case: gradients of rows in turn", types, rows, E, rms, flush=True)
    i = make((rows, E), *types, seed=rows + E)
    check_bwd(i, rms=rms)


@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
@pytest.mark.parametrize("types", TYPES, ids=IDS)
@pytest.mark.parametrize("E", [300, 511, 768, 1025, 4099, 8192, 8200, 16392, 40001])
def test_dropout_inside_rows(types, E, rms):
    """Rows of teams of 64 lanes, of workgroups, of two pieces a lane, and those that are read again for each pass."""
    print("case: dropout inside rows", types, E, rms, flush=True)
    kw = dict(rms=rms, p=0.3, seed=(5 << 40) + E, call=7)
    i = make((7, E), *types, seed=E)
    check_fwd(i, **kw)
    check_bwd(i, **kw)
    check_fwd(dict(i, residual=None), **kw)
    if types[0] == types[1]:
        check_bwd(i, residual=False, **kw)
    if E < 2000:  # several rows for a team
        check_bwd(make((1500, E), *types, seed=E + 1), **kw)
