"""What the recurrent layers write lies apart from what they read, parameters, bounds and
workspaces among it (no GPU needed: the calls are refused before the device is touched)."""
import pytest

import chunked_gated_delta_11_gb300 as kda
from test_recurrent_args import FAKE, FAR, INVALID, WORKSPACE, conv, lib, ssm  # noqa: F401

HERE = 1 << 40  # apart from FAKE and FAR


@pytest.mark.parametrize("kw", [
    dict(out=HERE, w=HERE + 16), dict(out=HERE, bias=HERE + 64 * 128 - 16), dict(out=HERE, cu=HERE + 4),
    dict(fin=HERE, w=HERE + 2 * 3 * 64 - 16), dict(fin=HERE, bias=HERE), dict(fin=HERE, cu=HERE - 4),
    dict(T=0, x=0, out=0, fin=HERE, w=HERE),
])
def test_conv_rejects_overlaps(lib, kw):  # noqa: F811
    assert conv(lib, **kw) == INVALID


SSM = [dict(out=HERE, A=HERE + 16), dict(out=HERE, skip=HERE + 64 * 512 - 4), dict(out=HERE, bias=HERE), dict(out=HERE, cu=HERE - 4),
       dict(fin=HERE, A=HERE + 4 * 64 * 128 * 4 - 4), dict(fin=HERE, skip=HERE + 8), dict(fin=HERE, bias=HERE - 12),
       dict(fin=HERE, cu=HERE), dict(T=0, x=0, dt=0, B=0, C=0, out=0, fin=HERE, A=HERE)]


@pytest.mark.parametrize("entry,ws", [("kda_ssm_step", ()), ("kda_ssm_fwd", (None, 0))])
@pytest.mark.parametrize("kw", SSM)
def test_ssm_rejects_overlaps(lib, entry, ws, kw):  # noqa: F811
    assert ssm(lib, entry=entry, ws=ws, **kw) == INVALID


@pytest.mark.parametrize("name", ["x", "dt", "A", "B", "C", "skip", "bias", "cu", "init", "fin", "out"])
def test_ssm_rejects_a_workspace_over_the_rest(lib, name):  # noqa: F811
    need = kda.kda_ssm_workspace_size(8192, 4, 2, 1, 64, 128)
    assert need > 0
    far = dict(out=FAR, fin=FAR * 2)
    for at in (HERE, HERE + need - 16):
        assert ssm(lib, entry="kda_ssm_fwd", T=8192, ws=(HERE, need), **{**far, name: at}) == INVALID
    # one that is too small or skewed is refused as that
    assert ssm(lib, entry="kda_ssm_fwd", T=8192, ws=(HERE, need - 1), **{**far, name: HERE}) == WORKSPACE
    assert ssm(lib, entry="kda_ssm_fwd", T=8192, ws=(HERE + 8, need), **far) == WORKSPACE


@pytest.mark.parametrize("which", [0, 2, 3])
def test_ssm_fwd_rejects_strides_that_no_tensor_map_holds(lib, which):  # noqa: F811
    strides = tuple(i == which and 1 << 39 for i in range(4))
    kw = dict(T=2, strides=strides, out=1 << 50, fin=1 << 52)
    assert ssm(lib, entry="kda_ssm_fwd", ws=(None, 0), **kw) == INVALID
