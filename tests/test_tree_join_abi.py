"""gpt2_diag_tree_join on the host: invalid arguments are refused before anything
is launched (the addresses here are aligned and never read)."""
import pytest

from gpt_transformer_forward_gb300 import binding as ab
from gpt_transformer_forward_gb300 import build

FAKE = 1 << 20
A, S, AL, W, U = -1, -2, -3, -4, -7  # GPT2_ERR_ARG, _SHAPE, _ALIGN, _WORKSPACE, _UNSUPPORTED


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return ab.load(build_if_missing=False)


@pytest.mark.parametrize("change,code", [
    (dict(out=None), A), (dict(B=0), A), (dict(N=0), A), (dict(C=0), A), (dict(NH=0), A), (dict(precision=4), A),
    (dict(NH=3), S), (dict(N=65), S), (dict(B=65536), S), (dict(shares=0), S), (dict(shares=152 * 12 + 1), S),
    (dict(N=17, shares=152 * 6 + 1), S), (dict(N=33, shares=152 * 3 + 1), S), (dict(C=512), U),
    (dict(workspace=None), W), (dict(ws_bytes=1000), W), (dict(out=FAKE + 8), AL), (dict(workspace=FAKE + 8), AL),
])
def test_refuses(change, code):
    args = dict(out=FAKE, B=4, N=8, C=256, NH=4, shares=7, precision=ab.GPT2_FP16, workspace=FAKE, ws_bytes=1 << 30)
    args.update(change)
    with pytest.raises(ab.GPT2Error) as e:
        ab.gpt2_diag_tree_join(**args, stream=0)
    assert e.value.code == code
