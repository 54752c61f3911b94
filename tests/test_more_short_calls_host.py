"""The short calls of the norm, the 8-bit quantiser and products and the routing
with groups on the CPU, as the others are tested: the same source, built to take
host tensors, around entry points that do nothing."""

import pytest

from tests.test_short_calls_host import _run, module  # noqa: F401  (module: a fixture)

MORE = """
gain = torch.zeros(64, dtype=torch.bfloat16)
bias = torch.zeros(8)
codes = torch.zeros(3, 4, 64, dtype=torch.uint8)
"""

CALLS = {
    "quantize8": ("lambda x: calls.quantize8(x, True)", "x"),
    "rms_norm": ("lambda x: calls.rms_norm(x, gain, 1e-6, x, True, True)", "x"),
    "rms_norm_plain": ("lambda x: calls.rms_norm(x, gain, 1e-6, None, False, False)", "x"),
    "rms_norm_backward": ("lambda x: calls.rms_norm_backward(x, x, gain, 1e-6, x, True)", "x"),
    "moe_route": ("lambda z: calls.moe_route(z, 2, 1, bias, 4, 2, 2, True, 2.5)", "z"),
    "moe_route_backward": ("lambda w, z, ids: calls.moe_route_backward(w, z, ids, 1, False, 2.0)",
                           "w, z, ids"),
    "fp8_gemv": ("lambda c, xs, ids: calls.fp8_gemv(c, xs, *bank, ids, None, False, 0.0, 0.0)",
                 "codes, xs, ids"),
    "fp8_gemm": ("lambda c, xs: calls.fp8_gemm(c, xs, *bank, route, None, True, 1.0, 1.0)",
                 "codes, xs"),
}


def _with(code):
    """The test's code after this module's own tensors."""
    import textwrap
    return MORE + textwrap.dedent(code)


@pytest.mark.parametrize("name", sorted(CALLS))
def test_tensors_without_storage_are_left_to_the_python_code(module, name):  # noqa: F811
    f, args = CALLS[name]
    _run(module, _with(f"""
        f = {f}
        assert f(*[t[0] for t in ({args},)]) is not None      # the plain tensors are taken
        count = len(done)
        assert count
        got = []
        torch.func.vmap(lambda *a: got.append(f(*a)) or a[0])({args})
        assert got == [None], got
        assert not [n for n in done[count:] if not n.endswith(("_max_tiles", "_workspace"))]
    """))


@pytest.mark.parametrize("name", sorted(CALLS))
def test_outputs_without_storage_raise(module, name):  # noqa: F811
    f, args = CALLS[name]
    _run(module, _with(f"""
        f = {f}
        plain = [t[0] for t in ({args},)]
        got = []
        def inside(s):
            try:
                got.append(f(*plain))
            except RuntimeError as e:
                got.append(e)
            return s * 2
        torch.func.grad(inside)(torch.tensor(1.0))
        assert len(got) == 1 and got[0] is not None, got
        assert f(*plain) is not None                          # and works on after it
    """))


def test_outputs_that_are_not_asked_for_are_none(module):  # noqa: F811
    _run(module, _with("""
        y, h, c, s, v = calls.rms_norm(x[0], gain, 1e-6, None, False, False)
        assert y.shape == (4, 64) and h is c is s is v is None
        y, h, c, s, v = calls.rms_norm(x[0], gain, 1e-6, x[1], True, False)
        assert h.shape == (4, 64) and c.shape == (4, 64) and s.shape == (4, 2) and v is None
        dx, dw = calls.rms_norm_backward(x[0], x[1], gain, 1e-6, None, False)
        assert dx.shape == (4, 64) and dw is None
        dx, dw = calls.rms_norm_backward(x[0], x[1], gain.float(), 1e-6, None, True)
        assert dw.shape == (64,) and dw.dtype == torch.float32
    """))


def test_what_is_not_an_ordinary_call_is_left_to_the_python_code(module):  # noqa: F811
    _run(module, _with("""
        count = len(done)
        for bad in (lambda: calls.rms_norm(x[0], gain, "1", None, False, False),
                    lambda: calls.rms_norm(x[0], gain.half(), 1e-6, None, False, False),
                    lambda: calls.rms_norm(x[0], gain[:32], 1e-6, None, False, False),
                    lambda: calls.rms_norm(x[0], gain, 1e-6, x[0, :2], False, False),
                    lambda: calls.rms_norm(x[0], gain, 1e-6, x[0].float(), False, False),
                    lambda: calls.rms_norm(x[0], gain, 1e-6, None, False, True),
                    lambda: calls.rms_norm(x[0, :, :40], gain[:40], 1e-6, None, True, False),
                    lambda: calls.rms_norm(x.transpose(0, 1), gain, 1e-6, None, False, False),
                    lambda: calls.rms_norm_backward(None, x[0], gain, 1e-6, None, True),
                    lambda: calls.rms_norm_backward(x[0, :1], x[0], gain, 1e-6, None, True),
                    lambda: calls.moe_route(z[0], 9, 1, None, 1, 1, 1, True, 1.0),
                    lambda: calls.moe_route(z[0], 2, 1, None, 3, 1, 1, True, 1.0),
                    lambda: calls.moe_route(z[0], 2, 1, None, 0, 1, 1, True, 1.0),
                    lambda: calls.moe_route(z[0], 2, 1, None, 1 << 40, 1, 1, True, 1.0),
                    lambda: calls.moe_route(z[0], 2, 1, None, 1, 1 << 70, 1, True, 1.0),
                    lambda: calls.moe_route(z[0], 2, 1, bias[:7], 1, 1, 1, True, 1.0),
                    lambda: calls.moe_route(z[0], 2, 1, bias.half(), 1, 1, 1, True, 1.0),
                    lambda: calls.moe_route(z[0], 2, 1, None, 1, 1, 1, True, "x"),
                    lambda: calls.moe_route_backward(w[0], z[0], ids[0], 1, True, None),
                    lambda: calls.fp8_gemv(codes[0, :, :32], xs[0], *bank, ids[0], None, False, 0.0,
                                           0.0),
                    lambda: calls.fp8_gemv(xb[0], xs[0], *bank, ids[0], None, False, 0.0, 0.0)):
            assert bad() is None
        assert not [n for n in done[count:] if not n.endswith("_workspace")], done[count:]
    """))
