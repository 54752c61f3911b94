"""The short calls' host code on the CPU: the same source, built to take host
tensors, around entry points that do nothing.  Each test runs in a process of
its own, so that a crash fails the test that caused it."""

import os
import subprocess
import sys
import sysconfig
import textwrap

import pytest
import torch

import bit_grouped_moe_amd.build as build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PRELUDE = """
import ctypes, importlib.machinery, importlib.util, sys
import torch
loader = importlib.machinery.ExtensionFileLoader("_calls", sys.argv[1])
calls = importlib.util.module_from_spec(importlib.util.spec_from_loader("_calls", loader))
loader.exec_module(calls)
import bit_grouped_moe_amd as gq
done = []                                  # entry points that were called
def stub(name):
    def f(*a):
        done.append(name)
        return 3 if name == "gq_route_max_tiles" else 0
    return ctypes.CFUNCTYPE(*[gq._SIGNATURES[name][0]] + gq._SIGNATURES[name][1])(f)
stubs = {n: stub(n) for n in gq.EXPORTED_SYMBOLS if n != "gq_status_string"}
calls.bind({n: ctypes.cast(f, ctypes.c_void_p).value for n, f in stubs.items()},
           lambda: -1, lambda index: 0)    # the device index of a host tensor is -1
z = torch.zeros(3, 4, 8)
x = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
ids = torch.zeros(3, 4, 2, dtype=torch.int32)
w = torch.zeros(3, 4, 2)
xb, xs = torch.zeros(3, 4, 2, 16, dtype=torch.uint8), torch.zeros(3, 4, 2, dtype=torch.uint8)
bank = torch.zeros(5, 32, 2, 16, dtype=torch.uint8), torch.zeros(5, 32, 2, dtype=torch.uint8)
route = gq.Route(torch.zeros(6, dtype=torch.int32), torch.zeros(8, dtype=torch.int32),
                 torch.zeros(3, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32),
                 3, 256, 4, 2, 5)
layer = gq._LayerStruct(hidden=64)
address = ctypes.addressof(layer)
"""


@pytest.fixture(scope="module")
def module(tmp_path_factory):
    """csrc/binding/calls.cpp for host tensors."""
    d = tmp_path_factory.mktemp("calls")
    with open(build.CALLS_SRC) as f:
        text = f.read()
    assert text.count("t.is_cuda()") == 1
    text = text.replace("t.is_cuda()", "t.is_cpu()").replace("DispatchKey::CUDA", "DispatchKey::CPU")
    text = text.replace("../../../include/gq.h", os.path.join(ROOT, "include", "gq.h"))
    src, lib = d / "calls.cpp", d / "_calls.so"
    src.write_text(text)
    root = os.path.dirname(torch.__file__)
    inc = os.path.join(root, "include")
    subprocess.run(
        [os.environ.get("CXX", "g++"), "-O0", "-std=c++17", "-fPIC", "-shared", "-w",
         "-D__HIP_PLATFORM_AMD__", '-DGQ_TORCH_VERSION="host"', '-DGQ_HEADER_ID="host"',
         f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
         "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
         "-isystem", os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "include"),
         "-isystem", sysconfig.get_paths()["include"], str(src), "-o", str(lib),
         "-L" + os.path.join(root, "lib"), "-lc10", "-ltorch_cpu", "-ltorch_python"], check=True)
    return str(lib)


def _run(module, code):
    r = subprocess.run([sys.executable, "-c", PRELUDE + textwrap.dedent(code), module], cwd=ROOT,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (r.returncode, r.stdout[-2000:], r.stderr[-2000:])


# Each short call on the parts of the prelude's tensors that a function transform
# hands over: (call, its arguments).
CALLS = {
    "quantize": ("lambda x: calls.quantize(x, True)", "x"),
    "moe_topk": ("lambda z: calls.moe_topk(z, 2, True)", "z"),
    "moe_topk_backward": ("lambda w, z, ids: calls.moe_topk_backward(w, z, ids, False)", "w, z, ids"),
    "route_sort": ("lambda ids: calls.route_sort(ids, 5, 256)", "ids"),
    "moe_decode": ("lambda x: calls.moe_decode(address, -1, 64, x)", "x"),
    "fp4_gemv": ("lambda xb, xs, ids: calls.fp4_gemv(xb, xs, *bank, ids, None, False, 0.0, 0.0)",
                 "xb, xs, ids"),
    "fp4_gemm": ("lambda xb, xs: calls.fp4_gemm(xb, xs, *bank, route, None, True, 1.0, 1.0)",
                 "xb, xs"),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_tensors_without_storage_are_left_to_the_python_code(module, name):
    """A tensor inside torch.func.vmap is exactly a torch.Tensor and has no
    memory: the short call leaves it alone, as anything else that is not a
    plain device tensor, and launches nothing."""
    f, args = CALLS[name]
    _run(module, f"""
        f = {f}
        assert f(*[t[0] for t in ({args},)]) is not None      # the plain tensors are taken
        count = len(done)
        assert count
        got = []
        torch.func.vmap(lambda *a: got.append(f(*a)) or a[0])({args})
        assert got == [None], got
        assert not [n for n in done[count:] if n != "gq_route_max_tiles"]
    """)


@pytest.mark.parametrize("name", sorted(CALLS))
def test_outputs_without_storage_raise(module, name):
    """Plain tensors used inside torch.func.grad, whose allocations torch
    wraps: an error, as with the Python code, or outputs, and no crash."""
    f, args = CALLS[name]
    _run(module, f"""
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
    """)


@pytest.mark.parametrize("name", ["quantize", "moe_topk", "route_sort"])
def test_outputs_have_their_own_storage(module, name):
    """An output may grow in place, be saved and be kept without its siblings:
    it shares no memory with them."""
    f, args = CALLS[name]
    _run(module, f"""
        outs = ({f})(*[t[0] for t in ({args},)])
        assert len({{t.untyped_storage().data_ptr() for t in outs}}) == len(outs)
        for t in outs:
            assert t.untyped_storage().nbytes() == t.numel() * t.element_size()
        for i, t in enumerate(outs):
            rest = [o for j, o in enumerate(outs) if j != i]
            for o in rest:
                o.fill_(1)
            t.resize_(4096)
            t.zero_()
            assert all((o == 1).all() for o in rest)
    """)


def test_bind_takes_all_or_nothing(module):
    """A binding that lacks an entry point leaves the earlier one as it was."""
    _run(module, """
        for bad in ({}, {"gq_mxfp4_quantize": 16}, {"gq_mxfp4_quantize": 0}, None):
            try:
                calls.bind(bad, None, None)
                raise SystemExit("bound")
            except (KeyError, TypeError):
                pass
            count = len(done)
            assert calls.quantize(x[0], False) is not None and len(done) == count + 1
    """)


@pytest.mark.parametrize("name", sorted(CALLS))
def test_modes_see_the_allocations(module, name):
    """A dispatch mode is told of the outputs, as of torch's own; without one
    they are what torch.empty makes, in and out of inference mode."""
    f, args = CALLS[name]
    _run(module, f"""
        from torch.utils._python_dispatch import TorchDispatchMode
        f = {f}
        plain = [t[0] for t in ({args},)]
        seen = []
        class Mode(TorchDispatchMode):
            def __torch_dispatch__(self, func, types, args=(), kwargs=None):
                seen.append(str(func))
                return func(*args, **(kwargs or {{}}))
        flat = lambda r: r if isinstance(r, tuple) else (r,)
        first = flat(f(*plain))
        with Mode():
            under = flat(f(*plain))
        assert sum("empty" in s for s in seen) >= len(first), seen
        with torch.inference_mode():
            inference = flat(f(*plain))
        for a, b, c in zip(first, under, inference):
            like = torch.empty(a.shape, dtype=a.dtype)
            for t in (a, b):
                assert (t.dtype, t.shape, t.stride(), t.device, t.requires_grad, t.is_inference()) == (
                    like.dtype, like.shape, like.stride(), like.device, False, False)
                assert torch._C._dispatch_keys(t) == torch._C._dispatch_keys(like)
                assert t._version == 0 and t.untyped_storage().resizable()
            assert c.is_inference() and not c.requires_grad
    """)


def test_route_sizes_past_32_bits_are_left_to_the_python_code(module):
    """A tile height or count whose low half would pass is not passed on."""
    _run(module, """
        call = lambda r: calls.fp4_gemm(xb[0], xs[0], *bank, r, None, False, 0.0, 0.0)
        assert call(route) is not None
        count = len(done)
        for bad in (route._replace(tile_m=256 - (1 << 32)), route._replace(tile_m=256 + (1 << 32)),
                    route._replace(max_tiles=3 + (1 << 32)), route._replace(max_tiles=3 - (1 << 32)),
                    route._replace(topk=2 + (1 << 32)), route._replace(topk=2 - (1 << 32))):
            assert call(bad) is None
        assert len(done) == count
    """)
