"""Every call runs with its tensors' device as the current one (a launch goes to the current device, and the handle of a
default stream does not tell which it is)."""
import ast

import pytest
import torch


@pytest.fixture
def calls(monkeypatch):
    """The binding on CPU tensors that stand for those of device 1, with device 0 the current one: what it does, in order."""
    import fine_grained_blockwise_amd as fgb
    seen, current, real = [], [0], fgb.lib()

    class Device:
        def __init__(self, d):
            self.d = d

        def __enter__(self):
            current.append(self.d)
            seen.append("enter")

        def __exit__(self, *a):
            current.pop()
            seen.append("exit")

    class Lib:
        def __getattr__(self, name):
            if name.endswith("_size") or name == "fgb_last_error":
                return getattr(real, name)

            def entry(*a):
                seen.append((name, a[-1], type(a[-1])))
                return 0
            return entry
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(fgb, "_current_device", lambda: current[-1] if current[-1] == 0 else current[-1].index)
    monkeypatch.setattr(fgb, "_raw_stream", lambda index: 77)
    monkeypatch.setattr(fgb, "_check_dev", lambda *t: torch.device("cpu"))
    monkeypatch.setattr(fgb, "_lib", Lib())
    return fgb, seen


def ran(seen, *names):
    want = []
    for n in names:
        want += ["enter", (n, 77, int), "exit"]
    return seen == want


def test_router(calls):
    fgb, seen = calls
    z, b = torch.zeros(4, 8), torch.zeros(8)
    idx, w, counts, _ = fgb.moe_router(z, 2)
    fgb.moe_router(z, 2, bias=b)
    fgb.moe_router(z, 2, groups=4, topk_groups=2)
    fgb.moe_router_backward(z, idx, counts)
    fgb.moe_bias_update(b, counts, 1e-3)
    assert ran(seen, "moe_router", "moe_router_grouped", "moe_router_grouped", "moe_router_backward", "moe_bias_update")


def test_quantizers_and_products(calls):
    fgb, seen = calls
    x = torch.zeros(128, 256)
    q, s = fgb.fp8_quant_rowwise(x)
    wq, ws = fgb.fp8_quant_blockwise(x)
    fgb.fp8_dequant(q, s, fgb.ROW1x128)
    fgb.fp8_block_gemm(q, s, fgb.ROW1x128, wq, ws, fgb.BLOCK128)
    q4, s4 = fgb.mxfp4_quant(x)
    fgb.mxfp4_gemm(q4, s4, q4, s4)
    assert ran(seen, "fp8_quant_rowwise", "fp8_quant_blockwise", "fp8_dequant", "fp8_block_gemm", "mxfp4_quant", "mxfp4_gemm")


def test_on_the_current_device_nothing_is_entered(calls, monkeypatch):
    fgb, seen = calls
    monkeypatch.setattr(fgb, "_current_device", lambda: -1)  # (what a CPU tensor says)
    fgb.moe_router(torch.zeros(4, 8), 2)
    assert seen == [("moe_router", 77, int)]


def test_every_entry_goes_through_it():
    """Nothing in the binding launches but _call, whose last argument is a stream's handle of _stream."""
    import fine_grained_blockwise_amd as fgb
    tree = ast.parse(open(fgb.__file__).read())
    found = 0
    for f in tree.body:
        if not isinstance(f, ast.FunctionDef):
            continue
        source = ast.unparse(f)
        for node in ast.walk(f):
            if isinstance(node, ast.Call) and isinstance(node.func, ast.Name) and node.func.id == "_call":
                if f.name in ("_call", "_call_on"):
                    continue
                last = ast.unparse(node.args[-1])
                assert last.startswith("_stream(") or (last == "*out" and "_stream(logits))" in source), (f.name, last)
                found += 1
            if isinstance(node, ast.Attribute) and ast.unparse(node.value) == "_lib":
                assert node.attr.endswith("_size") or node.attr in ("fgb_last_error", "mxfp4_gemm_tiled"), (f.name, node.attr)
    assert found >= 40
