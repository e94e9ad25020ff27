"""Host-side checks of the expert feed-forward and MXFP4 entry points (no GPU
needed): refusals with every reason before any device work, workspace sizes,
the calls that launch nothing, and the Python layer's argument checks."""
from __future__ import annotations

import copy
import ctypes
import os
import pickle
import re
import subprocess
import threading
import time
import types
import weakref

import pytest

from moe_router_top_gb300 import _lib
from moe_router_top_gb300._lib import ExpertDownArgs, ExpertUpArgs

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    from moe_router_top_gb300 import build
    build.build()
    return _lib.load()


@pytest.fixture(scope="module")
def smr(lib):
    import moe_router_top_gb300
    return moe_router_top_gb300


P = 0x10000


def _up(**over):
    a = ExpertUpArgs(4, 11, 256, 128, 65, 64, P, 256, None, P, None, P, 44 + 65 * 63, P, P, P)
    for k, v in over.items():
        setattr(a, k, v)
    return a


def _down(**over):
    a = ExpertDownArgs(4, 11, 256, 128, 65, 64, P, None, P, None, P, P, 65, P, 44 + 65 * 63, P, P, P)
    for k, v in over.items():
        setattr(a, k, v)
    return a


def _refused(lib, fn, a, status, *frags):
    assert fn(ctypes.byref(a), P, 1 << 40, None) == status
    msg = lib.smr_last_error().decode()
    for f in frags:
        assert f in msg, msg
    assert lib.smr_last_launch_count() == 0


def test_struct_layouts():
    assert ctypes.sizeof(ExpertUpArgs) == 6 * 4 + 10 * 8 and ExpertUpArgs.x.offset == 24
    assert ctypes.sizeof(ExpertDownArgs) == 6 * 4 + 12 * 8 and ExpertDownArgs.num_logical.offset == 72


INVALID, UNSUP, WORKSPACE = _lib.SMR_ERR_INVALID_ARG, _lib.SMR_ERR_UNSUPPORTED, _lib.SMR_ERR_WORKSPACE


@pytest.mark.parametrize("over,status,frag", [
    (dict(num_tokens=-1), INVALID, "num_tokens must be >= 0"),
    (dict(width=0), INVALID, "width must be >= 1"),
    (dict(H=250), INVALID, "multiple of 16"),
    (dict(H=16400), INVALID, "16384"),
    (dict(I=8), INVALID, "multiple of 16"),
    (dict(num_experts=0), INVALID, "num_experts must be in [1, 1025]"),
    (dict(num_experts=1026), INVALID, "num_experts must be in [1, 1025]"),
    (dict(block_size=32), UNSUP, "block_size must be 64 or 128"),
    (dict(x=None), INVALID, "x must be"),
    (dict(x=P + 8), INVALID, "x must be"),
    (dict(w=P + 4), INVALID, "w must be"),
    (dict(x_scales=P), INVALID, "both be set"),
    (dict(w_scales=P), INVALID, "both be set"),
    (dict(sorted_token_ids=None), INVALID, "must be set"),
    (dict(expert_ids=P + 2), INVALID, "4-byte aligned"),
    (dict(num_tokens_post_padded=None), INVALID, "must be set"),
    (dict(sorted_cap=0), INVALID, "sorted_cap must be >= 1"),
    (dict(sorted_cap=1 << 31), UNSUP, "int32 indexing"),
    (dict(num_tokens=1 << 27), UNSUP, "2^30"),
])
def test_product_refusals(lib, over, status, frag):
    _refused(lib, lib.smr_expert_up, _up(**over), status, "smr_expert_up", frag)
    _refused(lib, lib.smr_expert_down, _down(**over), status, "smr_expert_down", frag)


def test_own_refusals(lib):
    _refused(lib, lib.smr_expert_up, _up(ld_x=248), INVALID, "ld_x must be >= H")
    _refused(lib, lib.smr_expert_up, _up(ld_x=260), INVALID, "multiple of 8")
    _refused(lib, lib.smr_expert_up, _up(ld_x=1 << 31), UNSUP, "2^30")
    _refused(lib, lib.smr_expert_up, _up(act=None), INVALID, "act must be")
    _refused(lib, lib.smr_expert_down, _down(out=P + 8), INVALID, "out must be")
    _refused(lib, lib.smr_expert_down, _down(topk_ids=None), INVALID, "topk_ids must be")
    _refused(lib, lib.smr_expert_down, _down(topk_weights=P + 1), INVALID, "topk_weights must be")
    _refused(lib, lib.smr_expert_down, _down(num_logical=0), INVALID, "num_logical must be in")
    # every reason in one message
    _refused(lib, lib.smr_expert_up, _up(width=0, H=7, I=0), INVALID, "width must", "H must", "I must")
    # blocks x weight tiles
    _refused(lib, lib.smr_expert_up, _up(I=16384, sorted_cap=(1 << 31) - 1), UNSUP, "blocks x weight tiles")


def test_mxfp4_products_ask_for_whole_scale_groups(lib):
    mx = dict(x_scales=P, w_scales=P)
    _refused(lib, lib.smr_expert_up, _up(H=192, ld_x=192, **mx), INVALID, "H must be a multiple of 128")
    _refused(lib, lib.smr_expert_down, _down(I=160, **mx), INVALID, "I must be a multiple of 128")
    _refused(lib, lib.smr_expert_up, _up(x_scales=P + 2, w_scales=P), INVALID, "x_scales must be 4-byte")
    _refused(lib, lib.smr_expert_up, _up(x_scales=P, w_scales=P + 8), INVALID, "w_scales must be 16-byte")


def test_workspaces(lib):
    up, down = _up(), _down()
    assert lib.smr_expert_up_workspace_size(ctypes.byref(up)) == 256
    # the rows sit behind a small route's keys (16 tokens x 1024 experts x 8 bytes)
    need = 256 + 16 * 1024 * 8 + 44 * 256 * 4  # fp32 rows
    assert lib.smr_expert_down_workspace_size(ctypes.byref(down)) == need
    many = _down(num_tokens=4096)  # above 2^23 values: bf16 rows
    assert lib.smr_expert_down_workspace_size(ctypes.byref(many)) == 256 + 16 * 1024 * 8 + 4096 * 11 * 256 * 2
    assert lib.smr_expert_up(ctypes.byref(up), None, 0, None) == WORKSPACE
    assert lib.smr_expert_down(ctypes.byref(down), P, need - 1, None) == WORKSPACE
    assert lib.smr_expert_down(ctypes.byref(down), P + 128, need, None) == WORKSPACE
    assert lib.smr_expert_up(None, P, 256, None) == INVALID
    assert lib.smr_expert_down(None, P, 256, None) == INVALID
    assert lib.smr_expert_down_workspace_size(None) == 0


def test_nothing_to_do(lib):
    for fn, a in ((lib.smr_expert_up, ExpertUpArgs(0, 1, 16, 16, 1, 64)),
                  (lib.smr_expert_down, ExpertDownArgs(0, 1, 16, 16, 1, 64, num_logical=1))):
        assert fn(ctypes.byref(a), None, 0, None) == _lib.SMR_OK
        assert lib.smr_last_launch_count() == 0
    assert lib.smr_quantize_mxfp4(None, 0, 32, 32, None, None, None) == _lib.SMR_OK
    assert lib.smr_dequantize_mxfp4(None, None, 0, 32, None, None) == _lib.SMR_OK


@pytest.mark.parametrize("args,frag", [
    ((P, -1, 32, 32, P, P), "rows must be >= 0"),
    ((P, 4, 48, 48, P, P), "multiple of 32"),
    ((P, 4, 0, 32, P, P), "multiple of 32"),
    ((P, 4, 64, 32, P, P), "ld_x must be >= K"),
    ((P, 4, 64, 68, P, P), "multiple of 8"),
    ((P + 2, 4, 64, 64, P, P), "x must be a 16-byte"),
    ((P, 4, 64, 64, P + 2, P), "codes must be a 4-byte"),
    ((P, 4, 64, 64, P, None), "scales is NULL"),
    ((P, 1 << 40, 64, 64, P, P), "2^34"),
])
def test_quantize_refusals(lib, args, frag):
    assert lib.smr_quantize_mxfp4(*args, None) in (INVALID, UNSUP)
    assert frag in lib.smr_last_error().decode()


def test_dequantize_and_layout_refusals(lib):
    assert lib.smr_dequantize_mxfp4(P, P, 4, 64, P + 8, None) == INVALID
    assert "out must be a 16-byte" in lib.smr_last_error().decode()
    assert lib.smr_tile_mxfp4_scales(P, 2, 48, 128, 1, P, None) == INVALID
    assert "multiple of 32" in lib.smr_last_error().decode()
    assert lib.smr_tile_mxfp4_scales(P, 2, 64, 96, 0, P, None) == INVALID
    assert lib.smr_tile_mxfp4_scales(P + 1, 2, 64, 128, 2, None, None) == INVALID
    msg = lib.smr_last_error().decode()
    assert "gated must" in msg and "scales must" in msg and "tiled must" in msg
    assert lib.smr_mxfp4_tiled_scale_bytes(3, 160, 256, 0) == 3 * 2 * 2 * 512
    assert lib.smr_mxfp4_tiled_scale_bytes(3, 160, 256, 1) == 3 * 2 * 2 * 512  # 80 features: two tiles of 64
    assert lib.smr_mxfp4_tiled_scale_bytes(3, 160, 96, 0) == 0


def _align_outputs(T, width, E, A):
    cap = T * width + E * (A - 1)
    return (torch.zeros(cap, dtype=torch.int32), torch.zeros((cap + A - 1) // A, dtype=torch.int32),
            torch.zeros(1, dtype=torch.int32))


def test_python_checks(smr):
    T, width, E, H, I, A = 3, 2, 4, 64, 32, 64
    x, w = torch.zeros(T, H, dtype=torch.bfloat16), torch.zeros(E, 2 * I, H, dtype=torch.bfloat16)
    al = _align_outputs(T, width, E, A)
    kw = dict(width=width, block_size=A)
    with pytest.raises(ValueError, match="CUDA device"):
        smr.expert_up(x, w, *al, **kw)
    for bad, frag in ((dict(x=x.float()), "x must be"), (dict(x=x[:, ::2]), "x must be"), (dict(x=x[0]), "x must be"),
                      (dict(w=w[:, :, :32]), "w must be"), (dict(w=w.transpose(1, 2)), "must be"),
                      (dict(w=w[:, :33]), "2 I")):
        with pytest.raises(ValueError, match=frag):
            smr.expert_up(bad.get("x", x), bad.get("w", w), *al, **kw)
    with pytest.raises(ValueError, match="int32"):
        smr.expert_up(x, w, al[0].long(), al[1], al[2], **kw)
    with pytest.raises(ValueError, match="entry for every block"):
        smr.expert_up(x, w, al[0], al[1][:1], al[2], **kw)
    with pytest.raises(ValueError, match="both be given"):
        smr.expert_up(x, w, *al, x_scales=x, **kw)
    with pytest.raises(ValueError, match="width must be"):
        smr.expert_up(x, w, *al, width=0, block_size=A)
    ids, wts = torch.zeros(T, width, dtype=torch.int32), torch.zeros(T, width)
    act, w2 = torch.zeros(T * width, I, dtype=torch.bfloat16), torch.zeros(E, H, I, dtype=torch.bfloat16)
    for bad, frag in ((dict(ids=ids.long()), "topk_ids"), (dict(wts=wts.double()), "topk_weights"),
                      (dict(act=act[:-1]), "x must be"), (dict(wts=wts[:2]), "topk_weights")):
        with pytest.raises(ValueError, match=frag):
            smr.expert_down(bad.get("act", act), w2, bad.get("ids", ids), bad.get("wts", wts), *al, block_size=A)
    with pytest.raises(ValueError, match="CUDA device"):
        smr.expert_down(act, w2, ids, wts, *al, block_size=A)


def test_python_mxfp4_checks(smr):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA device"):
        smr.quantize_mxfp4(x)
    with pytest.raises(ValueError, match="multiple of 32"):
        smr.quantize_mxfp4(x[:, :48])
    with pytest.raises(ValueError, match="bfloat16"):
        smr.quantize_mxfp4(x.float())
    with pytest.raises(ValueError, match="contiguous"):
        smr.quantize_mxfp4(x.t())
    c, s = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    with pytest.raises(ValueError, match="scales must be"):
        smr.dequantize_mxfp4(c, s[:, :1])
    with pytest.raises(ValueError, match="CUDA device"):
        smr.dequantize_mxfp4(c, s)
    with pytest.raises(ValueError, match="scales must be"):
        smr.tile_mxfp4_scales(c)
    # MXFP4 operands of a product: types, scale shapes
    al = _align_outputs(4, 1, 2, 64)
    codes, sc = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.uint8)
    w = torch.zeros(2, 64, 64, dtype=torch.uint8)
    ws = torch.zeros(2, 1, 1, 512, dtype=torch.uint8)
    with pytest.raises(ValueError, match="x_scales must be"):
        smr.expert_up(codes, w, *al, width=1, block_size=64, x_scales=sc[:, :2], w_scales=ws)
    with pytest.raises(ValueError, match="w_scales must be"):
        smr.expert_up(codes, w, *al, width=1, block_size=64, x_scales=sc, w_scales=ws[:1])
    with pytest.raises(ValueError, match="CUDA device"):
        smr.expert_up(codes, w, *al, width=1, block_size=64, x_scales=sc, w_scales=ws)


def test_disabled(smr, monkeypatch):
    monkeypatch.setenv("SMR_DISABLE", "1")
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for call in (lambda: smr.quantize_mxfp4(x), lambda: smr.dequantize_mxfp4(x, x), lambda: smr.tile_mxfp4_scales(x),
                 lambda: smr.expert_up(x, x, x, x, x, width=1, block_size=64),
                 lambda: smr.expert_down(x, x, x, x, x, x, x, block_size=64)):
        with pytest.raises(smr.SmrUnsupported):
            call()


class _Buffer:
    """Stands in for device memory."""
    device = "cuda:0"

    def __init__(self, n, dev=0, dense=True):
        self.n, self.nbytes, self.dev, self.dense = n, n, dev, dense

    def get_device(self):
        return self.dev

    def is_contiguous(self):
        return self.dense

    def numel(self):
        return self.n

    def data_ptr(self):
        return P


@pytest.fixture
def fake_device(smr, monkeypatch):
    """A device that the Python layer can 'launch' on: memory and streams are stand-ins."""
    c = types.SimpleNamespace(_cuda_getCurrentRawStream=lambda dev: 7, _cuda_isCurrentStreamCapturing=lambda: False)
    monkeypatch.setattr(smr, "_torch_module", types.SimpleNamespace(
        _C=c, device=torch.device, uint8=torch.uint8, zeros=lambda n, dtype, device: _Buffer(n)))
    monkeypatch.setattr(smr, "_stream_ws", {})
    return smr


def test_workspace_must_be_writable_there(fake_device):
    smr, args, calls = fake_device, ExpertUpArgs(), []

    def fn(*a):
        calls.append(a)
        return _lib.SMR_OK

    for bad, frag in ((torch.zeros(256, dtype=torch.uint8), "device"), (_Buffer(256, dev=1), "device"),
                      (_Buffer(256, dense=False), "contiguous")):
        holder = smr.Workspace(0, torch.device("cuda", 0))
        holder.buf = bad
        for ws in (bad, holder):
            with pytest.raises(ValueError, match=frag):
                smr._run_product(fn, lambda ref: 256, args, ws, 0)
    assert not calls
    smr._run_product(fn, lambda ref: 256, args, _Buffer(512), 0)
    smr._run_product(fn, lambda ref: 256, args, smr.Workspace(0, torch.device("cuda", 0)), 0)
    assert [a[1:] for a in calls] == [(P, 512, 7), (P, 256, 7)]


def test_threads_on_one_stream_take_turns(fake_device):
    """Calls of several threads on one stream share a workspace: the product
    and the sum of one call are launched with no other call's between them."""
    smr, busy, mixed = fake_device, [], []

    def fn(ref, ptr, n, s):
        if n < 1024:
            return WORKSPACE
        busy.append(1)
        mixed.append(len(busy) > 1)
        time.sleep(0.002)
        busy.pop()
        return _lib.SMR_OK

    threads = [threading.Thread(target=lambda: [smr._run_product(fn, lambda ref: 1024, ExpertDownArgs(), None, 0)
                                                for _ in range(10)]) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(mixed) == 40 and not any(mixed) and len(smr._stream_ws) == 1


def test_sizes_past_32_bits_are_refused(smr):
    """They would be cut off on the way into the library."""
    big = 1 << 32
    al = _align_outputs(3, 2, 4, 64)
    x, w = torch.zeros(3, 64, dtype=torch.bfloat16), torch.zeros(4, 64, 64, dtype=torch.bfloat16)
    for width, block_size in ((big + 2, 64), (2, big + 64)):
        with pytest.raises(ValueError, match="below 2"):
            smr.expert_up(x, w, *al, width=width, block_size=block_size)
    ids, wts, w2 = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2), torch.zeros(4, 64, 32, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="below 2"):
        smr.expert_down(torch.zeros(6, 32, dtype=torch.bfloat16), w2, ids, wts, *al, block_size=64, num_logical=big + 4)
    # (meta tensors: shapes without memory)
    with pytest.raises(ValueError, match="below 2"):
        smr.quantize_mxfp4(torch.empty(1, big + 32, dtype=torch.bfloat16, device="meta"))
    with pytest.raises(ValueError, match="below 2"):
        smr.dequantize_mxfp4(torch.empty(1, big // 2 + 16, dtype=torch.uint8, device="meta"),
                             torch.empty(1, big // 32 + 1, dtype=torch.uint8, device="meta"))
    with pytest.raises(ValueError, match="below 2"):
        smr.tile_mxfp4_scales(torch.empty(1, 1, big // 32 + 4, dtype=torch.uint8, device="meta"))


def test_growing_keeps_the_error_bits(smr):
    ws = smr.Workspace(256, "cpu")
    ws.buf[4], ws.buf[8] = 5, 9  # error bits; another word of the header
    ws.ensure(4096)
    assert ws.nbytes == 4096 and ws.buf.nonzero().flatten().tolist() == [4] and ws.buf[4] == 5
    ws.ensure(100)
    assert ws.nbytes == 4096


def test_growing_is_ordered_on_the_calls_stream(smr, monkeypatch):
    """A route on another stream than the current one zeroes its workspace there."""
    seen = []

    class Stream:
        cuda_stream = 7

    class Context:
        def __init__(self, s):
            self.s = s

        def __enter__(self):
            seen.append(self.s)

        def __exit__(self, *a):
            seen.append(None)

    def zeros(n, dtype, device):
        seen.append("zeros")
        return torch.zeros(n, dtype=dtype)

    monkeypatch.setattr(smr, "_torch_module", types.SimpleNamespace(
        cuda=types.SimpleNamespace(stream=Context), device=torch.device, uint8=torch.uint8, zeros=zeros,
        _C=types.SimpleNamespace(_cuda_isCurrentStreamCapturing=lambda: False)))
    ws, s = smr.Workspace(0, "cuda:0"), Stream()
    calls = []

    def fn(*args):
        calls.append(args)
        return _lib.SMR_OK

    smr._launch(fn, ("a",), ws, 512, torch.device("cuda", 0), s)
    assert seen == [s, "zeros", None] and calls == [("a", ws.ptr, 512, 7)]
    smr._launch(fn, (), ws, 512, torch.device("cuda", 0), s)
    assert len(seen) == 3 and calls[1] == (ws.ptr, 512, 7)


@pytest.fixture
def captured_device(smr, monkeypatch):
    """A stand-in device whose stream can be put under capture; memory is the host's."""
    state = types.SimpleNamespace(capturing=False)
    c = types.SimpleNamespace(_cuda_getCurrentRawStream=lambda dev: 7,
                              _cuda_isCurrentStreamCapturing=lambda: state.capturing)
    monkeypatch.setattr(smr, "_torch_module", types.SimpleNamespace(
        _C=c, device=torch.device, uint8=torch.uint8, zeros=lambda n, dtype, device: torch.zeros(n, dtype=dtype),
        cuda=types.SimpleNamespace(current_stream=lambda: types.SimpleNamespace(cuda_stream=7))))
    monkeypatch.setattr(smr, "_default_ws", {})
    monkeypatch.setattr(smr, "_check_buffer", lambda ws, dev: None)
    return state


def test_no_growth_under_capture(smr, captured_device):
    calls = []

    def fn(ref, ptr, n, s):
        calls.append(n)
        return _lib.SMR_OK if n >= 1024 else WORKSPACE

    captured_device.capturing = True
    dev = torch.device("cuda", 0)
    for ws in (smr.Workspace(0, dev), smr.Workspace(0, dev)):
        captured_device.capturing = False
        ws.ensure(512)
        captured_device.capturing = True
        before = ws.buf
        with pytest.raises(smr.SmrError, match="being captured"):
            smr._run_product(fn, lambda ref: 1024, ExpertDownArgs(), ws, 0)
        with pytest.raises(smr.SmrError, match="being captured"):
            smr._launch(fn, (None,), ws, 1024, dev, None)
        assert ws.buf is before
    with pytest.raises(smr.SmrError, match="being captured"):
        smr.Workspace(256, dev)
    assert calls == [512, 512]
    # a route without a workspace: the capture gets memory of its own, the shared one is left alone
    assert smr._launch(fn, (None,), None, 2048, dev, 7) == _lib.SMR_OK
    assert calls[2:] == [2048] and smr._default_ws["cuda", 0].buf is None
    captured_device.capturing = False
    smr._launch(fn, (None,), None, 2048, dev, None)
    assert calls[3:] == [2048] and smr._default_ws["cuda", 0].nbytes == 2048


def test_memory_of_a_capture_is_kept(smr, captured_device):
    """A graph goes on writing to the memory that it was captured with."""
    ws = smr.Workspace(1024, torch.device("cuda", 0))
    captured_device.capturing = True
    smr._run_product(lambda *a: _lib.SMR_OK, lambda ref: 1024, ExpertDownArgs(), ws, 0)
    captured_device.capturing = False
    old = weakref.ref(ws.buf)
    ws.ensure(4096)
    assert old() is not None and old() is not ws.buf
    free = weakref.ref(ws.buf)
    ws.ensure(8192)  # no capture has used these
    assert free() is None and old() is not None
    captured_device.capturing = True
    smr._launch(lambda *a: _lib.SMR_OK, (), ws, 8192, torch.device("cuda", 0), 7)
    captured_device.capturing = False
    used = weakref.ref(ws.buf)
    ws.ensure(16384)
    assert used() is not None


def test_expert_error_word_refusals(lib):
    assert lib.smr_get_expert_error(None, None) == INVALID
    assert "code_out is NULL" in lib.smr_last_error().decode()


def test_launches_of_a_call_stay_together(tmp_path):
    """Through the C interface, two threads, one workspace: every product is
    followed by its own sum."""
    from moe_router_top_gb300 import build
    exe, here = tmp_path / "launch_order", os.path.dirname(__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(build.nvcc())), "include")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-I" + build.INCLUDE, "-I" + build.CSRC, "-I" + cuda, "-o", str(exe),
                           os.path.join(here, "launch_order.cpp"), os.path.join(build.CSRC, "smr_api.cpp"),
                           "-Wl,--unresolved-symbols=ignore-all", "-lpthread"])
    lines = subprocess.run([str(exe)], check=True, capture_output=True, text=True, timeout=60).stdout.split("\n")[:-1]
    assert [ln.split()[0] for ln in lines] == ["product", "sum"] * 20
    assert len({ln.split()[1] for ln in lines}) == 1


def test_threads_on_one_workspace_take_turns(fake_device):
    """A caller's workspace, like the ones that the layer keeps: no call's
    launches between another's, and none on memory that has been replaced."""
    smr, busy, bad = fake_device, [], []
    ws = smr.Workspace(0, torch.device("cuda", 0))

    def fn(ref, ptr, n, s):
        busy.append(1)
        bad.append(len(busy) > 1 or n != ws.buf.numel())
        time.sleep(0.002)
        bad.append(len(busy) > 1 or n != ws.buf.numel())
        busy.pop()
        return _lib.SMR_OK

    def work(k):
        for _ in range(10):
            smr._run_product(fn, lambda ref: 1024, ExpertDownArgs(), ws, 0)
            smr._launch(fn, (None,), ws, 1024, ws.device, 7)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(bad) == 160 and not any(bad)


def test_no_read_only_loads_behind_a_programmatic_launch():
    """The experts' and MXFP4 kernels start while the kernel before them may
    still write what they read (the product's rows, the values to quantise,
    fresh scales): none of it may come through the read-only path."""
    from moe_router_top_gb300 import build
    for name in ("smr_ffn.cu", "smr_mxfp4.cu"):
        text = open(os.path.join(build.CSRC, name)).read()
        code = re.sub(r"//[^\n]*", "", text)
        for bad in (".nc", "ld_stream_v4", "__ldg"):
            assert bad not in code, (name, bad)
        # a plain load through a const restrict pointer may become one as well
        kernels = re.findall(r"__global__.*?\n}\n", code, re.S)
        assert kernels
        for kernel in kernels:
            head, body = kernel.split("{", 1)
            for ptr in re.findall(r"const (?:uint\w+|int\w+|float) \*__restrict__ (\w+)", head):
                assert not re.search(rf"\b{ptr}\[", body), (name, ptr)


def test_blocks_of_the_sum_fit_beside_the_product(tmp_path):
    """By the compiler's register counts: a block of the sum fits on an SM
    that holds a CTA of the product whose rows it waits for, in every variant."""
    from moe_router_top_gb300 import build
    out = subprocess.run([build.nvcc()] + build.ARCH + build.FLAGS + ["-Xptxas", "-v", "-c", os.path.join(build.CSRC, "smr_ffn.cu"),
                         "-o", str(tmp_path / "ffn.o")], check=True, capture_output=True, text=True)
    used = dict(re.findall(r"Compiling entry function '(\w+)'.*?Used (\d+) registers", out.stdout + out.stderr, re.S))
    source = open(os.path.join(build.CSRC, "smr_ffn.cu")).read()
    threads = int(re.search(r"kCombineThreads = (\d+);", source).group(1))

    def alloc(name, threads):  # registers are handed out to warps in units of 8 a thread
        return -(-int(used[name]) // 8) * 8 * threads

    combine = {f: next(n for n in used if f"expert_combine_kernelILb{f}" in n) for f in (0, 1)}
    seen = 0
    for name in used:
        m = re.search(r"expert_ffn_kernelILb(\d)ELb0ELb(\d)ELi(\d)ELb(\d)E", name)  # (MX, not gated, PAIR, SUB, F32)
        if not m:
            continue
        mx, pair, sub, f32 = map(int, m.groups())
        seen += 1
        product, block = alloc(name, 480 if sub == 2 else 544), alloc(combine[f32], threads)
        assert product + block <= 65536, (name, product, block)
    assert seen >= 10


def test_streams_of_another_device_are_refused(smr, monkeypatch):
    """Not taken for the operands' device's current stream."""
    entered = []
    cuda = types.SimpleNamespace(stream=lambda s: entered.append(s) or "context", ExternalStream=lambda p, device: (p, device))
    monkeypatch.setattr(smr, "_torch_module", types.SimpleNamespace(cuda=cuda))
    other, same = (types.SimpleNamespace(device=torch.device("cuda", i)) for i in (1, 0))
    with pytest.raises(ValueError, match="stream must be on the operands' device, cuda:0"):
        smr._elsewhere(0, other)
    assert entered == []
    assert smr._elsewhere(0, same) == "context" and smr._elsewhere(0, 7) == "context" and entered == [same, (7, 0)]


def test_every_stream_has_a_workspace_of_its_own(fake_device, monkeypatch):
    """Also where threads name different streams by one handle, their own default streams."""
    smr, stream = fake_device, []
    monkeypatch.setattr(smr._torch_module._C, "_cuda_getCurrentRawStream", lambda dev: stream[-1])

    def call():
        smr._run_product(lambda *a: _lib.SMR_OK, lambda ref: 1024, ExpertDownArgs(), None, 0)

    for s in (7, 9, 7, 0):
        stream.append(s)
        call()
    assert len(smr._stream_ws) == 3 and len({id(w.buf) for w in smr._stream_ws.values()}) == 3
    stream.append(2)
    gate = threading.Barrier(3)

    def work():
        gate.wait()  # (three threads at a time: idents are not reused)
        call()
        call()
        gate.wait()

    threads = [threading.Thread(target=work) for _ in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(smr._stream_ws) == 6


def test_kept_workspaces_can_be_released(fake_device):
    smr = fake_device
    sizes = []
    for need in (4096, 512):
        smr._run_product(lambda ref, ptr, n, s: sizes.append(n) or _lib.SMR_OK, lambda ref: need, ExpertDownArgs(), None, 0)
        kept = weakref.ref(next(iter(smr._stream_ws.values())).buf)
        assert kept() is not None
        smr.release_workspaces()
        assert kept() is None and smr._stream_ws == {}
    assert sizes == [4096, 512]


def test_fp32_rows(lib):
    size, size32 = lib.smr_expert_down_workspace_size, lib.smr_expert_down_fp32_workspace_size
    few, many = _down(), _down(num_tokens=4096)
    assert size32(ctypes.byref(few)) == size(ctypes.byref(few))  # fp32 anyway
    need = 256 + 16 * 1024 * 8 + 4096 * 11 * 256 * 4
    assert size32(ctypes.byref(many)) == need
    assert lib.smr_expert_down_fp32(ctypes.byref(many), P, need - 1, None) == WORKSPACE
    assert "smr_expert_down_fp32" in lib.smr_last_error().decode()
    assert lib.smr_expert_down_fp32(None, P, need, None) == INVALID and size32(None) == 0
    _refused(lib, lib.smr_expert_down_fp32, _down(num_logical=0), INVALID, "smr_expert_down_fp32", "num_logical must be in")
    empty = ExpertDownArgs(0, 1, 16, 16, 1, 64, num_logical=1)
    assert lib.smr_expert_down_fp32(ctypes.byref(empty), None, 0, None) == _lib.SMR_OK


def test_workspaces_can_be_copied(smr):
    """As part of a model that is copied or stored, say."""
    ws = smr.Workspace(512, "cpu")
    ws.buf[4] = 2
    for other in (copy.deepcopy(ws), pickle.loads(pickle.dumps(ws))):
        assert other.nbytes == 512 and other.buf[4] == 2 and other.buf is not ws.buf and other.lock is not ws.lock
        other.ensure(1024)
        assert other.nbytes == 1024 and ws.nbytes == 512
