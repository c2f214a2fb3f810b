"""Host side of the operators around the recurrent step at the borders of
what they accept: no GPU is needed, fakes stand in for streams and the library."""

from __future__ import annotations

import contextlib
import ctypes
import types

import numpy as np
import pytest
import torch

from linear_attention_recurrent_deltalog_b200 import build
from linear_attention_recurrent_deltalog_b200 import deltalog as dl


# ------------------------------------------- the workspace of a prompt's scan

class FakeStream:
    device_index = 0

    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.fixture
def fake_device(monkeypatch):
    """A device 0 whose current stream is 11 until torch.cuda.stream() says
    otherwise; records (stream of the call, stream its workspace came from)."""
    now, made, calls = [11], [], []

    @contextlib.contextmanager
    def on(stream):
        now.append(stream.cuda_stream)
        yield
        now.pop()

    empty = torch.empty

    def allocate(*a, **kw):
        made.append(now[-1])
        return empty(*a, **kw)

    def bytes_(cfg, n, at, out):
        out._obj.value = 512
        return 0

    def prompt(cfg, n, at, io, s0, s1, ws, nbytes, stream):
        assert ws and nbytes == 512
        calls.append((stream, made[-1]))
        return 0

    monkeypatch.setattr(dl, "_on_device", lambda names, *t: 0)
    monkeypatch.setattr(dl, "_lib", types.SimpleNamespace(dl_ssm_bytes=bytes_, dl_ssm_prompt=prompt))
    monkeypatch.setattr(torch, "empty", allocate)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: FakeStream(handle))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: FakeStream(0))
    monkeypatch.setattr(dl, "_current_stream", lambda dev: now[-1])
    return calls


def prompt_on(stream, **kw):
    cfg = dl.SsmConfig(2, 1, 64, 64, "f32")
    q, v = torch.zeros(3, 64), torch.zeros(3, 128)
    dl.dl_ssm_prompt(cfg, [0, 3], q, q, v, torch.zeros(3, 2), torch.zeros(2), None, None, None, None,
                     torch.zeros(3, 128), stream=stream, **kw)


@pytest.mark.parametrize("stream", [None, 11, 4096, FakeStream(4096), 0, FakeStream(0)])
def test_workspace_comes_from_the_stream_of_the_call(fake_device, stream):
    # memory that the allocator hands out on one stream may be in use there
    # before the call, and is handed out again there after it
    prompt_on(stream)
    want = 11 if stream is None else getattr(stream, "cuda_stream", stream)
    assert fake_device == [(want, want)]


def test_workspace_of_the_special_stream_handles(fake_device):
    # 1 is the legacy default stream by another name; what 2 means depends on the
    # thread, so no memory can be tied to it
    prompt_on(1)
    assert fake_device == [(1, 0)]
    with pytest.raises(ValueError, match="workspace"):
        prompt_on(2)
    prompt_on(2, workspace=torch.empty(512, dtype=torch.uint8))
    assert fake_device[1:] == [(2, 11)]


def test_call_without_a_workspace_takes_any_stream_handle(fake_device):
    def none(cfg, n, at, out):
        out._obj.value = 0
        return 0

    called = []
    dl._lib.dl_ssm_bytes = none
    dl._lib.dl_ssm_prompt = lambda *a: called.append((a[6], a[7], a[8])) or 0
    prompt_on(2)
    assert called == [(None, 0, 2)]


# ------------------------------------------------ rows up to the last int32s

P = 1 << 20  # fake, aligned addresses: nothing here reaches a launch
TOP = 2 ** 31 - 1024  # the last row number that a call may end at


@pytest.mark.parametrize("start", [0, TOP - 3])
@pytest.mark.parametrize("end", [TOP + 1, 2 ** 31 - 5, 2 ** 31 - 1])
def test_row_numbers_near_the_end_of_int32_are_refused(start, end):
    # the kernels form row numbers past the last one, of a batch or a tile
    st = np.array([start, end], dtype=np.int32)
    at, lib, n = st.ctypes.data, dl._lib, ctypes.c_size_t()
    for dtype in ("bf16", "f32"):
        conv, ssm = dl.ConvConfig(64, 4, dtype), dl.SsmConfig(2, 1, 64, 64, dtype)
        x = dl.dl_ssm_io(q=P, k=P, v=P, dt=P, a=P, o=2 * P, ldq=64, ldk=64, ldv=128, lddt=2, ldo=128)
        assert lib.dl_conv_prompt(conv.ref, 1, at, P, 64, P, None, None, None, 2 * P, 64, None) == dl.DL_ERR_ARG
        assert lib.dl_ssm_bytes(ssm.ref, 1, at, ctypes.byref(n)) == dl.DL_ERR_ARG
        assert lib.dl_ssm_prompt(ssm.ref, 1, at, ctypes.byref(x), None, None, P, 1 << 50, None) == dl.DL_ERR_ARG
        assert lib.dl_conv_step(conv.ref, end, P, 64, P, None, P, 2 * P, 64, None) == dl.DL_ERR_ARG


def test_row_numbers_up_to_the_limit_are_planned():
    st = np.array([TOP - 300, TOP], dtype=np.int32)
    n = ctypes.c_size_t()
    ssm = dl.SsmConfig(2, 1, 64, 64)
    assert dl._lib.dl_ssm_bytes(ssm.ref, 1, st.ctypes.data, ctypes.byref(n)) == dl.DL_OK
    assert n.value == dl.dl_ssm_bytes(ssm, [0, 300])


# ------------------------------------------------- streams of another device

def test_stream_of_another_device_is_refused(fake_device):
    other = FakeStream(4096)
    other.device_index = 1
    for kw in ({}, {"workspace": torch.empty(512, dtype=torch.uint8)}):
        with pytest.raises(ValueError, match="stream: .*current CUDA device"):
            prompt_on(other, **kw)
    assert fake_device == []
    bare = types.SimpleNamespace(cuda_stream=4096)  # another library's: a handle and no more
    prompt_on(bare)
    assert fake_device == [(4096, 4096)]


# --------------------------------------------------- a torch without shortcuts

def test_current_device_and_stream_by_torchs_public_calls(monkeypatch):
    # the quick forms are private names of torch: without them the public ones serve
    for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
        monkeypatch.delattr(torch._C, name, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: FakeStream(100 + dev))
    device, stream = dl._cuda_calls()
    assert device() == 3 and stream(3) == 103
    monkeypatch.setattr(dl, "_current_device", device)
    monkeypatch.setattr(dl, "_current_stream", stream)
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    assert dl._stream(None) == 103 and dl._stream_on(2, None) == 102
    with pytest.raises(ValueError, match="x: .*current CUDA device"):
        dl._on_device("x", torch.zeros(1))


# ------------------------------------- registers that the scan's roles share out

PTXAS = """ptxas info    : Compiling entry function '_ZN2dl19dl_ssm_chunk_kernelILi128EEEv' for 'sm_100a'
ptxas info    : Function properties for _ZN2dl19dl_ssm_chunk_kernelILi128EEEv
    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads
ptxas info    : Used {} registers, used 1 barriers
ptxas info    : Compiling entry function '_ZN2dl18dl_ssm_join_kernelEv' for 'sm_100a'
ptxas info    : Used 32 registers, used 0 barriers
"""


def test_build_refuses_a_scan_kernel_with_too_few_registers():
    # the launch would refuse it: its warps' shares add up against what a block starts with
    need = build.start_registers()
    assert need >= 24 and need % 8 == 0
    build.check_registers(PTXAS.format(need))
    for text in (PTXAS.format(need - 8), PTXAS.format(need).replace("chunk", "other")):
        with pytest.raises(RuntimeError, match="registers"):
            build.check_registers(text)
