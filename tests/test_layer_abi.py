"""Refusals of the operators around the recurrent step, on the host: nothing
here reaches a launch, so no GPU is needed and fake addresses stand in for
device memory."""

from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

from linear_attention_recurrent_deltalog_b200 import deltalog as dl

lib = dl._lib
P = 1 << 20  # fake, aligned addresses
Q, R, S, O = P + (1 << 16), P + (2 << 16), P + (3 << 16), P + (4 << 16)


def starts(*v):
    return np.array(v, dtype=np.int32)


def conv_prompt(cfg, st, x=P, ldx=None, w=Q, bias=None, h0=None, h1=None, y=R, ldy=None, n=None):
    return lib.dl_conv_prompt(ctypes.byref(cfg.c), len(st) - 1 if n is None else n,
                              None if st is None else st.ctypes.data, x,
                              cfg.C if ldx is None else ldx, w, bias, h0, h1, y,
                              cfg.C if ldy is None else ldy, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), dl.DL_ERR_ARG), (dict(w=None), dl.DL_ERR_ARG), (dict(y=None), dl.DL_ERR_ARG),
    (dict(y=P), dl.DL_ERR_ARG), (dict(ldx=63), dl.DL_ERR_ARG), (dict(ldy=63), dl.DL_ERR_ARG),
    (dict(x=P + 1), dl.DL_ERR_ALIGN), (dict(w=Q + 2), dl.DL_ERR_ALIGN),
    (dict(h0=S + 1), dl.DL_ERR_ALIGN), (dict(h1=P), dl.DL_ERR_ARG), (dict(n=-1), dl.DL_ERR_ARG),
    (dict(bias=S + 2), dl.DL_ERR_ALIGN), (dict(n=0), dl.DL_OK),
])
def test_conv_prompt_arguments(kw, code):
    assert conv_prompt(dl.ConvConfig(64, 4), starts(0, 5, 9), **kw) == code


@pytest.mark.parametrize("st", [(0, 5, 4), (-1, 5), (7, 3)])
def test_bad_starts(st):
    st = starts(*st)
    assert conv_prompt(dl.ConvConfig(64, 4), st) == dl.DL_ERR_ARG
    cfg = dl.SsmConfig(2, 1, 64, 64)
    b = ctypes.c_size_t()
    assert lib.dl_ssm_bytes(ctypes.byref(cfg.c), len(st) - 1, st.ctypes.data,
                            ctypes.byref(b)) == dl.DL_ERR_ARG
    assert lib.dl_ssm_bytes(ctypes.byref(cfg.c), 1, None, ctypes.byref(b)) == dl.DL_ERR_ARG


@pytest.mark.parametrize("cfg,code", [
    (dl.ConvConfig(0, 4), dl.DL_ERR_ARG), (dl.ConvConfig(8, 1), dl.DL_ERR_UNSUPPORTED),
    (dl.ConvConfig(8, 5), dl.DL_ERR_UNSUPPORTED), (dl.ConvConfig(8, 0), dl.DL_ERR_ARG)])
def test_conv_config(cfg, code):
    assert conv_prompt(cfg, starts(0, 3), ldx=64, ldy=64) == code
    c = dl.ConvConfig(8, 4).c
    bad = dl.dl_conv_config(c.C, c.W, 2, c.flags)
    assert lib.dl_conv_step(ctypes.byref(bad), 1, P, 8, Q, None, S, R, 8, None) == dl.DL_ERR_ARG
    bad = dl.dl_conv_config(c.C, c.W, 0, 6)
    assert lib.dl_conv_step(ctypes.byref(bad), 1, P, 8, Q, None, S, R, 8, None) == dl.DL_ERR_ARG
    assert lib.dl_conv_step(ctypes.byref(c), 1, P, 8, Q, None, None, R, 8, None) == dl.DL_ERR_ARG
    assert lib.dl_conv_step(ctypes.byref(c), -1, P, 8, Q, None, S, R, 8, None) == dl.DL_ERR_ARG
    assert lib.dl_conv_step(ctypes.byref(c), 0, P, 8, Q, None, S, R, 8, None) == dl.DL_OK


def io(cfg, **kw):
    nk, nv = cfg.G * cfg.d_k, cfg.H * cfg.d_v
    f = dict(q=P, k=Q, v=R, dt=S, a=S, d=None, dt_bias=None, o=O, ldq=nk, ldk=nk, ldv=nv,
             lddt=cfg.H, ldo=nv)
    f.update(kw)
    return dl.dl_ssm_io(**f)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), dl.DL_ERR_ARG), (dict(k=None), dl.DL_ERR_ARG), (dict(v=None), dl.DL_ERR_ARG),
    (dict(dt=None), dl.DL_ERR_ARG), (dict(a=None), dl.DL_ERR_ARG), (dict(o=None), dl.DL_ERR_ARG),
    (dict(o=R), dl.DL_ERR_ARG), (dict(ldq=64), dl.DL_ERR_ARG), (dict(ldv=128), dl.DL_ERR_ARG),
    (dict(lddt=3), dl.DL_ERR_ARG), (dict(ldk=132), dl.DL_ERR_ALIGN),
    (dict(q=P + 8), dl.DL_ERR_ALIGN), (dict(o=O + 2), dl.DL_ERR_ALIGN),
    (dict(dt=S + 2), dl.DL_ERR_ALIGN), (dict(d=S + 1), dl.DL_ERR_ALIGN),
])
def test_ssm_arguments(kw, code):
    cfg = dl.SsmConfig(4, 2, 64, 64)
    st, x = starts(0, 5), io(cfg, **kw)
    assert lib.dl_ssm_step(ctypes.byref(cfg.c), 1, ctypes.byref(x), O + (1 << 16), None) == code
    assert lib.dl_ssm_prompt(ctypes.byref(cfg.c), 1, st.ctypes.data, ctypes.byref(x), None, None,
                             1 << 24, 1 << 30, None) == code


def test_ssm_states_and_counts():
    cfg = dl.SsmConfig(4, 2, 64, 64)
    st, x = starts(0, 5), io(cfg)
    step, prompt = lib.dl_ssm_step, lib.dl_ssm_prompt
    c, xp = ctypes.byref(cfg.c), ctypes.byref(x)
    assert step(c, 1, xp, None, None) == dl.DL_ERR_ARG
    assert step(c, -1, xp, P, None) == dl.DL_ERR_ARG
    assert step(c, 1, xp, P + 4, None) == dl.DL_ERR_ALIGN
    assert step(c, 0, xp, P, None) == dl.DL_OK
    assert prompt(c, 1, st.ctypes.data, xp, P + 4, None, None, 0, None) == dl.DL_ERR_ALIGN
    assert prompt(c, 1, st.ctypes.data, xp, None, P + 8, None, 0, None) == dl.DL_ERR_ALIGN
    assert prompt(c, 1, st.ctypes.data, xp, None, None, (1 << 24) + 16, 1 << 30, None) == \
        dl.DL_ERR_ALIGN
    assert prompt(c, -1, st.ctypes.data, xp, None, None, None, 0, None) == dl.DL_ERR_ARG
    assert prompt(c, 0, st.ctypes.data, xp, None, None, None, 0, None) == dl.DL_OK
    assert prompt(c, 1, st.ctypes.data, None, None, None, None, 0, None) == dl.DL_ERR_ARG


@pytest.mark.parametrize("cfg,code", [
    (dl.SsmConfig(4, 3, 64, 64), dl.DL_ERR_ARG), (dl.SsmConfig(0, 1, 64, 64), dl.DL_ERR_ARG),
    (dl.SsmConfig(4, 0, 64, 64), dl.DL_ERR_ARG), (dl.SsmConfig(4, 2, 96, 64), dl.DL_ERR_UNSUPPORTED),
    (dl.SsmConfig(4, 2, 64, 32), dl.DL_ERR_UNSUPPORTED)])
def test_ssm_config(cfg, code):
    st, x = starts(0, 5), io(dl.SsmConfig(4, 2, 64, 64))
    assert lib.dl_ssm_step(ctypes.byref(cfg.c), 1, ctypes.byref(x), P, None) == code
    b = ctypes.c_size_t()
    assert lib.dl_ssm_bytes(ctypes.byref(cfg.c), 1, st.ctypes.data, ctypes.byref(b)) == code


def norm(cfg, rows=2, x=P, ldx=64, res=None, ldr=64, w=Q, res_out=None, ldro=64, out=R, ldo=64,
         scales=None):
    return lib.dl_norm(ctypes.byref(cfg.c), rows, x, ldx, res, ldr, w, res_out, ldro, out, ldo,
                       scales, None)


@pytest.mark.parametrize("cfg,kw,code", [
    (dl.NormConfig(64), dict(x=None), dl.DL_ERR_ARG), (dl.NormConfig(64), dict(w=None), dl.DL_ERR_ARG),
    (dl.NormConfig(64), dict(out=None), dl.DL_ERR_ARG), (dl.NormConfig(64), dict(out=P), dl.DL_ERR_ARG),
    (dl.NormConfig(64), dict(rows=-1), dl.DL_ERR_ARG), (dl.NormConfig(64), dict(rows=0), dl.DL_OK),
    (dl.NormConfig(64), dict(ldx=63), dl.DL_ERR_ARG), (dl.NormConfig(64), dict(ldo=1), dl.DL_ERR_ARG),
    (dl.NormConfig(64), dict(res=S, ldr=8), dl.DL_ERR_ARG),
    (dl.NormConfig(64), dict(res_out=S, ldro=8), dl.DL_ERR_ARG),
    (dl.NormConfig(64), dict(res_out=P, ldro=72), dl.DL_ERR_ARG),
    (dl.NormConfig(64), dict(res=S, ldr=64, res_out=S, ldro=72), dl.DL_ERR_ARG),
    (dl.NormConfig(64), dict(x=P + 1), dl.DL_ERR_ALIGN), (dl.NormConfig(64), dict(w=Q + 2), dl.DL_ERR_ALIGN),
    (dl.NormConfig(0), {}, dl.DL_ERR_ARG), (dl.NormConfig(16385), dict(ldx=20000, ldo=20000), dl.DL_ERR_UNSUPPORTED),
    (dl.NormConfig(64, eps=-1.0), {}, dl.DL_ERR_ARG), (dl.NormConfig(64, eps=float("nan")), {}, dl.DL_ERR_ARG),
    (dl.NormConfig(64, block=128), {}, dl.DL_ERR_ARG),
    (dl.NormConfig(64, "bf16", "e4m3", block=64), dict(scales=S), dl.DL_ERR_ARG),
    (dl.NormConfig(64, "bf16", "e4m3", block=128), {}, dl.DL_ERR_ARG),
    (dl.NormConfig(64, "bf16", "e4m3", block=128), dict(scales=S + 2), dl.DL_ERR_ALIGN),
])
def test_norm_arguments(cfg, kw, code):
    assert norm(cfg, **kw) == code


def test_binding_checks_tensors():
    cfg = dl.NormConfig(64, "f32", "f32")
    x, w, out = torch.zeros(3, 64), torch.ones(64), torch.zeros(3, 64)
    for bad in (torch.zeros(3, 65), torch.zeros(3, 128)[:, ::2], torch.zeros(2, 64),
                torch.zeros(1, 64).expand(3, 64)):
        with pytest.raises(ValueError):
            dl.dl_norm(cfg, x, w, bad)
    with pytest.raises(TypeError):
        dl.dl_norm(cfg, x, w, out.half())
    with pytest.raises(TypeError):
        dl.dl_norm(cfg, x, None, out)
    with pytest.raises(TypeError):
        dl.dl_norm(dl.NormConfig(64, "f32", "e4m3"), x, w, out.to(torch.float8_e4m3fn))
    with pytest.raises(ValueError, match="current CUDA device"):
        dl.dl_norm(cfg, x, w, out)
    assert dl._rows(torch.zeros(5, 3, 64)[:, :2], "x", 5, 128, torch.float32) == 192
    assert dl._rows(torch.zeros(5, 200)[:, 8:72], "x", 5, 64, torch.float32) == 200
    with pytest.raises(ValueError):
        dl._rows(torch.zeros(5, 3, 64)[:, :, :32], "x", 5, 96, torch.float32)
    conv = dl.ConvConfig(8, 4, "f32")
    y, cw, h = torch.zeros(3, 8), torch.zeros(8, 4), torch.zeros(3, 3, 8)
    with pytest.raises(ValueError):
        dl.dl_conv_step(conv, y, cw, None, torch.zeros(2, 3, 8), torch.zeros(3, 8))
    with pytest.raises(ValueError):
        dl.dl_conv_prompt(conv, [0, 4], y, cw, None, None, None, torch.zeros(3, 8))
    for bad in ([0.0, 3.0], [[0, 3]], [0, 1 << 40], torch.zeros(0, dtype=torch.int32)):
        with pytest.raises(ValueError):
            dl.dl_conv_prompt(conv, bad, y, cw, None, None, None, torch.zeros(3, 8))
    s = dl.SsmConfig(2, 1, 64, 64, "f32")
    q, v = torch.zeros(3, 64), torch.zeros(3, 128)
    args = dict(q=q, k=q.clone(), v=v, dt=torch.zeros(3, 2), a=torch.zeros(2), d=None, dt_bias=None,
                S=torch.zeros(3, 2, 64, 64), o=torch.zeros(3, 128))
    for name, bad in (("q", torch.zeros(3, 128)), ("dt", torch.zeros(3, 3)), ("a", torch.zeros(1)),
                      ("S", torch.zeros(2, 2, 64, 64)), ("o", torch.zeros(2, 128))):
        with pytest.raises(ValueError):
            dl.dl_ssm_step(s, **{**args, name: bad})
    with pytest.raises(ValueError, match="current CUDA device"):
        dl.dl_ssm_step(s, **args)


def test_calls_without_rows_need_no_row_buffers():
    conv, ssm = dl.ConvConfig(64, 4), dl.SsmConfig(4, 2, 64, 64)
    assert conv_prompt(conv, starts(0), x=None, y=None) == dl.DL_OK
    assert conv_prompt(conv, starts(0), x=None, y=None, w=None) == dl.DL_ERR_ARG
    assert lib.dl_conv_step(ctypes.byref(conv.c), 0, None, 64, Q, None, None, None, 64, None) == dl.DL_OK
    x = io(ssm, q=None, k=None, v=None, dt=None, o=None)
    c, xp, st = ctypes.byref(ssm.c), ctypes.byref(x), starts(3)
    assert lib.dl_ssm_step(c, 0, xp, None, None) == dl.DL_OK
    assert lib.dl_ssm_step(c, 1, xp, P, None) == dl.DL_ERR_ARG
    assert lib.dl_ssm_prompt(c, 0, st.ctypes.data, xp, None, None, None, 0, None) == dl.DL_OK
    x = io(ssm, a=None)
    assert lib.dl_ssm_step(c, 0, ctypes.byref(x), None, None) == dl.DL_ERR_ARG
    assert norm(dl.NormConfig(64), rows=0, x=None, out=None) == dl.DL_OK
