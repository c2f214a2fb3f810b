"""The operators around the recurrent step on the GPU against 64-bit
references, at the sizes and inputs where they can go wrong."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from linear_attention_recurrent_deltalog_b200 import deltalog as dl
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu

T16, T32 = torch.bfloat16, torch.float32
DT = {"bf16": T16, "f32": T32}


def rnd(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def close(got, want, tol, what):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), what
    worst = ((got - want).abs() / tol.clamp_min(1e-300)).max() if want.numel() else torch.tensor(0.0)
    assert float(worst) <= 1.0, f"{what}: {float(worst):.3g} of its tolerance"


def starts_of(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


# ------------------------------------------------------------------ conv

LENS = [[1], [2, 0, 1, 3], [5, 31, 32, 33, 1], [64, 97], [3] * 70, [1] * 1025 + [40]]


@pytest.mark.parametrize("dtype,C,W,act", [
    ("bf16", 64, 4, True), ("bf16", 136, 3, False), ("bf16", 77, 4, True), ("f32", 36, 2, True),
    ("f32", 33, 4, False), ("f32", 1, 3, True)])
@pytest.mark.parametrize("lens", LENS, ids=[f"n{len(v)}" for v in LENS])
def test_conv_prompt(dtype, C, W, act, lens):
    t, st = DT[dtype], starts_of(lens)
    n, T = len(lens), int(st[-1])
    x, w, b = rnd(1, T, C).to(t), rnd(2, C, W), rnd(3, C)
    h0 = rnd(4, n, W - 1, C).to(t)
    y = torch.full((T + 3, C), 7.0, dtype=t, device="cuda")  # three rows behind the last sequence
    h1 = torch.empty(n, W - 1, C, dtype=t, device="cuda")
    dl.dl_conv_prompt(dl.ConvConfig(C, W, dtype, silu=act), st, x.cuda(), w.cuda(), b.cuda(),
                      h0.cuda(), h1, y)
    want, mag, hw = ref.conv(x, st, w, b, h0, act)
    close(y[:T], want, ref.conv_tol(mag, W, t), "y")
    assert torch.equal(h1.double().cpu(), hw)
    assert (y[T:] == 7).all()


def test_conv_prompt_of_many_rows_a_thread():
    # enough rows that a thread walks down more than one batch of them, and
    # sequences that end inside a batch
    C, W, st = 1536, 4, starts_of([1, 2985, 3, 31])
    x, w, b = rnd(1, 3020, C).to(T16), rnd(2, C, W), rnd(3, C)
    h = rnd(4, 4, W - 1, C).to(T16)
    y, h1 = torch.empty(3020, C, dtype=T16, device="cuda"), torch.empty_like(h, device="cuda")
    dl.dl_conv_prompt(dl.ConvConfig(C, W, "bf16"), st, x.cuda(), w.cuda(), b.cuda(), h.cuda(), h1, y)
    want, mag, hw = ref.conv(x, st, w, b, h, True)
    close(y, want, ref.conv_tol(mag, W, T16), "y")
    assert torch.equal(h1.double().cpu(), hw)


def test_conv_strides_in_place_state_and_no_state():
    # channel ranges of wider rows; x with an odd stride takes the narrow path
    C, W, st = 64, 4, starts_of([9, 0, 40])
    n, T = 3, 49
    for ld in (200, 201):
        big = rnd(1, T, ld).to(T16)
        x = big.cuda()[:, 8:8 + C]
        w, b, h = rnd(2, C, W), None, rnd(3, n, W - 1, C).to(T16)
        yb = torch.full((T, ld), 3.0, dtype=T16, device="cuda")
        y, hg = yb[:, 16:16 + C], h.cuda()
        cfg = dl.ConvConfig(C, W, "bf16")
        dl.dl_conv_prompt(cfg, st, x, w.cuda(), b, hg, hg, y)
        want, mag, hw = ref.conv(big[:, 8:8 + C], st, w, b, h, True)
        close(y, want, ref.conv_tol(mag, W, T16), "y")
        assert torch.equal(hg.double().cpu(), hw)
        assert (yb[:, :16] == 3).all() and (yb[:, 16 + C:] == 3).all()
        dl.dl_conv_prompt(cfg, st, x, w.cuda(), b, None, None, y)
        want, mag, _ = ref.conv(big[:, 8:8 + C], st, w, b, None, True)
        close(y, want, ref.conv_tol(mag, W, T16), "y without states")


def test_conv_neighbours_and_extremes_stay_apart():
    # NaN and infinities in one sequence do not reach another, and large
    # negative values leave silu at -0, not NaN
    C, st = 8, starts_of([5, 40, 6])
    x = rnd(1, 51, C)
    x[5:45] = float("nan")
    x[45, 0], x[46, 1] = -3e4, -3e38
    w, h = torch.ones(C, 2), torch.zeros(3, 1, C)
    y = torch.empty(51, C, device="cuda")
    dl.dl_conv_prompt(dl.ConvConfig(C, 2, "f32"), st, x.cuda(), w.cuda(), None, h.cuda(), None, y)
    y = y.cpu()
    assert torch.isnan(y[5:45]).all()
    assert torch.isfinite(y[:5]).all() and torch.isfinite(y[45:]).all()
    assert y[45, 0] == 0 and y[46, 1] == 0


@pytest.mark.parametrize("dtype,B,C,W", [("bf16", 1, 64, 4), ("bf16", 7, 200, 3), ("bf16", 3, 33, 4),
                                         ("f32", 5, 20, 2), ("f32", 130, 9, 4)])
def test_conv_step_continues_a_prompt(dtype, B, C, W):
    t, steps = DT[dtype], 6
    x, w, b = rnd(1, steps, B, C).to(t), rnd(2, C, W), rnd(3, C)
    h = rnd(4, B, W - 1, C).to(t)
    cfg = dl.ConvConfig(C, W, dtype)
    hg, y = h.cuda(), torch.empty(B, C, dtype=t, device="cuda")
    st = starts_of([steps] * B)
    want, mag, hw = ref.conv(x.transpose(0, 1).reshape(-1, C), st, w, b, h, True)
    want, mag = (z.view(B, steps, C) for z in (want, mag))
    xg, wg, bg = x.cuda(), w.cuda(), b.cuda()
    for i in range(steps):
        dl.dl_conv_step(cfg, xg[i], wg, bg, hg, y)
        close(y, want[:, i], ref.conv_tol(mag[:, i], W, t), f"step {i}")
    assert torch.equal(hg.double().cpu(), hw)


# ------------------------------------------------------------------ scan

def ssm_inputs(seed, T, n, H, G, dk, dv, dtype, pad=0):
    t = DT[dtype]
    f = lambda i, *s: torch.nn.functional.silu(rnd(seed + i, *s)).to(t)
    return dict(q=f(1, T + pad, G, dk), k=f(2, T + pad, G, dk), v=f(3, T + pad, H, dv),
                dt=rnd(seed + 4, T + pad, H) * 0.5, a=-torch.exp(rnd(seed + 5, H)),
                d=rnd(seed + 6, H), bias=rnd(seed + 7, H) - 2.0, S0=0.3 * rnd(seed + 8, n, H, dv, dk))


def run_prompt(cfg, st, z, S0=True, S1=True, in_place=False, pad=0):
    g = {k: v.cuda() for k, v in z.items()}
    n, T = len(st) - 1, int(st[-1])
    s0 = g["S0"] if S0 else None
    s1 = s0 if in_place else (torch.empty(n, cfg.H, cfg.d_v, cfg.d_k, device="cuda") if S1 else None)
    o = torch.full((T + pad, cfg.H, cfg.d_v), 5.0, dtype=cfg.torch_in_dtype, device="cuda")
    dl.dl_ssm_prompt(cfg, st, g["q"], g["k"], g["v"], g["dt"], g["a"], g["d"], g["bias"], s0, s1, o)
    torch.cuda.synchronize()
    assert dl.dl_device_error(None) == (0, 0)
    return o, s1


def check_prompt(cfg, st, z, **kw):
    pad = kw.get("pad", 0)
    o, s1 = run_prompt(cfg, st, z, **kw)
    T = int(st[-1])
    t = cfg.torch_in_dtype
    cut = {k: (v[:T] if k in ("q", "k", "v", "dt") else v) for k, v in z.items()}
    S0 = cut["S0"] if kw.get("S0", True) else None
    ow, sw, mo, ms, top = ref.ssm(st, cut["q"], cut["k"], cut["v"], cut["dt"], cut["a"], cut["d"],
                                  cut["bias"], S0, cfg.softplus)
    to, ts = ref.ssm_tol(mo, ms, top, int(np.diff(st).max()), cfg.d_k, t)
    close(o[:T], ow, to, "o")
    if s1 is not None:
        close(s1, sw, ts, "S1")
    assert (o[T:] == 5).all()
    return o, s1


SSM_LENS = [[1], [2, 0, 1], [127, 1, 128, 129], [300], [16, 17, 0, 255]]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,G,dk,dv", [(2, 1, 128, 64), (3, 1, 64, 64), (2, 2, 128, 128),
                                       (6, 2, 64, 128), (5, 5, 128, 64)])
@pytest.mark.parametrize("lens", SSM_LENS, ids=["-".join(map(str, v)) for v in SSM_LENS])
def test_ssm_prompt(dtype, H, G, dk, dv, lens):
    st = starts_of(lens)
    z = ssm_inputs(10, int(st[-1]), len(lens), H, G, dk, dv, dtype, pad=2)
    check_prompt(dl.SsmConfig(H, G, dk, dv, dtype), st, z, pad=2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ssm_prompt_states_optional_and_in_place(dtype):
    st = starts_of([40, 0, 200])
    cfg = dl.SsmConfig(4, 2, 128, 64, dtype)
    z = ssm_inputs(20, 240, 3, 4, 2, 128, 64, dtype)
    o, s1 = check_prompt(cfg, st, z)
    oi, si = run_prompt(cfg, st, z, in_place=True)
    assert torch.equal(o, oi) and torch.equal(s1, si)
    on, none = run_prompt(cfg, st, z, S1=False)
    assert none is None and torch.equal(o, on)
    check_prompt(cfg, st, z, S0=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ssm_prompt_large_batch_of_short_sequences(dtype):
    lens = [int(v) for v in np.random.default_rng(3).integers(0, 5, 1100)]
    st = starts_of(lens)
    z = ssm_inputs(30, int(st[-1]), len(lens), 1, 1, 64, 64, dtype)
    check_prompt(dl.SsmConfig(1, 1, 64, 64, dtype), st, z)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ssm_prompt_long_and_uneven(dtype):
    # long enough to be cut along its length; another sequence beside it
    st = starts_of([2900, 70])
    z = ssm_inputs(40, 2970, 2, 2, 1, 128, 64, dtype)
    check_prompt(dl.SsmConfig(2, 1, 128, 64, dtype), st, z)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,G,dk,dv", [(2, 1, 64, 128), (10, 2, 64, 64)])
def test_ssm_prompt_many_sequences_some_cut(dtype, H, G, dk, dv):
    # more sequences than the small table holds, empty ones among them, some
    # long enough to be cut, and several work items for each block of threads
    lens = [int(v) for v in np.random.default_rng(4).integers(0, 6, 80)]
    lens[7], lens[50], lens[79] = 1500, 130, 300
    st = starts_of(lens)
    z = ssm_inputs(45, int(st[-1]), len(lens), H, G, dk, dv, dtype, pad=1)
    cfg = dl.SsmConfig(H, G, dk, dv, dtype)
    assert dl.dl_ssm_bytes(cfg, st) > 0
    o, s1 = check_prompt(cfg, st, z, pad=1)
    oi, si = run_prompt(cfg, st, z, in_place=True, pad=1)
    assert torch.equal(o, oi) and torch.equal(s1, si)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ssm_prompt_states_aligned_to_16_bytes_only(dtype):
    st = starts_of([150, 20])
    z = ssm_inputs(47, 170, 2, 2, 1, 128, 64, dtype)
    cfg = dl.SsmConfig(2, 1, 128, 64, dtype)
    o, s1 = run_prompt(cfg, st, z)
    g = {k: v.cuda() for k, v in z.items()}
    n = z["S0"].numel()
    S0, S1 = (torch.empty(n + 4, device="cuda")[4:].view(z["S0"].shape) for _ in range(2))
    S0.copy_(g["S0"])
    o2 = torch.empty_like(o)
    dl.dl_ssm_prompt(cfg, st, g["q"], g["k"], g["v"], g["dt"], g["a"], g["d"], g["bias"], S0, S1, o2)
    assert torch.equal(o, o2) and torch.equal(s1, S1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rate", [0.0, 1e-4, 3.0, 400.0])
def test_ssm_prompt_decay_range(dtype, rate):
    # no decay at all, hardly any, strong, and all but total forgetting
    st = starts_of([200, 9])
    z = ssm_inputs(50, 209, 2, 2, 1, 128, 64, dtype)
    z["a"] = torch.full((2,), -rate)
    check_prompt(dl.SsmConfig(2, 1, 128, 64, dtype), st, z)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ssm_prompt_raw_steps_with_zeros_and_strided_rows(dtype):
    # without softplus; dt = 0 leaves the state alone; q, k, v are columns of one row
    H, G, dk, dv, T = 4, 1, 128, 64, 150
    t = DT[dtype]
    st = starts_of([100, 50])
    z = ssm_inputs(60, T, 2, H, G, dk, dv, dtype)
    z["dt"] = z["dt"].abs() * 0.1
    z["dt"][20:60] = 0.0
    z["bias"] = torch.zeros(H)
    row = torch.cat([z["v"].reshape(T, -1), z["k"].reshape(T, -1), z["q"].reshape(T, -1),
                     torch.zeros(T, 8, dtype=t)], 1).cuda()
    v, k, q = row[:, :H * dv], row[:, H * dv:H * dv + dk], row[:, H * dv + dk:H * dv + 2 * dk]
    cfg = dl.SsmConfig(H, G, dk, dv, dtype, softplus=False)
    ob = torch.full((T, H * dv + 64), 5.0, dtype=t, device="cuda")
    S1 = torch.empty(2, H, dv, dk, device="cuda")
    dtb = torch.full((T, 11), float("nan"))
    dtb[:, 3:3 + H] = z["dt"]
    dl.dl_ssm_prompt(cfg, st, q, k, v, dtb.cuda()[:, 3:3 + H], z["a"].cuda(), None, None,
                     z["S0"].cuda(), S1, ob[:, :H * dv])
    ow, sw, mo, ms, top = ref.ssm(st, z["q"], z["k"], z["v"], z["dt"], z["a"], None, None, z["S0"],
                                  False)
    to, ts = ref.ssm_tol(mo, ms, top, 100, dk, t)
    close(ob[:, :H * dv].reshape(T, H, dv), ow, to, "o")
    close(S1, sw, ts, "S1")
    assert (ob[:, H * dv:] == 5).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("what", ["q", "k", "v", "dt"])
def test_ssm_prompt_bad_values_stay_in_their_sequence(dtype, what):
    st = starts_of([130, 60, 77])
    z = ssm_inputs(70, 267, 3, 2, 1, 128, 64, dtype, pad=40)
    cfg = dl.SsmConfig(2, 1, 128, 64, dtype)
    good, sg = run_prompt(cfg, st, z, pad=40)
    bad = dict(z)
    bad[what] = z[what].clone()
    bad[what][130:190] = float("nan")
    bad[what][267:] = float("inf")  # rows behind the last sequence
    o, s = run_prompt(cfg, st, bad, pad=40)
    assert torch.equal(o[:130], good[:130]) and torch.equal(o[190:], good[190:])
    assert torch.equal(s[0], sg[0]) and torch.equal(s[2], sg[2])
    assert torch.isnan(o[130:190].float()).any()


@pytest.mark.parametrize("dtype,B,H,G,dk,dv", [
    ("bf16", 1, 2, 1, 128, 64), ("bf16", 5, 6, 2, 64, 128), ("bf16", 3, 3, 3, 64, 64),
    ("f32", 4, 2, 1, 128, 128), ("f32", 33, 1, 1, 64, 64)])
def test_ssm_step_continues_a_prompt(dtype, B, H, G, dk, dv):
    steps, t = 5, DT[dtype]
    st = starts_of([steps] * B)
    z = ssm_inputs(80, B * steps, B, H, G, dk, dv, dtype)
    ow, sw, mo, ms, top = ref.ssm(st, z["q"], z["k"], z["v"], z["dt"], z["a"], z["d"], z["bias"],
                                  z["S0"])
    to, ts = ref.ssm_tol(mo, ms, top, steps, dk, t)
    cfg = dl.SsmConfig(H, G, dk, dv, dtype)
    S = z["S0"].cuda()
    cut = lambda x: x.view((B, steps) + x.shape[1:]).transpose(0, 1).contiguous().cuda()
    q, k, v, dt = (cut(z[m]) for m in ("q", "k", "v", "dt"))
    a, d, bias = (z[m].cuda() for m in ("a", "d", "bias"))
    o = torch.empty(B, H, dv, dtype=t, device="cuda")
    for i in range(steps):
        dl.dl_ssm_step(cfg, q[i], k[i], v[i], dt[i], a, d, bias, S, o)
        close(o, ow.view(B, steps, H, dv)[:, i], to.view(B, steps, H, dv)[:, i], f"step {i}")
    close(S, sw, ts, "S")


# ------------------------------------------------------------------ norm

def check_norm(rows, D, dtype, out, block, res, seed=5, ld=0, scale=1.0):
    t, to = DT[dtype], {"bf16": T16, "f32": T32, "e4m3": torch.float8_e4m3fn}[out]
    x = (scale * rnd(seed, rows, D + ld)).to(t)[:, :D]
    r = (scale * rnd(seed + 1, rows, D + ld)).to(t)[:, :D] if res else None
    w = 1 + 0.2 * rnd(seed + 2, D)
    cfg = dl.NormConfig(D, dtype, out, block=block, eps=1e-5)
    wide = lambda ty: torch.zeros(rows, D + ld, dtype=ty, device="cuda")[:, :D]
    og, ro = wide(to), (wide(t) if res else None)
    sc = torch.full((rows, cfg.scales_per_row), -1.0, device="cuda") if out == "e4m3" else None
    back = torch.empty(rows, D + ld, dtype=t, device="cuda")
    xg = back[:, :D]
    xg.copy_(x)
    rg = None
    if res:
        rg = torch.empty(rows, D + ld, dtype=t, device="cuda")[:, :D]
        rg.copy_(r)
    dl.dl_norm(cfg, xg, w.cuda(), og, res=rg, res_out=ro, scales=sc)
    h, n = ref.norm(x, r, w, 1e-5)
    f = U32 = ref.U[T32]
    if res:
        # one fp32 sum, one rounding to the type
        close(ro, h, h.abs() * (ref.U[t] * (t != T32) + 1.01 * U32) + 1e-300, "res_out")
    # h: 1 rounding of what its addends are; the mean of squares: D roundings of
    # positive terms, halved by the root; 1/sqrt, two products: 4 more
    add = (x.double().abs() + (r.double().abs() if res else 0)) / h.abs().clamp_min(1e-30)
    rel = f * (0.5 * D + 6 + add.clamp_max(1e6)) * n.abs()
    if out != "e4m3":
        close(og, n, rel + n.abs() * ref.U[to] * (to != T32) + 1e-30, "out")
        return
    step = block or D
    amax = torch.stack([p.abs().max(1).values for p in n.split(step, 1)], 1)
    close(sc, amax / 448, amax / 448 * f * (0.5 * D + 12 + float(add.max().clamp_max(1e6))) + 1e-30,
          "scales")
    s = sc.double().cpu().repeat_interleave(step, 1)[:, :D]
    # codes: half a step of 3 mantissa bits, or half the smallest step 2^-9
    close(og.double().cpu() * s, n, 1.001 * (n.abs() * ref.U[to] + s * 2.0 ** -10) + 2 * rel + 1e-30,
          "codes")
    assert float(og.float().abs().max()) == 448.0


@pytest.mark.parametrize("dtype,out,block", [("bf16", "bf16", 0), ("bf16", "e4m3", 128),
                                             ("bf16", "e4m3", 0), ("f32", "f32", 0),
                                             ("f32", "bf16", 0), ("f32", "e4m3", 128)])
@pytest.mark.parametrize("rows,D", [(1, 1), (3, 128), (5, 129), (2, 256), (9, 1000), (3, 1024),
                                    (2, 2047), (4, 4096), (2, 6152), (1, 8192), (2, 16384), (3, 9001)])
def test_norm(dtype, out, block, rows, D):
    check_norm(rows, D, dtype, out, block, res=True)


@pytest.mark.parametrize("ld", [8, 3])
@pytest.mark.parametrize("dtype,out,block", [("bf16", "e4m3", 128), ("f32", "bf16", 0)])
def test_norm_strides_without_residual(dtype, out, block, ld):
    check_norm(7, 264, dtype, out, block, res=False, ld=ld)
    check_norm(6, 4096, dtype, out, block, res=True, ld=ld)


def test_norm_in_place_residual():
    x, r, w = rnd(1, 5, 512).to(T16), rnd(2, 5, 512).to(T16), torch.ones(512)
    cfg = dl.NormConfig(512, "bf16", "bf16")
    out, ro = torch.empty(5, 512, dtype=T16, device="cuda"), torch.empty(5, 512, dtype=T16, device="cuda")
    dl.dl_norm(cfg, x.cuda(), w.cuda(), out, res=r.cuda(), res_out=ro)
    for into in ("x", "res"):
        xg, rg, o2 = x.cuda(), r.cuda(), torch.empty_like(out)
        dl.dl_norm(cfg, xg, w.cuda(), o2, res=rg, res_out=xg if into == "x" else rg)
        assert torch.equal(o2, out) and torch.equal(xg if into == "x" else rg, ro)


def test_norm_zero_tiny_and_bad_rows():
    x = torch.zeros(5, 300)
    x[1] = 1e-30          # its square vanishes: n = x / sqrt(eps)
    x[2, 7] = 3e38        # the sum of squares is infinite: n = 0
    x[3, 200] = float("nan")
    x[4] = rnd(1, 300)
    w = torch.ones(300)
    w[128:256] = 0.0      # a block that is zero in every row
    cfg = dl.NormConfig(300, "f32", "e4m3", block=128, eps=1e-6)
    out = torch.empty(5, 300, dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.empty(5, 3, device="cuda")
    dl.dl_norm(cfg, x.cuda(), w.cuda(), out, scales=sc)
    o, sc = out.float().cpu(), sc.cpu()
    assert (o[0] == 0).all() and (sc[0] == 0).all()
    assert (o[1, :128] == 448).all() and sc[1, 0] > 0
    assert (o[2] == 0).all() and (sc[2] == 0).all()
    assert torch.isnan(o[3]).all()
    assert (o[[0, 1, 2, 4], 128:256] == 0).all() and (sc[[0, 1, 2, 4], 1] == 0).all()
    assert torch.isfinite(o[4]).all()


@pytest.mark.parametrize("block", [0, 128])
@pytest.mark.parametrize("rows,D", [(2500, 4096), (9000, 520)])
def test_norm_several_rows_a_team(rows, D, block):
    # more rows than run at once: a team takes one after the other
    check_norm(rows, D, "bf16", "e4m3", block, res=True)


def test_norm_many_rows():
    # more rows than one dimension of blocks of the short-row kernel covers evenly
    check_norm(70001, 24, "f32", "bf16", 0, res=False)


# ------------------------------------------------------- streams and graphs

def test_calls_on_a_side_stream_and_in_a_replayed_graph():
    H, G, dk, dv, B = 4, 1, 128, 64, 3
    C = H * dv + 2 * G * dk
    z = {k: v.cuda() for k, v in ssm_inputs(90, B, B, H, G, dk, dv, "bf16").items()}
    conv, ssm = dl.ConvConfig(C, 4, "bf16"), dl.SsmConfig(H, G, dk, dv, "bf16")
    nrm = dl.NormConfig(H * dv, "bf16", "e4m3", block=128)
    x, w, b = rnd(1, B, C).to(T16).cuda(), rnd(2, C, 4).cuda(), rnd(3, C).cuda()
    h, wn = rnd(4, B, 3, C).to(T16).cuda(), torch.ones(H * dv, device="cuda")

    def bufs():
        return dict(h=h.clone(), S=z["S0"].clone(), row=torch.empty(B, C, dtype=T16, device="cuda"),
                    o=torch.empty(B, H * dv, dtype=T16, device="cuda"),
                    out=torch.empty(B, H * dv, dtype=torch.float8_e4m3fn, device="cuda"),
                    sc=torch.empty(B, nrm.scales_per_row, device="cuda"))

    def step(u):
        dl.dl_conv_step(conv, x, w, b, u["h"], u["row"])
        dl.dl_ssm_step(ssm, u["row"][:, H * dv + dk:], u["row"][:, H * dv:H * dv + dk],
                       u["row"][:, :H * dv], z["dt"], z["a"], z["d"], z["bias"], u["S"], u["o"])
        dl.dl_norm(nrm, u["o"], wn, u["out"], scales=u["sc"])

    one, two, three = bufs(), bufs(), bufs()
    for _ in range(4):
        step(one)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(4):
            step(two)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(three)
    three["h"].copy_(h)
    three["S"].copy_(z["S0"])
    for _ in range(4):
        graph.replay()
    torch.cuda.synchronize()
    for name in one:
        a = one[name].float()
        assert torch.equal(a, two[name].float()), name
        assert torch.equal(a, three[name].float()), name


def test_prompt_in_a_graph_and_twice_the_same():
    st = starts_of([700, 3, 260])
    z = {k: v.cuda() for k, v in ssm_inputs(95, 963, 3, 2, 1, 128, 64, "bf16").items()}
    cfg = dl.SsmConfig(2, 1, 128, 64, "bf16")
    ws = torch.empty(dl.dl_ssm_bytes(cfg, st), dtype=torch.uint8, device="cuda")

    def call(o, s1):
        dl.dl_ssm_prompt(cfg, st, z["q"], z["k"], z["v"], z["dt"], z["a"], z["d"], z["bias"],
                         z["S0"], s1, o, ws)

    outs = [(torch.empty(963, 2, 64, dtype=T16, device="cuda"), torch.empty_like(z["S0"]))
            for _ in range(3)]
    call(*outs[0])
    call(*outs[1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(*outs[2])
    graph.replay()
    torch.cuda.synchronize()
    for o, s in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(s, outs[0][1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompts_at_the_same_time(dtype):
    # two streams, a workspace each
    st = [starts_of([900, 40]), starts_of([30, 1200])]
    cfg = dl.SsmConfig(2, 1, 128, 64, dtype)
    z = [{k: v.cuda() for k, v in ssm_inputs(97 + i, int(s[-1]), 2, 2, 1, 128, 64, dtype).items()}
         for i, s in enumerate(st)]
    ws = [torch.empty(dl.dl_ssm_bytes(cfg, s), dtype=torch.uint8, device="cuda") for s in st]
    alone = [(torch.empty(int(s[-1]), 2, 64, dtype=DT[dtype], device="cuda"), torch.empty_like(u["S0"]))
             for s, u in zip(st, z)]
    both = [[torch.empty_like(v) for v in pair] for pair in alone]

    def call(i, out):
        u = z[i]
        dl.dl_ssm_prompt(cfg, st[i], u["q"], u["k"], u["v"], u["dt"], u["a"], u["d"], u["bias"], u["S0"],
                         out[1], out[0], ws[i])

    for i in range(2):
        call(i, alone[i])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                call(i, both[i])
    torch.cuda.synchronize()
    assert dl.dl_device_error(None) == (0, 0)
    for a, b in zip(alone, both):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ------------------------------------------------------------ empty calls

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_calls_without_rows(dtype):
    # empty batches do nothing; prompts of no tokens pass their states on
    t = DT[dtype]
    z = lambda *s: torch.zeros(*s, dtype=t, device="cuda")
    f = lambda *s: torch.zeros(*s, device="cuda")
    dl.dl_norm(dl.NormConfig(64, dtype, "e4m3"), z(0, 64), f(64),
               z(0, 64).to(torch.float8_e4m3fn), scales=f(0, 1))
    conv = dl.ConvConfig(24, 4, dtype)
    dl.dl_conv_step(conv, z(0, 24), f(24, 4), None, z(0, 3, 24), z(0, 24))
    h0, h1 = rnd(1, 2, 3, 24).to(t).cuda(), z(2, 3, 24)
    dl.dl_conv_prompt(conv, [0, 0, 0], z(0, 24), f(24, 4), None, h0, h1, z(0, 24))
    assert torch.equal(h0, h1)
    ssm = dl.SsmConfig(2, 1, 64, 128, dtype)
    row = (z(0, 64), z(0, 64), z(0, 256), f(0, 2), f(2) - 1, None, None)
    dl.dl_ssm_step(ssm, *row, f(0, 2, 128, 64), z(0, 256))
    S0, S1 = rnd(2, 2, 2, 128, 64).cuda(), f(2, 2, 128, 64)
    dl.dl_ssm_prompt(ssm, [0, 0, 0], *row, S0, S1, z(0, 256))
    assert torch.equal(S0, S1)
    dl.dl_ssm_prompt(ssm, [0, 0, 0], *row, None, S1, z(0, 256))
    assert (S1 == 0).all()


# --------------------------------------------------- the operators together

def test_prompt_then_tokens_as_one_layer():
    # conv -> scan -> norm over a packed prompt, then token by token from the
    # states it leaves, against one run over all tokens in 64 bits
    H, G, dk, dv, W, B, extra = 4, 2, 64, 64, 4, 3, 4
    C = H * dv + 2 * G * dk
    lens = [130, 1, 47]
    st, stf = starts_of(lens), starts_of([n + extra for n in lens])
    T, Tf = int(st[-1]), int(stf[-1])
    x = rnd(1, Tf, C)
    w, b = 0.5 * rnd(2, C, W), 0.1 * rnd(3, C)
    z = ssm_inputs(7, Tf, B, H, G, dk, dv, "f32")
    gain = 1 + 0.1 * rnd(4, H * dv)
    conv, ssm = dl.ConvConfig(C, W, "f32"), dl.SsmConfig(H, G, dk, dv, "f32")
    nrm = dl.NormConfig(H * dv, "f32", "f32", eps=1e-5)
    parts = lambda r: (r[:, H * dv + G * dk:], r[:, H * dv:H * dv + G * dk], r[:, :H * dv])
    where = np.concatenate([np.arange(stf[s], stf[s] + lens[s]) for s in range(B)])
    cu = lambda v: v.contiguous().cuda()
    h, S = torch.empty(B, W - 1, C, device="cuda"), torch.empty(B, H, dv, dk, device="cuda")
    wg, bg, a, d, bias, gg = (cu(v) for v in (w, b, z["a"], z["d"], z["bias"], gain))

    def buffers(n):
        return (torch.empty(n, C, device="cuda"), torch.empty(n, H * dv, device="cuda"),
                torch.empty(n, H * dv, device="cuda"))

    row, o, out = buffers(T)
    dl.dl_conv_prompt(conv, st, cu(x[where]), wg, bg, None, h, row)
    dl.dl_ssm_prompt(ssm, st, *parts(row), cu(z["dt"][where]), a, d, bias, None, S, o)
    dl.dl_norm(nrm, o, gg, out)
    got = torch.empty(Tf, H * dv)
    got[where] = out.cpu()
    row, o, out = buffers(B)
    for i in range(extra):
        at = np.array([stf[s] + lens[s] + i for s in range(B)])
        dl.dl_conv_step(conv, cu(x[at]), wg, bg, h, row)
        dl.dl_ssm_step(ssm, *parts(row), cu(z["dt"][at]), a, d, bias, S, o)
        dl.dl_norm(nrm, o, gg, out)
        got[at] = out.cpu()
    y, _, _ = ref.conv(x, stf, w, b, None, True)
    q, k, v = (p.reshape(Tf, -1, m) for p, m in zip(parts(y), (dk, dk, dv)))
    ow, sw, mo, ms, top = ref.ssm(stf, q, k, v, z["dt"], z["a"], z["d"], z["bias"], None)
    _, want = ref.norm(ow.reshape(Tf, -1), None, gain, 1e-5)
    # each stage's own bound, the convolution's (a few 2^-24 of each factor) met
    # three times by the scan's products; the norm scales errors of a row by its r
    r = (want / ow.reshape(Tf, -1)).abs().clamp_max(1e6)
    f = ref.U[T32]
    err = mo.reshape(Tf, -1) * f * (max(lens) * (6 + 8 * top) + dk + 8 + 3 * (W + 10) * 4)
    tol = r * err + want.abs() * (f * (H * dv + 8) + (err.norm(dim=1) / ow.reshape(Tf, -1).norm(dim=1))[:, None])
    close(got, want, tol, "layer")
    _, ts = ref.ssm_tol(mo, ms, top, max(lens) + extra, dk, T32)
    close(S, sw, ts + ms * f * 2 * (W + 10) * 4, "S")


def test_conv_feeds_the_decode_step_and_norm_takes_its_output():
    # q, k, v of the existing GDN step through the convolution, its fp32 output
    # through the per-head norm
    B, H, d = 3, 2, 128
    C = 3 * H * d
    x, w = rnd(1, B, C).to(T16), rnd(2, C, 4)
    conv = dl.ConvConfig(C, 4, "bf16")
    h, row = torch.zeros(B, 3, C, dtype=T16, device="cuda"), torch.empty(B, C, dtype=T16, device="cuda")
    dl.dl_conv_step(conv, x.cuda(), w.cuda(), None, h, row)
    unit = lambda m: torch.nn.functional.normalize(m.float().view(B * H, d), dim=1).to(T16)
    q, k = (unit(row[:, i * H * d:(i + 1) * H * d]) for i in range(2))
    v = row[:, 2 * H * d:].contiguous()
    alpha, beta = torch.full((B * H,), 0.9, device="cuda"), torch.full((B * H,), 0.5, device="cuda")
    cfg = dl.Config("gdn", B, H, d, d, 4, "bf16", fused_merge=True)
    S0 = 0.1 * rnd(3, B * H, d, d).cuda()
    st = dl.DeltaLogState(cfg)
    st.reset(S0.reshape(-1))
    o = st.step(q, k, v, alpha, beta).view(B * H, d)
    out = torch.empty(B * H, d, dtype=T16, device="cuda")
    dl.dl_norm(dl.NormConfig(d, "f32", "bf16", eps=1e-6), o, torch.ones(d, device="cuda"), out)
    S, kd, qd = S0.double().cpu(), k.double().cpu(), q.double().cpu()
    vd = v.double().cpu().view(B * H, d)
    S = 0.9 * S
    S = S + 0.5 * (vd - (S * kd[:, None]).sum(-1))[..., None] * kd[:, None]
    ow = (S * qd[:, None]).sum(-1)
    assert float((o.double().cpu() - ow).abs().max()) <= 1e-5 * float(ow.abs().max())
    _, n = ref.norm(o.cpu(), None, torch.ones(d), 1e-6)
    close(out, n, n.abs() * (2.0 ** -8 + 2.0 ** -24 * (d + 8)) + 1e-30, "norm")
    st.close()


def test_prompt_state_loads_into_the_framework_layout():
    # the scan's S1 has the layout dl_state_load_seqs takes
    cfg = dl.SsmConfig(2, 1, 128, 128, "bf16")
    z = ssm_inputs(99, 60, 2, 2, 1, 128, 128, "bf16")
    _, s1 = run_prompt(cfg, starts_of([20, 40]), z)
    st = dl.DeltaLogState(dl.Config("gdn", 4, 2, 128, 128, 4, "bf16"))
    st.reset()
    st.load_seqs([3, 1], s1)
    S = st.materialize().view(4, 2, 128, 128)
    assert torch.equal(S[3], s1[0]) and torch.equal(S[1], s1[1]) and (S[0] == 0).all()
    st.close()
