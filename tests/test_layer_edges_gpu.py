"""The operators around the recurrent step on the GPU at the borders of their
number formats and of their launch forms, against 64-bit definitions."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from linear_attention_recurrent_deltalog_b200 import deltalog as dl
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu

T16, T32, T8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
U = 2.0 ** -24


def rnd(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


# ------------------------------------------------------------------ norm

# largest magnitudes of a block around the ones where 448 / amax leaves fp32's
# range (below 1.75 * 2^-120) and where a block is stored as zeros (below 2^-120)
PEAKS = [2.0 ** -121, 2.0 ** -120 * (1 - U), 2.0 ** -120, 1.2 * 2.0 ** -120, 1.74 * 2.0 ** -120,
         1.75 * 2.0 ** -120, 2.0 ** -119, 1.5 * 2.0 ** -100, 2.0 ** -65, 1.1 * 2.0 ** -64, 1.0, 2.0 ** 100]


def peaked(n, peak, seed):
    """n values whose largest magnitude is `peak`: zeros, the peak, and values down to its 2^-20."""
    g = torch.Generator().manual_seed(seed)
    v = peak * torch.exp2(-20 * torch.rand(n, generator=g)) * torch.sign(torch.randn(n, generator=g))
    v[::5] = 0.0
    v[1] = -peak
    return v.to(T32)


def check_codes(codes, scale, n):
    """Codes and scale of one block of exact values n: the scale is amax / 448
    rounded once (half a step: 2^-24 of it, or of the smallest normal below
    that); a code's value is n * (448 / amax) after two roundings to 24 bits,
    then half a step of e4m3 (2^-4 of it, at least half of 2^-9)."""
    n = n.double()
    amax = float(n.abs().max())
    codes = codes.double()
    assert torch.isfinite(codes).all()
    if amax < 2.0 ** -120:
        assert (codes == 0).all() and float(scale) == 0.0
        return
    assert abs(float(scale) - amax / 448) <= amax / 448 * U + 2.0 ** -150
    want = n * (448 / amax)
    pre = want.abs() * 2.1 * U
    assert ((codes - want).abs() <= torch.clamp((want.abs() + pre) * 2.0 ** -4, min=2.0 ** -10) + pre).all()
    assert (codes[n == 0] == 0).all() and float(codes.abs().max()) == 448.0


@pytest.mark.parametrize("tail", [0, 3])  # 3: rows that take the element-wise path
def test_norm_codes_of_small_blocks(tail):
    # rows of ones and eps = 0 have the root 1 exactly: n is the weight
    D = 128 * len(PEAKS) + tail
    w = torch.cat([peaked(128, p, i) for i, p in enumerate(PEAKS)] +
                  ([peaked(tail, 1.0, 99)] if tail else []))
    out, sc = torch.empty(2, D, dtype=T8, device="cuda"), torch.empty(2, -(-D // 128), device="cuda")
    dl.dl_norm(dl.NormConfig(D, "f32", "e4m3", block=128, eps=0.0), torch.ones(2, D, device="cuda"), w.cuda(),
               out, scales=sc)
    o, sc = out.float().cpu(), sc.cpu()
    for row in range(2):
        for b in range(len(PEAKS)):
            check_codes(o[row, 128 * b:128 * b + 128], sc[row, b], w[128 * b:128 * b + 128])


@pytest.mark.parametrize("D", [64, 1024, 4099])
@pytest.mark.parametrize("peak", PEAKS)
def test_norm_codes_of_small_rows(peak, D):
    w = peaked(D, peak, 7)
    out, sc = torch.empty(3, D, dtype=T8, device="cuda"), torch.empty(3, 1, device="cuda")
    dl.dl_norm(dl.NormConfig(D, "bf16", "e4m3", eps=0.0), torch.ones(3, D, dtype=T16, device="cuda"), w.cuda(),
               out, scales=sc)
    for row in range(3):
        check_codes(out[row].float().cpu(), sc[row].cpu(), w)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("block", [0, 128])
@pytest.mark.parametrize("rows,D", [(3, 1), (5, 129), (9, 1000), (4, 4096), (2, 6152), (2, 16384), (3, 9001),
                                    (9000, 520)])
def test_norm_scales_and_codes_tightly(rows, D, block, dtype):
    # In units of 2^-24 of the value: x + res is rounded once, whatever cancels.
    # The mean of squares: 2 of each square, D of the sum of positive terms, 1 each
    # of the division and of eps, halved by the root; root, reciprocal, two products
    # and the sum's own 1: D / 2 + 7 for n, one more for the scale.  The mean's part
    # is the whole row's and leaves n / amax as it is: 3 of n, 3 of amax, the
    # quotient and the product make 8 before the code's rounding, half a step of
    # e4m3 (2^-4 of it, at least half of 2^-9).
    t = {"bf16": T16, "f32": T32}[dtype]
    x, r, w = rnd(1, rows, D).to(t), rnd(2, rows, D).to(t), 1 + 0.2 * rnd(3, D)
    step = block or D
    out = torch.empty(rows, D, dtype=T8, device="cuda")
    sc = torch.empty(rows, -(-D // step), device="cuda")
    dl.dl_norm(dl.NormConfig(D, dtype, "e4m3", block=block, eps=1e-5), x.cuda(), w.cuda(), out, res=r.cuda(),
               scales=sc)
    _, n = ref.norm(x, r, w, 1e-5)
    amax = torch.stack([p.abs().max(1).values for p in n.split(step, 1)], 1)
    assert ((sc.double().cpu() - amax / 448).abs() <= amax / 448 * ((0.5 * D + 8.1) * U)).all()
    want = n * (448 / amax).repeat_interleave(step, 1)[:, :D]
    pre = want.abs() * (8.1 * U)
    err = (out.double().cpu() - want).abs()
    assert (err <= torch.clamp((want.abs() + pre) * 2.0 ** -4, min=2.0 ** -10) + pre).all()


# ------------------------------------------------------------------ scan

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["stream", "handle"])
def test_prompt_on_a_given_stream_without_a_workspace(dtype, kind):
    # the workspace of a call on a stream that is not the current one may not go
    # to the current stream's next tensor while the call still uses it
    t, T, H = {"bf16": T16, "f32": T32}[dtype], 4000, 2
    cfg = dl.SsmConfig(H, 1, 128, 64, dtype)
    z = dict(q=rnd(1, T, 128).to(t), k=rnd(2, T, 128).to(t), v=rnd(3, T, H * 64).to(t),
             dt=0.1 * rnd(4, T, H).abs(), a=-rnd(5, H).abs())
    z = {k: v.cuda() for k, v in z.items()}
    nbytes = dl.dl_ssm_bytes(cfg, [0, T])
    assert nbytes > 0

    def call(**kw):
        o, S1 = torch.empty(T, H * 64, dtype=t, device="cuda"), torch.empty(1, H, 64, 128, device="cuda")
        torch.cuda.synchronize()
        dl.dl_ssm_prompt(cfg, [0, T], z["q"], z["k"], z["v"], z["dt"], z["a"], None, None, None, S1, o, **kw)
        return o, S1

    want = call(workspace=torch.empty(nbytes, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(20):
        got = call(stream=side if kind == "stream" else side.cuda_stream)
        after = [torch.empty(nbytes, dtype=torch.uint8, device="cuda").fill_(0x7f) for _ in range(4)]
        torch.cuda.synchronize()
        assert all(bool((x == 0x7f).all()) for x in after)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert dl.dl_device_error(None) == (0, 0)


# ------------------------------------------------------------------ convolution

@pytest.mark.parametrize("C", [1, 4])  # element by element, four channels at a time
def test_conv_of_the_last_row_numbers(C):
    # offsets past 32 bits, and row numbers up to the last one allowed
    top, W, lens = 2 ** 31 - 1024, 4, [300, 0, 37]
    st = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64) + top - sum(lens)
    x = torch.empty(top, C, dtype=T16, device="cuda")
    y = torch.empty(top, C, dtype=T16, device="cuda")
    rows = rnd(1, sum(lens), C).to(T16)
    x[-sum(lens):] = rows.cuda()
    y[-500:] = 7.0
    w, h = rnd(2, C, W), rnd(3, 3, W - 1, C).to(T16)
    h1 = torch.empty(3, W - 1, C, dtype=T16, device="cuda")
    dl.dl_conv_prompt(dl.ConvConfig(C, W, "bf16", silu=False), st, x, w.cuda(), None, h.cuda(), h1, y)
    want, mag, hw = ref.conv(rows, st - st[0], w, None, h, False)
    got = y[-sum(lens):].double().cpu()
    assert ((got - want).abs() <= ref.conv_tol(mag, W, T16)).all()
    assert torch.equal(h1.double().cpu(), hw)
    assert (y[-500:-sum(lens)] == 7).all()


def test_conv_silu_of_fp32_rows_over_its_range():
    # one tap of 1: the sum is x itself, so y is the activation alone.  Its
    # roundings, in units of 2^-24 of the value: the exponential 4 (2 ulp), which
    # counts half to whole, and one each for 1 + e, the quotient and the product:
    # 8 in all.  Below -87.3 e^x has no normal fp32: half a step of 2^-149, times |x|.
    x = torch.cat([torch.linspace(-106, 106, 40001), torch.linspace(-89, -87, 4001),
                   torch.tensor([0.0, -0.0, 1e-30, -1e-30, 3e38, -3e38, 1e-45])]).to(T32)
    for C in (1, 4):
        n = x.numel() // C * C
        xg = x[:n].view(-1, C).cuda()
        w = torch.zeros(C, 2, device="cuda")
        w[:, 1] = 1.0
        y = torch.empty_like(xg)
        dl.dl_conv_prompt(dl.ConvConfig(C, 2, "f32"), [0, n // C], xg, w, None, None, None, y)
        xd = x[:n].double()
        want = xd / (1 + torch.exp(-xd))
        tol = want.abs() * 8 * U + (xd.abs() + 1) * 4 * 2.0 ** -149
        bad = (y.double().cpu().view(-1) - want).abs() > tol
        assert not bad.any(), (x[:n][bad][:5], y.cpu().view(-1)[bad][:5], int(bad.sum()))


@pytest.mark.parametrize("dtype,B,C,W", [("bf16", 509, 4352, 4), ("bf16", 67, 8191, 4), ("bf16", 1030, 1024, 3),
                                         ("bf16", 250, 8191, 2), ("f32", 301, 4352, 4), ("f32", 131, 4353, 2)])
def test_conv_step_of_several_sequences_a_thread(dtype, B, C, W):
    # more than the 113,664 threads of a wave at four channels (or one) each: a
    # thread takes 2 to 8 sequences, four at a time, with a rest in the last batch
    # and a shorter share in the last thread
    t = {"bf16": T16, "f32": T32}[dtype]
    x, w, b, h = rnd(1, B, C).to(t), rnd(2, C, W), rnd(3, C), rnd(4, B, W - 1, C).to(t)
    hg, y = h.cuda(), torch.full((B + 1, C), 7.0, dtype=t, device="cuda")
    dl.dl_conv_step(dl.ConvConfig(C, W, dtype), x.cuda(), w.cuda(), b.cuda(), hg, y[:B])
    rows = torch.cat([h, x[:, None]], 1).double()
    s = b.double() + (rows * w.double().t()).sum(1)
    mag = b.double().abs() + (rows * w.double().t()).abs().sum(1)
    want = ref.silu(s)
    tol = ref.conv_tol(1.1 * mag + want.abs(), W, t)
    assert ((y[:B].double().cpu() - want).abs() <= tol).all()
    assert torch.equal(hg.double().cpu(), rows[:, 1:]) and (y[B] == 7).all()
