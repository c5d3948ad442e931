"""Rotary embedding: api.rotary, its inverse and its gradient against the fp64 oracle.

Tolerance of an output element y of the pair (a, b), T the element type:
    eps(T)/2·|y|  its one rounding, and 2^-25 for fp16's smallest steps,
  + 1e-6·(|a| + |b|)  the angle (2^-32 turns, and its conversion to fp32, 2^-25 half turns:
    1e-7 rad), sincospif (2 ulp, 1.2e-7), and four fp32 roundings of products and the sum
    (2.4e-7), about doubled.
"""
import math

import numpy as np
import pytest
import torch

from oracle import cache as ref
from scaled_dot_product_flash_gb300 import _lib, api, autograd, build
from scaled_dot_product_flash_gb300.inputs import as_f64

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
INVALID, UNSUPPORTED = 1, 2


def frequencies(rot, base=10000.0):
    n = rot // 2
    return torch.from_numpy((base ** (-np.arange(n) / n)).astype(np.float32))


def draw(rng, shape, dtype):
    return torch.from_numpy(rng.standard_normal(shape)).to(TYPES[dtype])


def check(y, x, positions, inv, axes, adjacent, inverse, what=""):
    """y (torch) is the rotation of x (torch) within the tolerance above."""
    want = ref.rotary(as_f64(x), positions, inv.numpy(), axes, adjacent, inverse)
    n = len(inv)
    pair = np.abs(as_f64(x))
    size = pair.copy()
    for p in range(n):
        a, b = (2 * p, 2 * p + 1) if adjacent else (p, p + n)
        size[..., a] = size[..., b] = pair[..., a] + pair[..., b]
    size[..., 2 * n:] = 0
    tol = torch.finfo(y.dtype).eps / 2 * np.abs(want) + 1e-6 * size + (2.0 ** -25 if y.dtype == torch.float16 else 0)
    off = np.abs(as_f64(y) - want) - tol
    assert off.max() <= 0, f"{what} off by {off.max():.3e} more than its tolerance"
    assert np.array_equal(as_f64(y)[..., 2 * n:], as_f64(x)[..., 2 * n:])


# ---- without a GPU


def test_oracle_turns_by_the_angle():
    x = np.zeros((1, 1, 1, 4))
    x[..., 0], x[..., 1] = 1.0, 2.0
    y = ref.rotary(x, np.array([[[3]]]), np.array([0.5, 0.25]))
    assert np.allclose(y[0, 0, 0], [math.cos(1.5), 2 * math.cos(0.75), math.sin(1.5), 2 * math.sin(0.75)])
    y = ref.rotary(x, np.array([[[3]]]), np.array([0.5, 0.25]), adjacent=True)
    assert np.allclose(y[0, 0, 0], [math.cos(1.5) - 2 * math.sin(1.5), 2 * math.cos(1.5) + math.sin(1.5), 0, 0])


def test_axes_of_sections():
    assert api.rotary_axes([2, 0, 3], device="cpu").tolist() == [0, 0, 2, 2, 2]
    with pytest.raises(ValueError):
        api.rotary_axes([0, 0], device="cpu")
    with pytest.raises(ValueError):
        api.rotary_axes([2, -1], device="cpu")


@pytest.mark.parametrize("shape,want", [
    ((7,), (1, [0, 0, 1])), ((2, 7), (1, [0, 7, 1])), ((1, 7), (1, [0, 0, 1])),
    ((3, 2, 7), (3, [14, 7, 1])), ((3, 1, 7), (3, [7, 0, 1])),
])
def test_positions(shape, want):
    assert api._positions(torch.zeros(shape, dtype=torch.int32), 2, 7) == want


@pytest.mark.parametrize("bad", [
    torch.zeros(6, dtype=torch.int32), torch.zeros(3, 7, dtype=torch.int32),
    torch.zeros(1, 1, 2, 7, dtype=torch.int32), torch.zeros(7), torch.zeros(7, dtype=torch.int16),
    torch.zeros(0, 2, 7, dtype=torch.int32),
])
def test_positions_refused(bad):
    with pytest.raises(ValueError):
        api._positions(bad, 2, 7)


def test_host_tensors_are_refused():
    q = torch.zeros(1, 2, 3, 64)
    with pytest.raises(ValueError):
        api.rotary(q, None, torch.zeros(3, dtype=torch.int32), frequencies(64))
    with pytest.raises(NotImplementedError):
        autograd.rotary_embedding(q, None, torch.zeros(3, dtype=torch.int32), frequencies(64).requires_grad_())


# Fake, 16-byte aligned addresses: every case is rejected before anything is launched.
Q, K, QO, KO, POS, INV, AX = (0x10000000 * (n + 1) for n in range(7))


def call(q=Q, k=K, q_out=QO, k_out=KO, pos=POS, bits=32, pos_strides=(128, 64, 1), inv=INV, axes=AX, naxes=2, B=2, Hq=4, Hkv=2, L=64, D=64,
         rot=64, flags=0, dtype=2, lay=None):
    def dense(H):
        return (H * L * D, L * D, D)
    lay = lay or (*dense(Hq), *dense(Hkv), *dense(Hq), *dense(Hkv))
    build.build()
    return _lib.sdpa_rotary(q, k, q_out, k_out, pos, bits, _lib.Int64x3(*pos_strides), inv, axes, naxes, B, Hq, Hkv, L, D, rot, flags, dtype,
                            _lib.Int64x12(*lay), None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=0), INVALID), (dict(q_out=0), INVALID), (dict(pos=0), INVALID), (dict(inv=0), INVALID),
    (dict(k_out=0), INVALID), (dict(k=0), INVALID),            # one of k and k_out
    (dict(q=Q + 8), INVALID), (dict(k_out=KO + 2), INVALID), (dict(inv=INV + 2), INVALID), (dict(axes=AX + 1), INVALID),
    (dict(pos=POS + 4, bits=64), INVALID), (dict(bits=16), INVALID), (dict(pos_strides=(0, -1, 1)), INVALID),
    (dict(rot=63), INVALID), (dict(rot=0), INVALID), (dict(rot=66), INVALID), (dict(naxes=0), INVALID), (dict(flags=4), INVALID),
    (dict(B=0), INVALID), (dict(L=0), INVALID), (dict(Hkv=0), INVALID),
    (dict(D=48, rot=32), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED), (dict(B=70000), UNSUPPORTED),
    (dict(q_out=Q + 64), INVALID),                             # overlaps q without being in place
    (dict(q_out=K), INVALID), (dict(k_out=QO + 16), INVALID), (dict(q_out=POS), INVALID), (dict(k_out=INV), INVALID), (dict(k_out=AX), INVALID),
    # views of one token buffer that share heads, or whose tokens run into each other
    (dict(q=Q, k=Q + 4 * 128 - 16, q_out=Q, lay=(24576, 64, 384, 24576, 64, 384, 24576, 64, 384, 8192, 4096, 64)), INVALID),
    (dict(q=Q, k=Q + 4 * 128, q_out=Q, lay=(20480, 64, 320, 20480, 64, 320, 20480, 64, 320, 8192, 4096, 64)), INVALID),
    (dict(q_out=Q, lay=(16384, 4096, 64, 8192, 4096, 64, 16384, 64, 256, 8192, 4096, 64)), INVALID),   # q's memory, other strides
])
def test_refused(kw, code):
    assert call(**kw) == code


# ---- on the GPU


@pytest.mark.gpu
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("dtype,B,Hq,Hkv,L,D,rot,axes", [
    ("bf16", 1, 1, 1, 1, 32, 32, 1),
    ("bf16", 2, 8, 2, 33, 128, 128, 3),
    ("f16", 3, 6, 3, 17, 96, 96, 2),
    ("f16", 1, 5, 1, 130, 64, 42, 1),      # no 16-byte pieces: the one-pair form
    ("f32", 2, 4, 4, 9, 256, 256, 4),
    ("f32", 1, 3, 1, 70, 96, 24, 2),
    ("bf16", 1, 40, 8, 5, 256, 2, 1),
    ("f32", 1, 2, 2, 3, 32, 6, 1),
])
def test_rotary(dtype, B, Hq, Hkv, L, D, rot, axes, adjacent):
    rng = np.random.default_rng(B + L + D)
    q, k = draw(rng, (B, Hq, L, D), dtype), draw(rng, (B, Hkv, L, D), dtype)
    positions = rng.integers(-50, 100000, (axes, B, L))
    inv, of = frequencies(rot), rng.integers(0, axes, rot // 2).astype(np.int32)
    args = (torch.from_numpy(positions).to(torch.int32).cuda(), inv.cuda(), torch.from_numpy(of).cuda(), adjacent)
    qo, ko = api.rotary(q.cuda(), k.cuda(), *args)
    dq, dk = api.rotary_backward(q.cuda(), k.cuda(), *args)
    alone, nothing = api.rotary(q.cuda(), None, *args)
    api.poll_status()
    check(qo, q, positions, inv, of, adjacent, False, "q")
    check(ko, k, positions, inv, of, adjacent, False, "k")
    check(dq, q, positions, inv, of, adjacent, True, "dq")
    check(dk, k, positions, inv, of, adjacent, True, "dk")
    assert nothing is None and torch.equal(alone, qo)


@pytest.mark.gpu
def test_far_positions_keep_their_angles():
    """Positions near 2^31 and beyond, where position·inv_freq in fp32 has lost every digit.
    The angle's error is |position|·(1 + inv_freq)·2^-64 turns beside the usual, 7.5e-7 rad at 2^40."""
    rng = np.random.default_rng(5)
    positions = np.array([[[2**31 - 1, -2**31, 2**40, -(2**40) - 12345, 0, 1]]])
    q = draw(rng, (1, 2, 6, 64), "f32")
    inv = frequencies(64)
    from fractions import Fraction
    two_pi = Fraction("6.283185307179586476925286766559005768394338798750211641949889184615632812572417997256069650684234135964296173026564613")
    out, _ = api.rotary(q.cuda(), None, torch.from_numpy(positions[0, 0]).cuda(), inv.cuda())
    api.poll_status()
    want = as_f64(q)
    for i, pos in enumerate(positions[0, 0].tolist()):
        for p in range(32):
            turn = Fraction(pos) * Fraction(float(inv[p])) / two_pi
            angle = float((turn - round(turn)) * two_pi)
            a, b = want[..., i, p].copy(), want[..., i, p + 32].copy()
            want[..., i, p], want[..., i, p + 32] = a * math.cos(angle) - b * math.sin(angle), b * math.cos(angle) + a * math.sin(angle)
    assert np.abs(as_f64(out) - want).max() <= 1e-6 * 2 * np.abs(as_f64(q)).max() + 2e-6


@pytest.mark.gpu
def test_frequencies_of_any_size():
    """Frequencies above one turn a step, tiny ones, negative ones, 0 and a NaN in one call."""
    inv = torch.tensor([1000.0, 3.0e-39, -0.37, 0.0, float("nan"), float("inf"), 2.0 ** -60, 1.0])
    positions = np.array([[[5, 1234567]]])
    q = draw(np.random.default_rng(6), (1, 1, 2, 32), "f32")
    out, _ = api.rotary(q.cuda(), None, torch.from_numpy(positions[0]).cuda(), inv.cuda())
    api.poll_status()
    bad = [4, 5, 12, 13]
    assert torch.isnan(out[..., bad]).all()
    good = [p for p in range(8) if p not in (4, 5)]
    got, want = as_f64(out), ref.rotary(as_f64(q), positions, np.where(np.isfinite(inv.numpy()), inv.numpy(), 0))
    cols = good + [p + 8 for p in good]
    # 1000 rad a step: the fp64 oracle's own angle, 1.2e9 rad, is good to 1.2e-7 rad.
    assert np.abs(got[..., cols] - want[..., cols]).max() <= 2e-6 * np.abs(as_f64(q)).max() * 2


@pytest.mark.gpu
def test_layouts_in_place_and_streams():
    rng = np.random.default_rng(7)
    B, Hq, Hkv, L, D = 2, 6, 2, 37, 64
    packed = draw(rng, (B, L, Hq + Hkv, D), "bf16").cuda()           # a fused projection's output
    q, k = packed[:, :, :Hq].transpose(1, 2), packed[:, :, Hq:].transpose(1, 2)
    positions = torch.arange(100, 100 + L).cuda()
    inv = frequencies(D).cuda()
    want = api.rotary(q.contiguous(), k.contiguous(), positions.to(torch.int32), inv)
    got = api.rotary(q, k, positions.expand(B, L), inv, q_out=torch.empty(B, L, Hq, D, dtype=q.dtype, device="cuda").transpose(1, 2))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = api.rotary(q, k, positions, inv, stream=side)
    side.synchronize()
    assert torch.equal(other[0], want[0]) and torch.equal(other[1], want[1])
    same = api.rotary(q, k, positions, inv, q_out=q, k_out=k)
    assert torch.equal(same[0], want[0]) and torch.equal(packed[:, :, Hq:].transpose(1, 2), want[1])
    api.poll_status()
    with pytest.raises(_lib.SdpaError):
        api.rotary(q, k, positions, inv, q_out=torch.empty_like(q), k_out=q[:, :Hkv])


@pytest.mark.gpu
def test_an_axis_out_of_range_is_reported():
    q = draw(np.random.default_rng(8), (1, 2, 3, 32), "f32").cuda()
    positions = torch.arange(6, dtype=torch.int32).view(2, 1, 3).cuda()
    axes = torch.zeros(16, dtype=torch.int32)
    want, _ = api.rotary(q, None, positions, frequencies(32).cuda(), axes.cuda())
    axes[3], axes[9] = 2, -1
    got, _ = api.rotary(q, None, positions, frequencies(32).cuda(), axes.cuda())
    with pytest.raises(_lib.SdpaError) as e:
        api.poll_status()
    assert e.value.status == 6 and torch.equal(got, want)
    api.poll_status()


@pytest.mark.gpu
@pytest.mark.parametrize("adjacent", [False, True])
def test_gradients(adjacent):
    """Against the formula (the inverse rotation) and against differences of the forward."""
    rng = np.random.default_rng(9)
    q, k = draw(rng, (1, 4, 5, 32), "f32"), draw(rng, (1, 2, 5, 32), "f32")
    gq, gk = draw(rng, (1, 4, 5, 32), "f32"), draw(rng, (1, 2, 5, 32), "f32")
    positions = rng.integers(0, 50, (2, 1, 5))
    inv, axes = frequencies(24), np.array([0] * 5 + [1] * 7, dtype=np.int32)
    args = (torch.from_numpy(positions).cuda(), inv.cuda(), torch.from_numpy(axes).cuda(), adjacent)
    qd, kd = q.cuda().requires_grad_(), k.cuda().requires_grad_()
    qo, ko = autograd.rotary_embedding(qd, kd, *args)
    dq, dk = torch.autograd.grad((qo, ko), (qd, kd), (gq.cuda(), gk.cuda()), create_graph=True)
    check(dq.detach(), gq, positions, inv, axes, adjacent, True, "dq")
    check(dk.detach(), gk, positions, inv, axes, adjacent, True, "dk")
    # The map is linear: the difference quotient along any direction is exact.
    step = as_f64(draw(rng, (1, 4, 5, 32), "f32"))
    turned = ref.rotary(step, positions, inv.numpy(), axes, adjacent)
    assert abs((turned * as_f64(gq)).sum() - (step * as_f64(dq)).sum()) <= 1e-5 * np.abs(step * as_f64(gq)).sum()
    # One output alone, an expanded gradient, and the second derivative (in the gradients).
    only, = torch.autograd.grad(autograd.rotary_embedding(qd, kd, *args)[1].sum(), kd)
    check(only, torch.ones_like(k), positions, inv, axes, adjacent, True, "dk alone")
    back = torch.ones_like(gq.cuda()).requires_grad_()
    first, = torch.autograd.grad(autograd.rotary_embedding(qd, None, *args), qd, back, create_graph=True)
    again, = torch.autograd.grad(first, back, q.cuda())
    check(again, q, positions, inv, axes, adjacent, False, "second")
    api.poll_status()


@pytest.mark.gpu
def test_captured_forward_and_backward():
    rng = np.random.default_rng(10)
    q, k = draw(rng, (2, 4, 16, 64), "bf16").cuda(), draw(rng, (2, 2, 16, 64), "bf16").cuda()
    positions = torch.arange(16, dtype=torch.int32).cuda()
    inv = frequencies(64).cuda()
    api.rotary(q, k, positions, inv)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = api.rotary(q, k, positions, inv)
        back = api.rotary_backward(*out, positions, inv)
    positions += 1000
    graph.replay()
    want = api.rotary(q, k, positions, inv)
    api.poll_status()
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    # There and back: the first rounding reaches an element through both of its pair, at most
    # 2^-8·(|y_a| + |y_b|) <= 2^-8·2·max, the second adds 2^-8·max (fp32 terms are 2^-15 of it).
    assert float((back[0].float() - q.float()).abs().max()) <= 3.01 * 2**-8 * float(q.float().abs().max())


# The kernel's sines are no longer CUDA's, which the terms at the top of this file name, but
# series: 5·2^-24 = 3e-7 of themselves.  With four fp32 roundings of products and the sum, 2.4e-7,
# an output is off by 5.4e-7·(|a| + |b|) at most, which the 1e-6 there covers.


@pytest.mark.gpu
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("adjacent", [False, True])
def test_sines_and_cosines_keep_their_digits(adjacent, inverse):
    """Unit pairs (1, 0) and (0, 1) turn into a cosine and a sine without another rounding.  Both
    are within 6·2^-24 of themselves (x to the nearest quarter turn: rounded to fp32, times a
    constant that is rounded, rounded, 3·2^-24; series to 2e-9·x^2; two more roundings), small ones
    too, beside the angle's own |position|·(1 + inv_freq)·2^-64 turns."""
    from fractions import Fraction
    pi = Fraction("3.141592653589793238462643383279502884197169399375105820974944592307816406286208998628034825342117067982148086513282306647")
    rng = np.random.default_rng(13)
    n = 32
    inv = np.exp2(rng.uniform(-50, 1, n)).astype(np.float32)
    inv[0], inv[1], inv[2] = 2e-6, 1.0, np.float32(float(pi / 2))       # the last one is close to quarter turns
    positions = np.array([0, 1, -1, 2, 3, 355, -710, 103993, 1000003, 2**31 - 1, -2**20])
    x = torch.zeros(1, 2, len(positions), 2 * n)
    if adjacent:
        x[0, 0, :, 0::2], x[0, 1, :, 1::2] = 1, 1
    else:
        x[0, 0, :, :n], x[0, 1, :, n:] = 1, 1
    turn = api.rotary_backward if inverse else api.rotary
    out, _ = turn(x.cuda(), None, torch.from_numpy(positions).cuda(), torch.from_numpy(inv).cuda(), adjacent=adjacent)
    api.poll_status()
    got = as_f64(out)
    for i, pos in enumerate(positions.tolist()):
        for p in range(n):
            a, b = (2 * p, 2 * p + 1) if adjacent else (p, p + n)
            angle = Fraction(pos) * Fraction(float(inv[p])) * (-1 if inverse else 1)
            quarter = round(angle / (pi / 2))
            r = float(angle - quarter * (pi / 2))
            c, s = [(math.cos(r), math.sin(r)), (-math.sin(r), math.cos(r)), (-math.cos(r), -math.sin(r)), (math.sin(r), -math.cos(r))][quarter % 4]
            off = abs(pos) * (1 + float(inv[p])) * 2.0**-64 * 2 * math.pi
            for y, want in ((got[0, 0, i, a], c), (got[0, 0, i, b], s), (got[0, 1, i, a], -s), (got[0, 1, i, b], c)):
                assert abs(y - want) <= 6 * 2.0**-24 * abs(want) + off, (pos, float(inv[p]), y, want)
