"""Tensors of more than 2^31 values: rows on both sides of the border, and the last ones,
against the 64-bit forms; sums over all rows against 64-bit sums."""
from types import SimpleNamespace

import pytest
import torch

from tests import _block_reference as R
from tests._ffn_reference import HALF
from tests._harness import built_library
from tests.test_gpu_adamw import BETAS, DECAY, EPS, LR, _check_step

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
T, D = (1 << 18) + 1029, 8192
ROWS = torch.cat([torch.arange(4), torch.arange((1 << 18) - 3, (1 << 18) + 3), torch.arange(T - 5, T)])


@pytest.fixture(scope="module")
def ops():
    built_library()
    import latent_mixture_experts_gb300 as P
    yield P
    torch.cuda.empty_cache()


def _rnd(g, *s, dt=BF):
    return torch.randn(*s, device="cuda", generator=g, dtype=dt)


def test_gated_norm(ops):
    g = torch.Generator(device="cuda").manual_seed(1)
    y, s, w1, w2, gate = _rnd(g, T, D), _rnd(g, T, D), 1 + 0.3 * _rnd(g, D), 1 - 0.3 * _rnd(g, D), _rnd(g, T, D)
    i = ROWS.cuda()
    o, _, h = ops.lmoe_gated_add_norm(y, s, w1, w2, 1e-6, gate=gate)
    want, size = R.gated(y[i], s[i], w1, w2, 1e-6, gate[i])
    assert bool(((h[i].to(R.D) - want).abs() <= HALF[BF] * want.abs() * (1 + R.F32) + R.F32 * size + R.TINY).all())
    ref = R.norm_of(h[i], w2, 1e-6)
    assert bool(((o[i].to(R.D) - ref).abs() <= (HALF[BF] + R.F32) * ref.abs() + R.TINY).all())
    got = ops.lmoe_gated_add_norm_backward(o, y, h, w1, w2, 1e-6, gate=gate, dh=s)
    want, size = R.gated_backward(o[i], y[i], h[i], w1, w2, 1e-6, gate[i], gh=s[i])
    for k in (0, 1, 4):
        tol = HALF[BF] * want[k].abs() * (1 + R.F32) + 2 * R.F32 * size[k] + R.TINY
        assert bool(((got[k][i].to(R.D) - want[k]).abs() <= tol).all()), k
    dw, terms = torch.zeros(D, device="cuda", dtype=R.D), torch.zeros(D, device="cuda", dtype=R.D)
    for at in range(0, T, 1 << 14):
        hd, od = h[at:at + (1 << 14)].to(R.D), o[at:at + (1 << 14)].to(R.D)
        v = od * hd / torch.sqrt((hd * hd).mean(-1, keepdim=True) + 1e-6)
        dw += v.sum(0)
        terms += v.abs().sum(0)
    # a CTA adds 1732 rows one after the other, and 152 sums meet: 2^-24 of the running sum each, 2^-13 at most
    assert bool(((got.next_w.to(R.D) - dw).abs() <= 2.0 ** -13 * terms).all())


def test_linear(ops):
    g = torch.Generator(device="cuda").manual_seed(2)
    x, r = _rnd(g, T, 64), _rnd(g, T, D, dt=F32)
    w, b = (_rnd(g, D, 64, dt=F32) / 8).to(BF), _rnd(g, D)
    layer = ops.Linear(w, b, "gelu", max_tokens=T, training=True)
    y, z = layer.lmoe_linear_forward(x, residual=r, save=True)
    i = ROWS.cuda()
    yr, ye, zr, ze = R.linear(x[i], w, b, "gelu", r[i])
    assert bool(((y[i].to(R.D) - yr).abs() <= ye).all()) and bool(((z[i].to(R.D) - zr).abs() <= ze).all())
    dx, dw, db = layer.lmoe_linear_backward(x, r, z)
    want, err = R.linear_backward(x[i], w, r[i], z[i], "gelu")
    assert bool(((dx[i].to(R.D) - want[0]).abs() <= err[0]).all())
    s, e = torch.zeros(D, device="cuda", dtype=R.D), torch.zeros(D, device="cuda", dtype=R.D)
    for at in range(0, T, 1 << 14):
        dy = r[at:at + (1 << 14)].to(R.D)
        dz = dy * R.slope(z[at:at + (1 << 14)].to(R.D), "gelu")
        s += dz.sum(0)
        e += 2.0 ** -16 * (dz.abs().sum(0) + dy.abs().sum(0))
    assert bool(((db.to(R.D) - s).abs() <= e).all())
    layer.lmoe_linear_sync_status()


@pytest.mark.parametrize("states", ["fp32", "mxfp8"])
def test_adamw(ops, states):
    """The first and the last values of a tensor of 2^31 and more, and a small tensor behind it."""
    n, k = (1 << 31) + 4097, 1 << 14
    g = torch.Generator(device="cuda").manual_seed(3)
    p, q = _rnd(g, n), _rnd(g, 1000)
    gp, gq = _rnd(g, n), _rnd(g, 1000)
    opt = ops.AdamW([p, q], lr=LR, betas=BETAS, eps=EPS, weight_decay=DECAY, states=states, masters=False, seed=7)
    parts = [(0, slice(0, k)), (0, slice(n - 4097 - k, n - 4097 - k + 2 * k)), (0, slice((n - 2000) // 32 * 32, n)),
             (1, slice(0, 1000))]
    zero = [torch.zeros(s.stop - s.start if s.stop <= (n if j == 0 else 1000) else n - s.start, device="cuda",
                        dtype=R.D) for j, s in parts]
    before = [((p if j == 0 else q)[s].to(R.D), z, z) for (j, s), z in zip(parts, zero)]
    opt.step([gp, gq])

    def state(i):
        j, s = parts[i]
        full, blocks = opt.state(j), slice(s.start // 32, (s.stop + 31) // 32)
        return {name: v[blocks] if name.endswith("scales") else v[s] for name, v in full.items()}
    seen = SimpleNamespace(params=[(p if j == 0 else q)[s] for j, s in parts], states=states, seed=7,
                           offsets=[opt.offsets[j] + s.start for j, s in parts], state=state)
    _check_step(seen, before, [(gp if j == 0 else gq)[s] for j, s in parts], [DECAY] * len(parts), 1)
