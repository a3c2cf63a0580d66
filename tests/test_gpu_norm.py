"""GPU tests of the residual stream's norms against float64, forward and backward."""
from __future__ import annotations

import sys

import pytest

torch = pytest.importorskip("torch")
import block_ops_ref as R  # noqa: E402

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
TYPES = [(BF, BF), (HF, HF), (F32, F32), (F32, BF), (F32, HF)]
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def P():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import post_weight_quantization_29_amd as P
    P.lib()
    return P


def rows(m, d, dtype, seed, std=1.0, pitch=0, offset=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn((m, d + pitch), generator=g, device="cuda") * std).to(dtype)
    return x[:, offset:offset + d]


def vector(d, seed, mean=1.0):
    return mean + 0.3 * torch.randn(d, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def f64(t):
    return None if t is None else t.double()


def both_ways(P, m, d, ht, dt, branch, post, gate, alpha, pitch=0, offset=0, extra=True, seed=1):
    r, b = rows(m, d, ht, seed, 2.0, pitch, offset), rows(m, d, dt, seed + 1, 0.5, pitch, offset) if branch else None
    gamma = vector(d, 3)
    pw, gw = vector(d, 4, 0.4) if post else None, vector(d, 5, 0.0) if gate else None
    h = torch.full((m, d + pitch), 7.0, dtype=ht, device="cuda")[:, offset:offset + d] if branch else None
    whole = torch.full((m + 1, d + pitch), 7.0, dtype=dt, device="cuda")
    y = whole[:m, offset:offset + d]
    P.gptq_residual_rmsnorm(r, y, B=b, H=h, gamma=gamma, post_gamma=pw, gate=gw, alpha=alpha, eps=EPS)
    ref = R.norm64(f64(r), f64(b), f64(gamma), f64(pw), f64(gw), alpha, EPS)
    R.within(y, *ref["y"], "y")
    if branch:
        R.within(h, *ref["h"], "h")
    # what lies between and behind the rows stays
    assert bool((whole[m] == 7).all()) and bool((whole[:m, :offset] == 7).all()) and bool((whole[:m, offset + d:] == 7).all())
    dy, dh = rows(m, d, dt, seed + 2, 0.1, pitch, offset), rows(m, d, ht, seed + 3, 0.1, pitch, offset) if extra else None
    stored = h if branch else r
    dr, db = torch.empty((m, d), dtype=ht, device="cuda"), torch.empty((m, d), dtype=dt, device="cuda") if branch else None
    new = lambda on: torch.full((d,), 7.0, device="cuda") if on else None  # noqa: E731
    dg, dp, dw = new(True), new(post), new(gate)
    P.gptq_residual_rmsnorm_backward(dy, stored, dr, dH=dh, B=b, dB=db, gamma=gamma, post_gamma=pw, gate=gw, alpha=alpha, eps=EPS,
                                     dgamma=dg, dpost_gamma=dp, dgate=dw)
    ref = R.norm_backward64(f64(dy), f64(stored), f64(dh), f64(b), f64(gamma), f64(pw), f64(gw), alpha, EPS)
    for name, got in (("dr", dr), ("db", db), ("dgamma", dg), ("dpost", dp), ("dgate", dw)):
        if got is not None:
            R.within(got, *ref[name], name)


@pytest.mark.parametrize("ht,dt", TYPES)
@pytest.mark.parametrize("m,d", [(1, 8), (3, 1), (2, 63), (5, 64), (33, 511), (70, 520), (300, 1024), (17, 4096), (2, 5120), (9, 8200)])
def test_sizes_and_types(P, ht, dt, m, d):
    both_ways(P, m, d, ht, dt, True, True, True, 0.7)
    both_ways(P, m, d, ht, dt, True, False, False, 1.0, extra=False)


@pytest.mark.parametrize("d", [8192, 8193, 12000, 16383, 16384])
def test_wide_rows(P, d):
    both_ways(P, 3, d, BF, BF, True, True, True, 0.5)
    both_ways(P, 3, d, F32, HF, True, False, False, 1.0)


@pytest.mark.parametrize("branch,post,gate", [(False, False, False), (True, True, False), (True, False, True)])
def test_parts(P, branch, post, gate):
    both_ways(P, 40, 384, BF, BF, branch, post, gate, -1.5 if branch else 1.0)


@pytest.mark.parametrize("pitch,offset", [(8, 0), (16, 8), (5, 0), (8, 3)])
def test_pitched_and_unaligned_rows(P, pitch, offset):
    both_ways(P, 21, 256, BF, BF, True, True, True, 0.5, pitch, offset)
    both_ways(P, 21, 256, F32, HF, True, True, True, 0.5, pitch, offset)


def test_many_rows(P):
    both_ways(P, 5000, 96, BF, BF, True, True, True, 0.5)


def test_in_place_and_optional_outputs(P):
    m, d = 37, 640
    r, b, gamma, post = rows(m, d, BF, 1), rows(m, d, BF, 2), vector(d, 3), vector(d, 4)
    h, y = torch.empty_like(r), torch.empty_like(r)
    P.gptq_residual_rmsnorm(r, y, B=b, H=h, gamma=gamma, post_gamma=post)
    r2, b2 = r.clone(), b.clone()
    P.gptq_residual_rmsnorm(r2, b2, B=b2, H=r2, gamma=gamma, post_gamma=post)
    assert torch.equal(r2, h) and torch.equal(b2, y)
    only_h, only_y = torch.empty_like(r), torch.empty_like(r)
    P.gptq_residual_rmsnorm(r, None, B=b, H=only_h, post_gamma=post)
    P.gptq_residual_rmsnorm(r, only_y, B=b, gamma=gamma, post_gamma=post)
    assert torch.equal(only_h, h) and torch.equal(only_y, y)
    dy, dh = rows(m, d, BF, 5), rows(m, d, BF, 6)
    dr, db, dg, dp = torch.empty_like(r), torch.empty_like(r), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    P.gptq_residual_rmsnorm_backward(dy, h, dr, dH=dh, B=b, dB=db, gamma=gamma, post_gamma=post, dgamma=dg, dpost_gamma=dp)
    dr2, db2, one, two = dh.clone(), dy.clone(), torch.empty_like(dg), torch.empty_like(dp)
    P.gptq_residual_rmsnorm_backward(db2, h, dr2, dH=dr2, B=b, dB=db2, gamma=gamma, post_gamma=post)
    assert torch.equal(dr2, dr) and torch.equal(db2, db)
    P.gptq_residual_rmsnorm_backward(dy, h, None, dH=dh, B=b, gamma=gamma, post_gamma=post, dgamma=one, dpost_gamma=two)
    assert torch.equal(one, dg) and torch.equal(two, dp)


def test_no_rows(P):
    e, v = torch.empty((0, 64), dtype=BF, device="cuda"), vector(64, 1)
    P.gptq_residual_rmsnorm(e, e.clone(), gamma=v)
    s = [torch.full((64,), 7.0, device="cuda") for _ in range(3)]
    P.gptq_residual_rmsnorm_backward(e, e, e.clone(), B=e, dB=e.clone(), gamma=v, post_gamma=v, gate=v, dgamma=s[0], dpost_gamma=s[1],
                                     dgate=s[2])
    assert all(bool((t == 0).all()) for t in s)


def test_rows_keep_to_themselves(P):
    """A row that is no number, and one of zeros, leave the others as they are."""
    m, d = 9, 512
    r, b, gamma = rows(m, d, BF, 1), rows(m, d, BF, 2), vector(d, 3)
    y, h = torch.empty_like(r), torch.empty_like(r)
    P.gptq_residual_rmsnorm(r, y, B=b, H=h, gamma=gamma, post_gamma=gamma)
    r2, b2 = r.clone(), b.clone()
    r2[2, 5], b2[4, 7], r2[6], b2[6] = float("nan"), float("inf"), 0, 0
    y2, h2 = torch.empty_like(r), torch.empty_like(r)
    P.gptq_residual_rmsnorm(r2, y2, B=b2, H=h2, gamma=gamma, post_gamma=gamma)
    same = [i for i in range(m) if i not in (2, 4, 6)]
    assert torch.equal(y2[same], y[same]) and torch.equal(h2[same], h[same])
    assert bool(y2[2].isnan().all()) and bool(y2[4].isnan().any()) and bool((y2[6] == 0).all()) and bool((h2[6] == 0).all())


def test_gradient_against_differences(P):
    """The kernel's gradients along a direction, and the difference of float64 values there."""
    m, d, alpha = 6, 40, 0.6
    r, b = rows(m, d, F32, 1), rows(m, d, F32, 2)
    ws = [vector(d, k, mean) for k, mean in ((3, 1.0), (4, 0.5), (5, 0.0))]
    dy, dh = rows(m, d, F32, 6), rows(m, d, F32, 7)

    def loss(r, b, gamma, post, gate):
        ref = R.norm64(r, b, gamma, post, gate, alpha, EPS)
        return (ref["y"][0] * dy.double()).sum() + (ref["h"][0] * dh.double()).sum()

    h, y = torch.empty_like(r), torch.empty_like(r)
    P.gptq_residual_rmsnorm(r, y, B=b, H=h, gamma=ws[0], post_gamma=ws[1], gate=ws[2], alpha=alpha, eps=EPS)
    grads = [torch.empty_like(r), torch.empty_like(b)] + [torch.empty_like(w) for w in ws]
    P.gptq_residual_rmsnorm_backward(dy, h, grads[0], dH=dh, B=b, dB=grads[1], gamma=ws[0], post_gamma=ws[1], gate=ws[2], alpha=alpha,
                                     eps=EPS, dgamma=grads[2], dpost_gamma=grads[3], dgate=grads[4])
    at = [t.double() for t in (r, b, *ws)]
    for k, g in enumerate(grads):
        v = torch.randn(g.shape, generator=torch.Generator(device="cuda").manual_seed(20 + k), device="cuda").double()
        step = 1e-5
        up, down = [t.clone() for t in at], [t.clone() for t in at]
        up[k] += step * v
        down[k] -= step * v
        diff = (loss(*up) - loss(*down)) / (2 * step)
        # central differences are off by step^2 times a third derivative of order 1 to 100 here, and by 2^-53 |loss| / step
        assert abs(float((g.double() * v).sum() - diff)) <= 1e-6 * float((g.double() * v).abs().sum()) + 1e-6


@pytest.mark.parametrize("ht,dt", [(BF, BF), (F32, HF)])
@pytest.mark.parametrize("m,d", [(1, 8), (1, 4096), (3, 64), (3, 640), (5, 8), (33, 513), (4095, 520), (3, 9000)])
def test_without_eps(P, monkeypatch, ht, dt, m, d):
    """eps 0: the rows that a workgroup's last step does not have add nothing to the sums over rows."""
    monkeypatch.setattr(sys.modules[__name__], "EPS", 0.0)
    both_ways(P, m, d, ht, dt, True, True, True, 0.7)
    both_ways(P, m, d, ht, dt, True, False, True, 0.7)
    both_ways(P, m, d, ht, dt, False, False, False, 1.0)


@pytest.mark.parametrize("m,d", [(4101, 520), (4101, 1000), (4099, 5120), (4097, 8200), (1025, 16384), (6201, 2048)])
@pytest.mark.parametrize("ht,dt,post,gate", [(F32, BF, True, True), (BF, BF, True, False), (HF, HF, False, True), (F32, F32, False, False)])
def test_many_wide_rows(P, ht, dt, post, gate, m, d):
    """Workgroups that walk several rows, of one chunk a thread and of two, the last step with rows that do not exist."""
    both_ways(P, m, d, ht, dt, True, post, gate, 0.6)


@pytest.mark.parametrize("m,d", [(1101, 4096), (2051, 640), (601, 8200), (515, 16384)])
@pytest.mark.parametrize("ht,dt", [(BF, BF), (F32, F32)])
def test_many_rows_in_place(P, ht, dt, m, d):
    """As above, over the inputs: the next row is on its way while one is written."""
    r, b, gamma, post, gate = rows(m, d, ht, 1), rows(m, d, dt, 2), vector(d, 3), vector(d, 4), vector(d, 5)
    h, y = torch.empty_like(r), torch.empty_like(b)
    P.gptq_residual_rmsnorm(r, y, B=b, H=h, gamma=gamma, post_gamma=post, gate=gate, alpha=0.5, eps=EPS)
    r2, b2 = r.clone(), b.clone()
    P.gptq_residual_rmsnorm(r2, b2, B=b2, H=r2, gamma=gamma, post_gamma=post, gate=gate, alpha=0.5, eps=EPS)
    assert torch.equal(r2, h) and torch.equal(b2, y)
    dy, dh = rows(m, d, dt, 6), rows(m, d, ht, 7)
    outs = [torch.empty_like(r), torch.empty_like(b)] + [torch.empty(d, device="cuda") for _ in range(3)]
    P.gptq_residual_rmsnorm_backward(dy, h, outs[0], dH=dh, B=b, dB=outs[1], gamma=gamma, post_gamma=post, gate=gate, alpha=0.5, eps=EPS,
                                     dgamma=outs[2], dpost_gamma=outs[3], dgate=outs[4])
    ref = R.norm_backward64(f64(dy), f64(h), f64(dh), f64(b), f64(gamma), f64(post), f64(gate), 0.5, EPS)
    for name, got in zip(("dr", "db", "dgamma", "dpost", "dgate"), outs):
        R.within(got, *ref[name], name)
    dr2, db2, sums = dh.clone(), dy.clone(), [torch.empty(d, device="cuda") for _ in range(3)]
    P.gptq_residual_rmsnorm_backward(db2, h, dr2, dH=dr2, B=b, dB=db2, gamma=gamma, post_gamma=post, gate=gate, alpha=0.5, eps=EPS,
                                     dgamma=sums[0], dpost_gamma=sums[1], dgate=sums[2])
    for a, x in zip([dr2, db2, *sums], outs):
        assert torch.equal(a, x)
