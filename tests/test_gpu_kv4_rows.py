"""GPU tests of the attention over the 4-bit cache, each row and head against a
bound of its own: what a row does not see, or sees with no weight to speak of,
costs it nothing.

The probabilities (or what stands for them) are rounded once to 16 bits, by half
a step d_j each, in the sum over the values and in the one that normalizes it, so
the output moves by |sum_j p_j d_j (v_j - out)| <= eps sum_j p_j |v_j - out|, and
its own rounding is eps |out|; what fp32 adds is in attention64's bound."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
import packed_ops_ref as R  # noqa: E402
from test_gpu_kv4 import BF, HF, i32, plan, random_cache  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def P():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import post_weight_quantization_29_amd as P
    P.lib()
    return P


def spread(q, c, b, t0, first, n_q, scale):
    """sum_j p_j |v_j - out| of sequence b's rows [n_q, heads, hd] in float64 on the GPU, over the pages that exist."""
    n_kv, page, hd = c.n_kv_heads, c.page_size, c.head_dim
    rep = q.shape[1] // n_kv
    pos = torch.arange(first + n_q, device="cuda")
    pg = c.page_table[b, pos // page].long()
    keep = (pg >= 0) & (pg < len(c.k_codes))
    pos, pg = pos[keep], pg[keep]
    out = torch.zeros((n_q, q.shape[1], hd), dtype=torch.float64, device="cuda")
    for h in range(q.shape[1]):
        k, v = (R.cache_values(x[pg, h // rep, pos % page], g[pg, h // rep, pos % page])[0]
                for x, g in ((c.k_codes, c.k_grid), (c.v_codes, c.v_grid)))
        for i in range(n_q):
            n = int((pos <= first + i).sum())
            if n:
                p = torch.softmax(k[:n] @ q[t0 + i, h] * scale, 0)
                out[i, h] = p @ (v[:n] - p @ v[:n]).abs()
    return out


def check_rows(P, c, Q, q_lens, kv_lens, dtype, scale=None):
    T, H, hd = Q.shape
    scale = hd ** -0.5 if scale is None else scale
    start = [0]
    for n in q_lens:
        start.append(start[-1] + n)
    out = torch.full_like(Q, 5.0)
    P.gptq_kv4_attention(Q, c, i32(start), i32(kv_lens), max(q_lens), max(kv_lens), out, scale=scale)
    q = Q.double()
    ref, err, _ = R.attention64(q.cpu(), *(t.cpu() for t in (c.k_codes, c.k_grid, c.v_codes, c.v_grid, c.page_table)),
                                torch.tensor(start), torch.tensor(kv_lens), scale)
    eps, tiny = R.EPS[dtype], 2.0 ** -25 if dtype == HF else 1e-38
    far = torch.cat([spread(q, c, b, start[b], kv_lens[b] - n, n, scale) for b, n in enumerate(q_lens)]).cpu()
    d = (out.cpu().double() - ref).abs()
    tol = err + eps * (1 + 4 * eps) * (ref.abs() + far) + tiny
    row = d.norm(dim=-1) / (err.norm(dim=-1) + eps * (1 + 4 * eps) * (ref.norm(dim=-1) + far.norm(dim=-1)) + tiny * hd ** 0.5)
    print(f"  worst |d| / tol {float((d / tol).max()):.3f}, norm of a row and head {float(row.max()):.3f}", flush=True)
    assert float((d / tol).max()) <= 1.0 and float(row.max()) <= 1.0
    return out


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("n_q", [2, 60, 250])
@pytest.mark.parametrize("small,wide", [((0.0005, 0.004), 4000.0), ((0.005, 0.04), 4000.0), ((0.0005, 0.004), 100.0)])
def test_wide_values_of_a_later_token(P, dtype, hd, n_q, small, wide):
    """One token's values span a million times what the others' do: the tokens before it keep their accuracy."""
    kv = n_q + 30
    n_pages, table, _, _ = plan([n_q], [kv], 16, 1)
    c = random_cache(P, n_pages, 1, 16, hd, table, 2)
    g = torch.Generator(device="cuda").manual_seed(3)
    s = small[0] + (small[1] - small[0]) * torch.rand(c.v_grid.shape[:-1], generator=g, device="cuda")
    c.v_grid[..., 0], c.v_grid[..., 1] = s, -s * 7.5
    at = 30 + n_q // 2
    c.v_grid[int(table[0, at // 16]), 0, at % 16] = torch.tensor([wide, -8 * wide])
    Q = torch.randn((n_q, 2, hd), device="cuda", generator=g).to(dtype)
    check_rows(P, c, Q, [n_q], [kv], dtype)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("n_q", [2, 60, 250])
def test_wide_values_of_no_weight(P, dtype, n_q):
    """The same in a token that all rows see with a probability of e^-100 and less."""
    kv = n_q + 30
    n_pages, table, _, _ = plan([n_q], [kv], 16, 1)
    c = random_cache(P, n_pages, 1, 16, 128, table, 2, step=(0.0005, 0.004))
    for grid, row in ((c.v_grid, [4000.0, -32000.0]), (c.k_grid, [0.0, -30.0])):
        grid[int(table[0, 0]), 0, 5] = torch.tensor(row)
    Q = torch.randn((n_q, 2, 128), device="cuda", generator=torch.Generator(device="cuda").manual_seed(3)).abs().to(dtype)
    check_rows(P, c, Q, [n_q], [kv], dtype)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("n_q", [1, 48, 200])
@pytest.mark.parametrize("scale", [30.0, 0.0, -0.3, None])
def test_steps_over_five_orders_of_magnitude(P, dtype, n_q, scale):
    """Peaked and flat scores, values whose steps go from 1e-4 to 10 along every page and to 0 in one key."""
    n_pages, table, _, _ = plan([n_q], [400], 16, 1)
    c = random_cache(P, n_pages, 1, 16, 128, table, 2)
    s = torch.logspace(-4, 1, 16, device="cuda").half()
    c.v_grid[..., 0], c.v_grid[..., 1] = s, -8 * s
    c.v_grid[int(table[0, 3]), 0, 7] = torch.tensor([0.0, 0.25])
    Q = torch.randn((n_q, 2, 128), device="cuda", generator=torch.Generator(device="cuda").manual_seed(5)).to(dtype)
    check_rows(P, c, Q, [n_q], [400], dtype, scale)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("n_q", [1, 40, 130])
def test_garbage_behind_the_end(P, dtype, n_q):
    """Every row of the sequences' pages from kv_len on is NaN or infinite, the rows that no token has yet among
    them; a sequence ends inside a page, at a page's end, and a page is missing."""
    page, hd = 16, 64
    kv = [n_q + 5, n_q + 16 - n_q % 16, n_q + 37]
    n_pages, table, _, _ = plan([n_q] * 3, kv, page, 1, extra_pages=2)
    table[2, 1] = -1
    table[:, -2:] = torch.arange(2, device="cuda", dtype=torch.int32)       # pages of other sequences, past the end
    c = random_cache(P, n_pages, 2, page, hd, table, 3)
    before = [t.clone() for t in (c.k_grid, c.v_grid)]
    Q = torch.randn((3 * n_q, 4, hd), device="cuda", generator=torch.Generator(device="cuda").manual_seed(5)).to(dtype)
    want = check_rows(P, c, Q, [n_q] * 3, kv, dtype)
    free = torch.ones(c.k_grid.shape[0], page, dtype=torch.bool, device="cuda")
    for b, n in enumerate(kv):
        for p in range(n):
            if int(table[b, p // page]) >= 0:
                free[int(table[b, p // page]), p % page] = False
    assert int(free.sum()) > 16
    for bad in (float("nan"), float("inf"), float("-inf")):
        for t, old in zip((c.k_grid, c.v_grid), before):
            t.copy_(torch.where(free[:, None, :, None], torch.tensor(bad, dtype=HF, device="cuda"), old))
        got = torch.full_like(want, 5.0)
        start = i32([0, n_q, 2 * n_q, 3 * n_q])
        P.gptq_kv4_attention(Q, c, start, i32(kv), n_q, max(kv), got)
        assert torch.isfinite(got).all() and torch.equal(got, want)
