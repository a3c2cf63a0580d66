"""GPU tests of the cache held in 4 bits: append and read against the fp32
definition (exact), attention against float64 over the cached values."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
import packed_ops_ref as R  # noqa: E402

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def P():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import post_weight_quantization_29_amd as P
    P.lib()
    return P


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def plan(q_lens, kv_lens, page, seed, spare=2, extra_pages=0):
    """Page table with the pool's pages in random order."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-max(k, 0) // page) for k in kv_lens]
    n_pages = sum(need) + spare
    order = torch.randperm(n_pages, generator=g).tolist()
    width = max(max(need), 1) + extra_pages
    table = [[order.pop() if j < n else -1 for j in range(width)] for n in need]
    start = [0]
    for n in q_lens:
        start.append(start[-1] + n)
    return n_pages, i32(table), i32(start), i32(kv_lens)


def random_cache(P, n_pages, n_kv, page, hd, table, seed, step=(0.05, 0.4)):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = P.KV4Cache.empty(n_pages, n_kv, page, hd, table)
    for codes, grid in ((c.k_codes, c.k_grid), (c.v_codes, c.v_grid)):
        codes.copy_(torch.randint(-2 ** 31, 2 ** 31, codes.shape, generator=g, device="cuda", dtype=torch.int64))
        s = step[0] + (step[1] - step[0]) * torch.rand(grid.shape[:-1], generator=g, device="cuda")
        grid[..., 0] = s
        grid[..., 1] = -s * (6 + 3 * torch.rand(s.shape, generator=g, device="cuda"))
    return c


# ---------------------------------------------------------------- append and read

@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("hd,n_kv,page,q_lens,kv_lens", [
    (128, 1, 16, [1], [1]),
    (64, 3, 16, [5, 0, 17], [5, 9, 40]),
    (128, 8, 64, [70, 1, 3], [200, 65, 3]),
    (64, 5, 48, [33], [97]),
    (128, 2, 32, [1] * 70, list(range(1, 71))),
])
def test_append_and_read(P, dtype, hd, n_kv, page, q_lens, kv_lens):
    n_pages, table, start, kvl = plan(q_lens, kv_lens, page, 1)
    c = random_cache(P, n_pages, n_kv, page, hd, table, 2)
    before = [t.clone() for t in (c.k_codes, c.v_codes, c.k_grid, c.v_grid)]
    T = sum(q_lens)
    g = torch.Generator(device="cuda").manual_seed(3)
    rows = torch.randn((T + 2, 2 * n_kv, hd), generator=g, device="cuda")
    rows[0, 0] = 0.0                                 # a row of zeros, a constant row, a wide one, a large offset
    rows[0, -1] = -3.7
    if T > 2:
        rows[1, 0] *= 1e4
        rows[2, -1] = rows[2, -1] * 1e-3 + 100
    rows = rows.to(dtype)
    K, V = rows[:, :n_kv], rows[:, n_kv:]            # two rows more than the batch has
    P.gptq_kv4_append(c, K, V, start, kvl)
    want = [t.clone() for t in before]
    back = [torch.full((T + 2, n_kv, hd), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
    P.gptq_kv4_read(c, back[0], back[1], start, kvl)
    sh = 4 * torch.arange(8, device="cuda")
    for x, codes, grid, r in ((K, want[0], want[2], back[0]), (V, want[1], want[3], back[1])):
        step, lo, q = R.grid_rows(x)
        w = (q.long().view(*q.shape[:-1], hd // 8, 8) << sh).sum(-1)
        w = torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)
        t = 0
        for b, n in enumerate(q_lens):
            for i in range(n):
                p = kv_lens[b] - n + i
                at = (int(table[b, p // page]), slice(None), p % page)
                codes[at], grid[at] = w[t], torch.cat([step, lo], -1)[t].half()
                t += 1
        assert torch.equal(r[:T], (lo + step * q)[:T].to(dtype))
        assert bool((r[T:] == 7).all())              # rows behind the last sequence
    for got, exp in zip((c.k_codes, c.v_codes, c.k_grid, c.v_grid), want):
        assert torch.equal(got, exp)                 # the new rows, and nothing else


def test_append_values_out_of_range(P):
    """NaNs, infinities and values beyond fp16."""
    n_pages, table, start, kvl = plan([4], [4], 16, 1)
    c = random_cache(P, n_pages, 1, 16, 64, table, 2)
    x = torch.randn((4, 1, 64), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    x[0, 0, 3] = float("nan")
    x[1, 0, 5], x[1, 0, 6] = float("inf"), -1e30
    x[2] = float("nan")
    x[3] = float("-inf")
    P.gptq_kv4_append(c, x, x, start, kvl)
    step, lo, q = R.grid_rows(x)
    got = torch.empty_like(x)
    P.gptq_kv4_read(c, None, got, start, kvl)
    assert torch.equal(got, lo + step * q) and torch.isfinite(got).all()
    assert bool((got[2] == 0).all()) and bool((got[3] == -65504).all())


def test_append_skips_what_has_no_place(P):
    """Positions below 0, pages that do not exist, positions past the table: nothing is written, zeros are read."""
    n_kv, hd, page = 2, 64, 16
    table = i32([[0, 99], [1, -5], [2, 3]])
    c = random_cache(P, 5, n_kv, page, hd, table, 2)
    before = c.k_codes.clone()
    # sequence 0 writes positions 14..17 (16, 17 on page 99), 1: -2, -1, 0, 2: 31..33 (32, 33 past the table)
    start, kvl = i32([0, 4, 7, 10]), i32([18, 1, 34])
    x = torch.randn((10, n_kv, hd), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(HF)
    P.gptq_kv4_append(c, x, x, start, kvl)
    changed = (c.k_codes != before).any(-1).nonzero().cpu().tolist()
    assert {(p, r) for p, _, r in changed} <= {(0, 14), (0, 15), (1, 0), (3, 15)}
    out = torch.full_like(x, 9.0)
    P.gptq_kv4_read(c, out, None, start, kvl)
    gone = [2, 3, 4, 5, 8, 9]
    assert bool((out[gone] == 0).all())
    step, lo, q = R.grid_rows(x)
    stay = [0, 1, 6, 7]
    assert torch.equal(out[stay], (lo + step * q)[stay].to(HF))


# ---------------------------------------------------------------- attention

def check(P, c, Q, start, kvl, max_q, max_kv, dtype, scale=None, out=None):
    T, H, hd = Q.shape
    out = torch.full((T, H, hd), 5.0, dtype=dtype, device="cuda") if out is None else out
    P.gptq_kv4_attention(Q, c, start, kvl, max_q, max_kv, out, scale=scale)
    cpu = [t.cpu() for t in (c.k_codes, c.k_grid, c.v_codes, c.v_grid, c.page_table)]
    ref, err, touched = R.attention64(Q.cpu().double(), *cpu, start.cpu(), kvl.cpu(),
                                      hd ** -0.5 if scale is None else scale, max_q, max_kv)
    got = out.cpu().double()
    assert bool((got[~touched] == 5).all())
    # the probabilities' rounding: half a step of each of the terms p (16 + code - 16) step
    eps = R.EPS[dtype]
    vx, vs, _ = R.cache_values(cpu[2], cpu[3])
    prob = eps * 15 * float(vs[torch.isfinite(vs)].abs().max()) if touched.any() else 0.0
    tol = err + prob + eps * ref.abs() + 1e-7
    bad = ((got - ref).abs() / tol)[touched]
    print(f"  worst |d| / tol {float(bad.max()) if bad.numel() else 0:.3f}", flush=True)
    assert bad.numel() == 0 or float(bad.max()) <= 1.0
    # and in the mean, where a wrong key or channel cannot hide behind the largest step
    d, n = (got - ref)[touched].norm(), ref[touched].norm()
    assert float(d) <= 2 * eps * float(n) + 1e-6
    return out


ATTENTION = [
    # q_lens, kv_lens, heads, kv heads, hd, page
    ([1], [1], 1, 1, 64, 16),
    ([1], [17], 2, 2, 128, 16),
    ([1], [129], 4, 4, 128, 16),
    ([1, 1, 1], [5, 700, 33], 8, 2, 128, 64),
    ([1, 0, 2, 1], [40, 90, 2, 513], 6, 2, 64, 48),
    ([3], [1500], 16, 2, 128, 32),
    ([2, 2], [4100, 31], 8, 1, 64, 256),
    ([1], [9000], 24, 1, 128, 128),
    ([20], [20], 4, 2, 128, 16),
    ([70, 1, 33], [170, 600, 33], 4, 1, 64, 32),
    ([130], [1100], 8, 8, 128, 64),
    ([257, 64], [300, 64], 6, 2, 128, 64),
]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("q_lens,kv_lens,H,n_kv,hd,page", ATTENTION)
def test_attention(P, dtype, q_lens, kv_lens, H, n_kv, hd, page):
    n_pages, table, start, kvl = plan(q_lens, kv_lens, page, 1)
    c = random_cache(P, n_pages, n_kv, page, hd, table, 2)
    T = sum(q_lens)
    g = torch.Generator(device="cuda").manual_seed(4)
    rows = torch.randn((T + 1, H + n_kv, hd), generator=g, device="cuda").to(dtype)
    Q = rows[:, :H]                                 # pitched, and a row behind the last sequence
    out = check(P, c, Q, start, kvl, max(q_lens), max(kv_lens), dtype)
    again = torch.full_like(out, 5.0)
    P.gptq_kv4_attention(Q, c, start, kvl, max(q_lens), max(kv_lens), again)
    assert torch.equal(out, again)
    # generous bounds change the split, not the result's accuracy
    check(P, c, Q, start, kvl, max(q_lens) + 40, max(kv_lens) + 5000, dtype)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("n_q", [1, 40])
def test_attention_rows_that_see_nothing(P, dtype, n_q):
    """Empty sequences, positions below 0, missing pages, a batch cut by its bounds; garbage in unused rows."""
    page, hd, n_kv, H = 16, 128, 1, 2
    table = i32([[0, 1, 2, 3], [4, -1, 5, 77], [-1, -1, -1, -1], [6, 6, 6, 6]])
    c = random_cache(P, 7, n_kv, page, hd, table, 3)
    start = i32([0, n_q, 2 * n_q, 3 * n_q, 4 * n_q])
    kvl = i32([n_q // 2, 64, 60, 50])               # 0: some positions below 0 (or an empty cache)
    for t in (c.k_grid, c.v_grid):
        t[0, :, n_q // 2:] = float("nan")           # behind sequence 0's end
        t[6, :, 15] = float("inf") if n_q == 1 else t[6, :, 15]
    if n_q == 1:
        kvl[3] = 15                                 # right before a row of infinities
    Q = torch.randn((4 * n_q, H, hd), device="cuda", generator=torch.Generator(device="cuda").manual_seed(5)).to(dtype)
    out = check(P, c, Q, start, kvl, n_q, 64, dtype)
    assert torch.isfinite(out).all()
    assert bool((out[2 * n_q:3 * n_q] == 0).all())
    assert bool((out[:n_q - n_q // 2] == 0).all())


@pytest.mark.parametrize("n_q", [1, 24])
def test_attention_bounds_cut_the_batch(P, n_q):
    """Tokens past max_q_len are left alone, positions past max_kv_len and rows past the tensors' end are not there."""
    n_pages, table, start, kvl = plan([n_q, n_q], [200, 90], 16, 1)
    c = random_cache(P, n_pages, 2, 16, 64, table, 2)
    Q = torch.randn((2 * n_q, 4, 64), device="cuda", generator=torch.Generator(device="cuda").manual_seed(5)).to(BF)
    check(P, c, Q, start, kvl, max(1, n_q - 5), 100, BF)
    check(P, c, Q[: 2 * n_q - 1], start, kvl, n_q, 200, BF)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("n_q", [1, 48])
def test_attention_peaked_scores_and_scales(P, dtype, n_q):
    """Scores of many hundreds (one key takes all), and values whose steps span orders of magnitude."""
    n_pages, table, start, kvl = plan([n_q], [400], 16, 1)
    c = random_cache(P, n_pages, 1, 16, 128, table, 2)
    s = torch.logspace(-4, 1, c.v_grid.shape[2], device="cuda").half()
    c.v_grid[..., 0] = s
    c.v_grid[..., 1] = -8 * s
    Q = torch.randn((n_q, 2, 128), device="cuda", generator=torch.Generator(device="cuda").manual_seed(5)).to(dtype)
    check(P, c, Q, start, kvl, n_q, 400, dtype, scale=30.0)
    check(P, c, Q, start, kvl, n_q, 400, dtype, scale=0.0)
    check(P, c, Q, start, kvl, n_q, 400, dtype, scale=-0.3)


def test_attention_over_more_than_2_gib_of_codes(P):
    """Rows whose byte offsets pass 32 bits."""
    page, hd, n_kv = 256, 128, 8
    n_pages = 20000                                  # 41 million rows, 2.6 GB of codes for keys
    table = i32([[n_pages - 1, 3, n_pages - 2]])
    c = P.KV4Cache.empty(n_pages, n_kv, page, hd, table)
    small = random_cache(P, 3, n_kv, page, hd, i32([[0, 1, 2]]), 9)
    for big, few in ((c.k_codes, small.k_codes), (c.v_codes, small.v_codes), (c.k_grid, small.k_grid), (c.v_grid, small.v_grid)):
        big[n_pages - 1], big[3], big[n_pages - 2] = few[0], few[1], few[2]
    start, kvl = i32([0, 1]), i32([700])
    Q = torch.randn((1, 8, hd), device="cuda", generator=torch.Generator(device="cuda").manual_seed(5)).to(BF)
    a, b = torch.empty_like(Q), torch.empty_like(Q)
    P.gptq_kv4_attention(Q, c, start, kvl, 1, 700, a)
    P.gptq_kv4_attention(Q, small, start, kvl, 1, 700, b)
    assert torch.equal(a, b)
    x = torch.randn((1, n_kv, hd), device="cuda").to(BF)
    r = [torch.empty_like(x) for _ in range(2)]
    P.gptq_kv4_append(c, x, x, start, kvl)
    P.gptq_kv4_append(small, x, x, start, kvl)
    P.gptq_kv4_read(c, r[0], None, start, kvl)
    P.gptq_kv4_read(small, r[1], None, start, kvl)
    assert torch.equal(r[0], r[1]) and torch.equal(c.k_codes[n_pages - 2], small.k_codes[2])
