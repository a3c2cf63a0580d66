"""GPU tests of the packed layer's operators and the 4-bit cache as a program
uses them: a decoder layer served step by step, captured graphs, other streams,
one workspace for all calls, and the sizes at which a call changes its way."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
import packed_ops_ref as R  # noqa: E402
from test_gpu_kv4 import check as check_attention, i32, plan, random_cache  # noqa: E402
from test_gpu_packed_ops import (BF, F32, HF, acts, backward_ref, close, gated_ref, linear_ref,  # noqa: E402
                                 weight)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def P():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import post_weight_quantization_29_amd as P
    P.lib()
    return P


def poisoned(nbytes):
    """A workspace of exactly that size, full of NaN patterns, and a view of the bytes behind it."""
    buf = torch.full((nbytes + 512,), 0xFF, dtype=torch.uint8, device="cuda")
    assert buf.data_ptr() % 256 == 0
    return buf[:nbytes], buf[nbytes:]


# ---------------------------------------------------------------- sizes at which a call changes its way

# m, d_out, d_in, G, dtype, y, perm
WAYS = [
    (16, 4608, 8192, 128, BF, BF, False),       # few tokens and much work: activations shared by eight waves
    (16, 4616, 8192, 64, HF, F32, True),
    (65, 140, 2080, 32, BF, BF, False),         # a second block of one token
    (100, 260, 4096, 128, HF, HF, False),
    (128, 77, 1056, 96, BF, F32, True),
    (127, 64, 264, 24, HF, BF, False),          # groups that the direct way does not take
    (129, 130, 4096, 128, BF, BF, False),       # few tiles: every one split over k
    (200, 5, 2368, -1, HF, F32, False),
    (577, 1000, 1088, 64, BF, HF, True),
    (1500, 3000, 1600, 64, BF, BF, False),      # full rounds and a split rest
]


@pytest.mark.parametrize("m,d_out,d_in,G,xt,yt,perm", WAYS)
def test_linear_ways(P, m, d_out, d_in, G, xt, yt, perm):
    L = R.layer(d_out, d_in, G, m + d_in, "cuda", perm=perm)
    X, bias, Rs = acts(m, d_in, xt, 1), acts(1, d_out, xt, 2)[0], acts(m, d_out, yt, 3)
    w = weight(P, L)
    ws, behind = poisoned(P.gptq_w4_linear_workspace_size(m, w))
    Y = torch.full((m + 2, d_out), 7.0, dtype=yt, device="cuda")
    P.gptq_w4_linear(X, w, Y[:m], bias=bias, act="silu", R=Rs, ws=ws)
    ref, err = linear_ref(X, L, bias, "silu", Rs)
    close(Y[:m], ref, err, yt)
    assert bool((Y[m:] == 7).all()) and bool((behind == 0xFF).all())
    again = torch.empty_like(Rs)
    P.gptq_w4_linear(X, w, again, bias=bias, act="silu", R=Rs, ws=ws)     # over what the first call left there
    assert torch.equal(again, Y[:m])


@pytest.mark.parametrize("m,d_in,G,shift", [(3, 32776, 8, 0), (3, 32768, 32, 1), (70, 264, 8, 1), (600, 136, 8, 3), (5000, 64, 32, 0)])
def test_linear_act_order(P, m, d_in, G, shift):
    """Rows that fit LDS and longer ones, aligned or not, brought into processing order."""
    L = R.layer(24, d_in, G, 7, "cuda", perm=True)
    X = acts(m, d_in + 8, BF, 1)[:, shift:shift + d_in]
    Y = torch.full((m, 24), float("nan"), dtype=F32, device="cuda")
    w = weight(P, L)
    ws, behind = poisoned(P.gptq_w4_linear_workspace_size(m, w))
    P.gptq_w4_linear(X, w, Y, ws=ws)
    ref, err = linear_ref(X, L, None, "none", None)
    close(Y, ref, err, F32)
    assert bool((behind == 0xFF).all())


@pytest.mark.parametrize("m,d,f,G,dtype", [
    (16, 8192, 13760, 128, BF), (70, 512, 100, 64, HF), (128, 1056, 70, 32, BF), (300, 1024, 200, 128, HF),
    (1100, 640, 1500, 64, BF)])
def test_gated_ways(P, m, d, f, G, dtype):
    Lg, Lu = R.layer(f, d, G, m, "cuda"), R.layer(f, d, G, m + 1, "cuda")
    X = acts(m, d, dtype, 1)
    g, u = weight(P, Lg), weight(P, Lu)
    ws, behind = poisoned(P.gptq_w4_gated_workspace_size(m, g, u))
    out = [torch.full((m + 2, f), 7.0, dtype=dtype, device="cuda") for _ in range(3)]
    P.gptq_w4_gated(X, g, u, out[0][:m], G=out[1][:m], U=out[2][:m], ws=ws)
    for t, (ref, err) in zip(out, gated_ref(X, Lg, Lu, "silu")):
        close(t[:m], ref, err, dtype)
        assert bool((t[m:] == 7).all())
    assert bool((behind == 0xFF).all())


@pytest.mark.parametrize("m,d,f,dtype,outs", [(300, 264, 1000, HF, True), (257, 128, 2048, BF, False), (40, 520, 1344, BF, True)])
def test_backward_ways(P, m, d, f, dtype, outs):
    Lg, Lu = R.layer(f, d, 8, m, "cuda", perm=True), R.layer(f, d, 8, m + 1, "cuda")
    Lu["perm"] = Lg["perm"]
    g, u = weight(P, Lg), weight(P, Lu)
    dM, Gt, Ut = acts(m, f, dtype, 1), acts(m, f, dtype, 2, 2.0), acts(m, f, dtype, 3)
    dX = torch.full((m + 2, d), 7.0, dtype=dtype, device="cuda")
    dG, dU = (torch.empty_like(dM) if outs else None for _ in range(2))
    ws, behind = poisoned(P.gptq_w4_gated_backward_workspace_size(m, g, u))
    P.gptq_w4_gated_backward(dM, Gt, Ut, g, u, dX[:m], dG=dG, dU=dU, ws=ws)
    for t, (ref, err) in zip((dX[:m], dG, dU), backward_ref(dM, Gt, Ut, Lg, Lu, "silu", dtype)):
        if t is not None:
            close(t, ref, err, dtype)
    assert bool((dX[m:] == 7).all()) and bool((behind == 0xFF).all())


@pytest.mark.parametrize("rows", [48, 49])
def test_attention_ways(P, rows):
    """Around the number of rows from which tiles are unpacked, with a workspace of exactly the size."""
    n_pages, table, start, kvl = plan([rows, 3], [1400, 900], 32, 1)
    c = random_cache(P, n_pages, 2, 32, 128, table, 2)
    Q = acts((rows + 3) * 2, 128, BF, 5).view(rows + 3, 2, 128)
    ws, behind = poisoned(P.gptq_kv4_attention_workspace_size(rows + 3, 2, c, rows, 1400))
    a, b = torch.empty_like(Q), torch.empty_like(Q)
    P.gptq_kv4_attention(Q, c, start, kvl, rows, 1400, a, ws=ws)
    assert bool((behind == 0xFF).all())
    P.gptq_kv4_attention(Q, c, start, kvl, rows, 1400, b, ws=ws)
    assert torch.equal(a, b)
    check_attention(P, c, Q, start, kvl, rows, 1400, BF)


def test_no_tokens(P):
    L = R.layer(16, 64, 32, 1, "cuda")
    w, none = weight(P, L), torch.empty((0, 64), dtype=BF, device="cuda")
    small = torch.empty((0, 16), dtype=BF, device="cuda")
    P.gptq_w4_linear(none, w, small)
    P.gptq_w4_gated(none, w, w, small)
    P.gptq_w4_gated_backward(small, small, small, w, w, none)
    c = random_cache(P, 2, 1, 16, 64, i32([[0], [1]]), 2)
    before = c.k_codes.clone()
    rows = torch.empty((0, 1, 64), dtype=BF, device="cuda")
    start, kvl = i32([0, 0, 0]), i32([5, 0])
    P.gptq_kv4_append(c, rows, rows, start, kvl)
    P.gptq_kv4_read(c, rows, None, start, kvl)
    P.gptq_kv4_attention(rows, c, start, kvl, 1, 16, rows)
    torch.cuda.synchronize()
    assert torch.equal(c.k_codes, before)


# ---------------------------------------------------------------- a layer served

class Layer:
    """A decoder layer whose seven projections are packed: q, k, v in one product, the residuals in the
    products' epilogues, one workspace for every call."""

    def __init__(self, P, dtype, d=256, H=4, n_kv=2, hd=64, f=352, G=64, max_tokens=80, max_kv=128):
        self.P, self.dtype, self.d, self.H, self.n_kv, self.hd, self.f, self.max_kv = P, dtype, d, H, n_kv, hd, f, max_kv
        perm = R.layer(8, d, G, 1, "cuda", perm=True)["perm"]
        self.L = {n: R.layer(o, i, G, k, "cuda") for k, (n, o, i) in enumerate(
            [("qkv", (H + 2 * n_kv) * hd, d), ("o", d, H * hd), ("gate", f, d), ("up", f, d), ("down", d, f)], 30)}
        for n in ("qkv", "gate", "up"):
            self.L[n]["perm"] = perm
        for v in self.L.values():
            v["scales"] *= 0.05
        self.w = {n: weight(P, v) for n, v in self.L.items()}
        page = 16
        self.table = i32([[5, 0, 3, 9, 11, 2, 14, 7], [1, 4, 8, 6, 10, 12, 13, 15], [17, 16, 18, 19, 20, 21, 22, 23]])
        self.cache = P.KV4Cache.empty(24, n_kv, page, hd, self.table)
        for t in (self.cache.k_codes, self.cache.v_codes):
            t.fill_(-1)
        for t in (self.cache.k_grid, self.cache.v_grid):
            t.fill_(float("nan"))                        # nothing that was not appended may be seen
        w, m = self.w, max_tokens
        need = max(P.gptq_w4_linear_workspace_size(m, w["qkv"]), P.gptq_w4_linear_workspace_size(m, w["o"]),
                   P.gptq_w4_linear_workspace_size(m, w["down"]), P.gptq_w4_gated_workspace_size(m, w["gate"], w["up"]),
                   P.gptq_kv4_attention_workspace_size(m, H, self.cache, m, max_kv))
        self.ws, self.behind = poisoned(need)

    def norm(self, x):
        y = torch.empty(x.shape, dtype=F32, device="cuda")
        self.P.gptq_rmsnorm(x, y)
        return y.to(self.dtype)

    def step(self, x, start, kvl, max_q):
        """x [T, d]; returns every intermediate, each an operator's output."""
        P, w, T, dt = self.P, self.w, x.shape[0], self.dtype
        new = lambda *s: torch.full(s, float("nan"), dtype=dt, device="cuda")  # noqa: E731
        x1 = self.norm(x)
        qkv = new(T, self.H + 2 * self.n_kv, self.hd)
        P.gptq_w4_linear(x1, w["qkv"], qkv.view(T, -1), ws=self.ws)
        q, k, v = qkv.split([self.H, self.n_kv, self.n_kv], 1)
        P.gptq_kv4_append(self.cache, k, v, start, kvl)
        a = new(T, self.H, self.hd)
        P.gptq_kv4_attention(q, self.cache, start, kvl, max_q, self.max_kv, a, ws=self.ws)
        h = x.clone()
        P.gptq_w4_linear(a.view(T, -1), w["o"], h, R=h, ws=self.ws)       # onto the residual stream
        x2 = self.norm(h)
        m = new(T, self.f)
        P.gptq_w4_gated(x2, w["gate"], w["up"], m, ws=self.ws)
        y = h.clone()
        P.gptq_w4_linear(m, w["down"], y, R=y, ws=self.ws)
        return dict(x=x, x1=x1, qkv=qkv, a=a, h=h, x2=x2, m=m, y=y)

    def check(self, s, start, kvl, max_q):
        """Every step against float64 with the inputs it had, right after it ran."""
        dt, T = self.dtype, s["x"].shape[0]
        close(s["qkv"].view(T, -1), *linear_ref(s["x1"], self.L["qkv"], None, "none", None), dt)
        check_attention(self.P, self.cache, s["qkv"][:, :self.H], start, kvl, max_q, self.max_kv, dt, out=s["a"])
        close(s["h"], *linear_ref(s["a"].view(T, -1), self.L["o"], None, "none", s["x"]), dt)
        close(s["m"], *gated_ref(s["x2"], self.L["gate"], self.L["up"], "silu")[0], dt)
        close(s["y"], *linear_ref(s["m"], self.L["down"], None, "none", s["h"]), dt)
        assert bool((self.behind == 0xFF).all())


@pytest.mark.parametrize("dtype", [BF, HF])
def test_layer_served(P, dtype):
    """Prompts of three sequences, single tokens, and a step in which one sequence rests and one brings several."""
    layer = Layer(P, dtype)
    lens = [0, 0, 0]
    for k, new in enumerate(([40, 17, 3], [1, 1, 1], [1, 1, 1], [1, 0, 6])):
        lens = [a + b for a, b in zip(lens, new)]
        start = [0]
        for n in new:
            start.append(start[-1] + n)
        st, kv = i32(start), i32(lens)
        s = layer.step(acts(start[-1], layer.d, dtype, 50 + k), st, kv, max(new))
        layer.check(s, st, kv, max(new))


def test_tokens_one_by_one_or_at_once(P):
    """The same tokens as one prompt and one at a time give the same cache up to the products' order of
    additions, and attention that differs by the rounding of each only."""
    dtype, n = BF, 30
    n_pages, table, start, kvl = plan([n], [n], 16, 1)
    K, V, Q = (acts(n * h, 64, dtype, s).view(n, h, 64) for h, s in ((2, 1), (2, 2), (4, 3)))
    one, all_ = (P.KV4Cache.empty(n_pages, 2, 16, 64, table) for _ in range(2))
    a, b = torch.empty_like(Q), torch.empty_like(Q)
    P.gptq_kv4_append(all_, K, V, start, kvl)
    P.gptq_kv4_attention(Q, all_, start, kvl, n, n, a)
    for t in range(n):
        s, l = i32([0, 1]), i32([t + 1])
        P.gptq_kv4_append(one, K[t:t + 1], V[t:t + 1], s, l)
        P.gptq_kv4_attention(Q[t:t + 1], one, s, l, 1, t + 1, b[t:t + 1])
    used = sorted(table.flatten().tolist())
    for x, y in ((one.k_codes, all_.k_codes), (one.v_codes, all_.v_codes)):
        for j, pg in enumerate(table[0].tolist()):
            rows = min(16, n - 16 * j)
            assert torch.equal(x[pg, :, :rows], y[pg, :, :rows]), used
    d = (a.double() - b.double())
    assert float(d.norm()) <= 4 * R.EPS[dtype] * float(a.double().norm())


# ---------------------------------------------------------------- graphs and streams

def calls(P, dtype, seed):
    """(name, call, inputs, outputs) of every operator, each with a workspace of its own."""
    G, d, f = 64, 256, 320
    Lg, Lu = R.layer(f, d, G, seed, "cuda", perm=True), R.layer(f, d, G, seed + 1, "cuda")
    Lu["perm"] = Lg["perm"]
    g, u = weight(P, Lg), weight(P, Lu)
    out = []
    e = lambda *s: torch.empty(s, dtype=dtype, device="cuda")  # noqa: E731
    for m in (1, 20, 90, 200):
        x, y = acts(m, d, dtype, seed + m), e(m, f)
        ws = torch.empty(P.gptq_w4_linear_workspace_size(m, g), dtype=torch.uint8, device="cuda")
        out.append((f"linear {m}", lambda x=x, y=y, ws=ws: P.gptq_w4_linear(x, g, y, act="gelu", ws=ws), (x,), (y,)))
        M, Gt, Ut = e(m, f), e(m, f), e(m, f)
        ws = torch.empty(P.gptq_w4_gated_workspace_size(m, g, u), dtype=torch.uint8, device="cuda")
        out.append((f"gated {m}", lambda x=x, M=M, Gt=Gt, Ut=Ut, ws=ws: P.gptq_w4_gated(x, g, u, M, G=Gt, U=Ut, ws=ws), (x,), (M, Gt, Ut)))
        dM, gi, ui, dX, dG, dU = acts(m, f, dtype, 3), acts(m, f, dtype, 4), acts(m, f, dtype, 5), e(m, d), e(m, f), e(m, f)
        ws = torch.empty(P.gptq_w4_gated_backward_workspace_size(m, g, u), dtype=torch.uint8, device="cuda")
        out.append((f"gated backward {m}", lambda dM=dM, gi=gi, ui=ui, dX=dX, dG=dG, dU=dU, ws=ws: P.gptq_w4_gated_backward(
            dM, gi, ui, g, u, dX, dG=dG, dU=dU, ws=ws), (dM, gi, ui), (dX, dG, dU)))
    for new, ln in (([1, 1], [700, 33]), ([60, 2], [100, 1300])):
        n_pages, table, start, kvl = plan(new, ln, 16, seed)
        c = random_cache(P, n_pages, 2, 16, 64, table, seed)
        T = sum(new)
        K, V, Q = (acts(T * h, 64, dtype, seed + h).view(T, h, 64) for h in (2, 2, 4))
        rK, rV, o = torch.empty_like(K), torch.empty_like(V), torch.empty_like(Q)
        ws = torch.empty(P.gptq_kv4_attention_workspace_size(T, 4, c, max(new), max(ln)), dtype=torch.uint8, device="cuda")

        def run(c=c, K=K, V=V, Q=Q, rK=rK, rV=rV, o=o, ws=ws, start=start, kvl=kvl, mq=max(new), mk=max(ln)):
            P.gptq_kv4_append(c, K, V, start, kvl)
            P.gptq_kv4_read(c, rK, rV, start, kvl)
            P.gptq_kv4_attention(Q, c, start, kvl, mq, mk, o, ws=ws)
        out.append((f"cache {new}", run, (K, V, Q), (rK, rV, o)))
    return out


@pytest.mark.parametrize("dtype", [BF, HF])
def test_captured_calls_replay_like_eager_ones(P, dtype):
    """Each operator captured alone and replayed four times over new inputs, with eager runs in between."""
    for name, call, ins, outs in calls(P, dtype, 5):
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        for k in range(4):
            for t in ins:
                t.mul_(-0.75 if k % 2 else 1.25)
            for t in outs:
                t.fill_(float("nan"))
            call()
            torch.cuda.synchronize()
            want = [t.clone() for t in outs]
            for t in outs:
                t.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            print(f"  {name}, replay {k}", flush=True)
            for a, b in zip(outs, want):
                assert torch.equal(a, b), (name, k)


def test_two_graphs_and_an_eager_stream_at_once(P):
    """Two captures of the same operators with workspaces of their own, replayed on two streams while the
    default one runs a third set."""
    sets = [calls(P, BF, s) for s in (5, 40, 80)]
    want = []
    for s in sets:
        for _, call, _, _ in s:
            call()
        torch.cuda.synchronize()
        want.append([t.clone() for _, _, _, outs in s for t in outs])
    graphs, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for s in sets[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _, call, _, _ in s:
                call()
        graphs.append(g)
    for k in range(3):
        for s in sets:
            for _, _, _, outs in s:
                for t in outs:
                    t.fill_(float("nan"))
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        for _, call, _, _ in sets[2]:
            call()
        torch.cuda.synchronize()
        for s, w in zip(sets, want):
            for t, x in zip([t for _, _, _, outs in s for t in outs], w):
                assert torch.equal(t, x)


def test_other_stream_without_a_workspace(P):
    """A stream given by argument; the binding's own scratch is not handed out before the call's work is done."""
    L = R.layer(1024, 2048, 128, 3, "cuda", perm=True)
    w, X = weight(P, L), acts(300, 2048, BF, 1)
    want = torch.empty((300, 1024), dtype=BF, device="cuda")
    P.gptq_w4_linear(X, w, want)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for _ in range(3):
        Y = torch.full_like(want, float("nan"))
        st.wait_stream(torch.cuda.current_stream())
        P.gptq_w4_linear(X, w, Y, stream=st)
        torch.full((32 << 20,), 0xFF, dtype=torch.uint8, device="cuda")   # what the allocator would hand out again
        torch.cuda.current_stream().wait_stream(st)
        assert torch.equal(Y, want)


def test_binding_refuses_tensors_that_do_not_fit(P):
    L = R.layer(16, 64, 32, 1, "cuda")
    w, X, Y = weight(P, L), acts(3, 64, BF, 1), torch.empty((3, 16), dtype=BF, device="cuda")
    c = random_cache(P, 2, 1, 16, 64, i32([[0], [1]]), 2)
    rows, start, kvl = acts(2, 64, BF, 2).view(2, 1, 64), i32([0, 1, 2]), i32([1, 1])
    for call in (
        lambda: P.gptq_w4_linear(X.float(), w, Y),
        lambda: P.gptq_w4_linear(X[:, :56], w, Y),
        lambda: P.gptq_w4_linear(X.t(), w, Y),
        lambda: P.gptq_w4_linear(X.cpu(), w, Y),
        lambda: P.gptq_w4_linear(X, w, Y[:2]),
        lambda: P.gptq_w4_linear(X, w, Y, act="tanh"),
        lambda: P.gptq_w4_linear(X, w, Y, R=Y.float()),
        lambda: P.gptq_w4_linear(X, w, Y, bias=Y[0].float()),
        lambda: P.gptq_w4_linear(X, w, Y.double()),
        lambda: P.gptq_w4_gated(X, w, w, Y, G=Y.float(), U=Y),
        lambda: P.gptq_w4_gated(X, w, w, torch.empty((3, 20), dtype=BF, device="cuda")[:, :16]),
        lambda: P.gptq_w4_gated_backward(Y, Y, Y.half(), w, w, X),
        lambda: P.W4Weight(L["packed"], L["scales"][:, :1].contiguous(), L["zeros"], 32),
        lambda: P.W4Weight(L["packed"], L["scales"], L["zeros"], 12),
        lambda: P.gptq_kv4_append(c, rows, rows.half(), start, kvl),
        lambda: P.gptq_kv4_append(c, rows, rows[:1], start, kvl),
        lambda: P.gptq_kv4_append(c, rows, rows, start.long(), kvl),
        lambda: P.gptq_kv4_append(c, rows, rows, start[:2], kvl),
        lambda: P.gptq_kv4_read(c, rows[:, :, :32], None, start, kvl),
        lambda: P.gptq_kv4_attention(rows.float(), c, start, kvl, 1, 16, rows),
        lambda: P.gptq_kv4_attention(rows, c, start, kvl, 1, 16, rows[:1]),
        lambda: P.gptq_kv4_attention(rows, c, start, kvl, 1, (1 << 32) + 16, torch.empty_like(rows)),
        lambda: P.gptq_kv4_attention_workspace_size(2, 1, c, 1 << 31, 16),
        lambda: P.KV4Cache(c.k_codes, c.v_codes, c.k_grid, c.v_grid[:, :, :8].contiguous(), c.page_table),
    ):
        with pytest.raises(ValueError):
            call()
    for call in (
        lambda: P.gptq_w4_gated(X, w, w, Y, act="relu"),
        lambda: P.gptq_w4_gated(X, w, w, Y, G=torch.empty_like(Y)),
        lambda: P.gptq_w4_linear(X[:1].expand(3, 64), w, Y),
        lambda: P.gptq_kv4_attention(rows, c, start, kvl, 0, 16, torch.empty_like(rows)),
        lambda: P.gptq_kv4_attention(rows, c, start, kvl, 1, 16, torch.empty_like(rows), scale=float("nan")),
        lambda: P.gptq_w4_gated_backward(Y, Y, Y, w, w, X, ws=torch.empty(16, dtype=torch.uint8, device="cuda")),
    ):
        with pytest.raises(P.GPTQError):
            call()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("n_q", [1, 3, 60, 300])
@pytest.mark.parametrize("what", ["v step", "v lo", "k step", "k lo"])
def test_attention_a_row_that_is_no_number_reaches_only_those_that_see_it(P, dtype, n_q, what):
    """A cached row whose step or minimum is NaN or infinite, in the middle of the new tokens: the tokens
    before it are what they are without it, and it shows in itself and in those behind it.  Not to the bit:
    rows that are computed together change their reference maximum together, so an infinite score of one
    moves the others' roundings.  Both results are within the same bound of the exact one, half a step of p's
    type on terms of at most 15 steps and half a step of the output, so they differ by twice that at most
    (fp32's part, below 1e-4 here, beside it)."""
    n_pages, table, start, kvl = plan([n_q, n_q], [n_q + 37, n_q], 16, 1)
    c = random_cache(P, n_pages, 1, 16, 64, table, 2)
    Q = acts(2 * n_q * 2, 64, dtype, 5).view(2 * n_q, 2, 64)
    a, b = torch.empty_like(Q), torch.empty_like(Q)
    P.gptq_kv4_attention(Q, c, start, kvl, n_q, n_q + 37, a)
    grid = c.v_grid if what[0] == "v" else c.k_grid
    for value in (float("nan"), float("inf")):
        at = n_q // 2
        p = 37 + at
        grid[int(table[0, p // 16]), 0, p % 16, 0 if "step" in what else 1] = value
        P.gptq_kv4_attention(Q, c, start, kvl, n_q, n_q + 37, b)
        assert torch.equal(b[n_q:], a[n_q:])                       # another sequence shares nothing
        x, y, eps = a[:at].double(), b[:at].double(), R.EPS[dtype]
        assert torch.isfinite(y).all()
        assert bool(((x - y).abs() <= 2 * eps * (15 * 0.4 + x.abs() * (1 + eps)) + 1e-4).all())
        if what[0] == "v" or value != value:
            assert not torch.isfinite(b[at:n_q]).any()
