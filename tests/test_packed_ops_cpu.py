"""Refusals and size queries of the operators on the packed layer and of the
4-bit cache, without a GPU: every call here is turned down on the host."""
from __future__ import annotations

import ctypes

import pytest

torch = pytest.importorskip("torch")
import post_weight_quantization_29_amd as P  # noqa: E402
from post_weight_quantization_29_amd import _lib as M  # noqa: E402

vp, i64, i32, f32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
F32, F16, BF16 = 0, 1, 2
FAKE = 0x100000
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    assert M._DTYPE == {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
    return P.lib()


def weight(packed=FAKE, scales=FAKE, zeros=FAKE, perm=0, d_out=64, d_in=256, G=128, ng=None):
    ng = -(-d_in // (d_in if G == -1 else max(G, 1))) if ng is None else ng
    return M.gptq_w4_weight(packed, scales, zeros, perm or None, d_out, d_in, G, ng)


def cache(k=FAKE, v=FAKE, kg=FAKE, vg=FAKE, table=FAKE, n_pages=8, n_kv=2, page=16, hd=128, n_seqs=3, max_pages=4):
    return M.gptq_kv4_cache(k or None, v or None, kg or None, vg or None, table or None, n_pages, n_kv, page, hd, n_seqs, max_pages)


BAD_WEIGHTS = [dict(packed=None), dict(scales=None), dict(zeros=None), dict(packed=FAKE + 2), dict(scales=FAKE + 1), dict(perm=FAKE + 3),
               dict(d_out=0), dict(d_out=-1), dict(d_in=0, ng=0), dict(d_in=252), dict(d_in=(1 << 20) + 8), dict(G=0), dict(G=-2),
               dict(G=12), dict(ng=1), dict(ng=3)]


def linear(L, w=None, X=FAKE, xt=BF16, m=4, ldx=256, bias=None, act=0, R=None, ldr=0, Y=FAKE, yt=BF16, ldy=64, ws=FAKE, nb=BIG):
    w = weight() if w is None else w
    return L.gptq_w4_linear(vp(X), xt, i64(m), i64(ldx), ctypes.byref(w), vp(bias), act, vp(R), i64(ldr), vp(Y), yt, i64(ldy),
                            vp(ws), sz(nb), None)


def test_linear_refuses(L):
    for kw in BAD_WEIGHTS:
        assert linear(L, weight(**kw)) == M.ERR_INVALID_ARG, kw
        assert L.gptq_w4_linear_workspace_size(i64(100), ctypes.byref(weight(**kw))) == 0, kw
    for kw in (dict(X=None), dict(Y=None), dict(m=-1), dict(m=1 << 31), dict(xt=F32), dict(xt=3), dict(yt=3), dict(act=-1), dict(act=5),
               dict(ldx=255), dict(ldx=0), dict(ldy=63), dict(R=FAKE, ldr=63), dict(X=FAKE + 1), dict(Y=FAKE + 1),
               dict(Y=FAKE + 2, yt=F32), dict(bias=FAKE + 1), dict(R=FAKE + 1, ldr=64)):
        assert linear(L, **kw) == M.ERR_INVALID_ARG, kw
    perm = weight(perm=FAKE)
    need = L.gptq_w4_linear_workspace_size(i64(4), ctypes.byref(perm))
    assert need > 0
    for kw in (dict(ws=None), dict(nb=need - 1), dict(ws=FAKE + 16)):
        assert linear(L, perm, **kw) == M.ERR_WORKSPACE, kw
    assert linear(L, weight(), m=200, ws=None) == M.ERR_WORKSPACE
    assert linear(L, weight(), X=FAKE + 2, ws=None) == M.ERR_WORKSPACE       # rows off the 16-byte grid are copied
    assert linear(L, m=0, X=None, Y=None, ws=None) == M.OK


def gated(L, g=None, u=None, X=FAKE, xt=BF16, m=4, ldx=256, act=2, G=None, U=None, Mo=FAKE, ws=FAKE, nb=BIG):
    g, u = weight() if g is None else g, weight() if u is None else u
    return L.gptq_w4_gated(vp(X), xt, i64(m), i64(ldx), ctypes.byref(g), ctypes.byref(u), act, vp(G), vp(U), vp(Mo), vp(ws), sz(nb), None)


def backward(L, g=None, u=None, dM=FAKE, G=FAKE, U=FAKE, t=BF16, m=4, act=2, dG=None, dU=None, dX=FAKE, ws=FAKE, nb=BIG):
    g, u = weight() if g is None else g, weight() if u is None else u
    return L.gptq_w4_gated_backward(vp(dM), vp(G), vp(U), t, i64(m), ctypes.byref(g), ctypes.byref(u), act, vp(dG), vp(dU), vp(dX),
                                    vp(ws), sz(nb), None)


def test_gated_and_backward_refuse(L):
    pairs = [(weight(**kw), weight()) for kw in BAD_WEIGHTS] + [(weight(), weight(**kw)) for kw in BAD_WEIGHTS]
    pairs += [(weight(), weight(d_out=72)), (weight(), weight(d_in=512)), (weight(), weight(G=64)), (weight(perm=FAKE), weight()),
              (weight(perm=FAKE), weight(perm=FAKE + 64))]
    for a, b in pairs:
        assert gated(L, a, b) == M.ERR_INVALID_ARG and backward(L, a, b) == M.ERR_INVALID_ARG
        for q in (L.gptq_w4_gated_workspace_size, L.gptq_w4_gated_backward_workspace_size):
            assert q(i64(9), ctypes.byref(a), ctypes.byref(b)) == 0
    for kw in (dict(X=None), dict(Mo=None), dict(m=-1), dict(m=1 << 31), dict(xt=F32), dict(act=0), dict(act=1), dict(act=5), dict(ldx=255),
               dict(G=FAKE), dict(U=FAKE), dict(X=FAKE + 1), dict(Mo=FAKE + 1), dict(G=FAKE + 1, U=FAKE)):
        assert gated(L, **kw) == M.ERR_INVALID_ARG, kw
    for kw in (dict(dM=None), dict(G=None), dict(U=None), dict(dX=None), dict(m=-1), dict(t=F32), dict(act=0), dict(act=1),
               dict(dM=FAKE + 1), dict(dX=FAKE + 1), dict(dG=FAKE + 1), dict(dU=FAKE + 1)):
        assert backward(L, **kw) == M.ERR_INVALID_ARG, kw
    g = weight()
    assert gated(L, m=200, ws=None) == M.ERR_WORKSPACE
    need = L.gptq_w4_gated_backward_workspace_size(i64(4), ctypes.byref(g), ctypes.byref(g))
    for kw in (dict(ws=None), dict(nb=need - 1), dict(ws=FAKE + 16)):
        assert backward(L, **kw) == M.ERR_WORKSPACE, kw
    assert gated(L, m=0, X=None, Mo=None, ws=None) == M.OK and backward(L, m=0, dM=None, dX=None, ws=None) == M.OK
    # group_size -1 and the row's length say the same
    assert L.gptq_w4_gated_workspace_size(i64(9), ctypes.byref(weight(G=-1)), ctypes.byref(weight(G=256))) > 0


BAD_CACHES = [dict(k=0), dict(v=0), dict(kg=0), dict(vg=0), dict(table=0), dict(k=FAKE + 8), dict(vg=FAKE + 4), dict(table=FAKE + 2),
              dict(n_pages=0), dict(n_kv=0), dict(n_seqs=0), dict(max_pages=0), dict(page=0), dict(page=24), dict(page=-16), dict(hd=96),
              dict(hd=256), dict(max_pages=1 << 28), dict(n_pages=1 << 30)]


def append(L, c=None, K=FAKE, V=FAKE, t=BF16, n=5, ldk=256, ldv=256, qs=FAKE, kl=FAKE):
    c = cache() if c is None else c
    return L.gptq_kv4_append(ctypes.byref(c), vp(K), vp(V), t, i64(n), i64(ldk), i64(ldv), vp(qs), vp(kl), None)


def read(L, c=None, K=FAKE, V=FAKE, t=BF16, n=5, qs=FAKE, kl=FAKE):
    c = cache() if c is None else c
    return L.gptq_kv4_read(ctypes.byref(c), vp(K), vp(V), t, i64(n), vp(qs), vp(kl), None)


def attention(L, c=None, Q=FAKE, t=BF16, n=5, heads=4, ldq=512, qs=FAKE, kl=FAKE, mq=5, mk=64, scale=0.1, out=FAKE, ldo=512, ws=FAKE, nb=BIG):
    c = cache() if c is None else c
    return L.gptq_kv4_attention(vp(Q), t, i64(n), i32(heads), i64(ldq), ctypes.byref(c), vp(qs), vp(kl), i32(mq), i32(mk), f32(scale),
                                vp(out), i64(ldo), vp(ws), sz(nb), None)


def test_cache_calls_refuse(L):
    for kw in BAD_CACHES:
        c = cache(**kw)
        assert append(L, c) == M.ERR_INVALID_ARG and read(L, c) == M.ERR_INVALID_ARG and attention(L, c) == M.ERR_INVALID_ARG, kw
        assert L.gptq_kv4_attention_workspace_size(i64(5), i32(4), ctypes.byref(c), i32(5), i32(64)) == 0, kw
    for kw in (dict(K=None), dict(V=None), dict(qs=None), dict(kl=None), dict(t=3), dict(n=-1), dict(n=1 << 31), dict(ldk=255), dict(ldv=0),
               dict(K=FAKE + 1), dict(V=FAKE + 2, t=F32)):
        assert append(L, **kw) == M.ERR_INVALID_ARG, kw
    for kw in (dict(qs=None), dict(kl=None), dict(t=3), dict(n=-1), dict(K=FAKE + 1), dict(V=FAKE + 2, t=F32)):
        assert read(L, **kw) == M.ERR_INVALID_ARG, kw
    for kw in (dict(Q=None), dict(out=None), dict(qs=None), dict(kl=None), dict(t=F32), dict(t=3), dict(n=-1), dict(heads=0), dict(heads=3),
               dict(ldq=504), dict(ldo=504), dict(ldq=516), dict(ldo=516), dict(Q=FAKE + 8), dict(out=FAKE + 2), dict(mq=0), dict(mk=0),
               dict(mq=-1), dict(mk=-5), dict(scale=float("nan")), dict(scale=float("inf")), dict(mq=1 << 30, heads=8, ldq=1024, ldo=1024)):
        assert attention(L, **kw) == M.ERR_INVALID_ARG, kw
    long = cache(n_pages=4096, max_pages=4096)
    need = L.gptq_kv4_attention_workspace_size(i64(5), i32(4), ctypes.byref(long), i32(5), i32(65536))
    assert need > 0
    for kw in (dict(ws=None), dict(nb=need - 1), dict(ws=FAKE + 16)):
        assert attention(L, long, mk=65536, **kw) == M.ERR_WORKSPACE, kw
    assert append(L, n=0, K=None, V=None) == M.OK and read(L, n=0) == M.OK and read(L, K=None, V=None) == M.OK
    assert attention(L, n=0, Q=None, out=None, ws=None) == M.OK


def test_size_queries_cover_every_alignment(L):
    """A query knows neither X's address nor its pitch: it has room for X's copy whenever one may be made."""
    for m in (1, 16, 17, 64, 65, 128, 129, 1000):
        for d_in in (256, 264):
            w = weight(d_in=d_in, G=8 if d_in == 264 else 128)
            assert L.gptq_w4_linear_workspace_size(i64(m), ctypes.byref(w)) >= m * d_in * 2
    assert L.gptq_w4_linear_workspace_size(i64(0), ctypes.byref(weight())) == 0
    assert L.gptq_w4_linear_workspace_size(i64(-3), ctypes.byref(weight())) == 0


def test_binding_refuses(L):
    """Tensors that are not on a GPU, or of other types or shapes, before any library call."""
    packed, sc, z = torch.zeros((64, 32), dtype=torch.int32), torch.ones((64, 2)), torch.zeros((64, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="packed must be on cuda"):
        P.W4Weight(packed, sc, z, 128)
    codes, grid = torch.zeros((4, 2, 16, 16), dtype=torch.int32), torch.zeros((4, 2, 16, 2), dtype=torch.float16)
    with pytest.raises(ValueError, match="k_codes must be on cuda"):
        P.KV4Cache(codes, codes, grid, grid, torch.zeros((1, 4), dtype=torch.int32))
